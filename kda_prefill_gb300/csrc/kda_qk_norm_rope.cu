// Norms of queries and keys for each head with the rotary positions in the same pass:
//
//     y = x / sqrt(mean(x^2) + eps) * weight,   pairs of y's first rot dimensions turned
//
// Bound by reading and writing the heads once.  As in kda_rope a row is cut into units, 16
// bytes and their partners of the half layout, and a thread keeps its unit of its head and
// goes through a CTA's tokens, so that it reads its weights once.  A row's lanes lie beside
// each other in a warp and sum its squares by shuffles; the row stays in registers.  Longer
// rows, and rows that are not whole pieces, take a warp each, which reads them twice.

#include "kda_f32x2.cuh"
#include "kda_rope.cuh"

namespace kda {
namespace {

using rope::Unit;

constexpr int kMaxThreads = 512;
constexpr int kMaxTable = 2048;  // pairs times tokens a CTA holds (16 KB)

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int w = LANES / 2; w >= 1; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    return x;
}

template <int VE>
__device__ __forceinline__ void load_weights(float (&w)[VE], const float* p) {
#pragma unroll
    for (int j = 0; j < VE; ++j) w[j] = p ? p[j] : 1.f;
}
template <int VE>
__device__ __forceinline__ void pairs(f2 (&x)[VE / 2], const float (&f)[VE]) {
#pragma unroll
    for (int j = 0; j < VE / 2; ++j) x[j] = pack2(f[2 * j], f[2 * j + 1]);
}
template <int VE>
__device__ __forceinline__ void values(float (&f)[VE], const f2 (&x)[VE / 2]) {
#pragma unroll
    for (int j = 0; j < VE / 2; ++j) {
        const float2 y = unpack2(x[j]);
        f[2 * j] = y.x, f[2 * j + 1] = y.y;
    }
}

// The table's entries of two pairs, 16 bytes: (c, c, s, s) for the half layout, (c, s, c, s)
// for pairs beside each other. Units lie beside each other in it, so that a row's lanes
// read it without conflicts.
template <int VE, bool IL>
struct Entry {
    static constexpr int kPairs = IL ? VE / 2 : VE;  // of a unit
    static __device__ __forceinline__ void put(float* table, int j, int rot_units, float2 cs) {
        const int u = j / kPairs, k = j % kPairs, e = k & 1;
        float* at = table + ((k >> 1) * rot_units + u) * 4;
        at[IL ? 2 * e : e] = cs.x;
        at[IL ? 2 * e + 1 : 2 + e] = cs.y;
    }
};

// Rows ahead and registers: a unit and its partner with their weights take 80 registers for two
// rows, a unit alone 56 for four (16384 tokens, 12 + 12 heads, half layout: 37.1 us, 39.1 with
// 72 registers, 41.2 with 64; 12 + 2 heads, pairs beside each other: 21.7 us, 23.0 with 64
// registers, 24.9 with 48; each with the tokens of a CTA that suit it).  These times and those at
// the launch are of calls on one set of buffers, part of which stays in the L2: on alternating
// ones the same calls take 39.2 us for 37.1 and 25.1 for 21.7.
constexpr int regs_of(bool interleaved) { return interleaved ? 56 : 80; }

// `units` units a row, at most LANES, the first rot_units of them turned.
template <class E, int VE, bool IL, int LANES>
__global__ void __maxnreg__(regs_of(IL))
kda_qk_norm_rope(const __grid_constant__ NormRopeParams p, int tokens, int rot_units, int units) {
    using U = Unit<E, VE, IL>;
    using T = Entry<VE, IL>;
    __shared__ __align__(16) float table[2 * kMaxTable];
    __shared__ unsigned long long fraction[rope::kMaxPairs];
    constexpr int kAhead = IL ? 4 : 2, kH = VE / 2;
    const int half = p.rot >> 1;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, p.T - t0);
    const int h0 = p.x[0].heads, items = (h0 + p.x[1].heads) * LANES;
    const float per = 1.f / (float)p.D;
    bool made = false;
    // whole warps go on together
    for (int item = threadIdx.x; (item & ~31) < items || !made; item += blockDim.x) {
        int h = item / LANES;
        const int u = item % LANES;
        const bool live = item < items && u < units;
        const int which = h >= h0;
        const RopeTensor& r = p.x[which];
        if (which) h -= h0;
        const bool turned = live && u < rot_units;
        const bool two = U::kPaired && turned;
        const int at = U::one(p, u, rot_units), at2 = U::two(p, u);
        const int64_t in_st = r.in_st, out_st = r.out_st;
        const E* in = static_cast<const E*>(r.in) + t0 * in_st + (int64_t)h * r.in_sh;
        E* out = static_cast<E*>(r.out) + t0 * out_st + (int64_t)h * r.out_sh;
        const int n = live ? nt : 0;
        U x[kAhead] = {};
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < n) x[i].load(in + i * in_st, at, at2, turned);
        f2 w1[kH], w2[kH];
        {
            const float* weight = live && p.weight[which] ? p.weight[which] + (int64_t)h * p.weight_sh[which] : nullptr;
            float w[VE];
            load_weights<VE>(w, weight ? weight + at : nullptr);
            pairs<VE>(w1, w);
            load_weights<VE>(w, weight && two ? weight + at2 : nullptr);
            pairs<VE>(w2, w);
        }
        if (!made) {
            for (int j = threadIdx.x; j < half; j += blockDim.x) fraction[j] = rope::fraction_of(p, j);
            __syncthreads();
            for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
                const int t = i / half, j = i - t * half;
                T::put(table + 2 * t * half, j, rot_units, rope::turn_of(p, t0 + t, fraction[j]));
            }
            __syncthreads();
            made = true;
        }
        const float4* cs = reinterpret_cast<const float4*>(table) + u;
        for (int t = 0; t < nt; t += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                f2 f[kH], g[kH];
                float v[VE];
                x[i].a.get(v);
                pairs<VE>(f, v);
                f2 sum = 0;
#pragma unroll
                for (int j = 0; j < kH; ++j) sum = fma2(f[j], f[j], sum);
                if constexpr (U::kPaired) {
                    x[i].b.get(v);
                    pairs<VE>(g, v);
                    if (two) {
#pragma unroll
                        for (int j = 0; j < kH; ++j) sum = fma2(g[j], g[j], sum);
                    }
                }
                const float2 both = unpack2(sum);
                const float all = group_sum<LANES>(live ? both.x + both.y : 0.f);
                // (a sum that overflows leaves no row to give: infinity times zero makes it NaN, not zeros)
                const float inv = rsqrtf(fmaf(all, 0.f, fmaf(all, per, p.eps)));
                const f2 inv2 = pack2(inv, inv);
                if (t + i < n) {
#pragma unroll
                    for (int j = 0; j < kH; ++j) f[j] = mul2(f[j], mul2(inv2, w1[j]));
                    if constexpr (U::kPaired) {
#pragma unroll
                        for (int j = 0; j < kH; ++j) g[j] = mul2(g[j], mul2(inv2, w2[j]));
                    }
                    if (turned) {
                        const float4* k = cs + i * (half / 2);
#pragma unroll
                        for (int j = 0; j < T::kPairs / 2; ++j) {
                            const float4 y = k[j * rot_units];
                            if constexpr (U::kPaired) {
                                const f2 c = pack2(y.x, y.y), s = pack2(y.z, y.w), ms = pack2(-y.z, -y.w);
                                const f2 a = f[j];
                                f[j] = fma2(g[j], ms, mul2(a, c));
                                g[j] = fma2(a, s, mul2(g[j], c));
                            } else {
                                const float2 a = unpack2(f[2 * j]), b = unpack2(f[2 * j + 1]);
                                f[2 * j] = fma2(pack2(a.y, a.x), pack2(-y.y, y.y), mul2(f[2 * j], pack2(y.x, y.x)));
                                f[2 * j + 1] = fma2(pack2(b.y, b.x), pack2(-y.w, y.w), mul2(f[2 * j + 1], pack2(y.z, y.z)));
                            }
                        }
                    }
                    values<VE>(v, f);
                    x[i].a.set(v);
                    if constexpr (U::kPaired) {
                        values<VE>(v, g);
                        x[i].b.set(v);
                    }
                    x[i].store(out + i * out_st, at, at2, turned);
                }
            }
            cs += kAhead * (half / 2);
            in += kAhead * in_st;
            out += kAhead * out_st;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (t + kAhead + i < n) x[i].load(in + i * in_st, at, at2, turned);
        }
    }
}

// Rows of more units: a warp each, the row read again for its products.
template <class E, int VE, bool IL>
__global__ void __launch_bounds__(kMaxThreads)
kda_qk_norm_rope_long(const __grid_constant__ NormRopeParams p, int tokens, int rot_units, int units) {
    using U = Unit<E, VE, IL>;
    __shared__ float2 table[kMaxTable];
    __shared__ unsigned long long fraction[rope::kMaxPairs];
    const int half = p.rot >> 1;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, p.T - t0);
    for (int j = threadIdx.x; j < half; j += blockDim.x) fraction[j] = rope::fraction_of(p, j);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int t = i / half, j = i - t * half;
        table[i] = rope::turn_of(p, t0 + t, fraction[j]);
    }
    __syncthreads();
    const int h0 = p.x[0].heads, heads = h0 + p.x[1].heads, lane = threadIdx.x & 31;
    for (int row = threadIdx.x >> 5; row < nt * heads; row += blockDim.x >> 5) {
        const int t = row / heads;
        int h = row - t * heads;
        const int which = h >= h0;
        const RopeTensor& r = p.x[which];
        if (which) h -= h0;
        const E* in = static_cast<const E*>(r.in) + (t0 + t) * r.in_st + (int64_t)h * r.in_sh;
        E* out = static_cast<E*>(r.out) + (t0 + t) * r.out_st + (int64_t)h * r.out_sh;
        const float* weight = p.weight[which] ? p.weight[which] + (int64_t)h * p.weight_sh[which] : nullptr;
        float sum = 0.f;
        for (int c = lane * VE; c < p.D; c += 32 * VE) {
            float f[VE];
            rows::load<E, VE>(in + c).get(f);
#pragma unroll
            for (int j = 0; j < VE; ++j) sum = fmaf(f[j], f[j], sum);
        }
        sum = group_sum<32>(sum);
        const float inv = sum < INFINITY ? 1.f / sqrtf(sum / (float)p.D + p.eps) : NAN;
        __syncwarp();  // in place: all lanes have read the row
        for (int u = lane; u < units; u += 32) {
            const bool turned = u < rot_units;
            const int at = U::one(p, u, rot_units), at2 = U::two(p, u);
            U x = {};
            x.load(in, at, at2, turned);
            float f[VE], g[VE], w1[VE], w2[VE];
            load_weights<VE>(w1, weight ? weight + at : nullptr);
            load_weights<VE>(w2, weight && U::kPaired && turned ? weight + at2 : nullptr);
            x.a.get(f);
            if constexpr (U::kPaired) x.b.get(g);
#pragma unroll
            for (int j = 0; j < VE; ++j) f[j] *= inv * w1[j];
            if constexpr (U::kPaired) {
#pragma unroll
                for (int j = 0; j < VE; ++j) g[j] *= inv * w2[j];
            }
            if (turned) U::turn(f, g, table + t * half + (U::kPaired ? u * VE : u * VE / 2));
            x.a.set(f);
            if constexpr (U::kPaired) x.b.set(g);
            x.store(out, at, at2, turned);
        }
    }
}

template <class E, int VE, bool IL, int LANES>
cudaError_t launch(const NormRopeParams& p, int rot_units, int units, cudaStream_t s) {
    const int most = kMaxTable / max(1, p.rot / 2);  // tokens that the table holds
    const int heads = p.x[0].heads + p.x[1].heads;
    if constexpr (LANES == 0) {
        // eight tokens a CTA, and few enough that each SM has eight CTAs where there are so
        // many tokens
        const int tokens = (int)max((int64_t)1, min((int64_t)min(8, most), p.T / (8 * num_sms())));
        const int threads = (int)min((int64_t)kMaxThreads, (int64_t)heads * tokens * 32);
        kda_qk_norm_rope_long<E, VE, IL><<<(unsigned)((p.T + tokens - 1) / tokens), max(128, threads), 0, s>>>(p, tokens, rot_units, units);
    } else {
        // threads: as many as a token's units in the fewest rounds, in whole warps
        const int items = heads * LANES;
        const int rounds = (items + kMaxThreads - 1) / kMaxThreads;
        const int threads = max(128, ((items + rounds - 1) / rounds + 31) / 32 * 32);
        // tokens a CTA: all CTAs are on the SMs at once, or go there in the fewest whole waves
        // (16384 tokens, 12 + 2 heads: 21.7 us with 22 tokens, one wave; 23.3 with 8, 24.8 with
        // 16; 12 + 12 heads: 37.1 us with 27 tokens, 38.1 with 8, 47.5 with 24)
        const int resident = max(1, min(65536 / (regs_of(IL) * threads), min(2048 / threads, 10)));
        const int64_t ctas = (int64_t)resident * num_sms(), one = (p.T + ctas - 1) / ctas, waves = (one + most - 1) / most;
        const int tokens = (int)max((int64_t)1, (p.T + waves * ctas - 1) / (waves * ctas));
        kda_qk_norm_rope<E, VE, IL, LANES><<<(unsigned)((p.T + tokens - 1) / tokens), threads, 0, s>>>(p, tokens, rot_units, units);
    }
    return cudaGetLastError();
}

template <class E, int VE, bool IL>
cudaError_t by_units(const NormRopeParams& p, cudaStream_t s) {
    const int rot_units = IL && VE > 1 ? p.rot / VE : p.rot / 2 / VE;
    const int units = rot_units + (p.D - p.rot) / VE;
    if constexpr (VE > 1) {
        if (units <= 8) return launch<E, VE, IL, 8>(p, rot_units, units, s);
        if (units <= 16) return launch<E, VE, IL, 16>(p, rot_units, units, s);
        if (units <= 32) return launch<E, VE, IL, 32>(p, rot_units, units, s);
    }
    return launch<E, VE, IL, 0>(p, rot_units, units, s);
}

template <class E>
cudaError_t dispatch(const NormRopeParams& p, cudaStream_t s) {
    constexpr int VE = 16 / sizeof(E);
    // 16-byte units when the dimensions, strides and bases allow them
    bool vec = (p.interleaved ? p.rot : p.rot / 2) % VE == 0 && (p.D - p.rot) % VE == 0;
    for (const RopeTensor& x : p.x)
        if (x.heads)
            vec = vec && ((reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out)) & 15) == 0 &&
                  (x.in_st | x.in_sh | x.out_st | x.out_sh) % VE == 0;
    if (p.interleaved) return vec ? by_units<E, VE, true>(p, s) : by_units<E, 1, true>(p, s);
    return vec ? by_units<E, VE, false>(p, s) : by_units<E, 1, false>(p, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, cudaStream_t s) {
    if (p.dtype == KDA_F32) return dispatch<float>(p, s);
    if (p.dtype == KDA_BF16) return dispatch<__nv_bfloat16>(p, s);
    return dispatch<__half>(p, s);
}

}  // namespace kda
