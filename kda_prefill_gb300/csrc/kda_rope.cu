// Rotary positions: y1 = c x1 - s x2, y2 = c x2 + s x1 for each pair of a head's
// first rot dimensions, with (c, s) of one token and pair shared by all heads.
//
// The angle p f is wanted modulo one turn.  f / 2 pi is rounded to a 64-bit
// fraction of a turn F; then p F mod 2^64 is the phase, exactly, in one integer
// product (two's complement wraps as turns do), and its top 32 bits give the
// argument of sincospi.  A fp32 product p f would be off by p 2^-25 radians.
//
// Bound by reading and writing the heads once.  A token's heads are cut into units of
// 16 bytes and their partners (half layout: the 16 bytes rot / 2 further), or of 16
// bytes to copy.  A CTA takes a few tokens; a thread keeps its unit of its head and goes
// through the tokens, so that addresses only advance, four of them in flight, the
// first four read before the tokens' (c, s) are made.  16384 tokens, 12 + 12 heads of 128,
// half of each turned by interleaved pairs: 34.8 us, 85 % of a plain copy's rate; the rest is
// the start and the end of a launch.  All of each turned in the half layout: 46.4 us in bf16,
// 64 %, and 66.0 us in fp32, 90 %.

#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxTable = 2048;  // pairs times tokens a CTA holds (16 KB)

// One unit of a row: 16 bytes, and for pairs of the half layout (and for the narrow
// form's pairs) the partner's.
template <class E, int VE, bool IL>
struct Unit {
    rows::Piece<E, VE> a, b;
    static constexpr bool kPaired = !IL || VE == 1;

    // Offsets of the two in a row; units from rot_units on are copied.
    static __device__ __forceinline__ int one(const RopeParams& p, int u, int rot_units) {
        if (u >= rot_units) return p.rot + (u - rot_units) * VE;
        return IL && VE == 1 ? 2 * u : u * VE;
    }
    static __device__ __forceinline__ int two(const RopeParams& p, int u) {
        return IL ? 2 * u + 1 : (p.rot >> 1) + u * VE;
    }
    __device__ __forceinline__ void load(const E* in, int at, int at2, bool turned) {
        a = rows::load<E, VE>(in + at);
        if (kPaired && turned) b = rows::load<E, VE>(in + at2);
    }
    __device__ __forceinline__ void turn(const float2* cs) {
        float f[VE], g[VE];
        a.get(f);
        if constexpr (kPaired) {
            b.get(g);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float2 w = cs[j];
                const float x1 = f[j], x2 = g[j];
                f[j] = x1 * w.x - x2 * w.y;
                g[j] = x2 * w.x + x1 * w.y;
            }
            b.set(g);
        } else {
#pragma unroll
            for (int j = 0; j < VE; j += 2) {
                const float2 w = cs[j / 2];
                const float x1 = f[j], x2 = f[j + 1];
                f[j] = x1 * w.x - x2 * w.y;
                f[j + 1] = x2 * w.x + x1 * w.y;
            }
        }
        a.set(f);
    }
    __device__ __forceinline__ void store(E* out, int at, int at2, bool turned) const {
        rows::store<E, VE>(out + at, a);
        if (kPaired && turned) rows::store<E, VE>(out + at2, b);
    }
};

// `units` units a row, the first rot_units of them turned.
template <class E, int VE, bool IL>
__global__ void __maxnreg__(56) kda_rope(RopeParams p, int tokens, int rot_units, int units) {
    __shared__ float2 table[kMaxTable];
    constexpr int kAhead = 4;
    const int half = p.rot >> 1;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, p.T - t0);
    const int h0 = p.x[0].heads, items = (h0 + p.x[1].heads) * units;
    bool made = false;
    for (int item = threadIdx.x; item < items || !made; item += blockDim.x) {
        const bool live = item < items;
        int h = live ? item / units : 0;
        const int u = live ? item - h * units : 0;
        const RopeTensor& r = p.x[h >= h0];
        if (h >= h0) h -= h0;
        const bool turned = u < rot_units;
        const int at = Unit<E, VE, IL>::one(p, u, rot_units), at2 = Unit<E, VE, IL>::two(p, u);
        const int64_t in_st = r.in_st, out_st = r.out_st;
        const E* in = static_cast<const E*>(r.in) + t0 * in_st + (int64_t)h * r.in_sh;
        E* out = static_cast<E*>(r.out) + t0 * out_st + (int64_t)h * r.out_sh;
        const bool write = turned || in != out;
        Unit<E, VE, IL> x[kAhead];
        const int n = live ? nt : 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < n) x[i].load(in + i * in_st, at, at2, turned);
        if (!made) {
            for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
                const int t = i / half, j = i - t * half;
                const int64_t pos = p.pos64 ? static_cast<const int64_t*>(p.pos)[t0 + t]
                                            : (int64_t) static_cast<const int32_t*>(p.pos)[t0 + t];
                const double turns = p.inv_freq[j] * 0.15915494309189533577;  // 1 / 2 pi
                const long long F = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
                const unsigned long long phase = (unsigned long long)pos * (unsigned long long)F;
                const float a = (float)(int)(phase >> 32) * 4.656612873077392578125e-10f;  // 2^-31
                float s, c;
                sincospif(a, &s, &c);
                table[i] = make_float2(c * p.factor, s * p.factor * p.sign);
            }
            __syncthreads();
            made = true;
        }
        const float2* cs = table + (Unit<E, VE, IL>::kPaired ? u * VE : u * VE / 2);
        for (int t = 0; t < n; t += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (t + i < n) {
                    if (turned) x[i].turn(cs + i * half);
                    if (write) x[i].store(out + i * out_st, at, at2, turned);
                }
            cs += kAhead * half;
            in += kAhead * in_st;
            out += kAhead * out_st;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (t + kAhead + i < n) x[i].load(in + i * in_st, at, at2, turned);
        }
    }
}

template <class E, int VE, bool IL>
cudaError_t launch(const RopeParams& p, cudaStream_t s) {
    const int half = p.rot / 2;
    const int rot_units = IL && VE > 1 ? p.rot / VE : half / VE;
    const int units = rot_units + (p.D - p.rot) / VE;
    // tokens per CTA: eight, at most what the table holds, and few enough that each SM
    // has eight CTAs where there are so many tokens (16384 tokens, 12 + 12 heads: 34.8 us,
    // and 45.4 us with two a CTA; 512 tokens: 6.2 us with either)
    int tokens = max(1, min(8, kMaxTable / max(1, half)));
    tokens = (int)max((int64_t)1, min((int64_t)tokens, p.T / (8 * num_sms())));
    const int64_t grid = (p.T + tokens - 1) / tokens;
    // threads: as many as a token's units in the fewest rounds, in whole warps
    const int items = (p.x[0].heads + p.x[1].heads) * units;
    const int rounds = (items + kMaxThreads - 1) / kMaxThreads;
    const int threads = max(128, ((items + rounds - 1) / rounds + 31) / 32 * 32);
    kda_rope<E, VE, IL><<<(unsigned)grid, threads, 0, s>>>(p, tokens, rot_units, units);
    return cudaGetLastError();
}

template <class E>
cudaError_t dispatch(const RopeParams& p, cudaStream_t s) {
    constexpr int VE = 16 / sizeof(E);
    // 16-byte units when the dimensions, strides and bases allow them
    bool vec = (p.interleaved ? p.rot : p.rot / 2) % VE == 0 && (p.D - p.rot) % VE == 0;
    for (const RopeTensor& x : p.x)
        if (x.heads)
            vec = vec && ((reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out)) & 15) == 0 &&
                  (x.in_st | x.in_sh | x.out_st | x.out_sh) % VE == 0;
    if (p.interleaved) return vec ? launch<E, VE, true>(p, s) : launch<E, 1, true>(p, s);
    return vec ? launch<E, VE, false>(p, s) : launch<E, 1, false>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t s) {
    if (p.dtype == KDA_F32) return dispatch<float>(p, s);
    if (p.dtype == KDA_BF16) return dispatch<__nv_bfloat16>(p, s);
    return dispatch<__half>(p, s);
}

}  // namespace kda
