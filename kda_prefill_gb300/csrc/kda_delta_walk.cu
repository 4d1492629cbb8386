// The gated delta rule's walk over a sequence's chunks on the tensor cores (tcgen05,
// accumulators in tensor memory).  For a chunk of C = 64 tokens with incoming state S (V x K),
// with kda_delta_chunk's k, q, T and P T:
//
//     X = S [k q]^T                   128 x 128 x 128
//     R = beta (V - c X_k)            in registers
//     U = R T^T,  O = X_q + R (P T)^T 128 x 64 x 64
//     S' = e^{G_C} S + (w U) k        128 x 128 x 64
//
// All products have the value rows as their M: a thread keeps half a row of S in fp32
// registers, and everything it rounds, scales or stores belongs to that row.  Rows are
// independent of each other but for the keys, so nothing has to be summed across threads.
//
// One CTA walks one (sequence, head); two share an SM, and one's products run while the
// other's threads make operands.  Warps 0-7 make operands, two for each 32 rows, and write
// the outputs; warp 8 issues the copies and the products.
//
// Rounding.  Operands are fp16: k exactly, up to its row's power of two; S, R, U and T as
// the sum of two (22 bits; with one, a state would be off by 2^-12).  The outputs' own terms,
// q e^G and P T, have one: 11 bits, beside the 8 of out.  S, R and U of a row are scaled by
// one power of two, from a bound that holds for all three: with |v| <= m and beta <= b in the
// chunk, |R| <= b (m + |S|) and |U| <= b (m + |S| + 64 b m), since I - beta k k^T does not
// lengthen a row for beta in [0, 2] and a token adds at most b m; |S| itself is bounded by
// that of a chunk before and 64 b m of that chunk, so that no thread waits for another's
// maximum.  The bound is up to 2^10 too large; fp16's exponent has room for it: a term is kept to
// 2^-25 of 2^14, the bound.
//
// Infinities and NaN stay in their value row (in v or the state) or sequence and head (in k)
// from their token on: R's entries that are not finite become zero for the products and their
// rows get NaN afterwards, until a token clears the state.

#include "kda_device.cuh"
#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

using namespace dev;

constexpr int D = kD;
constexpr int C = kC;
constexpr int kThreads = 288;
constexpr int kMakers = 8;  // warps 0 .. 7

// Shared memory.
constexpr int kTileK = C * D * 2;
constexpr int kSmK = 0;                          // [2] k
constexpr int kSmQ = kSmK + 2 * kTileK;
constexpr int kSmT = kSmQ + kTileK;              // [2] T's parts, then P T
constexpr int kSmV = kSmT + 3 * C * C * 2;       // [2] v, rows of 128
constexpr int kSmScal = kSmV + 2 * kTileK;       // [2] scalars
constexpr int kSmVMax = kSmScal + 2 * kDeltaScalBytes;      // [2][128] largest |v| of a value row
constexpr int kSmSMax = kSmVMax + 2 * D * 4;     // [2][2][128] largest |S| of half a row
constexpr int kSmBad = kSmSMax + 4 * D * 4;      // [2][128] tokens whose R is not finite
constexpr int kSmBar = kSmBad + 2 * D * 4;
enum Bar {
    kFullK = 0,             // [2] k and scalars
    kFullV = kFullK + 2,    // [2]
    kFullQ = kFullV + 2,
    kFullT,
    kXDone,
    kUDone,
    kODone,
    kDDone,
    kSReady,
    kRReady,
    kUReady,
    kVMax,                  // [2]
    kEnd = kVMax + 2,
    kNumBars
};
constexpr int kSmMisc = kSmBar + kNumBars * 8;
constexpr int kSmemBytes = kSmMisc + 16;
static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs on an SM");
static_assert(kSmT % 1024 == 0 && kSmV % 1024 == 0 && kSmBar % 8 == 0, "alignment");

// Tensor memory columns.  Operands have, for 16 of their K, 8 columns of the high part and 8
// of the low one.  Half of S's operand, and then of dS, lies where a half's warps alone write.
constexpr uint32_t kTmCols = 256;
constexpr uint32_t kTmS = 0;      // S: keys 0-63, 64-127; R in its first half, U in its second
constexpr uint32_t kTmR = 0;
constexpr uint32_t kTmU = 64;
constexpr uint32_t kTmX = 128;    // X_k; then R T^T; then dS of keys 64-127
constexpr uint32_t kTmO = 192;
__host__ __device__ constexpr uint32_t ds_column(int half) { return half ? kTmX : 0; }

constexpr uint32_t kIdescKK = mma_idesc(0, 0, 0, 128, 64);  // B K-major
constexpr uint32_t kIdescKM = mma_idesc(0, 0, 1, 128, 64);  // B MN-major

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        asm volatile("" : "+r"(r[i]));  // read after the wait
        v[i] = __uint_as_float(r[i]);
    }
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Sixteen values as the sum of two fp16 each, as an operand's columns.
__device__ __forceinline__ void store_split(uint32_t a, const float* x) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2 hi = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        const float2 f = __half22float2(hi);
        r[i] = reinterpret_cast<const uint32_t&>(hi);
        r[8 + i] = pack_half2(x[2 * i] - f.x, x[2 * i + 1] - f.y);
    }
    tmem_st16(a, r);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// 2^(14 - e) for a bound below 2^e, and its inverse.
__device__ __forceinline__ float scale_of(float bound, float& inverse) {
    const int e = max(14, min(254, (int)(__float_as_uint(bound) >> 23)));
    inverse = __uint_as_float((uint32_t)(e - 13) << 23);
    return __uint_as_float((uint32_t)(267 - e) << 23);
}

struct Walk {
    uint8_t* smem;
    uint64_t* bar;
    volatile int* abort;
    uint32_t tmem;
    int n, h, slot, t0, len, chunks;
    const uint8_t* blocks;  // of the first chunk
    int64_t step;           // bytes between chunks' blocks
    bool init;

    // Waits for a phase; gives up after about a second, or once another warp has.  A whole
    // warp goes on or leaves together.
    __device__ bool wait(int b, uint32_t parity) const {
#pragma unroll 1
        for (uint32_t i = 0; i < kWaitLimit; ++i) {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar + b, parity & 1))) return true;
            if (__any_sync(0xffffffffu, *abort)) return false;
        }
        *abort = 1;
        return false;
    }
    // One arrival of a whole warp, its tensor-memory accesses before it.
    __device__ void arrive_warp(int b, int lane) const {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + b);
    }
    __device__ const DeltaScalars* scalars(int c) const {
        return reinterpret_cast<const DeltaScalars*>(smem + kSmScal + (c & 1) * kDeltaScalBytes);
    }
    __device__ float* vmax(int c) const { return reinterpret_cast<float*>(smem + kSmVMax) + (c & 1) * D; }
    __device__ volatile float* smax(int c, int half) const {
        return reinterpret_cast<volatile float*>(smem + kSmSMax) + ((c & 1) * 2 + half) * D;
    }
    __device__ volatile unsigned* bad(int half) const {
        return reinterpret_cast<volatile unsigned*>(smem + kSmBad) + half * D;
    }
};

// Warp 8: copies, products and the largest |v|.
struct Issuer {
    const Walk& w;
    const DeltaParams& p;
    const int lane;
    int k_loads = 0, v_loads = 0, q_loads = 0, t_loads = 0;

    __device__ const uint8_t* block(int c) const { return w.blocks + c * w.step; }
    __device__ void load_k(int c) {
        if (lane == 0) {
            uint64_t* b = w.bar + kFullK + (c & 1);
            mbar_arrive_expect_tx(b, kTileK + (uint32_t)sizeof(DeltaScalars));
            bulk_g2s(w.smem + kSmK + (c & 1) * kTileK, block(c) + kDeltaK, kTileK, b);
            bulk_g2s(w.smem + kSmScal + (c & 1) * kDeltaScalBytes, block(c) + kDeltaScal, sizeof(DeltaScalars), b);
        }
        ++k_loads;
    }
    __device__ void load_v(int c) {
        const int rows = min(C, w.len - c * C);
        uint64_t* b = w.bar + kFullV + (c & 1);
        if (lane == 0) mbar_arrive_expect_tx(b, rows * D * 2);
        __syncwarp();
        const __nv_bfloat16* v = p.v + (int64_t)(w.t0 + c * C) * p.v_st + (int64_t)w.h * p.v_sh;
        for (int r = lane; r < rows; r += 32)
            bulk_g2s(w.smem + kSmV + (c & 1) * kTileK + r * (D * 2), v + r * p.v_st, D * 2, b);
        ++v_loads;
    }
    __device__ void load_q(int c) {
        if (lane == 0) {
            mbar_arrive_expect_tx(w.bar + kFullQ, kTileK);
            bulk_g2s(w.smem + kSmQ, block(c) + kDeltaQ, kTileK, w.bar + kFullQ);
        }
        ++q_loads;
    }
    __device__ void load_t(int c) {
        if (lane == 0) {
            mbar_arrive_expect_tx(w.bar + kFullT, 3 * C * C * 2);
            bulk_g2s(w.smem + kSmT, block(c) + kDeltaT, 2 * C * C * 2, w.bar + kFullT);
            bulk_g2s(w.smem + kSmT + 2 * C * C * 2, block(c) + kDeltaPT, C * C * 2, w.bar + kFullT);
        }
        ++t_loads;
    }
    // The largest finite |v| of each value row of chunk c.
    __device__ bool largest_v(int c) {
        if (!w.wait(kFullV + (c & 1), c >> 1)) return false;
        const int rows = min(C, w.len - c * C);
        const uint2* v = reinterpret_cast<const uint2*>(w.smem + kSmV + (c & 1) * kTileK) + lane;
        __nv_bfloat162 a = __float2bfloat162_rn(0.f), b = a;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            const uint2 x = v[r * (D / 4)];
            a = __hmax2_nan(a, __habs2(reinterpret_cast<const __nv_bfloat162&>(x.x)));
            b = __hmax2_nan(b, __habs2(reinterpret_cast<const __nv_bfloat162&>(x.y)));
        }
        float4 m = make_float4(__low2float(a), __high2float(a), __low2float(b), __high2float(b));
        if (__any_sync(0xffffffffu, !(finite(m.x) && finite(m.y) && finite(m.z) && finite(m.w)))) {
            m = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < rows; ++r) {
                const uint2 x = v[r * (D / 4)];
                const float f[4] = {fabsf(__uint_as_float(x.x << 16)), fabsf(__uint_as_float(x.x & 0xFFFF0000u)),
                                    fabsf(__uint_as_float(x.y << 16)), fabsf(__uint_as_float(x.y & 0xFFFF0000u))};
                m.x = finite(f[0]) ? fmaxf(m.x, f[0]) : m.x;
                m.y = finite(f[1]) ? fmaxf(m.y, f[1]) : m.y;
                m.z = finite(f[2]) ? fmaxf(m.z, f[2]) : m.z;
                m.w = finite(f[3]) ? fmaxf(m.w, f[3]) : m.w;
            }
        }
        reinterpret_cast<float4*>(w.vmax(c))[lane] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(w.bar + kVMax + (c & 1));
        return true;
    }

    __device__ bool go() {
        const uint32_t tm = w.tmem;
        const uint32_t ks = smem_u32(w.smem + kSmK), qs = smem_u32(w.smem + kSmQ), ts = smem_u32(w.smem + kSmT);
        load_k(0);
        load_v(0);
        load_q(0);
        load_t(0);
        if (w.chunks > 1) {
            load_k(1);
            load_v(1);
        }
        if (!largest_v(0)) return false;
#pragma unroll 1
        for (int c = 0; c < w.chunks; ++c) {
            const uint32_t kt = ks + (c & 1) * kTileK;
            if (!w.wait(kFullK + (c & 1), c >> 1) || !w.wait(kFullQ, c) || !w.wait(kSReady, c)) return false;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        mma_f16_ts(tm + kTmX, tm + kTmS + 16 * s + 8 * part,
                                   sw128_desc(kt + (s >> 2) * (kTileK / 2) + (s & 3) * 32, 0, 1024), kIdescKK, s > 0 || part > 0);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_f16_ts(tm + kTmO, tm + kTmS + 16 * s,
                               sw128_desc(qs + (s >> 2) * (kTileK / 2) + (s & 3) * 32, 0, 1024), kIdescKK, s > 0);
                mma_commit(w.bar + kXDone);
            }
            __syncwarp();
            // the chunk before's k has been used
            if (c >= 1 && c + 1 < w.chunks) load_k(c + 1);
            if (c + 1 < w.chunks && !largest_v(c + 1)) return false;
            if (!w.wait(kFullT, c) || !w.wait(kRReady, c)) return false;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint64_t hi = sw128_desc(ts + s * 32, 0, 1024), lo = sw128_desc(ts + C * C * 2 + s * 32, 0, 1024);
                    mma_f16_ts(tm + kTmX, tm + kTmR + 16 * s, lo, kIdescKK, s > 0);
                    mma_f16_ts(tm + kTmX, tm + kTmR + 16 * s + 8, hi, kIdescKK, 1);
                    mma_f16_ts(tm + kTmX, tm + kTmR + 16 * s, hi, kIdescKK, 1);
                }
                mma_commit(w.bar + kUDone);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_f16_ts(tm + kTmO, tm + kTmR + 16 * s, sw128_desc(ts + 2 * C * C * 2 + s * 32, 0, 1024), kIdescKK, 1);
                mma_commit(w.bar + kODone);
            }
            __syncwarp();
            // the makers have read v, and X's products q
            if (c + 2 < w.chunks) load_v(c + 2);
            if (c + 1 < w.chunks) load_q(c + 1);
            if (!w.wait(kUReady, c)) return false;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint64_t b = sw128_desc(kt + half * (kTileK / 2) + s * 2048, 8192, 1024);
                        mma_f16_ts(tm + ds_column(half), tm + kTmU + 16 * s + 8, b, kIdescKM, s > 0);
                        mma_f16_ts(tm + ds_column(half), tm + kTmU + 16 * s, b, kIdescKM, 1);
                    }
                mma_commit(w.bar + kDDone);
            }
            __syncwarp();
            if (!w.wait(kODone, c)) return false;
            if (c + 1 < w.chunks) load_t(c + 1);
        }
        return true;
    }
    // Copies and products in flight end before the CTA does.
    __device__ void finish() {
        if (lane == 0) mma_commit(w.bar + kEnd);
        bool ok = mbar_wait(w.bar + kEnd, 0);
        for (int i = 0; i < 2; ++i) {
            // loads of slot i: chunks i, i + 2, ...
            const int nk = (k_loads + 1 - i) / 2, nv = (v_loads + 1 - i) / 2;
            if (nk > 0) ok = mbar_wait(w.bar + kFullK + i, (nk - 1) & 1) && ok;
            if (nv > 0) ok = mbar_wait(w.bar + kFullV + i, (nv - 1) & 1) && ok;
        }
        if (q_loads > 0) ok = mbar_wait(w.bar + kFullQ, (q_loads - 1) & 1) && ok;
        if (t_loads > 0) ok = mbar_wait(w.bar + kFullT, (t_loads - 1) & 1) && ok;
        if (!ok) *w.abort = 1;
    }
};

// Whether tokens up to i leave a row without a finite value: bit i of the result.  `bad` are
// the tokens that bring one in, `clears` those that clear the state.
__device__ __noinline__ uint2 poisoned(uint2 bad, uint2 clears) {
    uint2 r = make_uint2(0, 0);
    bool on = false;
    for (int i = 0; i < C; ++i) {
        const unsigned bit = 1u << (i & 31);
        if ((i < 32 ? clears.x : clears.y) & bit) on = false;
        if ((i < 32 ? bad.x : bad.y) & bit) on = true;
        if (on) (i < 32 ? r.x : r.y) |= bit;
    }
    return r;
}

// Warps 0-7: a thread has half of value row `row`: 64 keys, 32 of a chunk's tokens.
template <class S>
__device__ bool make(const Walk& w, const DeltaParams& p, int warp, int lane) {
    const int half = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t tm = w.tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    constexpr int N = 16 / sizeof(S);
    S* const state = static_cast<S*>(p.pool) + (w.slot >= 0 ? (size_t)w.slot * p.stride0 : 0) +
                     ((size_t)w.h * D + row) * D + half * 64;
    float s[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) s[i] = 0.f;
    if (w.init) {
#pragma unroll
        for (int i = 0; i < 64; i += N) {
            float f[N];
            rows::load<S, N>(state + i).get(f);
#pragma unroll
            for (int j = 0; j < N; ++j) s[i + j] = f[j];
        }
    }
    float smax = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) smax = max_nan(smax, fabsf(s[i]));
    w.smax(0, half)[row] = smax;
    asm volatile("bar.sync 1, %0;" ::"n"(kMakers * 32) : "memory");
    // the largest |S| a chunk ago; what the chunk adds to |S| at most
    float was = max_nan(smax, w.smax(0, half ^ 1)[row]), adds, scale, inv;
    if (!w.wait(kVMax, 0) || !w.wait(kFullK, 0)) return false;
    auto rescale = [&](int c, float grown) {
        const float s = 11.32f * (finite(was) ? was : 0.f) + grown;  // |S| <= sqrt(128) max
        const float b = w.scalars(c)->strongest, m = w.vmax(c)[row];
        adds = 64.f * b * m;
        // (v itself has to stay finite when it is scaled)
        scale = scale_of(fmaxf(fmaxf(s, b * (m + s + adds)), 0x1p-60f * m), inv);
    };
    rescale(0, 0.f);
    // S's operand; a row with infinities or NaN as zeros
    auto store_s = [&]() {
        const bool live = finite(smax);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = s[16 * b + i] * scale;
            if (!live) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = 0.f;
            }
            store_split(tm + kTmS + 64 * half + 16 * b, x);
        }
        tmem_wait_st();
    };
    store_s();
    w.arrive_warp(kSReady, lane);

    __nv_bfloat16* out = p.out + ((int64_t)w.t0 * p.H + w.h) * D + row;
#pragma unroll 1
    for (int c = 0; c < w.chunks; ++c) {
        const DeltaScalars* sc = w.scalars(c);
        const int live = min(C, w.len - c * C) - half * 32;  // of this half's tokens
        float x[32];
        // R
        if (!w.wait(kXDone, c) || !w.wait(kFullV + (c & 1), c >> 1)) return false;
        tc_fence_after();
        tmem_ld32(tm + kTmX + 32 * half, x);
        if (c > 0) {
            // both halves' largest of the state that the chunk starts from
            was = max_nan(smax, w.smax(c, half ^ 1)[row]);
        }
        const int clear = sc->first_clear;
        if (clear < C) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 32 * half + i < clear ? x[i] : 0.f;
        }
        const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(w.smem + kSmV + (c & 1) * kTileK) + half * 32 * D + row;
        float check = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 ci = *reinterpret_cast<const float4*>(sc->c + 32 * half + i);
            const float4 bi = *reinterpret_cast<const float4*>(sc->beta + 32 * half + i);
            const float cc[4] = {ci.x, ci.y, ci.z, ci.w}, bb[4] = {bi.x, bi.y, bi.z, bi.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float vv = i + u < live ? __bfloat162float(v[(i + u) * D]) * scale : 0.f;
                x[i + u] = bb[u] * fmaf(-cc[u], x[i + u], vv);
                check = fmaf(x[i + u], 0.f, check);
            }
        }
        unsigned bad = 0;
        const bool dead = !finite(was);
        if (__any_sync(0xffffffffu, check != 0.f || dead)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (!finite(x[i]) || (dead && 32 * half + i < clear)) {
                    bad |= 1u << i;
                    x[i] = 0.f;
                }
            }
        }
        w.bad(half)[row] = bad;
        store_split(tm + kTmR + 32 * half, x);
        store_split(tm + kTmR + 32 * half + 16, x + 16);
        tmem_wait_st();
        w.arrive_warp(kRReady, lane);
        // U
        if (!w.wait(kUDone, c)) return false;
        tc_fence_after();
        tmem_ld32(tm + kTmX + 32 * half, x);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 wi = *reinterpret_cast<const float4*>(sc->w + 32 * half + i);
            x[i] *= wi.x, x[i + 1] *= wi.y, x[i + 2] *= wi.z, x[i + 3] *= wi.w;
        }
        store_split(tm + kTmU + 32 * half, x);
        store_split(tm + kTmU + 32 * half + 16, x + 16);
        tmem_wait_st();
        w.arrive_warp(kUReady, lane);
        // outputs
        if (!w.wait(kODone, c)) return false;
        tc_fence_after();
        tmem_ld32(tm + kTmO + 32 * half, x);
        const unsigned other = w.bad(half ^ 1)[row];
        uint2 spoilt = make_uint2(0, 0);
        if (__any_sync(0xffffffffu, (bad | other) != 0)) {
            spoilt = poisoned(half ? make_uint2(other, bad) : make_uint2(bad, other), make_uint2(sc->clears[0], sc->clears[1]));
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if ((half ? spoilt.y : spoilt.x) >> i & 1) x[i] = NAN;
        }
        {
            const float f = inv * p.scale;
            __nv_bfloat16* o = out + (int64_t)(c * C + half * 32) * p.H * D;
            const int64_t st = (int64_t)p.H * D;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 di = *reinterpret_cast<const float4*>(sc->down + 32 * half + i);
                const float dd[4] = {di.x, di.y, di.z, di.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (i + u < live) *o = __float2bfloat16_rn(x[i + u] * dd[u] * f);
                    o += st;
                }
            }
        }
        // S
        const float gamma = sc->gamma, back = 2.f * inv;
        if (clear < C) {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = 0.f;
        }
        const bool more = c + 1 < w.chunks;
        if (more) {
            if (!w.wait(kVMax + ((c + 1) & 1), (c + 1) >> 1) || !w.wait(kFullK + ((c + 1) & 1), (c + 1) >> 1)) return false;
            rescale(c + 1, adds);
        }
        if (!w.wait(kDDone, c)) return false;
        tc_fence_after();
        smax = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            tmem_ld32(tm + ds_column(half) + 32 * b, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                s[32 * b + i] = fmaf(gamma, s[32 * b + i], x[i] * back);
                smax = max_nan(smax, fabsf(s[32 * b + i]));
            }
        }
        if (spoilt.y >> 31) {
            smax = NAN;
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = NAN;
        }
        if (more) {
            w.smax(c + 1, half)[row] = smax;
            store_s();
            w.arrive_warp(kSReady, lane);
        }
    }
    if (w.slot >= 0) {
#pragma unroll
        for (int i = 0; i < 64; i += N) {
            float f[N];
#pragma unroll
            for (int j = 0; j < N; ++j) f[j] = s[i + j];
            rows::Piece<S, N> x;
            x.set(f);
            rows::store<S, N>(state + i, x);
        }
    }
    return true;
}

template <class S>
__global__ void __launch_bounds__(kThreads, 2) kda_delta_walk(const __grid_constant__ DeltaParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Walk w;
    w.smem = smem;
    w.bar = reinterpret_cast<uint64_t*>(smem + kSmBar);
    w.abort = reinterpret_cast<volatile int*>(smem + kSmMisc);
    uint32_t* const base = reinterpret_cast<uint32_t*>(smem + kSmMisc + 8);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNumBars; ++i) mbar_init(w.bar + i, i >= kSReady && i <= kUReady ? kMakers : 1);
        *w.abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(base, kTmCols);
    w.h = blockIdx.x % p.H;
    w.n = p.long_list[blockIdx.x / p.H];
    w.t0 = p.cu[w.n];
    w.len = p.cu[w.n + 1] - w.t0;
    w.chunks = (w.len + C - 1) / C;
    w.step = (int64_t)p.H * kDeltaBlock;
    w.blocks = p.blocks + ((int64_t)p.seq_off[w.n] * p.H + w.h) * kDeltaBlock;
    const int slot = p.idx[w.n];
    w.slot = slot >= 0 && slot < p.num_slots ? slot : -1;
    w.init = w.slot >= 0 && p.has_init[w.n] != 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    w.tmem = *base;
    if (warp < kMakers) {
        make<S>(w, p, warp, lane);
        tc_fence_before();
        __syncthreads();
    } else {
        Issuer i{w, p, lane};
        i.go();
        i.finish();
        __syncthreads();
        __syncwarp();
        tc_fence_after();
        if (*w.abort && lane == 0) atomicOr(p.status, 1);
        tmem_dealloc(w.tmem, kTmCols);
    }
}

template <class S>
cudaError_t launch(const DeltaParams& p, cudaStream_t s) {
    static unsigned configured = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 32 || !(configured & (1u << dev))) {
        e = cudaFuncSetAttribute(kda_delta_walk<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 32) configured |= 1u << dev;
    }
    kda_delta_walk<S><<<(unsigned)(p.n_long * p.H), kThreads, kSmemBytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_walk(const DeltaParams& p, cudaStream_t s) {
    if (p.n_long <= 0) return cudaSuccess;
    if (p.st_dtype == KDA_STATE_F32) return launch<float>(p, s);
    if (p.st_dtype == KDA_STATE_BF16) return launch<__nv_bfloat16>(p, s);
    return launch<__half>(p, s);
}

}  // namespace kda
