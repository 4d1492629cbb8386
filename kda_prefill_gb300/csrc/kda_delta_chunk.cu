// The gated delta rule, each chunk of C = 64 tokens and head for itself: everything that does
// not need the state.  With G the prefix sums of the log decays, k^ and q^ of length one:
//
//     A_ij = beta_i e^{G_i - G_j} k^_i . k^_j  (j < i)      T = (1 + A)^-1
//     P_ij = e^{G_i - G_j} q^_i . k^_j  (j <= i)            P T
//
// so that for an incoming state S, with R = beta (V - e^G K^ S^T), the chunk's writes are
// U = T R and its outputs e^G Q^ S^T + (P T) R.
//
// A CTA takes a chunk and head.  Rows of k and q are scaled by powers of two, so that they
// are exact in fp16; their lengths are factors on sums.  The scores are products of 16-bit
// MMAs, exact but for the sums.  T is solved in fp32: the two 32 x 32 blocks on the diagonal
// column by column, a lane each (the block below them is T22 N21 T11, N = -A).  A power series of N
// would cancel: with equal keys its terms grow to 10^18.
//
// q e^G would leave fp16's range where a chunk's decays are strong, while P T, at most one,
// does not: rows of both are multiplied by a power of two, up to 2^15, that brings e^G near one.
//
// Decays are sums of the decays between two tokens, never differences of sums over the
// chunk, which lose the bits of weak decays behind strong ones.

#include "kda_device.cuh"
#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

using namespace dev;

constexpr int D = kD;
constexpr int C = kC;
constexpr int kThreads = 256;
constexpr int kLd = 68;  // floats of a row of the fp32 matrices

// Shared memory.
constexpr int kSmK = 0;                          // k, the block's tile
constexpr int kSmQ = kSmK + C * D * 2;           // q; then T in fp32
constexpr int kSmN = kSmQ + C * kLd * 4;         // transposed: e^{G_i - G_j}, then N; then T high
constexpr int kSmP = kSmN + C * kLd * 4;         // P; then P T
constexpr int kSmVec = kSmP + C * C * 2;         // a, ck, cq, beta, e^G up, up
constexpr int kSmemBytes = kSmVec + 6 * C * 4;
static_assert(C * kLd * 4 >= C * D * 2 && C * kLd * 4 >= 2 * C * C * 2 && kSmP % 1024 == 0 && kSmN % 1024 == 0, "room");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The fragments of rows r0 .. r0 + 15, columns c0 .. c0 + 15 of a swizzled tile of halves of
// R rows: an A operand, or two B operands of eight rows each (r0 .. r0 + 7: b[0], b[2]).
__device__ __forceinline__ void frag(uint32_t tile, int r0, int c0, int R, int lane, uint32_t (&a)[4]) {
    const int r = r0 + (lane & 15), c = c0 + (lane >> 4) * 8;
    ldsm_x4(tile + sw128_off(r, c, R), a[0], a[1], a[2], a[3]);
}

// One row's 32 values of this thread: scaled by a power of two so that the row's largest is
// in [1/2, 1), as fp16; the sum of their squares over the row.  Four threads have a row.
struct RowPart {
    uint4 h[4];
    float ssq, scale;  // of the row
    bool fine;         // no infinities or NaN in the row
};
__device__ __forceinline__ RowPart scaled_row(const __nv_bfloat16* row, int part, bool live) {
    rows::Piece<__nv_bfloat16, 8> p[4];
    float m = 0.f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i].v = live ? __ldg(reinterpret_cast<const uint4*>(row + (4 * i + part) * 8)) : make_uint4(0, 0, 0, 0);
    RowPart r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[8];
        p[i].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m = fmaxf(m, fabsf(f[j]));
            fine = fine && fabsf(f[j]) < INFINITY;
        }
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    int bad = !fine;
    bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
    bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
    r.fine = bad == 0;
    // 2^-e with 2^(e-1) <= m < 2^e; values of the smallest exponents stay below 1/2
    const int e = (int)(__float_as_uint(m) >> 23) - 126;
    r.scale = __uint_as_float((uint32_t)(127 - max(-126, min(e, 126))) << 23);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[8];
        p[i].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] *= r.scale;
            s = fmaf(f[j], f[j], s);
        }
        rows::Piece<__half, 8> h;
        h.set(f);
        r.h[i] = h.v;
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    r.ssq = s;
    return r;
}
// What a scaled row is multiplied by to have length one.
__device__ __forceinline__ float unit(const RowPart& r) {
    return 1.f / sqrtf(fmaf(1e-6f * r.scale, r.scale, r.ssq));
}

__global__ void __launch_bounds__(kThreads, 3) kda_delta_chunk(const __grid_constant__ DeltaParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    float* const q32 = reinterpret_cast<float*>(smem + kSmQ);  // T
    float* const n32 = reinterpret_cast<float*>(smem + kSmN);
    float* const va = reinterpret_cast<float*>(smem + kSmVec);
    float *const vck = va + C, *const vcq = vck + C, *const vb = vcq + C, *const veg = vb + C, *const vup = veg + C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t chunk = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H;
    if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && warp == 0) write_status(p, lane);
    const int n = p.chunk_seq[chunk], t0 = p.chunk_tok[chunk];
    const int len = min(C, p.cu[n + 1] - t0);
    uint8_t* const blk = p.blocks + (chunk * p.H + h) * (int64_t)kDeltaBlock;
    DeltaScalars* const scal = reinterpret_cast<DeltaScalars*>(blk);

    // k and q
    {
        const int r = tid >> 2, part = tid & 3;
        const bool live = r < len;
        const int64_t t = t0 + r;
        const RowPart k = scaled_row(p.k + t * p.k_st + (int64_t)(h / p.rep) * p.k_sh, part, live);
        const RowPart q = scaled_row(p.q + t * p.q_st + (int64_t)(h / p.rep) * p.q_sh, part, live);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t at = sw128_off(r, (4 * i + part) * 8, C);
            // (a row with infinities or NaN counts as zero, but for its own factor c)
            const uint4 kv = k.fine ? k.h[i] : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(smem + kSmK + at) = kv;
            *reinterpret_cast<uint4*>(blk + kDeltaK + at) = kv;
            *reinterpret_cast<uint4*>(smem + kSmQ + at) = q.h[i];
        }
        if (part == 0) {
            vck[r] = k.fine ? unit(k) : NAN;
            vcq[r] = unit(q);
        }
    }
    if (tid < C) {
        const bool live = tid < len;
        const int64_t t = t0 + tid;
        va[tid] = live ? p.g[t * p.g_st + h] : 0.f;
        vb[tid] = live ? p.beta[t * p.H + h] : 0.f;
    }
    __syncthreads();
    // scalars: G from the chunk's start and to its end
    if (tid < C) {
        const float b = vb[tid], ck = vck[tid];
        float g = 0.f, rest = 0.f;
#pragma unroll 8
        for (int m = 0; m < C; ++m) {
            const float a = va[m];
            g += m <= tid ? a : 0.f;
            rest += m > tid ? a : 0.f;
        }
        const float eg = g > -0.5f ? 1.f + expm1f(g) : expf(g);
        const bool clears = va[tid] < kMinDecay;
        const unsigned mask = __ballot_sync(0xffffffffu, clears);
        scal->c[tid] = eg * ck;
        scal->beta[tid] = b;
        scal->w[tid] = 0.5f * expf(rest) * (ck == ck ? ck : 0.f);
        // up: 2^-e with 2^e <= e^G < 2^(e+1), at most 2^15
        const int e = min(15, max(0, 127 - (int)(__float_as_uint(eg) >> 23)));
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        scal->down[tid] = __uint_as_float((uint32_t)(127 - e) << 23);
        veg[tid] = eg * up;
        vup[tid] = up;
        if (tid == C - 1) scal->gamma = eg;
        float most = b;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
        if (lane == 0) {
            scal->clears[warp] = mask;
            reinterpret_cast<volatile unsigned*>(smem + kSmP)[warp] = mask;
            reinterpret_cast<volatile float*>(smem + kSmP)[2 + warp] = most;
        }
    }
    // e^{G_i - G_j}, transposed: row j, column i
    {
        constexpr float kLog2e = 1.4426950408889634f;
        const int j = tid & (C - 1), i0 = (tid >> 6) * 16;
        float sum = 0.f;
        for (int m = 0; m < i0; ++m) {
            const float a = va[m];
            sum += m > j && a == a ? a : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int ii = i0 + i + u;
                const float a = va[ii];
                sum += ii > j && a == a ? a : 0.f;
                x[u] = ii >= j ? ex2(sum * kLog2e) : 0.f;
            }
            *reinterpret_cast<float4*>(n32 + j * kLd + i0 + i) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
    __syncthreads();
    if (tid == 0) {
        const unsigned lo = reinterpret_cast<volatile unsigned*>(smem + kSmP)[0];
        const unsigned hi = reinterpret_cast<volatile unsigned*>(smem + kSmP)[1];
        scal->strongest = fmaxf(reinterpret_cast<volatile float*>(smem + kSmP)[2], reinterpret_cast<volatile float*>(smem + kSmP)[3]);
        scal->first_clear = lo ? __ffs(lo) - 1 : hi ? 31 + __ffs(hi) : C;
    }
    // q^ e^G
    {
        const int r = tid >> 2, part = tid & 3;
        const float f = vcq[r] * veg[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t at = sw128_off(r, (4 * i + part) * 8, C);
            rows::Piece<__half, 8> x;
            x.v = *reinterpret_cast<const uint4*>(smem + kSmQ + at);
            float y[8];
            x.get(y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= f;
            x.set(y);
            *reinterpret_cast<uint4*>(blk + kDeltaQ + at) = x.v;
        }
    }
    // scores: 16 rows x 32 columns a warp
    const int r0 = (warp & 3) * 16, c0 = (warp >> 2) * 32;
    const bool below = c0 < r0 + 16;  // some column is not above the diagonal
    {
        float kk[4][4] = {}, qk[4][4] = {};
        if (below) {
            const uint32_t kt = smem_u32(smem + kSmK), qt = smem_u32(smem + kSmQ);
#pragma unroll
            for (int ks = 0; ks < D; ks += 16) {
                uint32_t a[4], q[4], b[2][4];
                frag(kt, r0, ks, C, lane, a);
                frag(qt, r0, ks, C, lane, q);
                frag(kt, c0, ks, C, lane, b[0]);
                frag(kt, c0 + 16, ks, C, lane, b[1]);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    mma_f16(kk[t], a, b[t >> 1][t & 1], b[t >> 1][2 + (t & 1)]);
                    mma_f16(qk[t], q, b[t >> 1][t & 1], b[t >> 1][2 + (t & 1)]);
                }
            }
        }
        __syncthreads();  // these words are read
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = r0 + half * 8 + (lane >> 2), j = c0 + t * 8 + (lane & 3) * 2;
                float pv[2];
                const float b = vb[i], ci = vck[i], cq = vcq[i];
                const float bi = b == b && ci == ci ? b * ci : 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float cj = vck[j + u];
                    const float l = n32[(j + u) * kLd + i] * (cj == cj ? cj : 0.f);
                    n32[(j + u) * kLd + i] = j + u < i ? -bi * l * kk[t][2 * half + u] : 0.f;
                    pv[u] = j + u <= i ? cq * l * qk[t][2 * half + u] : 0.f;
                }
                *reinterpret_cast<uint32_t*>(smem + kSmP + sw64_off(i, j)) = pack_half2(pv[0], pv[1]);
            }
    }
    __syncthreads();
    // the diagonal blocks of T: lane j has column j; once row m is known its multiples go to
    // the rows below
    if (warp < 2) {
        const int o = warp * 32;
        float t[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) t[i] = i == lane ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 31; ++m) {
#pragma unroll
            for (int i = (m + 1) & ~3; i < 32; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(n32 + (o + m) * kLd + o + i);
                if (i > m) t[i] = fmaf(x.x, t[m], t[i]);
                if (i + 1 > m) t[i + 1] = fmaf(x.y, t[m], t[i + 1]);
                if (i + 2 > m) t[i + 2] = fmaf(x.z, t[m], t[i + 2]);
                if (i + 3 > m) t[i + 3] = fmaf(x.w, t[m], t[i + 3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) q32[(o + i) * kLd + o + lane] = t[i];
    } else if (warp < 4) {  // above the diagonal
        for (int i = warp - 2; i < 32; i += 2) q32[i * kLd + 32 + lane] = 0.f;
    }
    __syncthreads();
    // Y = N21 T11, four rows a warp, into N's place above the diagonal (row 32 + j, column r)
    float* const y32 = n32 + 32 * kLd;
    {
        float y[4] = {};
#pragma unroll 8
        for (int m = 0; m < 32; ++m) {
            const float4 x = *reinterpret_cast<const float4*>(n32 + m * kLd + 32 + 4 * warp);
            const float t = q32[m * kLd + lane];
            y[0] = fmaf(x.x, t, y[0]), y[1] = fmaf(x.y, t, y[1]);
            y[2] = fmaf(x.z, t, y[2]), y[3] = fmaf(x.w, t, y[3]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) y32[(4 * warp + u) * kLd + lane] = y[u];
    }
    __syncthreads();
    {  // T21 = T22 Y
        float y[4] = {};
#pragma unroll
        for (int m = 0; m < 32; m += 4) {
            float4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const float4*>(q32 + (32 + 4 * warp + u) * kLd + 32 + m);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float t = y32[(m + v) * kLd + lane];
#pragma unroll
                for (int u = 0; u < 4; ++u) y[u] = fmaf(v == 0 ? x[u].x : v == 1 ? x[u].y : v == 2 ? x[u].z : x[u].w, t, y[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) q32[(32 + 4 * warp + u) * kLd + lane] = y[u];
    }
    __syncthreads();
    // T as the sum of two fp16
    {
        const int r = tid >> 2, part = tid & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = (4 * i + part) * 8;
            float f[8], lo[8];
            const float4 a = *reinterpret_cast<const float4*>(q32 + r * kLd + c);
            const float4 b = *reinterpret_cast<const float4*>(q32 + r * kLd + c + 4);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
            rows::Piece<__half, 8> hi, rest;
            hi.set(f);
            hi.get(lo);
#pragma unroll
            for (int j = 0; j < 8; ++j) lo[j] = f[j] - lo[j];
            rest.set(lo);
            const uint32_t at = sw64_off(r, c);
            *reinterpret_cast<uint4*>(smem + kSmN + at) = hi.v;
            *reinterpret_cast<uint4*>(blk + kDeltaT + at) = hi.v;
            *reinterpret_cast<uint4*>(blk + kDeltaT + C * C * 2 + at) = rest.v;
        }
    }
    __syncthreads();
    // P T
    {
        float d[4][4] = {};
        if (below) {
            const uint32_t pt = smem_u32(smem + kSmP), tt = smem_u32(smem + kSmN);
#pragma unroll
            for (int ks = 0; ks < C; ks += 16) {
                if (ks < r0 + 16 && ks + 16 > c0) {
                    uint32_t a[4], b[4];
                    frag(pt, r0, ks, C, lane, a);
#pragma unroll
                    for (int t = 0; t < 4; t += 2) {
                        // rows ks .. ks + 15 of T, columns c0 + 8 t .. + 15, transposed
                        const int r = ks + (lane & 15), c = c0 + 8 * t + (lane >> 4) * 8;
                        ldsm_x4_t(tt + sw64_off(r, c), b[0], b[1], b[2], b[3]);
                        mma_f16(d[t], a, b[0], b[1]);
                        mma_f16(d[t + 1], a, b[2], b[3]);
                    }
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = r0 + half * 8 + (lane >> 2), j = c0 + t * 8 + (lane & 3) * 2;
                *reinterpret_cast<uint32_t*>(smem + kSmP + sw64_off(i, j)) = pack_half2(vup[i] * d[t][2 * half], vup[i] * d[t][2 * half + 1]);
            }
    }
    __syncthreads();
#pragma unroll
    for (int i = tid; i < C * C * 2 / 16; i += kThreads)
        reinterpret_cast<uint4*>(blk + kDeltaPT)[i] = reinterpret_cast<const uint4*>(smem + kSmP)[i];
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaParams& p, cudaStream_t s) {
    if (p.n_chunks <= 0) return cudaSuccess;
    static unsigned configured = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 32 || !(configured & (1u << dev))) {
        e = cudaFuncSetAttribute(kda_delta_chunk, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 32) configured |= 1u << dev;
    }
    kda_delta_chunk<<<(unsigned)(p.n_chunks * p.H), kThreads, kSmemBytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
