// The gated delta rule, each chunk of C = 64 tokens and head for itself: everything that does
// not need the state.  With G the prefix sums of the log decays, k^ and q^ of length one:
//
//     A_ij = beta_i e^{G_i - G_j} k^_i . k^_j  (j < i)      T = (1 + A)^-1
//     P_ij = e^{G_i - G_j} q^_i . k^_j  (j <= i)
//
// so that for an incoming state S, with R = beta (V - e^G K^ S^T), the chunk's writes are
// U = T R and its outputs e^G Q^ S^T + P U.
//
// A CTA takes a chunk and head.  The scores are products of k and q as they come, exact but
// for the sums; their lengths are factors on them.  For the walk rows of k and q are scaled by powers
// of two: a bf16 value is exact in fp16 down to 2^-17 of its row's length, smaller ones are off
// by at most 2^-24 of it.  T is solved in the four 16 x 16 blocks on the diagonal in fp32,
// column by column, a lane each, then in blocks twice as large from the two on their diagonal,
// the one below being T22 N21 T11, N = -A: 16-bit MMAs of operands that are sums of two fp16 (22
// bits, as T's in the end).  A power series of N would cancel: with equal keys its terms
// grow to 10^18.
//
// Writing 59 KB a chunk (3.0 to 3.5 TB/s; 67 KB took 12 to 18 % longer), the shared-memory port (61 %
// of the cycles) and instructions are the bound: 16384 tokens of 12 heads take 60 us, 128 sequences
// of 117,555 tokens 388 us, 4.7 and 4.1 TB/s with what is read.  So all accesses are of whole lines, addresses of fragments come
// from a lane's own few, and T's blocks are products of MMAs (in fp32 they took 7.6 K cycles of
// that port); four CTAs an SM fill each other's waits.  With k and q left to the walk, to make
// the tiles itself, this kernel took 59 us instead of 69 then, but the walk 176 instead of 140.
//
// An output's two terms may cancel (a large value overwritten by a small one), so neither is rounded to
// 11 bits: q^ e^G is m 2^x q with 1 <= m < 2, and the row of q takes 2^x alone, P's row 1 / m and
// the output m; P is the sum of two fp16.  q^ e^G would leave fp16's range where a chunk's decays are
// strong, while P, at most one, does not: rows of both are multiplied by a power of two, up to
// 2^15, that brings e^G near one.  The quarters of T and P above the diagonal are not read: P's low
// part stands in them, so that the block is no larger for it (with 8 KB more this kernel took 72 us
// instead of 61, the last walk 76 instead of 70).
//
// Decays are sums of the decays between two tokens, never differences of sums over the
// chunk, which lose the bits of weak decays behind strong ones.  In the 16 x 16 blocks on the
// diagonal each sum is made; left of them e^{G_i - G_j} is e^{G_i - G_b} e^{G_b - G_j}, b the
// last token of column j's block: both factors are at most one, the first is one a row and
// block and the second one a token.

#include "kda_device.cuh"
#include "kda_f32x2.cuh"
#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

using namespace dev;

constexpr int D = kD;
constexpr int C = kC;
constexpr int B = 16;  // tokens of a block
constexpr int kThreads = 256;
constexpr int kLdE = 20; // floats of a row of the fp32 blocks on the diagonal

// Shared memory.
constexpr int kTile = C * C * 2;
constexpr int kSmK = 0;                   // k; then N below the diagonal blocks, high and low part; above them Y
constexpr int kSmQ = kSmK + C * D * 2;    // q; then T, high and low part
constexpr int kSmP = kSmQ + C * D * 2;    // P's high part
constexpr int kSmE = kSmP + kTile;        // blocks on the diagonal, transposed: e^{G_i - G_j}; then N
constexpr int kSmVec = kSmE + (C * kLdE + 4 * C / B) * 4;
struct Vecs {
    float a[C];       // decays in log2
    float ck[C];      // what makes k's length one (0 if k is not finite)
    float ks[C];      // the same for the scaled k (NaN)
    float rk[C];      // that and e^{G_b - G_j}
    float cq[C];      // what makes q's length one (NaN if q is not finite); then P's rows' factor
    float bk[C];      // beta ck
    float two[C];     // q's rows' power of two
    float f[3][C];    // e^{G_i - G_b} of the blocks before token i's
    float total[4];   // decays over a block
    unsigned clears[2];
    float strongest[2];
};
constexpr int kSmemBytes = kSmVec + (int)sizeof(Vecs);
static_assert(4 * (kSmemBytes + 1024) <= 233472, "four CTAs on an SM");
static_assert(2 * kTile <= C * D * 2 && kSmP % 1024 == 0 && kSmVec % 16 == 0, "room");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float zero_if_nan(float x) { return x == x ? x : 0.f; }
__device__ __forceinline__ uint32_t half2_of(f2 x) {
    const float2 f = unpack2(x);
    return pack_half2(f.x, f.y);
}
// D += A (16x16, row) * B (16x8, col), bf16 inputs, fp32 accumulation.
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A lane's places in 16 rows of a swizzled tile: its row's bytes, and its 16 bytes for each 16
// of 64 columns.
struct Lanes {
    uint32_t row, x[4];
    __device__ __forceinline__ explicit Lanes(int lane) : row((lane & 15) * 128) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ((2 * i + (lane >> 4)) ^ (lane & 7)) << 4;
    }
    // Rows r0 .. r0 + 15 (r0 a multiple of 8), columns c0 .. c0 + 15 (of 16) of a tile.
    __device__ __forceinline__ uint32_t at(uint32_t tile, int r0, int c0) const {
        return tile + r0 * 128 + (c0 >> 6) * kTile + row + x[c0 >> 4 & 3];
    }
    // Its fragments: an A operand, or two B operands of eight rows each (the first: a[0], a[2]).
    __device__ __forceinline__ void load(uint32_t tile, int r0, int c0, uint32_t (&a)[4]) const {
        ldsm_x4(at(tile, r0, c0), a[0], a[1], a[2], a[3]);
    }
};

// Row j of the fp32 blocks: two blocks' same rows in different banks.
__device__ __forceinline__ int e_at(int j) { return j * kLdE + j / B * 4; }

// Eight threads have two rows, four apart: of each two pieces of eight values, v[2 row + half].
// (With four threads a row every access is of half lines.)
__device__ __forceinline__ void fetch(uint4 (&v)[4], const __nv_bfloat16* from, int64_t st, int64_t rows) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = 4 * (i >> 1) < rows ? __ldg(reinterpret_cast<const uint4*>(from + 4 * (i >> 1) * st + 64 * (i & 1))) : make_uint4(0, 0, 0, 0);
}
// A row's sum of squares: the first one's in even lanes, the second one's in odd ones.
__device__ __forceinline__ float squares(const uint4 (&v)[4], int lane) {
    float sum[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        f2 s = 0;
#pragma unroll
        for (int i = 2 * r; i < 2 * r + 2; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) s = fma2(bf16x2(w[j]), bf16x2(w[j]), s);
        }
        const float2 t = unpack2(s);
        sum[r] = t.x + t.y;
    }
    const bool odd = lane & 1;
    float x = (odd ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, odd ? sum[0] : sum[1], 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    return x + __shfl_xor_sync(0xffffffffu, x, 4);
}
// e with |k| <= 2^e < 2 |k| or so, from k's square.
__device__ __forceinline__ int length_of(float kk) { return ((int)(__float_as_uint(kk) >> 23) - 127 + 2) >> 1; }
// Eight values times f, as fp16.
__device__ __forceinline__ uint4 times(uint4 v, float f) {
    const f2 ff = pack2(f, f);
    return make_uint4(half2_of(mul2(bf16x2(v.x), ff)), half2_of(mul2(bf16x2(v.y), ff)), half2_of(mul2(bf16x2(v.z), ff)),
                      half2_of(mul2(bf16x2(v.w), ff)));
}

// Two values as the sum of two fp16 each.
__device__ __forceinline__ void put_split(uint8_t* at, uint8_t* lo, f2 x) {
    const uint32_t hi = half2_of(x);
    const float2 f = __half22float2(reinterpret_cast<const __half2&>(hi));
    *reinterpret_cast<uint32_t*>(at) = hi;
    *reinterpret_cast<uint32_t*>(lo) = half2_of(fma2(pack2(f.x, f.y), pack2(-1.f, -1.f), x));
}
__device__ __forceinline__ void put_split(uint8_t* at, f2 x) { put_split(at, at + kTile, x); }
// 16 rows from r0 and 8 columns from n0 of a b, over K from a's column ca and b's row rb on, all
// of them sums of two fp16; into the tile `to` at row r1, column n1.
template <int K>
__device__ __forceinline__ void block_product(const Lanes& ln, uint8_t* a, int r0, int ca, uint8_t* b, int rb, int n0, uint8_t* to,
                                              int r1, int n1, int lane) {
    float d[4] = {};
    const uint32_t at = smem_u32(a);
    const uint32_t bt = smem_u32(b) + (lane >> 4) * kTile + rb * 128 + ln.row + (((n0 >> 3) ^ (lane & 7)) << 4);
#pragma unroll
    for (int ks = 0; ks < K; ks += 16) {
        uint32_t hi[4], lo[4], x[4];  // x: b's high part, then its low one
        ln.load(at, r0, ca + ks, hi);
        ln.load(at + kTile, r0, ca + ks, lo);
        ldsm_x4_t(bt + ks * 128, x[0], x[1], x[2], x[3]);
        mma_f16(d, lo, x[0], x[1]);
        mma_f16(d, hi, x[2], x[3]);
        mma_f16(d, hi, x[0], x[1]);
    }
    const int r = lane >> 2;
    uint8_t* const y = to + (r1 + r) * 128 + (((n1 >> 3) ^ r) << 4) + (lane & 3) * 4;
    put_split(y, pack2(d[0], d[1]));
    put_split(y + 8 * 128, pack2(d[2], d[3]));
}

__global__ void __launch_bounds__(kThreads, 4) kda_delta_chunk(const __grid_constant__ DeltaParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    float* const e32 = reinterpret_cast<float*>(smem + kSmE);
    uint8_t *const tt = smem + kSmQ, *const nt = smem + kSmK;
    Vecs& vec = *reinterpret_cast<Vecs*>(smem + kSmVec);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Lanes ln(lane);
    const int64_t chunk = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H;
    if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && warp == 0) write_status(p, lane);
    const int n = p.chunk_seq[chunk], t0 = p.chunk_tok[chunk];
    const int len = min(C, p.cu[n + 1] - t0);
    uint8_t* const blk = p.blocks + (chunk * p.H + h) * (int64_t)kDeltaBlock;
    DeltaScalars* const scal = reinterpret_cast<DeltaScalars*>(blk);
    const int r = warp * 8 + (lane >> 3), col = (lane & 7) * 8;  // of this thread's first piece

    uint4 q[4];
    float g = 0.f, beta = 0.f;
    {
        const int64_t t = t0 + r;
        uint4 k[4];
        // (rows past the sequence's end are another's: cleared once its end is there)
        fetch(k, p.k + t * p.k_st + (int64_t)(h / p.rep) * p.k_sh + col, p.k_st, p.T - t);
        fetch(q, p.q + t * p.q_st + (int64_t)(h / p.rep) * p.q_sh + col, p.q_st, p.T - t);
        if (tid < C && t0 + tid < p.T) {
            g = p.g[(int64_t)(t0 + tid) * p.g_st + h];
            beta = p.beta[(int64_t)(t0 + tid) * p.H + h];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r + 4 * (i >> 1) >= len) k[i] = q[i] = make_uint4(0, 0, 0, 0);
        if (tid >= len) g = beta = 0.f;
        const float mine = squares(k, lane), other = __shfl_xor_sync(0xffffffffu, mine, 1);
        const float kk[2] = {lane & 1 ? other : mine, lane & 1 ? mine : other};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (a row with infinities or NaN counts as zero, but for its own factor c; values of
            // the smallest exponents stay smaller)
            const float x = kk[i >> 1], down = __uint_as_float((uint32_t)(127 - length_of(x)) << 23);
            if (!(x < INFINITY)) k[i] = make_uint4(0, 0, 0, 0);
            const uint32_t at = sw128_off(r + 4 * (i >> 1), col + 64 * (i & 1), C);
            *reinterpret_cast<uint4*>(smem + kSmK + at) = k[i];
            *reinterpret_cast<uint4*>(blk + kDeltaK + at) = x < INFINITY ? times(k[i], down) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(smem + kSmQ + at) = q[i];
        }
        const float qq = squares(q, lane);
        if (col < 16) {
            const int row = r + 4 * (lane & 1);
            const bool fine = mine < INFINITY;
            const float one = 1.f / sqrtf(mine + 1e-6f);
            vec.ck[row] = fine ? one : 0.f;
            vec.ks[row] = fine ? one * __uint_as_float((uint32_t)(127 + length_of(mine)) << 23) : NAN;
            vec.cq[row] = qq < INFINITY ? 1.f / sqrtf(qq + 1e-6f) : NAN;
        }
    }
    // sums of decays within the block, up to the token and behind it
    float pre = 0.f, suf = 0.f;
    if (tid < C) {
        const int at = lane & 15;
        pre = g, suf = g;
#pragma unroll
        for (int d = 1; d < B; d <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, pre, d), y = __shfl_down_sync(0xffffffffu, suf, d);
            if (at >= d) pre += x;
            if (at + d < B) suf += y;
        }
        suf = __shfl_down_sync(0xffffffffu, suf, 1);
        if (at == B - 1) {
            suf = 0.f;
            vec.total[tid / B] = pre;
        }
        vec.a[tid] = zero_if_nan(g) * 1.4426950408889634f;
        const unsigned mask = __ballot_sync(0xffffffffu, g < kMinDecay);
        float most = beta;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
        if (lane == 0) vec.clears[warp] = mask, vec.strongest[warp] = most;
    }
    __syncthreads();
    // e^{G_i - G_j} on the diagonal: row j, column i - its block's first
    if (tid >= C && tid < 2 * C) {
        const int j = tid - C, o = j & ~(B - 1);
        float sum = 0.f;
#pragma unroll
        for (int i0 = 0; i0 < B; i0 += 4) {
            const float4 a = *reinterpret_cast<const float4*>(vec.a + o + i0);
            const float aa[4] = {a.x, a.y, a.z, a.w};
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u;
                sum += o + i > j ? aa[u] : 0.f;
                x[u] = o + i >= j ? ex2(sum) : 0.f;
            }
            *reinterpret_cast<float4*>(e32 + e_at(j) + i0) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
    if (tid < C) {
        constexpr float kLog2e = 1.4426950408889634f;
        const int blk_i = tid / B;
        const float ck = vec.ck[tid], ks = vec.ks[tid];
        // decays from each block's end up to the token, from the chunk's start, to its end
        float upto = pre, rest = suf;
#pragma unroll
        for (int b = 2; b >= 0; --b) {
            if (b < blk_i) {
                vec.f[b][tid] = zero_if_nan(ex2(upto * kLog2e));
                upto += vec.total[b];
            }
        }
#pragma unroll
        for (int b = 1; b < 4; ++b)
            if (b > blk_i) rest += vec.total[b];
        const float eg = upto > -0.5f ? 1.f + expm1f(upto) : expf(upto);
        // up: 2^-e with 2^e <= e^G < 2^(e+1), at most 2^15
        const int e = min(15, max(0, 127 - (int)(__float_as_uint(eg) >> 23)));
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        scal->c[tid] = eg * ks;
        scal->beta[tid] = beta;
        scal->w[tid] = 0.5f * expf(rest) * zero_if_nan(ks);
        // q^ e^G up = m 2^x q, 1 <= m < 2: the row of q takes 2^x, those of P and the output take 1 / m and m
        const uint32_t f = __float_as_uint(vec.cq[tid] * (eg * up));
        const float m = f < 0x7F800000u ? __uint_as_float((f & 0x007FFFFFu) | 0x3F800000u) : NAN;
        scal->down[tid] = m * __uint_as_float((uint32_t)(127 - e) << 23);
        vec.rk[tid] = zero_if_nan(ex2(suf * kLog2e)) * ck;
        vec.bk[tid] = -zero_if_nan(beta * ck);
        vec.two[tid] = __uint_as_float(f & 0x7F800000u);
        vec.cq[tid] = vec.cq[tid] * up / m;
        if (tid == C - 1) {
            scal->gamma = eg;
            const unsigned lo = vec.clears[0], hi = vec.clears[1];
            scal->first_clear = lo ? __ffs(lo) - 1 : hi ? 31 + __ffs(hi) : C;
            scal->clears[0] = lo, scal->clears[1] = hi;
            scal->strongest = fmaxf(vec.strongest[0], vec.strongest[1]);
        }
    }
    __syncthreads();
    // q
    {
        const float f[2] = {vec.two[r], vec.two[r + 4]};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(blk + kDeltaQ + sw128_off(r + 4 * (i >> 1), col + 64 * (i & 1), C)) = times(q[i], f[i >> 1]);
    }
    // scores: 16 rows x 32 columns a warp
    const int bi = warp & 3, r0 = bi * B, c0 = (warp >> 2) * 32;
    const bool below = c0 < r0 + B;  // some column is not above the diagonal
    {
        float kk[4][4] = {}, qk[4][4] = {};
        if (below) {
            const uint32_t kt = smem_u32(smem + kSmK), qt = smem_u32(smem + kSmQ);
#pragma unroll
            for (int ks = 0; ks < D; ks += 16) {
                uint32_t a[4], qa[4], b[4];
                ln.load(kt, r0, ks, a);
                ln.load(qt, r0, ks, qa);
#pragma unroll
                for (int t = 0; t < 4; t += 2) {
                    if (c0 + 8 * t > r0) continue;
                    ln.load(kt, c0 + 8 * t, ks, b);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        mma_bf16(kk[t + u], a, b[u], b[2 + u]);
                        mma_bf16(qk[t + u], qa, b[u], b[2 + u]);
                    }
                }
            }
        }
        // e^{G_i - G_j} of the block on the diagonal, before N takes its place
        const int ri = lane >> 2, cj = (lane & 3) * 2;
        float e[2][2][2] = {};  // [columns][rows][column]
        if (below && r0 - c0 < 32) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int u = 0; u < 2; ++u) e[t][half][u] = e32[e_at(r0 + 8 * t + cj + u) + 8 * half + ri];
        }
        __syncthreads();
        uint32_t y[4];  // in a row of a tile
#pragma unroll
        for (int t = 0; t < 4; ++t) y[t] = (((c0 >> 3) + t) ^ ri) << 4 | cj * 2;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = r0 + half * 8 + ri;
            const float b = vec.bk[i], cq = vec.cq[i];
            const f2 bb = pack2(b, b), cc = pack2(cq, cq);
            uint8_t *const nrow = nt + i * 128, *const prow = smem + kSmP + i * 128;
            // P's low part in the quarters above the diagonal
            uint8_t* const lrow = (c0 ? smem + kSmP : r0 < 32 ? tt : tt + kTile) + (i & 31) * 128;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int j = c0 + t * 8 + cj, bj = (c0 + t * 8) / B;
                f2 pv = 0;
                if (bj < bi) {
                    const float f = vec.f[bj][i];
                    const f2 l = mul2(pack2(f, f), *reinterpret_cast<const f2*>(vec.rk + j));
                    put_split(nrow + y[t], mul2(mul2(bb, l), pack2(kk[t][2 * half], kk[t][2 * half + 1])));
                    pv = mul2(mul2(cc, l), pack2(qk[t][2 * half], qk[t][2 * half + 1]));
                } else if (bj == bi) {
                    const f2 l = mul2(pack2(e[t & 1][half][0], e[t & 1][half][1]), *reinterpret_cast<const f2*>(vec.ck + j));
                    const float2 nv = unpack2(mul2(mul2(bb, l), pack2(kk[t][2 * half], kk[t][2 * half + 1])));
                    const float2 q = unpack2(mul2(mul2(cc, l), pack2(qk[t][2 * half], qk[t][2 * half + 1])));
                    e32[e_at(j) + i - r0] = j < i ? nv.x : 0.f;
                    e32[e_at(j + 1) + i - r0] = j + 1 < i ? nv.y : 0.f;
                    pv = pack2(j <= i ? q.x : 0.f, j + 1 <= i ? q.y : 0.f);
                }
                if (below) put_split(prow + y[t], lrow + (c0 ? y[t] : y[t] ^ 64), pv);
            }
        }
        // T is zero right of its diagonal blocks, within the quarters that are read
        if (tid < 128) {
            const int row = (tid >> 1 & 15) + (tid >> 5 & 1) * 32, c = (row & 32) + 16 + (tid & 1) * 8;
            *reinterpret_cast<uint4*>(tt + (tid >> 6) * kTile + sw64_off(row, c)) = make_uint4(0, 0, 0, 0);
        }
    }
    fence_proxy_async();
    __syncthreads();
    if (tid == kThreads - 1) {
        bulk_s2g(blk + kDeltaP, smem + kSmP, kTile);
        bulk_commit();
    }
    // the diagonal blocks of T, two a warp: a lane has a column; once row m is known its
    // multiples go to the rows below
    if (warp < 2) {
        const int o = (2 * warp + (lane >> 4)) * B, col = lane & 15;
        float t[B];
#pragma unroll
        for (int i = 0; i < B; ++i) t[i] = i == col ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < B - 1; ++m) {
#pragma unroll
            for (int i = (m + 1) & ~3; i < B; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(e32 + e_at(o + m) + i);
                if (i > m) t[i] = fmaf(x.x, t[m], t[i]);
                if (i + 1 > m) t[i + 1] = fmaf(x.y, t[m], t[i + 1]);
                if (i + 2 > m) t[i + 2] = fmaf(x.z, t[m], t[i + 2]);
                if (i + 3 > m) t[i + 3] = fmaf(x.w, t[m], t[i + 3]);
            }
        }
        const uint32_t piece = (o >> 3) + (col >> 3);
        uint8_t* const to = tt + o * 128 + (col & 7) * 2;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const __half hi = __float2half_rn(t[i]);
            uint8_t* const at = to + i * 128 + ((piece ^ (i & 7)) << 4);
            *reinterpret_cast<__half*>(at) = hi;
            *reinterpret_cast<__half*>(at + kTile) = __float2half_rn(t[i] - __half2float(hi));
        }
    }
    __syncthreads();
    // blocks of 32: Y = N21 T11, then T21 = T22 Y
    {
        const int o = (warp >> 1 & 1) * 32, n = (warp & 1) * 8;
        if (warp < 4) block_product<B>(ln, nt, o + B, o, tt, o, o + n, nt, o, o + B + n, lane);
        __syncthreads();
        if (warp < 4) block_product<B>(ln, tt, o + B, o + B, nt, o, o + B + n, tt, o + B, o + n, lane);
    }
    __syncthreads();
    // and of 64
    {
        const int o = (warp >> 2) * B, n = (warp & 3) * 8;
        block_product<32>(ln, nt, 32 + o, 0, tt, 0, n, nt, o, 32 + n, lane);
        __syncthreads();
        block_product<32>(ln, tt, 32 + o, 32, nt, 0, 32 + n, tt, 32 + o, n, lane);
    }
    fence_proxy_async();
    __syncthreads();
    if (tid == kThreads - 1) {
        bulk_s2g(blk + kDeltaT, tt, 2 * kTile);
        bulk_commit();
        bulk_wait_all();
    }
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaParams& p, cudaStream_t s) {
    if (p.n_long <= 0) return cudaSuccess;
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
