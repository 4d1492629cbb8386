// Linear attention with a decay for each head, token by token:
//
//     S_t = e^{g_t} S_{t-1} + v_t k_t^T,    o_t = scale S_t q_t
//
// A CTA of four warps holds 32 value rows of one (sequence, head) state, a warp eight
// rows.  A lane reads and writes 16 bytes: four key columns of each row in fp32 (a warp's
// access is a whole row), eight columns of every other row in 16 bits (two rows).  It
// needs only its own k and q values, and a token's eight outputs of a warp come from one
// halving butterfly.  The next token's values are read while one is worked on.  For single
// tokens the state's two trips through memory are the bound: 512 tokens x 12 heads with
// fp32 states take 121.5 us, 98 % of a plain copy's rate, with bf16 states 68.1 us, 88 %.
// A second token hides behind that (125 us); further ones are bound by instructions, scalar
// fp32 and four for each state value, about 22 us each: 512 sequences of 8 tokens take 260
// us, as long as the chunk kernel takes for 9 (257 us), which is where the two change over.

#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int D = kD;
constexpr int kWarps = 4;
constexpr int kRows = 8;                      // value rows per warp
constexpr int kSplit = D / (kWarps * kRows);  // CTAs per (sequence, head)

template <class S>
struct Lane {
    static constexpr int kCols = 16 / sizeof(S);  // columns of a row
    static constexpr int kAcross = D / kCols;     // lanes of a row
    static constexpr int kHeld = kRows * kAcross / 32;  // rows a lane has part of
};

// N bf16 values of a row (k and q), and this warp's eight of v, as they lie in memory.
template <int N>
struct Bf16s;
template <>
struct Bf16s<4> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void get(float (&f)[4]) const {
        f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
        f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
};
template <>
struct Bf16s<8> {
    rows::Piece<__nv_bfloat16, 8> p8;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { p8.v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&f)[8]) const { p8.get(f); }
};

template <class S>
__global__ void __launch_bounds__(kWarps * 32, 8) kda_lin_step(const __grid_constant__ LinParams p) {
    constexpr int N = Lane<S>::kCols, A = Lane<S>::kAcross, R = Lane<S>::kHeld;
    const int h = blockIdx.y;
    const int n = p.short_list[blockIdx.x / kSplit];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = (blockIdx.x % kSplit) * (kWarps * kRows) + warp * kRows;
    const int col = (lane % A) * N, part = lane / A;  // rows part, part + 32 / A, ... of the eight
    const int t0 = p.cu[n], t1 = p.cu[n + 1];
    const int slot = p.idx[n];
    const bool ok = slot >= 0 && slot < p.num_slots;
    const bool init = ok && p.has_init[n] != 0;
    S* state = static_cast<S*>(p.pool) + (ok ? (size_t)slot * p.stride0 : 0) +
               ((size_t)h * D + row0 + part) * D + col;
    const __nv_bfloat16* qp = p.q + (int64_t)(h / p.rep) * p.q_sh + col;
    const __nv_bfloat16* kp = p.k + (int64_t)(h / p.rep) * p.k_sh + col;
    const __nv_bfloat16* vp = p.v + (int64_t)h * p.v_sh + row0;
    Bf16s<N> q4, k4;
    Bf16s<8> v8;
    float g = 0.f;
    auto fetch = [&](int t) {
        k4.load(kp + (int64_t)t * p.k_st);
        q4.load(qp + (int64_t)t * p.q_st);
        v8.load(vp + (int64_t)t * p.v_st);
        g = p.g[(int64_t)t * p.g_st + h];
    };
    if (t0 < t1) fetch(t0);
    rows::Piece<S, N> piece[R] = {};
    if (init) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            reinterpret_cast<uint4&>(piece[r]) = __ldcs(reinterpret_cast<const uint4*>(state + r * (32 / A) * D));
    }
    float s[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r) piece[r].get(s[r]);
    for (int t = t0; t < t1; ++t) {
        float k[N], q[N], v[8];
        k4.get(k);
        q4.get(q);
        v8.get(v);
        // a decay near one as 1 + expm1(g): rounded to fp32, e^g alone would be off
        // by up to 2^-25 in the same direction at every token
        const bool slow = g > -0.5f;
        const float d = slow ? expm1f(g) : expf(g);
        const float one = slow ? 1.f : 0.f;
        if (g < kMinDecay) {  // cleared, whatever it held
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < N; ++j) s[r][j] = 0.f;
        }
        if (t + 1 < t1) fetch(t + 1);
        float o[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // this lane's row of v: 32 / A rows lie between its own
            float vr = v[r * (32 / A)];
#pragma unroll
            for (int u = 1; u < 32 / A; ++u) vr = part == u ? v[r * (32 / A) + u] : vr;
            o[r] = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                s[r][j] = fmaf(one, s[r][j], fmaf(d, s[r][j], vr * k[j]));
                o[r] = fmaf(s[r][j], q[j], o[r]);
            }
        }
        // sums over the A lanes of a row: lane l keeps that of its held row l % R
#pragma unroll
        for (int w = R / 2; w >= 1; w >>= 1) {
            const bool up = (lane & w) != 0;
#pragma unroll
            for (int j = 0; j < w; ++j) {
                const float give = up ? o[j] : o[j + w];
                const float keep = up ? o[j + w] : o[j];
                o[j] = keep + __shfl_xor_sync(0xffffffffu, give, w);
            }
        }
        float sum = o[0];
#pragma unroll
        for (int w = R; w < A; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        if (lane % A < R)
            p.out[((size_t)t * p.H + h) * D + row0 + (lane % A) * (32 / A) + part] =
                __float2bfloat16_rn(p.scale * sum);
    }
    if (ok && !(init && t1 <= t0)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            piece[r].set(s[r]);
            __stcs(reinterpret_cast<uint4*>(state + r * (32 / A) * D), reinterpret_cast<const uint4&>(piece[r]));
        }
    }
    // Launched beside the walk, this grid is over only once the walk is; otherwise the
    // wait returns at once.
    if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.n_long == 0 && blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) write_status(p, lane);
}

template <class S>
cudaError_t launch(const LinParams& p, bool beside, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.n_short * kSplit, (unsigned)p.H);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kda_lin_step<S>, p);
}

}  // namespace

cudaError_t launch_lin_step(const LinParams& p, bool beside, cudaStream_t s) {
    if (p.n_short <= 0) return cudaSuccess;
    if (p.st_dtype == KDA_STATE_F32) return launch<float>(p, beside, s);
    if (p.st_dtype == KDA_STATE_BF16) return launch<__nv_bfloat16>(p, beside, s);
    return launch<__half>(p, beside, s);
}

}  // namespace kda
