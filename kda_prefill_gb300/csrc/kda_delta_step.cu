// The gated delta rule with a decay for each head, token by token:
//
//     u_t = b_t (v_t - e^{g_t} S_{t-1} k_t),   S_t = e^{g_t} S_{t-1} + u_t k_t^T
//     o_t = scale S_t q_t = scale (e^{g_t} S_{t-1} q_t + u_t (k_t . q_t))
//
// with k and q divided by their lengths.  So both products with the state are with the one
// that is there, their sums over a row's lanes travel together, and the lengths are factors
// on sums.
//
// A CTA of four warps holds 32 value rows of one (sequence, head) state, a warp eight rows,
// sixteen lanes a row: a lane has eight key columns of every other row, in 16-byte pieces.

#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int D = kD;
constexpr int kWarps = 4;
constexpr int kRows = 8;                      // value rows per warp
constexpr int kSplit = D / (kWarps * kRows);  // CTAs per (sequence, head)
constexpr int kAcross = 16;                   // lanes of a row
constexpr int kHeld = kRows * kAcross / 32;   // rows a lane has part of
constexpr int kCols = D / kAcross;            // columns of a row a lane has

// A lane's eight columns of a state row: 16 bytes at its place in each 16 x 16 bytes.
template <class S>
struct Cols {
    static constexpr int kN = 16 / sizeof(S), kPieces = kCols / kN;
    static __device__ __forceinline__ int at(int lane, int i) { return i * kAcross * kN + lane * kN; }
    static __device__ __forceinline__ void load(const S* row, int lane, uint4 (&raw)[kPieces]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) raw[i] = __ldcs(reinterpret_cast<const uint4*>(row + at(lane, i)));
    }
    static __device__ __forceinline__ void get(const uint4 (&raw)[kPieces], float (&f)[kCols]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float x[kN];
            reinterpret_cast<const rows::Piece<S, kN>&>(raw[i]).get(x);
#pragma unroll
            for (int j = 0; j < kN; ++j) f[i * kN + j] = x[j];
        }
    }
    static __device__ __forceinline__ void store(S* row, int lane, const float (&f)[kCols]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float x[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) x[j] = f[i * kN + j];
            rows::Piece<S, kN> p;
            p.set(x);
            __stcs(reinterpret_cast<uint4*>(row + at(lane, i)), reinterpret_cast<const uint4&>(p));
        }
    }
    // the same columns of a bf16 row of k or q
    static __device__ __forceinline__ uint4 load16(const __nv_bfloat16* row, int lane) {
        if constexpr (kPieces == 1) {
            return __ldg(reinterpret_cast<const uint4*>(row + at(lane, 0)));
        } else {
            const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + at(lane, 0)));
            const uint2 b = __ldg(reinterpret_cast<const uint2*>(row + at(lane, 1)));
            return make_uint4(a.x, a.y, b.x, b.y);
        }
    }
};

__device__ __forceinline__ float row_sum(float x) {  // over the lanes of a row
#pragma unroll
    for (int w = kAcross / 2; w >= 1; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    return x;
}

template <class S>
__global__ void __launch_bounds__(kWarps * 32, 5)
kda_delta_step(const __grid_constant__ DeltaParams p) {
    using C = Cols<S>;
    const int h = blockIdx.y;
    const int n = p.short_list[blockIdx.x / kSplit];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int at = lane % kAcross, part = lane / kAcross;  // rows part, part + 2, ... of the eight
    const int own = at % kHeld;                            // the held row whose output this lane makes
    const int row0 = (blockIdx.x % kSplit) * (kWarps * kRows) + warp * kRows + part;
    const int t0 = p.cu[n], t1 = p.cu[n + 1];
    const int slot = p.idx[n];
    const bool ok = slot >= 0 && slot < p.num_slots;
    const bool init = ok && p.has_init[n] != 0;
    S* state = static_cast<S*>(p.pool) + (ok ? (size_t)slot * p.stride0 : 0) + ((size_t)h * D + row0) * D;
    const __nv_bfloat16* qp = p.q + (int64_t)(h / p.rep) * p.q_sh;
    const __nv_bfloat16* kp = p.k + (int64_t)(h / p.rep) * p.k_sh;
    const __nv_bfloat16* vp = p.v + (int64_t)h * p.v_sh + row0 + own * (32 / kAcross);
    rows::Piece<__nv_bfloat16, 8> k8, q8;
    __nv_bfloat16 v1;
    float g = 0.f, beta = 0.f;
    auto fetch = [&](int t) {
        k8.v = C::load16(kp + (int64_t)t * p.k_st, at);
        q8.v = C::load16(qp + (int64_t)t * p.q_st, at);
        v1 = vp[(int64_t)t * p.v_st];
        g = p.g[(int64_t)t * p.g_st + h];
        beta = p.beta[(int64_t)t * p.H + h];
    };
    if (t0 < t1) fetch(t0);
    uint4 raw[kHeld][C::kPieces] = {};
    if (init) {
#pragma unroll
        for (int r = 0; r < kHeld; ++r) C::load(state + r * (32 / kAcross) * D, at, raw[r]);
    }
    float s[kHeld][kCols];
#pragma unroll
    for (int r = 0; r < kHeld; ++r) C::get(raw[r], s[r]);
    for (int t = t0; t < t1; ++t) {
        float k[kCols], q[kCols];
        k8.get(k);
        q8.get(q);
        const float v = __bfloat162float(v1), b = beta;
        // a decay near one as 1 + expm1(g): rounded to fp32, e^g alone would be off
        // by up to 2^-25 in the same direction at every token
        const bool slow = g > -0.5f;
        const float d = slow ? expm1f(g) : expf(g);
        const float one = slow ? 1.f : 0.f;
        if (g < kMinDecay) {  // cleared, whatever it held
#pragma unroll
            for (int r = 0; r < kHeld; ++r)
#pragma unroll
                for (int j = 0; j < kCols; ++j) s[r][j] = 0.f;
        }
        if (t + 1 < t1) fetch(t + 1);
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            kk = fmaf(k[j], k[j], kk);
            qq = fmaf(q[j], q[j], qq);
            kq = fmaf(k[j], q[j], kq);
        }
        // sums over a row's lanes: lane l keeps x[l % 8], the state's product with k for the
        // held rows, then with q
        float x[2 * kHeld];
#pragma unroll
        for (int r = 0; r < kHeld; ++r) {
            x[r] = x[kHeld + r] = 0.f;
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                x[r] = fmaf(s[r][j], k[j], x[r]);
                x[kHeld + r] = fmaf(s[r][j], q[j], x[kHeld + r]);
            }
        }
#pragma unroll
        for (int w = kHeld; w >= 1; w >>= 1) {
            const bool up = (lane & w) != 0;
#pragma unroll
            for (int j = 0; j < w; ++j) {
                const float give = up ? x[j] : x[j + w];
                const float keep = up ? x[j + w] : x[j];
                x[j] = keep + __shfl_xor_sync(0xffffffffu, give, w);
            }
        }
        const float sum = x[0] + __shfl_xor_sync(0xffffffffu, x[0], 2 * kHeld);
        const float rk = 1.f / sqrtf(row_sum(kk) + 1e-6f), rq = 1.f / sqrtf(row_sum(qq) + 1e-6f);
        kq = row_sum(kq);
        const int first = lane - at;
        const float sk = __shfl_sync(0xffffffffu, sum, first + own);
        const float sq = __shfl_sync(0xffffffffu, sum, first + kHeld + own);
        const float e = one + d;
        const float uk = b * (v - e * (rk * sk)) * rk;
        if (at < kHeld)
            p.out[((size_t)t * p.H + h) * D + row0 + own * (32 / kAcross)] =
                __float2bfloat16_rn(p.scale * (rq * fmaf(uk, kq, e * sq)));
#pragma unroll
        for (int r = 0; r < kHeld; ++r) {
            const float ur = __shfl_sync(0xffffffffu, uk, first + r);
#pragma unroll
            for (int j = 0; j < kCols; ++j) s[r][j] = fmaf(one, s[r][j], fmaf(d, s[r][j], ur * k[j]));
        }
    }
    if (ok && !(init && t1 <= t0)) {
#pragma unroll
        for (int r = 0; r < kHeld; ++r) C::store(state + r * (32 / kAcross) * D, at, s[r]);
    }
    // Launched beside the walk, this grid may be over only once the walk is: its last CTA waits
    // (all of them waiting would keep their places on the SMs that the walk leaves free: 512
    // single tokens beside four prompts of 2048 then took 217 us)
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && threadIdx.x == 0)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.n_long == 0 && blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) write_status(p, lane);
}

template <class S>
cudaError_t launch(const DeltaParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.n_short * kSplit, (unsigned)p.H);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    // right behind the walk, beside its CTAs
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.n_long > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kda_delta_step<S>, p);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaParams& p, cudaStream_t s) {
    if (p.n_short <= 0) return cudaSuccess;
    if (p.st_dtype == KDA_STATE_F32) return launch<float>(p, s);
    if (p.st_dtype == KDA_STATE_BF16) return launch<__nv_bfloat16>(p, s);
    return launch<__half>(p, s);
}

}  // namespace kda
