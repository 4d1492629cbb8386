// Linear attention with a decay for each head, token by token:
//
//     S_t = e^{g_t} S_{t-1} + v_t k_t^T,    o_t = scale S_t q_t
//
// A CTA of four warps holds 32 value rows of one (sequence, head) state, a warp
// eight rows, a lane four key columns of each: rows are read and written as
// whole 512-byte (fp32) lines, every lane needs only its own four k and q
// values, and a token's eight outputs of a warp come from one halving butterfly.
// For single tokens the state's two trips through memory are the bound.

#include "kda_ops.h"

namespace kda {
namespace {

constexpr int D = kD;
constexpr int kWarps = 4;
constexpr int kRows = 8;                      // value rows per warp
constexpr int kSplit = D / (kWarps * kRows);  // CTAs per (sequence, head)

template <class S>
struct Quad;  // four state values of one row
template <>
struct Quad<float> {
    static __device__ __forceinline__ float4 load(const float* p) {
        return __ldcs(reinterpret_cast<const float4*>(p));
    }
    static __device__ __forceinline__ void store(float* p, float4 x) {
        __stcs(reinterpret_cast<float4*>(p), x);
    }
};
template <>
struct Quad<__nv_bfloat16> {
    static __device__ __forceinline__ float4 load(const __nv_bfloat16* p) {
        const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
        const float2 a = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(r.x));
        const float2 b = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(r.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, float4 x) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(reinterpret_cast<const uint32_t&>(a),
                                                       reinterpret_cast<const uint32_t&>(b)));
    }
};
template <>
struct Quad<__half> {
    static __device__ __forceinline__ float4 load(const __half* p) {
        const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
        const float2 a = __half22float2(reinterpret_cast<const __half2&>(r.x));
        const float2 b = __half22float2(reinterpret_cast<const __half2&>(r.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    static __device__ __forceinline__ void store(__half* p, float4 x) {
        const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(reinterpret_cast<const uint32_t&>(a),
                                                       reinterpret_cast<const uint32_t&>(b)));
    }
};

__device__ __forceinline__ float4 load_bf16x4(const __nv_bfloat16* p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(r.x));
    const float2 b = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(r.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

// Sums of x[0..7] over the warp's 32 lanes; lane l gets that of row l & 7.
__device__ __forceinline__ float sum_rows8(float (&x)[8], int lane) {
#pragma unroll
    for (int w = 4; w >= 1; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int j = 0; j < w; ++j) {
            const float give = up ? x[j] : x[j + w];
            const float keep = up ? x[j + w] : x[j];
            x[j] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
    float s = x[0];
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    return s;
}

template <class S>
__global__ void __launch_bounds__(kWarps * 32) kda_lin_step(LinParams p, const int32_t* list) {
    const int h = blockIdx.y;
    const int n = list[blockIdx.x / kSplit];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = (blockIdx.x % kSplit) * (kWarps * kRows) + warp * kRows;
    const int t0 = p.cu[n], t1 = p.cu[n + 1];
    const int slot = p.idx[n];
    const bool ok = slot >= 0 && slot < p.num_slots;
    const bool init = ok && p.has_init[n] != 0;
    if (!ok && threadIdx.x == 0) atomicOr(p.status, 4);
    S* state = static_cast<S*>(p.pool) + (ok ? (size_t)slot * p.stride0 : 0) +
               ((size_t)h * D + row0) * D + 4 * lane;
    float4 s[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        s[r] = init ? Quad<S>::load(state + r * D) : make_float4(0.f, 0.f, 0.f, 0.f);
    const __nv_bfloat16* qp = p.q + (int64_t)(h / p.rep) * p.q_sh + 4 * lane;
    const __nv_bfloat16* kp = p.k + (int64_t)(h / p.rep) * p.k_sh + 4 * lane;
    const __nv_bfloat16* vp = p.v + (int64_t)h * p.v_sh + row0;
    for (int t = t0; t < t1; ++t) {
        const float4 k = load_bf16x4(kp + (int64_t)t * p.k_st);
        const float4 q = load_bf16x4(qp + (int64_t)t * p.q_st);
        const float4 va = load_bf16x4(vp + (int64_t)t * p.v_st);
        const float4 vb = load_bf16x4(vp + (int64_t)t * p.v_st + 4);
        const float v[kRows] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
        const float g = p.g[(int64_t)t * p.g_st + h];
        // a decay near one as 1 + expm1(g): rounded to fp32, e^g alone would be off
        // by up to 2^-25 in the same direction at every token
        const bool slow = g > -0.5f;
        const float d = slow ? expm1f(g) : expf(g);
        float o[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float4 w = make_float4(v[r] * k.x, v[r] * k.y, v[r] * k.z, v[r] * k.w);
            if (slow) {
                s[r].x += fmaf(d, s[r].x, w.x);
                s[r].y += fmaf(d, s[r].y, w.y);
                s[r].z += fmaf(d, s[r].z, w.z);
                s[r].w += fmaf(d, s[r].w, w.w);
            } else if (d == 0.f) {  // cleared, whatever it held
                s[r] = w;
            } else {
                s[r].x = fmaf(d, s[r].x, w.x);
                s[r].y = fmaf(d, s[r].y, w.y);
                s[r].z = fmaf(d, s[r].z, w.z);
                s[r].w = fmaf(d, s[r].w, w.w);
            }
            o[r] = fmaf(s[r].x, q.x, s[r].y * q.y) + fmaf(s[r].z, q.z, s[r].w * q.w);
        }
        const float sum = sum_rows8(o, lane);
        if (lane < kRows)
            p.out[((size_t)t * p.H + h) * D + row0 + lane] = __float2bfloat16_rn(p.scale * sum);
    }
    if (ok && !(init && t1 <= t0)) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) Quad<S>::store(state + r * D, s[r]);
    }
}

}  // namespace

cudaError_t launch_lin_step(const LinParams& p, const int32_t* list, int n, cudaStream_t s) {
    if (n <= 0) return cudaSuccess;
    const dim3 grid((unsigned)n * kSplit, (unsigned)p.H);
    if (p.st_dtype == KDA_STATE_F32)
        kda_lin_step<float><<<grid, kWarps * 32, 0, s>>>(p, list);
    else if (p.st_dtype == KDA_STATE_BF16)
        kda_lin_step<__nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(p, list);
    else
        kda_lin_step<__half><<<grid, kWarps * 32, 0, s>>>(p, list);
    return cudaGetLastError();
}

}  // namespace kda
