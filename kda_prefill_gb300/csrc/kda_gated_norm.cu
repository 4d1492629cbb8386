// Root-mean-square norm of each row with a weight and a gate:
//
//     y = x / sqrt(mean(x^2) + eps) * weight * act(gate)
//
// Bound by reading x and the gate and writing y once.  A group of lanes takes a
// row.  Rows of at most one 16-byte vector a lane stay in registers between the
// sum of squares and the product; longer ones are read again, from the caches.

#include "kda_ops.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <class E> __device__ __forceinline__ E from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

template <class E, int VE>
struct alignas(sizeof(E) * VE) Vec {
    E e[VE];
};

__device__ __forceinline__ float gate_of(float z, int act) {
    if (act == KDA_ACT_NONE) return z;
    const float s = 1.f / (1.f + expf(-z));
    // z s for z at -inf is 0, its limit
    return act == KDA_ACT_SIGMOID ? s : (s > 0.f ? z * s : (z < 0.f ? 0.f : z));
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int w = LANES / 2; w >= 1; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    return x;
}

// LANES lanes a row, `steps` vectors of VE elements a lane.
template <class E, int VE, int LANES>
__global__ void __launch_bounds__(kThreads) kda_gated_norm(NormParams p, int64_t rows) {
    const int lane = threadIdx.x % LANES;
    const int64_t step = (int64_t)gridDim.x * (kThreads / LANES);
    // the same number of rounds for all lanes: the sums are taken by whole warps
    for (int64_t base = (int64_t)blockIdx.x * (kThreads / LANES); base < rows; base += step) {
        const int64_t row = base + threadIdx.x / LANES;
        const bool live = row < rows;
        const int64_t t = live ? row / p.H : 0;
        const int h = live ? (int)(row - t * p.H) : 0;
        const E* x = static_cast<const E*>(p.x) + t * p.x_st + (int64_t)h * p.x_sh;
        const E* g = static_cast<const E*>(p.gate) + (p.gate ? t * p.g_st + (int64_t)h * p.g_sh : 0);
        E* y = static_cast<E*>(p.out) + t * p.o_st + (int64_t)h * p.o_sh;
        const int end = live ? p.D : 0;
        Vec<E, VE> first{};
        float sum = 0.f;
        for (int c = lane * VE; c < end; c += LANES * VE) {
            const Vec<E, VE> a = *reinterpret_cast<const Vec<E, VE>*>(x + c);
            if (c == lane * VE) first = a;
#pragma unroll
            for (int j = 0; j < VE; ++j) sum = fmaf(to_f(a.e[j]), to_f(a.e[j]), sum);
        }
        sum = group_sum<LANES>(sum);
        const float inv = 1.f / sqrtf(sum / (float)p.D + p.eps);
        for (int c = lane * VE; c < end; c += LANES * VE) {
            const Vec<E, VE> a = c == lane * VE ? first : *reinterpret_cast<const Vec<E, VE>*>(x + c);
            Vec<E, VE> z{}, b;
            if (p.gate) z = *reinterpret_cast<const Vec<E, VE>*>(g + c);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                float r = to_f(a.e[j]) * inv;
                if (p.weight) r *= p.weight[c + j];
                if (p.gate) r *= gate_of(to_f(z.e[j]), p.act);
                b.e[j] = from_f<E>(r);
            }
            *reinterpret_cast<Vec<E, VE>*>(y + c) = b;
        }
    }
}

template <class E, int VE, int LANES>
cudaError_t launch(const NormParams& p, cudaStream_t s) {
    const int64_t rows = p.T * p.H;
    const int64_t per_cta = kThreads / LANES;
    const int64_t grid = (rows + per_cta - 1) / per_cta;
    kda_gated_norm<E, VE, LANES><<<(unsigned)(grid < INT32_MAX ? grid : INT32_MAX), kThreads, 0, s>>>(p, rows);
    return cudaGetLastError();
}

template <class E>
cudaError_t dispatch(const NormParams& p, cudaStream_t s) {
    constexpr int VE = 16 / sizeof(E);
    // 16-byte vectors when the row length, strides and bases allow them
    const uintptr_t bases = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out) |
                            reinterpret_cast<uintptr_t>(p.gate);
    const int64_t strides = p.x_st | p.x_sh | p.o_st | p.o_sh | (p.gate ? p.g_st | p.g_sh : 0);
    if (p.D % VE != 0 || (bases & 15) != 0 || strides % VE != 0) return launch<E, 1, 32>(p, s);
    if (p.D <= 8 * VE) return launch<E, VE, 8>(p, s);
    if (p.D <= 16 * VE) return launch<E, VE, 16>(p, s);
    return launch<E, VE, 32>(p, s);
}

}  // namespace

cudaError_t launch_gated_norm(const NormParams& p, cudaStream_t s) {
    if (p.dtype == KDA_F32) return dispatch<float>(p, s);
    if (p.dtype == KDA_BF16) return dispatch<__nv_bfloat16>(p, s);
    return dispatch<__half>(p, s);
}

}  // namespace kda
