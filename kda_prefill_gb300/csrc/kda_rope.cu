// Rotary positions: y1 = c x1 - s x2, y2 = c x2 + s x1 for each pair of a head's
// first rot dimensions, with (c, s) of one token and pair shared by all heads.
//
// The angle p f is wanted modulo one turn.  f / 2 pi is rounded to a 64-bit
// fraction of a turn F; then p F mod 2^64 is the phase, exactly, in one integer
// product (two's complement wraps as turns do), and its top 32 bits give the
// argument of sincospi.  A fp32 product p f would be off by p 2^-25 radians.
//
// Bound by reading and writing the heads once.  A CTA takes a few tokens,
// writes their (c, s) to shared memory, then its threads walk the tokens' units:
// 16 bytes of a head and their partners (half layout: the 16 bytes rot / 2
// further), or 16 bytes to copy.

#include "kda_ops.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTable = 2048;  // pairs times tokens a CTA holds (16 KB)

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

// Units of one head's row: `rot_units` of them turn, the others copy.
template <class E, int VE, bool IL>
__global__ void __launch_bounds__(kThreads) kda_rope(RopeParams p, int tokens, int rot_units,
                                                     int units) {
    __shared__ float2 table[kMaxTable];
    const int half = p.rot >> 1;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, p.T - t0);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
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
    const int h0 = p.x[0].heads, heads = h0 + p.x[1].heads;
    const int per_token = heads * units;
    for (int i = threadIdx.x; i < nt * per_token; i += kThreads) {
        const int t = i / per_token, r = i - t * per_token;
        int h = r / units;
        const int u = r - h * units;
        const RopeTensor& x = p.x[h >= h0];
        if (h >= h0) h -= h0;
        const E* in = static_cast<const E*>(x.in) + (t0 + t) * x.in_st + (int64_t)h * x.in_sh;
        E* out = static_cast<E*>(x.out) + (t0 + t) * x.out_st + (int64_t)h * x.out_sh;
        const float2* cs = table + t * half;
        if (u >= rot_units) {
            if (in != out) {
                const int at = p.rot + (u - rot_units) * VE;
                *reinterpret_cast<Vec<E, VE>*>(out + at) = *reinterpret_cast<const Vec<E, VE>*>(in + at);
            }
        } else if (IL && VE > 1) {
            Vec<E, VE> a = *reinterpret_cast<const Vec<E, VE>*>(in + u * VE);
#pragma unroll
            for (int j = 0; j + 1 < VE; j += 2) {
                const float2 w = cs[u * (VE / 2) + j / 2];
                const float x1 = to_f(a.e[j]), x2 = to_f(a.e[j + 1]);
                a.e[j] = from_f<E>(x1 * w.x - x2 * w.y);
                a.e[j + 1] = from_f<E>(x2 * w.x + x1 * w.y);
            }
            *reinterpret_cast<Vec<E, VE>*>(out + u * VE) = a;
        } else {
            const int one = IL ? 2 * u : u * VE, two = IL ? 2 * u + 1 : half + u * VE;
            Vec<E, VE> a = *reinterpret_cast<const Vec<E, VE>*>(in + one);
            Vec<E, VE> b = *reinterpret_cast<const Vec<E, VE>*>(in + two);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float2 w = cs[u * VE + j];
                const float x1 = to_f(a.e[j]), x2 = to_f(b.e[j]);
                a.e[j] = from_f<E>(x1 * w.x - x2 * w.y);
                b.e[j] = from_f<E>(x2 * w.x + x1 * w.y);
            }
            *reinterpret_cast<Vec<E, VE>*>(out + one) = a;
            *reinterpret_cast<Vec<E, VE>*>(out + two) = b;
        }
    }
}

template <class E, int VE, bool IL>
cudaError_t launch(const RopeParams& p, cudaStream_t s) {
    const int half = p.rot / 2;
    const int rot_units = IL && VE > 1 ? p.rot / VE : half / VE;
    const int units = rot_units + (p.D - p.rot) / VE;
    const int heads = p.x[0].heads + p.x[1].heads;
    // tokens per CTA: about eight units for each thread, at most what the table holds
    int tokens = kThreads * 8 / max(1, heads * units);
    tokens = max(1, min(tokens, kMaxTable / max(1, half)));
    // and at least four CTAs for each SM, where there are so many tokens
    tokens = (int)max((int64_t)1, min((int64_t)tokens, p.T / (4 * num_sms())));
    const int64_t grid = (p.T + tokens - 1) / tokens;
    kda_rope<E, VE, IL><<<(unsigned)grid, kThreads, 0, s>>>(p, tokens, rot_units, units);
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
