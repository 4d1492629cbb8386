// Rows of fp32, bf16 or fp16 values in 16-byte pieces or one by one, for the
// operators that stream over rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace kda {
namespace rows {

// A piece of N values: 16 bytes of them, or one.
template <class E, int N>
struct Piece;

template <>
struct Piece<float, 4> {
    float4 v;
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w; }
    __device__ __forceinline__ void set(const float (&f)[4]) { v = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Piece<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = reinterpret_cast<const uint32_t&>(h);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Piece<__half, 8> {
    uint4 v;
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = __half22float2(reinterpret_cast<const __half2&>(w[i]));
            f[2 * i] = a.x, f[2 * i + 1] = a.y;
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = reinterpret_cast<const uint32_t&>(h);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Piece<float, 1> {
    float v;
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = v; }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = f[0]; }
};
template <>
struct Piece<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(v); }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = __float2bfloat16_rn(f[0]); }
};
template <>
struct Piece<__half, 1> {
    __half v;
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __half2float(v); }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = __float2half_rn(f[0]); }
};

template <class E, int N>
__device__ __forceinline__ Piece<E, N> load(const E* p) {
    return *reinterpret_cast<const Piece<E, N>*>(p);
}
template <class E, int N>
__device__ __forceinline__ void store(E* p, const Piece<E, N>& x) {
    *reinterpret_cast<Piece<E, N>*>(p) = x;
}

}  // namespace rows
}  // namespace kda
