// Root-mean-square norm of each row with a weight and a gate:
//
//     y = x / sqrt(mean(x^2) + eps) * weight * act(gate)
//
// Bound by reading x and the gate and writing y once.  A group of lanes takes a row.
// Rows of at most one 16-byte piece a lane stay in registers between the sum of squares
// and the product, and where there are enough of them a group has two in flight, with
// their gates.  Longer rows are read again, from the caches, by a warp each, with few loads
// in flight: 3000 rows of 8192 in bf16 47.3 us, 46 % of a plain copy's rate, 49152 of 512
// 39.0 us, 57 %.
// 16384 tokens x 12 heads of 128: 28.7 us in bf16, 77 % of a plain copy's rate, 53.3 us in
// fp32, 83 %; the rest is the start and the end of a launch and, in 16 bits, the
// conversions' instructions (63 % of the issue rate).

#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
enum Gate { kNoGate, kPlain, kSigmoid, kSilu };

// 1 / (1 + e^-z).  For fp32 rows to fp32's last bits; 16-bit rows take exp and the
// quotient from the special function unit (within 2^-21 for |z| < 16, then rounded to
// 2^-11 or 2^-8): otherwise they are bound by instructions (36 a value instead of 11).
template <class E>
__device__ __forceinline__ float sigmoid(float z) {
    if (sizeof(E) == 4) return 1.f / (1.f + expf(-z));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <class E, int GATE>
__device__ __forceinline__ float gate_of(float z) {
    if (GATE == kPlain) return z;
    const float s = sigmoid<E>(z);
    if (GATE == kSigmoid) return s;
    return s > 0.f ? z * s : (z < 0.f ? 0.f : z);  // z s at z = -inf is 0, its limit
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int w = LANES / 2; w >= 1; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    return x;
}

// Rows of at most one piece a lane, ROWS of them at a time.
template <class E, int VE, int LANES, int ROWS, int GATE>
__global__ void __launch_bounds__(kThreads, ROWS == 1 ? 12 : 10) kda_gated_norm_short(NormParams p, int64_t rows) {
    const int c = (threadIdx.x % LANES) * VE;
    const bool in_row = c < p.D;
    constexpr int kGroups = kThreads / LANES;
    const int64_t first = (int64_t)blockIdx.x * (kGroups * ROWS) + threadIdx.x / LANES;
    rows::Piece<E, VE> x[ROWS] = {}, z[ROWS] = {};
    E* out[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t row = first + i * kGroups;
        out[i] = nullptr;
        if (row < rows && in_row) {
            const int64_t t = rows <= INT32_MAX ? (int64_t)((uint32_t)row / (uint32_t)p.H) : row / p.H;
            const int64_t h = row - t * p.H;
            x[i] = rows::load<E, VE>(static_cast<const E*>(p.x) + t * p.x_st + h * p.x_sh + c);
            if (GATE != kNoGate) z[i] = rows::load<E, VE>(static_cast<const E*>(p.gate) + t * p.g_st + h * p.g_sh + c);
            out[i] = static_cast<E*>(p.out) + t * p.o_st + h * p.o_sh + c;
        }
    }
    float w[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) w[j] = p.weight && in_row ? p.weight[c + j] : 1.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        float f[VE];
        x[i].get(f);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < VE; ++j) sum = fmaf(f[j], f[j], sum);
        sum = group_sum<LANES>(sum);
        const float inv = 1.f / sqrtf(sum / (float)p.D + p.eps);
#pragma unroll
        for (int j = 0; j < VE; ++j) f[j] *= inv * w[j];
        if (GATE != kNoGate) {
            float g[VE];
            z[i].get(g);
#pragma unroll
            for (int j = 0; j < VE; ++j) f[j] *= gate_of<E, GATE>(g[j]);
        }
        x[i].set(f);
        if (out[i]) rows::store<E, VE>(out[i], x[i]);
    }
}

// Longer rows, and rows that are not whole pieces: a warp each.
template <class E, int VE, int GATE>
__global__ void __launch_bounds__(kThreads) kda_gated_norm(NormParams p, int64_t rows) {
    const int lane = threadIdx.x % 32;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; row < rows; row += step) {
        const int64_t t = row / p.H;
        const int64_t h = row - t * p.H;
        const E* x = static_cast<const E*>(p.x) + t * p.x_st + h * p.x_sh;
        const E* g = static_cast<const E*>(p.gate) + (GATE != kNoGate ? t * p.g_st + h * p.g_sh : 0);
        E* y = static_cast<E*>(p.out) + t * p.o_st + h * p.o_sh;
        float sum = 0.f;
        for (int c = lane * VE; c < p.D; c += 32 * VE) {
            float f[VE];
            rows::load<E, VE>(x + c).get(f);
#pragma unroll
            for (int j = 0; j < VE; ++j) sum = fmaf(f[j], f[j], sum);
        }
        sum = group_sum<32>(sum);
        const float inv = 1.f / sqrtf(sum / (float)p.D + p.eps);
        for (int c = lane * VE; c < p.D; c += 32 * VE) {
            float f[VE], z[VE];
            rows::load<E, VE>(x + c).get(f);
            if (GATE != kNoGate) rows::load<E, VE>(g + c).get(z);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                f[j] *= inv * (p.weight ? p.weight[c + j] : 1.f);
                if (GATE != kNoGate) f[j] *= gate_of<E, GATE>(z[j]);
            }
            rows::Piece<E, VE> b;
            b.set(f);
            rows::store<E, VE>(y + c, b);
        }
    }
}

template <class E, int VE, int LANES, int GATE>
cudaError_t launch_short(const NormParams& p, cudaStream_t s) {
    const int64_t rows = p.T * p.H;
    constexpr int kGroups = kThreads / LANES;
    // two rows a group where that still gives each SM sixteen CTAs (16384 tokens x 12 heads
    // of 128: 28.8 us, and 32.1 us with one; 512 tokens: 4.1 us with either)
    if (rows >= (int64_t)32 * kGroups * num_sms())
        kda_gated_norm_short<E, VE, LANES, 2, GATE>
            <<<(unsigned)((rows + 2 * kGroups - 1) / (2 * kGroups)), kThreads, 0, s>>>(p, rows);
    else
        kda_gated_norm_short<E, VE, LANES, 1, GATE>
            <<<(unsigned)((rows + kGroups - 1) / kGroups), kThreads, 0, s>>>(p, rows);
    return cudaGetLastError();
}

template <class E, int VE, int GATE>
cudaError_t launch_long(const NormParams& p, cudaStream_t s) {
    const int64_t rows = p.T * p.H;
    const int64_t grid = (rows + kThreads / 32 - 1) / (kThreads / 32);
    kda_gated_norm<E, VE, GATE><<<(unsigned)(grid < INT32_MAX ? grid : INT32_MAX), kThreads, 0, s>>>(p, rows);
    return cudaGetLastError();
}

template <class E, int GATE>
cudaError_t dispatch(const NormParams& p, cudaStream_t s) {
    constexpr int VE = 16 / sizeof(E);
    // 16-byte pieces when the row length, strides and bases allow them
    const uintptr_t bases = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out) |
                            reinterpret_cast<uintptr_t>(p.gate);
    const int64_t strides = p.x_st | p.x_sh | p.o_st | p.o_sh | (p.gate ? p.g_st | p.g_sh : 0);
    if (p.D % VE != 0 || (bases & 15) != 0 || strides % VE != 0) return launch_long<E, 1, GATE>(p, s);
    // (a CTA of the short forms takes at least a KB of rows: the grid stays within 2^31)
    if (p.D <= 8 * VE) return launch_short<E, VE, 8, GATE>(p, s);
    if (p.D <= 16 * VE) return launch_short<E, VE, 16, GATE>(p, s);
    if (p.D <= 32 * VE) return launch_short<E, VE, 32, GATE>(p, s);
    return launch_long<E, VE, GATE>(p, s);
}

template <class E>
cudaError_t by_gate(const NormParams& p, cudaStream_t s) {
    if (!p.gate) return dispatch<E, kNoGate>(p, s);
    if (p.act == KDA_ACT_SIGMOID) return dispatch<E, kSigmoid>(p, s);
    if (p.act == KDA_ACT_SILU) return dispatch<E, kSilu>(p, s);
    return dispatch<E, kPlain>(p, s);
}

}  // namespace

cudaError_t launch_gated_norm(const NormParams& p, cudaStream_t s) {
    if (p.dtype == KDA_F32) return by_gate<float>(p, s);
    if (p.dtype == KDA_BF16) return by_gate<__nv_bfloat16>(p, s);
    return by_gate<__half>(p, s);
}

}  // namespace kda
