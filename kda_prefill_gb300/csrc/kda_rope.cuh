// What the rotary positions' kernels share: a token's (c, s) of a pair, and the units of
// a head that a thread turns.
//
// The angle p f is wanted modulo one turn.  f / 2 pi is rounded to a 64-bit
// fraction of a turn F; then p F mod 2^64 is the phase, exactly, in one integer
// product (two's complement wraps as turns do), and its top 32 bits give the
// argument of sincospi.  A fp32 product p f would be off by p 2^-25 radians.
#pragma once

#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace rope {

// F of pair j.  (64-bit floating point is slow: one for each pair and CTA, not for each token.)
__device__ __forceinline__ unsigned long long fraction_of(const RopeParams& p, int j) {
    const double turns = p.inv_freq[j] * 0.15915494309189533577;  // 1 / 2 pi
    return (unsigned long long)__double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
}
// (c, s) of token t and a pair.
__device__ __forceinline__ float2 turn_of(const RopeParams& p, int64_t t, unsigned long long fraction) {
    const int64_t pos = p.pos64 ? static_cast<const int64_t*>(p.pos)[t]
                                : (int64_t) static_cast<const int32_t*>(p.pos)[t];
    const unsigned long long phase = (unsigned long long)pos * fraction;
    const float a = (float)(int)(phase >> 32) * 4.656612873077392578125e-10f;  // 2^-31
    float s, c;
    sincospif(a, &s, &c);
    return make_float2(c * p.factor, s * p.factor * p.sign);
}
constexpr int kMaxPairs = 512;  // of a head

// One unit of a row: 16 bytes, and for pairs of the half layout (and for the narrow
// form's pairs) the partner's.
template <class E, int VE, bool IL>
struct Unit {
    rows::Piece<E, VE> a, b;
    static constexpr bool kPaired = !IL || VE == 1;

    // Offsets of the two in a row; units from rot_units on are copied.
    static __device__ __forceinline__ int one(const RopeParams& p, int u, int rot_units) {
        if (u >= rot_units) return p.rot + (u - rot_units) * VE;
        return IL && VE == 1 ? 2 * u : u * VE;
    }
    static __device__ __forceinline__ int two(const RopeParams& p, int u) {
        return IL ? 2 * u + 1 : (p.rot >> 1) + u * VE;
    }
    __device__ __forceinline__ void load(const E* in, int at, int at2, bool turned) {
        a = rows::load<E, VE>(in + at);
        if (kPaired && turned) b = rows::load<E, VE>(in + at2);
    }
    // Its values f and the partners' g, turned.
    static __device__ __forceinline__ void turn(float (&f)[VE], float (&g)[VE], const float2* cs) {
        if constexpr (kPaired) {
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float2 w = cs[j];
                const float x1 = f[j], x2 = g[j];
                f[j] = x1 * w.x - x2 * w.y;
                g[j] = x2 * w.x + x1 * w.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < VE; j += 2) {
                const float2 w = cs[j / 2];
                const float x1 = f[j], x2 = f[j + 1];
                f[j] = x1 * w.x - x2 * w.y;
                f[j + 1] = x2 * w.x + x1 * w.y;
            }
        }
    }
    __device__ __forceinline__ void turn(const float2* cs) {
        float f[VE], g[VE];
        a.get(f);
        if constexpr (kPaired) b.get(g);
        turn(f, g, cs);
        if constexpr (kPaired) b.set(g);
        a.set(f);
    }
    __device__ __forceinline__ void store(E* out, int at, int at2, bool turned) const {
        rows::store<E, VE>(out + at, a);
        if (kPaired && turned) rows::store<E, VE>(out + at2, b);
    }
};

}  // namespace rope
}  // namespace kda
