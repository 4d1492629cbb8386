// The gated delta rule with a decay for each head, token by token:
//
//     u_t = b_t (v_t - e^{g_t} S_{t-1} k_t),   S_t = e^{g_t} S_{t-1} + u_t k_t^T
//     o_t = scale S_t q_t = scale (e^{g_t} S_{t-1} q_t + u_t (k_t . q_t))
//
// with k and q divided by their lengths.  So both products with the state are with the one
// that is there, their sums over a row's lanes travel together, and the lengths are factors
// on sums.
//
// Memory is the bound for single tokens: 512 of them, 12 heads, take 122.8 us with an fp32 pool (97 %
// of a copy's rate) and 67.6 us with a bf16 one (89 %); 2 and 4 tokens a sequence take 124 and
// 133 us, and behind the fourth each costs about 23 us, instructions (with a bf16 pool about 23.5).
//
// A CTA of four warps has 32 or 128 value rows of one (sequence, head) state, a warp eight
// rows at a time, eight lanes a row: a lane has sixteen key columns of every fourth row, in 16-byte
// pieces, and the next eight rows' pieces are on their way.  What belongs to a token is made once
// a CTA, in shared memory: k, q and v in fp32, the lengths, the decay.

#include "kda_f32x2.cuh"
#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int D = kD;
constexpr int kWarps = 4;
constexpr int kRows = 8;                      // value rows per warp
constexpr int kParts = D / (kWarps * kRows);  // a CTA's least share of a (sequence, head)
constexpr int kAcross = 8;                    // lanes of a row
constexpr int kStep = 32 / kAcross;           // rows between a lane's
constexpr int kHeld = kRows / kStep;          // rows a lane has part of
constexpr int kPairs = D / kAcross / 2;       // pairs of columns of a row a lane has

struct alignas(16) Token {
    float k[D], q[D];  // a row's lanes' first four columns beside each other, then their next
    float v[D];
    float d, one;  // e^g = one + d
    float rk, rq;  // 1 / |k|, 1 / |q|
    float kq, beta;
    bool clears;
};

// A lane's columns of a state row: 16 bytes at its place in each 8 x 16 bytes.
template <class S>
struct Cols {
    static constexpr int kN = 16 / sizeof(S), kPieces = 2 * kPairs / kN;
    static __device__ __forceinline__ int at(int lane, int i) { return (i * kAcross + lane) * kN; }
    static __device__ __forceinline__ void load(const S* row, int lane, uint4 (&raw)[kPieces]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) raw[i] = __ldcs(reinterpret_cast<const uint4*>(row + at(lane, i)));
    }
    static __device__ __forceinline__ void get(const uint4 (&raw)[kPieces], f2 (&f)[kPairs]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float x[kN];
            reinterpret_cast<const rows::Piece<S, kN>&>(raw[i]).get(x);
#pragma unroll
            for (int j = 0; j < kN; j += 2) f[(i * kN + j) / 2] = pack2(x[j], x[j + 1]);
        }
    }
    static __device__ __forceinline__ void store(S* row, int lane, const f2 (&f)[kPairs]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float x[kN];
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
                const float2 y = unpack2(f[(i * kN + j) / 2]);
                x[j] = y.x, x[j + 1] = y.y;
            }
            rows::Piece<S, kN> p;
            p.set(x);
            __stcs(reinterpret_cast<uint4*>(row + at(lane, i)), reinterpret_cast<const uint4&>(p));
        }
    }
};

// A lane's share of a token's rows; a warp makes the token of it.
struct Rows {
    uint2 k, q, v;
    float g, beta;
};
__device__ __forceinline__ Rows load_token(const DeltaParams& p, int64_t t, int h, int lane) {
    const auto row = [&](const __nv_bfloat16* x, int64_t st, int64_t off) {
        return __ldg(reinterpret_cast<const uint2*>(x + t * st + off + 4 * lane));
    };
    return {row(p.k, p.k_st, (int64_t)(h / p.rep) * p.k_sh), row(p.q, p.q_st, (int64_t)(h / p.rep) * p.q_sh),
            row(p.v, p.v_st, (int64_t)h * p.v_sh), p.g[t * p.g_st + h], p.beta[t * p.H + h]};
}
template <class C>
__device__ __forceinline__ void make_token(const Rows& x, int lane, Token& to) {
    // its four columns are the `four`-th of lane `of`'s
    constexpr int kFours = C::kN / 4;  // of a piece
    const int piece = lane / (kFours * kAcross), of = lane / kFours % kAcross, four = piece * kFours + lane % kFours;
    const int at = (four * kAcross + of) * 4;
    const auto row = [&](uint2 w, float* out, f2 (&f)[2]) {
        f[0] = bf16x2(w.x), f[1] = bf16x2(w.y);
        *reinterpret_cast<ulonglong2*>(out) = make_ulonglong2(f[0], f[1]);
    };
    const float g = x.g;
    f2 k[2], q[2], v[2];
    row(x.k, to.k + at, k);
    row(x.q, to.q + at, q);
    row(x.v, to.v + 4 * lane, v);
    const auto dot = [](const f2 (&a)[2], const f2 (&b)[2]) {
        const float2 s = unpack2(fma2(a[0], b[0], mul2(a[1], b[1])));
        return s.x + s.y;
    };
    float kk = dot(k, k), qq = dot(q, q), kq = dot(k, q);
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
        kk += __shfl_xor_sync(0xffffffffu, kk, w);
        qq += __shfl_xor_sync(0xffffffffu, qq, w);
        kq += __shfl_xor_sync(0xffffffffu, kq, w);
    }
    // a decay near one as 1 + expm1(g): rounded to fp32, e^g alone would be off
    // by up to 2^-25 in the same direction at every token
    const bool slow = g > -0.5f;
    if (lane == 0) {
        to.d = slow ? expm1f(g) : expf(g);
        to.one = slow ? 1.f : 0.f;
        // (a sum that overflows has no length to divide by: as if the row were not finite)
        to.rk = kk < INFINITY ? 1.f / sqrtf(kk + 1e-6f) : NAN;
        to.rq = qq < INFINITY ? 1.f / sqrtf(qq + 1e-6f) : NAN;
        to.kq = kq;
        to.beta = x.beta;
        to.clears = g < kMinDecay;
    }
}

template <class S, int kPasses>
__global__ void __launch_bounds__(kWarps * 32, kPasses == 1 ? 6 : sizeof(S) == 4 ? 4 : 5)
kda_delta_step(const __grid_constant__ DeltaParams p) {
    using C = Cols<S>;
    extern __shared__ Token tokens[];  // of a sequence
    const int h = blockIdx.y, ctas = kParts / kPasses;
    const int n = p.short_list[blockIdx.x / ctas];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int at = lane % kAcross, part = lane / kAcross;  // rows part, part + 4 of the eight
    const int own = at % kHeld;                            // the held row whose output this lane makes
    int row = ((blockIdx.x % ctas) * kWarps + warp) * kRows * kPasses + part;
    const int t0 = p.cu[n], t1 = p.cu[n + 1], slot = p.idx[n];
    const bool has = p.has_init[n] != 0;
    const bool ok = slot >= 0 && slot < p.num_slots, init = ok && has;
    S* state = static_cast<S*>(p.pool) + (ok ? (size_t)slot * p.stride0 : 0) + ((size_t)h * D + row) * D;
    uint4 raw[kHeld][C::kPieces] = {};
    const auto load = [&](const S* from) {
#pragma unroll
        for (int r = 0; r < kHeld; ++r) C::load(from + r * kStep * D, at, raw[r]);
    };
    // (the token's rows first: its sums are made while the state is on its way)
    Rows rows = {};
    if (t0 + warp < t1) rows = load_token(p, t0 + warp, h, lane);
    if (init) load(state);
    for (int t = t0 + warp; t < t1; t += kWarps) {
        make_token<C>(rows, lane, tokens[t - t0]);
        if (t + kWarps < t1) rows = load_token(p, t + kWarps, h, lane);
    }
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass, row += kRows, state += kRows * D) {
        f2 s[kHeld][kPairs];
#pragma unroll
        for (int r = 0; r < kHeld; ++r) C::get(raw[r], s[r]);
        if (init && pass + 1 < kPasses) load(state + kRows * D);
#pragma unroll 1
        for (int t = t0; t < t1; ++t) {
            const Token& x = tokens[t - t0];
            if (x.clears) {  // whatever it held
#pragma unroll
                for (int r = 0; r < kHeld; ++r)
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) s[r][j] = 0;
            }
            // the state's products with k for the held rows, then with q
            f2 k[kPairs], sum[2 * kHeld] = {};
#pragma unroll
            for (int i = 0; i < kPairs; i += 2) {
                const int c = (i / 2 * kAcross + at) * 4;
                const ulonglong2 kk = *reinterpret_cast<const ulonglong2*>(x.k + c), qq = *reinterpret_cast<const ulonglong2*>(x.q + c);
                k[i] = kk.x, k[i + 1] = kk.y;
#pragma unroll
                for (int r = 0; r < kHeld; ++r) {
                    sum[r] = fma2(s[r][i + 1], kk.y, fma2(s[r][i], kk.x, sum[r]));
                    sum[kHeld + r] = fma2(s[r][i + 1], qq.y, fma2(s[r][i], qq.x, sum[kHeld + r]));
                }
            }
            // summed over a row's lanes: lane l keeps y[l % 4]
            float y[2 * kHeld];
#pragma unroll
            for (int i = 0; i < 2 * kHeld; ++i) {
                const float2 f = unpack2(sum[i]);
                y[i] = f.x + f.y;
            }
#pragma unroll
            for (int w = kHeld; w >= 1; w >>= 1) {
                const bool up = (lane & w) != 0;
#pragma unroll
                for (int j = 0; j < w; ++j) {
                    const float give = up ? y[j] : y[j + w];
                    const float keep = up ? y[j + w] : y[j];
                    y[j] = keep + __shfl_xor_sync(0xffffffffu, give, w);
                }
            }
            float all = y[0];
#pragma unroll
            for (int w = 2 * kHeld; w < kAcross; w <<= 1) all += __shfl_xor_sync(0xffffffffu, all, w);
            const int first = lane - at;
            const float sk = __shfl_sync(0xffffffffu, all, first + own);
            const float sq = __shfl_sync(0xffffffffu, all, first + kHeld + own);
            const int mine = row + own * kStep;
            const float e = x.one + x.d;
            const float uk = x.beta * (x.v[mine] - e * (x.rk * sk)) * x.rk;
            if (at < kHeld)
                p.out[((size_t)t * p.H + h) * D + mine] = __float2bfloat16_rn(p.scale * (x.rq * fmaf(uk, x.kq, e * sq)));
            const f2 d = pack2(x.d, x.d), one = pack2(x.one, x.one);
#pragma unroll
            for (int r = 0; r < kHeld; ++r) {
                const float ur = __shfl_sync(0xffffffffu, uk, first + r);
                const f2 u = pack2(ur, ur);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[r][j] = fma2(one, s[r][j], fma2(d, s[r][j], mul2(u, k[j])));
            }
        }
        if (ok && !(init && t1 <= t0)) {
#pragma unroll
            for (int r = 0; r < kHeld; ++r) C::store(state + r * kStep * D, at, s[r]);
        }
    }
    // Launched beside the walk, this grid may be over only once the walk is: its last CTA waits
    // (all of them waiting would keep their places on the SMs that the walk leaves free: 512
    // single tokens beside four prompts of 2048 then took 217 us)
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && threadIdx.x == 0)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.n_long == 0 && blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) write_status(p, lane);
}

template <class S, int kPasses>
cudaError_t launch(const DeltaParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.n_short * (kParts / kPasses), (unsigned)p.H);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = sizeof(Token) * (p.n_mid > 0 ? kDeltaStepMax : kShortMax);
    cfg.stream = s;
    // right behind the walk, beside its CTAs
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.n_long > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kda_delta_step<S, kPasses>, p);
}
template <class S>
cudaError_t launch(const DeltaParams& p, cudaStream_t s) {
    // Few states: 32 rows a CTA, for the latency; many: 128, whose loads overlap and which share
    // what belongs to a token.  12 heads, fp32 pool: 16 sequences of 4 tokens 10.4 and 12.5 us, 50
    // of them 18.6 and 16.8; 512 single tokens, bf16 pool: 82 and 68 us
    if ((int64_t)p.n_short * p.H * kParts <= 8 * num_sms()) return launch<S, 1>(p, s);
    return launch<S, kParts>(p, s);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaParams& p, cudaStream_t s) {
    if (p.n_short <= 0) return cudaSuccess;
    if (p.st_dtype == KDA_STATE_F32) return launch<float>(p, s);
    if (p.st_dtype == KDA_STATE_BF16) return launch<__nv_bfloat16>(p, s);
    return launch<__half>(p, s);
}

}  // namespace kda
