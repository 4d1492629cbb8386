// Internal interface of the operators beside the KDA forward (linear attention and the
// gated delta rule with a decay for each head, rotary positions alone and behind a norm of
// q and k, gated norm): the parameters
// their host checks (kda_ops_api.cu) hand to their kernels, and the services of
// kda_api.cu they share.
#pragma once

#include "kda.h"
#include "kda_internal.h"

namespace kda {

// Records the message kda_last_error() returns and gives back `code`.
int set_error(int code, const char* fmt, ...);

// The cached tables of a call's bounds (see kda_api.cu).  The tables stay valid
// on `stream` for work enqueued while the lock is held.
struct SeqTables {
    const int32_t* cu;          // [N + 1]
    const int32_t* long_list;   // sequences of more than step_max tokens, longest first
    const int32_t* short_list;  // the others
    int n_long, n_short;
    int n_mid;                  // of the others, those of more than kShortMax tokens
    // chunks of kC tokens of the long sequences: the first of each sequence [N + 1], and
    // each one's sequence and first token
    const int32_t *seq_off, *chunk_seq, *chunk_tok;
    int64_t n_chunks;
    // host: the bounds, and the long sequences and their lengths in long_list's order
    const int32_t* bounds;
    const int32_t* long_seqs;
    const int32_t* long_lens;
};
// Looks the bounds up (reading them back once without cu_host), calls
// enqueue(arg, tables) with the cache locked and marks the tables' use.  Sequences of at
// most step_max tokens are the short ones.
int with_seq_tables(const int32_t* cu_dev, const int32_t* cu_host, int32_t N, int64_t T,
                    int step_max, cudaStream_t stream, int (*enqueue)(void*, const SeqTables&), void* arg);
// The bounds' host check (message set on failure).
int check_bounds(const int32_t* cu_host, int32_t N, int64_t T);

struct LinParams {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;  // elements between tokens, between heads
    const float* g;   // log decays
    int64_t g_st;     // elements between tokens' decays: H, or 0 for one decay per head
    __nv_bfloat16* out;
    float scale;
    int H, rep, N;    // heads, heads per q/k head, sequences
    int64_t T;
    const int32_t* cu;
    const int32_t *long_list, *short_list;
    int n_long, n_short;
    // the first n_cut long sequences are cut into n_seg segments of seg_len tokens
    int n_cut, n_seg, seg_len;
    float* planes;  // [kLinPlanes][128 x 128] states of the segments
    float* kept;    // [kLinPlanes] decays over them
    int* status;
    void* pool;
    int64_t stride0;  // elements between slots
    const int32_t* idx;
    const uint8_t* has_init;
    int num_slots;
    int st_dtype;
};

#ifdef __CUDACC__
// The call's status word, by one warp of the first CTA of its first kernel, whichever that
// is: whether a sequence's slot is outside the pool.  So nothing has to clear the word
// before (a memset ahead of the kernel: 512 single tokens x 12 heads 123.2 us instead of
// 121.5).
__device__ __forceinline__ void write_status(const LinParams& p, int lane) {
    bool bad = false;
#pragma unroll 4
    for (int i = lane; i < p.N; i += 32) {
        const int slot = p.idx[i];
        bad |= slot < 0 || slot >= p.num_slots;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) *p.status = bad ? 4 : 0;
}
#endif

// Values below kMinDecay, where exp() is 0 in fp32, clear the state whatever it held; the
// clamp keeps sums of them finite.
constexpr float kMinDecay = -104.f;

// Segment states a call's workspace holds: a cut needs at most two for each SM.
constexpr int kLinPlanes = 2 * 152;
// Chunks of 128 tokens of the shortest sequence that is cut.
constexpr int kLinMinCut = 3;
// The cut sequences, by value in the kernels' parameters: of sequence seq[r], which has
// len[r] tokens from t0[r] on, the segments are first[r] .. first[r + 1] - 1.
constexpr int kLinCuts = kLinPlanes / 2;
struct LinCuts {
    int seq[kLinCuts], t0[kLinCuts], len[kLinCuts], first[kLinCuts + 1];
};
// Chooses n_cut, n_seg, seg_len and the cuts.
void lin_cut(LinParams& p, LinCuts& cuts, const SeqTables& t);
// Long sequences chunk by chunk (kda_lin_walk.cu); short ones token by token.
cudaError_t launch_lin_walk(const LinParams& p, const LinCuts& cuts, cudaStream_t s);
// `beside`: right after the walk, beside its last CTAs.
cudaError_t launch_lin_step(const LinParams& p, bool beside, cudaStream_t s);

// The gated delta rule: linear attention's parameters, the strengths of the writes, and the
// long sequences' chunks of kC tokens.
struct DeltaParams : LinParams {
    const float* beta;  // [T][H]
    const int32_t *seq_off, *chunk_seq, *chunk_tok;
    int64_t n_chunks;
    int n_mid;  // short sequences of more than kShortMax tokens
    uint8_t* blocks;  // [n_chunks][H] of kDeltaBlock bytes
    // of the cut sequences' segments: `planes` has two of [128 x 128] for each segment and
    // head, its state from zero (then the one that the next starts from) and its transition,
    // `kept` what the transition is to be multiplied by, or -1 where a token clears the state
};
// Sequences of at most so many tokens go token by token: 512 of 9, 12 and 16 tokens of 12 heads
// take 250, 318 and 413 us (fp32 pool; bf16 232, 301 and 396) instead of 467 (401) in a chunk, one of
// them 8.4 to 12.5 us instead of 15.
constexpr int kDeltaStepMax = 16;
// What kda_delta_chunk leaves for the walk of a chunk and head: fp32 scalars, and fp16 tiles in
// the swizzled layout of kda_device.cuh.
//   k   [64][128]  k times a power of two for each row
//   t   [2][64][64] the triangular inverse's high and low part
//   q   [64][128]  q times a power of two for each row
//   p   [64][64]   the scores' high part, each row over down
// The upper right quarters of t and p are not read as theirs: the scores' low part stands in them, its
// upper left quarter in t's high part, the lower left one in t's low part, the lower right one in p.  A walk without outputs needs the first kDeltaQ bytes.
struct DeltaScalars {
    float c[kC];      // e^{G_i} and k's length: k^ e^{G_i} = c k
    float beta[kC];
    float w[kC];      // half of e^{G_C - G_i} and k's length
    float down[kC];   // of a token's output
    float gamma;      // e^{G_C}
    int first_clear;  // first token that clears the state, kC if none
    unsigned clears[2];  // all of them
    float strongest;     // largest beta
    float unused[3];
};
constexpr int kDeltaK = 2048;
constexpr int kDeltaT = kDeltaK + 16384;
constexpr int kDeltaQ = kDeltaT + 16384;
constexpr int kDeltaP = kDeltaQ + 16384;
constexpr int kDeltaBlock = kDeltaP + 8192;
static_assert(sizeof(DeltaScalars) <= kDeltaK, "room for the scalars");
// At most so many chunks: only sequences of more than kDeltaStepMax tokens have any.
inline int64_t delta_chunks(int64_t T, int64_t N) {
    return T / kC + (T / (kDeltaStepMax + 1) < N ? T / (kDeltaStepMax + 1) : N);
}
// Segments times heads that a call's workspace holds: as many as are ever cut, or as there
// can be.  All segments but a sequence's last have kDeltaMinSeg chunks or more: m > 1
// segments have at least (m - 1) kDeltaMinSeg chunks' tokens, half as many each.
constexpr int kDeltaPlanes = 2 * 152;
constexpr int kDeltaMinSeg = 3;
inline int64_t delta_planes(int64_t T, int64_t H) {
    const int64_t n = T / (kDeltaMinSeg * kC / 2) * H;
    return n < kDeltaPlanes ? n : kDeltaPlanes;
}
// Chooses n_cut, n_seg, seg_len and the cuts.
void delta_cut(DeltaParams& p, LinCuts& cuts, const SeqTables& t);
// The sequences of at most kDeltaStepMax tokens (kda_delta_step.cu).
cudaError_t launch_delta_step(const DeltaParams& p, cudaStream_t s);
// The other sequences' chunks, each for itself (kda_delta_chunk.cu), and the walk over them
// (kda_delta_walk.cu).
cudaError_t launch_delta_chunk(const DeltaParams& p, cudaStream_t s);
cudaError_t launch_delta_walk(const DeltaParams& p, const LinCuts& cuts, cudaStream_t s);

struct RopeTensor {
    const void* in;
    void* out;
    int64_t in_st, in_sh, out_st, out_sh;
    int heads;
};
struct RopeParams {
    RopeTensor x[2];
    const void* pos;
    int pos64;
    const double* inv_freq;
    int64_t T;
    int D, rot;
    int interleaved;
    float factor;   // on cos and sin
    float sign;     // -1 for the inverse rotation
    int dtype;
};
cudaError_t launch_rope(const RopeParams& p, cudaStream_t s);
// Each row divided by the root of its mean square plus eps and multiplied by its head's
// weight before it is turned.
struct NormRopeParams : RopeParams {
    const float* weight[2];  // of the tensors' heads, or nullptr for ones
    int64_t weight_sh[2];    // elements between heads' weights, 0 for one of all
    float eps;
};
cudaError_t launch_qk_norm_rope(const NormRopeParams& p, cudaStream_t s);

struct NormParams {
    const void* x;
    const void* gate;
    const float* weight;
    void* out;
    int64_t x_st, x_sh, g_st, g_sh, o_st, o_sh;
    int64_t T;
    int H, D;
    float eps;
    int act;
    int dtype;
};
cudaError_t launch_gated_norm(const NormParams& p, cudaStream_t s);

}  // namespace kda
