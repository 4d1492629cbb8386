// Internal interface of the operators beside the KDA forward (linear attention
// with a decay for each head, rotary positions, gated norm): the parameters
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
    const int32_t* long_list;   // sequences of more than kShortMax tokens, longest first
    const int32_t* short_list;  // the others
    int n_long, n_short;
    // host: the bounds, and the long sequences and their lengths in long_list's order
    const int32_t* bounds;
    const int32_t* long_seqs;
    const int32_t* long_lens;
};
// Looks the bounds up (reading them back once without cu_host), calls
// enqueue(arg, tables) with the cache locked and marks the tables' use.
int with_seq_tables(const int32_t* cu_dev, const int32_t* cu_host, int32_t N, int64_t T,
                    cudaStream_t stream, int (*enqueue)(void*, const SeqTables&), void* arg);
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
