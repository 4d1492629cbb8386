// Host side of the operators beside the KDA forward: argument checks and launches.

#include <algorithm>
#include <numeric>

#include "kda_ops.h"

namespace {

using kda::set_error;

int cuda_error(cudaError_t e, const char* what) {
    return set_error(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Bytes [lo, hi) that a [T][H][D] view touches.
struct Span {
    const char* name;
    uintptr_t lo, hi;
};
Span span(const char* name, const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{name, lo, p ? lo + bytes : lo};
}
Span view(const char* name, const void* p, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh,
          size_t elt) {
    const bool any = T > 0 && H > 0 && D > 0;
    return span(name, p, any ? (size_t)((T - 1) * st + (H - 1) * sh + D) * elt : 0);
}
bool overlap(const Span& a, const Span& b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// A [T][H][D] view of rows in memory, in bytes.
struct Rows {
    uintptr_t lo;
    int64_t T, H, D, st, sh;
};
Rows rows_of(const void* p, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh, size_t elt) {
    const int64_t e = (int64_t)elt;
    return Rows{reinterpret_cast<uintptr_t>(p), T, H, D * e, T > 1 ? st * e : 0, H > 1 ? sh * e : 0};
}
// The same rows in the same places, as where out is in.
bool same_rows(const Rows& a, const Rows& b) { return a.lo == b.lo && a.st == b.st && a.sh == b.sh; }
// Whether two views may share a byte.  They do not where their extents lie apart, or where
// both consist of blocks (rows, tokens with all heads, or heads with all tokens) that
// begin a multiple of one step apart and fit beside each other in that step: so views of
// one projection's output are told apart.
bool may_share(const Rows& a, const Rows& b) {
    if (a.T <= 0 || a.H <= 0 || b.T <= 0 || b.H <= 0) return false;
    const auto apart = [&](int64_t step, int64_t in_a, int64_t in_b) {
        if (step == 0) return a.lo + in_a <= b.lo || b.lo + in_b <= a.lo;
        const int64_t gap = a.lo <= b.lo ? (int64_t)((b.lo - a.lo) % step) : (step - (int64_t)((a.lo - b.lo) % step)) % step;
        return in_a <= gap && in_b <= step - gap;
    };
    const int64_t heads_a = (a.H - 1) * a.sh + a.D, heads_b = (b.H - 1) * b.sh + b.D;
    const int64_t tokens_a = (a.T - 1) * a.st + a.D, tokens_b = (b.T - 1) * b.st + b.D;
    return !(apart(0, tokens_a + heads_a - a.D, tokens_b + heads_b - b.D) ||
             apart(std::gcd(a.st, b.st), heads_a, heads_b) || apart(std::gcd(a.sh, b.sh), tokens_a, tokens_b) ||
             apart(std::gcd(std::gcd(a.st, b.st), std::gcd(a.sh, b.sh)), a.D, b.D));
}

size_t dtype_size(int dtype) { return dtype == KDA_F32 ? 4 : 2; }

// A [T][H][D] view's strides: rows apart by at least their length, no token or
// head inside another's rows, and the extent within 62 bits.
int check_view(const char* name, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh) {
    if (st < 0 || sh < 0 || (H > 1 && sh < D) || (T > 1 && st < D))
        return set_error(KDA_ERR_INVALID_ARG, "%s: strides %lld, %lld are smaller than a row of %lld",
                         name, (long long)st, (long long)sh, (long long)D);
    const int64_t lim = int64_t(1) << 58;
    if ((T > 1 && st > lim / T) || (H > 1 && sh > lim / H))
        return set_error(KDA_ERR_INVALID_ARG, "%s: strides %lld, %lld are out of range", name,
                         (long long)st, (long long)sh);
    return KDA_OK;
}
// The rows of a view that is written may not lie in each other.
int check_written(const char* name, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh) {
    if (T > 1 && H > 1 && st < (H - 1) * sh + D && sh < (T - 1) * st + D)
        return set_error(KDA_ERR_INVALID_ARG, "%s: strides %lld, %lld make its rows overlap", name,
                         (long long)st, (long long)sh);
    return KDA_OK;
}

int check_tokens(int64_t T) {
    if (T < 0) return set_error(KDA_ERR_INVALID_ARG, "total_tokens = %lld < 0", (long long)T);
    if (T > INT32_MAX - 1024)
        return set_error(KDA_ERR_INVALID_ARG, "total_tokens = %lld exceeds the int32 token index",
                         (long long)T);
    return KDA_OK;
}

// A call over packed sequences and the pool of their states: linear attention's and the
// gated delta rule's.
struct PackedCall {
    const void *q, *k, *v;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;
    const float* g;
    int per_token;
    const float* beta;
    bool has_beta;
    const int32_t *cu, *cu_host;
    int N;
    int64_t T;
    int H, Hk;
    void* pool;
    int64_t stride0;
    int slots;
    const int32_t* idx;
    const uint8_t* has_init;
    void* out;
    float scale;
    int state_dtype;
    void* ws;
    size_t ws_bytes;
};

// Its checks; `need` bytes of workspace.  (A call without sequences is right and has nothing
// to do.)
int check_packed(const PackedCall& a, size_t need) {
    constexpr int D = kda::kD;
    const int64_t T = a.T;
    const int H = a.H, Hk = a.Hk, N = a.N;
    int rc = check_tokens(T);
    if (rc != KDA_OK) return rc;
    if (N < 0) return set_error(KDA_ERR_INVALID_ARG, "num_seqs = %d < 0", N);
    if (H <= 0 || H > 65535) return set_error(KDA_ERR_INVALID_ARG, "num_heads = %d out of range", H);
    if (Hk <= 0 || H % Hk != 0)
        return set_error(KDA_ERR_INVALID_ARG, "num_qk_heads = %d does not divide num_heads = %d", Hk, H);
    if (N == 0 && T != 0) return set_error(KDA_ERR_INVALID_ARG, "tokens without sequences");
    if (a.state_dtype < KDA_STATE_F32 || a.state_dtype > KDA_STATE_F16)
        return set_error(KDA_ERR_UNSUPPORTED, "state_dtype %d not supported (0 fp32, 1 bf16, 2 fp16)",
                         a.state_dtype);
    if (!a.cu && !a.cu_host)
        return set_error(KDA_ERR_INVALID_ARG, "cu_seqlens and cu_seqlens_host are both NULL");
    if (a.cu_host) {
        rc = kda::check_bounds(a.cu_host, N, T);
        if (rc != KDA_OK) return rc;
    }
    const size_t g_bytes = sizeof(float) * (size_t)H * (a.per_token ? (size_t)T : 1);
    const Span so = view("out", a.out, T, H, D, (int64_t)H * D, D, 2);
    Span ins[5] = {span("q", a.q, 0), span("k", a.k, 0), span("v", a.v, 0), span("log_decay", a.g, 0),
                   span("beta", a.beta, 0)};
    if (T > 0) {
        if (!a.q || !a.k || !a.v || !a.g || !a.out)
            return set_error(KDA_ERR_INVALID_ARG, "a q/k/v/log_decay/out pointer is NULL");
        if (a.has_beta && !a.beta) return set_error(KDA_ERR_INVALID_ARG, "beta is NULL");
        const void* base[3] = {a.q, a.k, a.v};
        const char* name[3] = {"q", "k", "v"};
        const int64_t st[3] = {a.q_st, a.k_st, a.v_st};
        const int64_t sh[3] = {a.q_sh, a.k_sh, a.v_sh};
        for (int i = 0; i < 3; ++i) {
            const int heads = i == 2 ? H : Hk;
            rc = check_view(name[i], T, heads, D, st[i], sh[i]);
            if (rc != KDA_OK) return rc;
            if (!aligned(base[i], 16) || st[i] % 8 != 0 || sh[i] % 8 != 0)
                return set_error(KDA_ERR_UNSUPPORTED,
                                 "%s and its strides must be 16-byte aligned", name[i]);
            ins[i] = view(name[i], base[i], T, heads, D, st[i], sh[i], 2);
        }
        if (!aligned(a.out, 16)) return set_error(KDA_ERR_UNSUPPORTED, "out is not 16-byte aligned");
        if (!aligned(a.g, 4))
            return set_error(KDA_ERR_UNSUPPORTED, "log_decay is not 4-byte aligned");
        if (!aligned(a.beta, 4)) return set_error(KDA_ERR_UNSUPPORTED, "beta is not 4-byte aligned");
        ins[3] = span("log_decay", a.g, g_bytes);
        ins[4] = span("beta", a.beta, sizeof(float) * (size_t)H * (size_t)T);
        for (const Span& r : ins)
            if (overlap(so, r)) return set_error(KDA_ERR_INVALID_ARG, "out overlaps %s", r.name);
    }
    if (N == 0) return KDA_OK;
    if (!a.ws || a.ws_bytes < need)
        return set_error(KDA_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed",
                         a.ws ? a.ws_bytes : (size_t)0, need);
    if (!aligned(a.ws, 256))
        return set_error(KDA_ERR_UNSUPPORTED, "workspace is not 256-byte aligned");
    const int64_t plane = (int64_t)H * D * D;
    if (!a.pool || !a.idx || !a.has_init)
        return set_error(KDA_ERR_INVALID_ARG,
                         "state_cache, state_indices and has_initial_state are required");
    if (a.slots < N)
        return set_error(KDA_ERR_INVALID_ARG, "num_slots %d < num_seqs %d (slots are distinct)",
                         a.slots, N);
    if (a.stride0 < plane || a.stride0 > (int64_t(1) << 58) / a.slots)
        return set_error(KDA_ERR_INVALID_ARG,
                         "state_stride0 %lld is smaller than the slot plane H*V*K = %lld, or out of range",
                         (long long)a.stride0, (long long)plane);
    const size_t elt = dtype_size(a.state_dtype);
    if (!aligned(a.pool, 16) || ((size_t)a.stride0 * elt) % 16 != 0)
        return set_error(KDA_ERR_UNSUPPORTED,
                         "state_cache and its slot stride must be 16-byte aligned");
    const Span sp = span("state_cache", a.pool,
                         ((size_t)(a.slots - 1) * (size_t)a.stride0 + (size_t)plane) * elt);
    const Span sw = span("workspace", a.ws, need);
    const Span with_pool[] = {ins[0], ins[1], ins[2], ins[3], ins[4], so, sw};
    for (const Span& r : with_pool)
        if (overlap(sp, r)) return set_error(KDA_ERR_INVALID_ARG, "state_cache overlaps %s", r.name);
    const Span with_ws[] = {ins[0], ins[1], ins[2], ins[3], ins[4], so};
    for (const Span& r : with_ws)
        if (overlap(sw, r)) return set_error(KDA_ERR_INVALID_ARG, "workspace overlaps %s", r.name);
    return KDA_OK;
}

void set_params(const PackedCall& a, kda::LinParams& p) {
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k = static_cast<const __nv_bfloat16*>(a.k);
    p.v = static_cast<const __nv_bfloat16*>(a.v);
    p.q_st = a.q_st, p.q_sh = a.q_sh;
    p.k_st = a.k_st, p.k_sh = a.k_sh;
    p.v_st = a.v_st, p.v_sh = a.v_sh;
    p.g = a.g;
    p.g_st = a.per_token ? a.H : 0;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.scale = a.scale;
    p.H = a.H, p.rep = a.H / a.Hk, p.N = a.N, p.T = a.T;
    p.status = static_cast<int*>(a.ws);
    p.pool = a.pool;
    p.stride0 = a.stride0;
    p.idx = a.idx;
    p.has_init = a.has_init;
    p.num_slots = a.slots;
    p.st_dtype = a.state_dtype;
}

struct LinCall {
    kda::LinParams p;
    cudaStream_t stream;
};

int enqueue_lin(void* arg, const kda::SeqTables& t) {
    LinCall& c = *static_cast<LinCall*>(arg);
    kda::LinParams& p = c.p;
    p.cu = t.cu;
    p.long_list = t.long_list;
    p.short_list = t.short_list;
    p.n_long = t.n_long;
    p.n_short = t.n_short;
    kda::LinCuts cuts;
    kda::lin_cut(p, cuts, t);
    cudaError_t e = kda::launch_lin_walk(p, cuts, c.stream);
    if (e == cudaSuccess) e = kda::launch_lin_step(p, p.n_long > 0, c.stream);
    return e == cudaSuccess ? KDA_OK : cuda_error(e, "kernel launch");
}

struct DeltaCall {
    kda::DeltaParams p;
    cudaStream_t stream;
};

// Whether the host's bounds say that no sequence has chunks, so that nothing of the workspace
// but the header is used.
bool token_by_token(const int32_t* cu_host, int32_t N) {
    if (!cu_host) return false;
    for (int32_t n = 0; n < N; ++n)
        if ((int64_t)cu_host[n + 1] - cu_host[n] > kda::kDeltaStepMax) return false;
    return true;
}

int enqueue_delta(void* arg, const kda::SeqTables& t) {
    DeltaCall& c = *static_cast<DeltaCall*>(arg);
    kda::DeltaParams& p = c.p;
    p.cu = t.cu;
    p.long_list = t.long_list;
    p.short_list = t.short_list;
    p.n_long = t.n_long;
    p.n_short = t.n_short;
    p.n_mid = t.n_mid;
    p.seq_off = t.seq_off;
    p.chunk_seq = t.chunk_seq;
    p.chunk_tok = t.chunk_tok;
    p.n_chunks = t.n_chunks;
    kda::LinCuts cuts;
    kda::delta_cut(p, cuts, t);
    cudaError_t e = kda::launch_delta_chunk(p, c.stream);
    if (e == cudaSuccess) e = kda::launch_delta_walk(p, cuts, c.stream);
    if (e == cudaSuccess) e = kda::launch_delta_step(p, c.stream);
    return e == cudaSuccess ? KDA_OK : cuda_error(e, "kernel launch");
}

// The checks of kda_rope and kda_qk_norm_rope, and their parameters; p.T stays 0 where there
// is nothing to do.  `weights` are read beside the tensors (two, empty ones where there are none).
int check_rope(const char* what, const kda_rope_tensor* tensors, int32_t num_tensors, const Span* weights,
               const void* positions, int position_bytes, const double* inv_freq, int64_t total_tokens,
               int32_t head_dim, int32_t rot_dim, int layout, float factor, int inverse, int dtype,
               kda::RopeParams& p) {
    const int64_t T = total_tokens;
    int rc = check_tokens(T);
    if (rc != KDA_OK) return rc;
    if (!tensors || num_tensors < 1 || num_tensors > 2)
        return set_error(KDA_ERR_INVALID_ARG, "%s takes 1 or 2 tensors, got %d", what, num_tensors);
    if (head_dim < 1 || head_dim > 1024)
        return set_error(KDA_ERR_UNSUPPORTED, "head_dim %d outside [1, 1024]", head_dim);
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 != 0)
        return set_error(KDA_ERR_INVALID_ARG, "rot_dim %d is not an even number in [0, head_dim = %d]",
                         rot_dim, head_dim);
    if (layout != KDA_ROPE_HALF && layout != KDA_ROPE_INTERLEAVED)
        return set_error(KDA_ERR_UNSUPPORTED, "layout %d not supported", layout);
    if (dtype < KDA_F32 || dtype > KDA_F16)
        return set_error(KDA_ERR_UNSUPPORTED, "dtype %d not supported (0 fp32, 1 bf16, 2 fp16)", dtype);
    if (position_bytes != 4 && position_bytes != 8)
        return set_error(KDA_ERR_UNSUPPORTED, "positions of %d bytes (4 or 8)", position_bytes);
    const size_t elt = dtype_size(dtype);
    Span out[2] = {};
    Rows from[2] = {}, to[2] = {};
    for (int i = 0; i < num_tensors; ++i) {
        const kda_rope_tensor& x = tensors[i];
        if (x.num_heads < 0 || x.num_heads > 65535)
            return set_error(KDA_ERR_INVALID_ARG, "num_heads = %d out of range", x.num_heads);
        if (x.num_heads == 0 || T == 0) continue;
        if (!x.in || !x.out) return set_error(KDA_ERR_INVALID_ARG, "tensor %d has a NULL pointer", i);
        if (!aligned(x.in, elt) || !aligned(x.out, elt))
            return set_error(KDA_ERR_UNSUPPORTED, "tensor %d is not %zu-byte aligned", i, elt);
        rc = check_view("in", T, x.num_heads, head_dim, x.in_stride_t, x.in_stride_h);
        if (rc == KDA_OK) rc = check_view("out", T, x.num_heads, head_dim, x.out_stride_t, x.out_stride_h);
        if (rc == KDA_OK) rc = check_written("out", T, x.num_heads, head_dim, x.out_stride_t, x.out_stride_h);
        if (rc != KDA_OK) return rc;
        out[i] = view("out", x.out, T, x.num_heads, head_dim, x.out_stride_t, x.out_stride_h, elt);
        from[i] = rows_of(x.in, T, x.num_heads, head_dim, x.in_stride_t, x.in_stride_h, elt);
        to[i] = rows_of(x.out, T, x.num_heads, head_dim, x.out_stride_t, x.out_stride_h, elt);
        if (!same_rows(from[i], to[i]) && may_share(from[i], to[i]))
            return set_error(KDA_ERR_INVALID_ARG, "out of tensor %d overlaps its in", i);
        p.x[i] = kda::RopeTensor{x.in, x.out, x.in_stride_t, x.in_stride_h,
                                 x.out_stride_t, x.out_stride_h, x.num_heads};
    }
    if (p.x[0].heads + p.x[1].heads == 0 || T == 0) return KDA_OK;
    // one launch reads and writes both tensors in any order
    for (int i = 0; i < 2; ++i)
        if (may_share(to[i], from[1 - i]))
            return set_error(KDA_ERR_INVALID_ARG, "out of tensor %d overlaps the in of tensor %d", i, 1 - i);
    if (may_share(to[0], to[1])) return set_error(KDA_ERR_INVALID_ARG, "the outs of the two tensors overlap");
    if (!positions || (rot_dim > 0 && !inv_freq))
        return set_error(KDA_ERR_INVALID_ARG, "positions and inv_freq are required");
    if (!aligned(positions, (size_t)position_bytes) || !aligned(inv_freq, 8))
        return set_error(KDA_ERR_UNSUPPORTED, "positions or inv_freq is not aligned to its type");
    const Span sp = span("positions", positions, (size_t)T * position_bytes);
    const Span sf = span("inv_freq", inv_freq, (size_t)(rot_dim / 2) * 8);
    for (int i = 0; i < num_tensors; ++i) {
        if (overlap(out[i], sp) || overlap(out[i], sf))
            return set_error(KDA_ERR_INVALID_ARG, "out of tensor %d overlaps the positions or inv_freq", i);
        for (int j = 0; j < num_tensors; ++j)
            if (overlap(out[i], weights[j]))
                return set_error(KDA_ERR_INVALID_ARG, "out of tensor %d overlaps a weight", i);
    }
    p.pos = positions;
    p.pos64 = position_bytes == 8;
    p.inv_freq = inv_freq;
    p.T = T;
    p.D = head_dim;
    p.rot = rot_dim;
    p.interleaved = layout == KDA_ROPE_INTERLEAVED;
    p.factor = factor;
    p.sign = inverse ? -1.f : 1.f;
    p.dtype = dtype;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_lin_attn_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t num_heads) {
    if (total_tokens < 0 || num_seqs <= 0 || num_heads <= 0) return 0;
    if (total_tokens <= (kda::kLinMinCut - 1) * 128) return kda::kWsHeader;  // nothing is cut
    return kda::kWsHeader + (size_t)kda::kLinPlanes * (kda::kD * kda::kD + 64) * sizeof(float);
}

int kda_lin_attn_fwd(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                     int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                     int64_t v_stride_h, const float* log_decay, int decay_per_token,
                     const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int32_t num_seqs,
                     int64_t total_tokens, int32_t num_heads, int32_t num_qk_heads,
                     void* state_cache, int64_t state_stride0, int32_t num_slots,
                     const int32_t* state_indices, const uint8_t* has_initial_state, void* out,
                     float scale, int state_dtype, void* workspace, size_t workspace_bytes,
                     kda_stream_t stream) {
    const PackedCall a{q, k, v, q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h,
                       log_decay, decay_per_token, nullptr, false, cu_seqlens, cu_seqlens_host, num_seqs,
                       total_tokens, num_heads, num_qk_heads, state_cache, state_stride0, num_slots,
                       state_indices, has_initial_state, out, scale, state_dtype, workspace, workspace_bytes};
    const int rc = check_packed(a, kda_lin_attn_workspace_size(total_tokens, num_seqs, num_heads));
    if (rc != KDA_OK || num_seqs == 0) return rc;
    LinCall c{};
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    set_params(a, c.p);
    c.p.kept = reinterpret_cast<float*>(static_cast<char*>(workspace) + kda::kWsHeader);
    c.p.planes = c.p.kept + 64 * kda::kLinPlanes;
    return kda::with_seq_tables(cu_seqlens, cu_seqlens_host, num_seqs, total_tokens, kda::kShortMax, c.stream, enqueue_lin, &c);
}

size_t kda_gated_delta_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t num_heads) {
    if (total_tokens < 0 || num_seqs <= 0 || num_heads <= 0) return 0;
    return kda::kWsHeader + (size_t)kda::delta_chunks(total_tokens, num_seqs) * num_heads * kda::kDeltaBlock +
           (size_t)kda::delta_planes(total_tokens, num_heads) * (2 * kda::kD * kda::kD + 64) * sizeof(float);
}

int kda_gated_delta_fwd(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                        int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                        int64_t v_stride_h, const float* log_decay, int decay_per_token, const float* beta,
                        const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int32_t num_seqs,
                        int64_t total_tokens, int32_t num_heads, int32_t num_qk_heads,
                        void* state_cache, int64_t state_stride0, int32_t num_slots,
                        const int32_t* state_indices, const uint8_t* has_initial_state, void* out,
                        float scale, int state_dtype, void* workspace, size_t workspace_bytes,
                        kda_stream_t stream) {
    const PackedCall a{q, k, v, q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h,
                       log_decay, decay_per_token, beta, true, cu_seqlens, cu_seqlens_host, num_seqs,
                       total_tokens, num_heads, num_qk_heads, state_cache, state_stride0, num_slots,
                       state_indices, has_initial_state, out, scale, state_dtype, workspace, workspace_bytes};
    size_t need = kda_gated_delta_workspace_size(total_tokens, num_seqs, num_heads);
    if (token_by_token(cu_seqlens_host, num_seqs)) need = std::min(need, (size_t)kda::kWsHeader);
    const int rc = check_packed(a, need);
    if (rc != KDA_OK || num_seqs == 0) return rc;
    DeltaCall c{};
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    set_params(a, c.p);
    c.p.beta = beta;
    c.p.blocks = static_cast<uint8_t*>(workspace) + kda::kWsHeader;
    c.p.planes = reinterpret_cast<float*>(
        c.p.blocks + (size_t)kda::delta_chunks(total_tokens, num_seqs) * num_heads * kda::kDeltaBlock);
    c.p.kept = c.p.planes + (size_t)kda::delta_planes(total_tokens, num_heads) * 2 * kda::kD * kda::kD;
    return kda::with_seq_tables(cu_seqlens, cu_seqlens_host, num_seqs, total_tokens, kda::kDeltaStepMax, c.stream, enqueue_delta, &c);
}

int kda_rope(const kda_rope_tensor* tensors, int32_t num_tensors, const void* positions,
             int position_bytes, const double* inv_freq, int64_t total_tokens, int32_t head_dim,
             int32_t rot_dim, int layout, float factor, int inverse, int dtype,
             kda_stream_t stream) {
    kda::RopeParams p{};
    const Span none[2] = {};
    const int rc = check_rope("kda_rope", tensors, num_tensors, none, positions, position_bytes, inv_freq,
                              total_tokens, head_dim, rot_dim, layout, factor, inverse, dtype, p);
    if (rc != KDA_OK || p.T == 0) return rc;
    const cudaError_t e = kda::launch_rope(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_error(e, "kda_rope");
}

int kda_qk_norm_rope(const kda_norm_rope_tensor* tensors, int32_t num_tensors, float eps,
                     const void* positions, int position_bytes, const double* inv_freq,
                     int64_t total_tokens, int32_t head_dim, int32_t rot_dim, int layout, float factor,
                     int dtype, kda_stream_t stream) {
    if (!tensors || num_tensors < 1 || num_tensors > 2)
        return set_error(KDA_ERR_INVALID_ARG, "kda_qk_norm_rope takes 1 or 2 tensors, got %d", num_tensors);
    if (!(eps >= 0.f)) return set_error(KDA_ERR_INVALID_ARG, "eps %g is negative", (double)eps);
    kda::NormRopeParams p{};
    kda_rope_tensor x[2] = {};
    Span weights[2] = {};
    for (int i = 0; i < num_tensors; ++i) {
        const kda_norm_rope_tensor& t = tensors[i];
        x[i] = t.x;
        if (!t.weight || t.x.num_heads <= 0 || head_dim < 1) continue;
        if (!aligned(t.weight, 4)) return set_error(KDA_ERR_UNSUPPORTED, "weight %d is not 4-byte aligned", i);
        const int64_t sh = t.x.num_heads > 1 ? t.weight_stride_h : 0;
        if (sh < 0 || sh > (int64_t(1) << 40))
            return set_error(KDA_ERR_INVALID_ARG, "weight_stride_h %lld is out of range", (long long)sh);
        weights[i] = span("weight", t.weight, (size_t)((t.x.num_heads - 1) * sh + head_dim) * 4);
        p.weight[i] = t.weight;
        p.weight_sh[i] = sh;
    }
    p.eps = eps;
    const int rc = check_rope("kda_qk_norm_rope", x, num_tensors, weights, positions, position_bytes, inv_freq,
                              total_tokens, head_dim, rot_dim, layout, factor, 0, dtype, p);
    if (rc != KDA_OK || p.T == 0) return rc;
    const cudaError_t e = kda::launch_qk_norm_rope(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_error(e, "kda_qk_norm_rope");
}

int kda_gated_norm(const void* x, int64_t x_stride_t, int64_t x_stride_h, const void* gate,
                   int64_t gate_stride_t, int64_t gate_stride_h, const float* weight, void* out,
                   int64_t out_stride_t, int64_t out_stride_h, int64_t total_tokens,
                   int32_t num_heads, int32_t head_dim, float eps, int activation, int dtype,
                   kda_stream_t stream) {
    const int64_t T = total_tokens;
    const int H = num_heads, D = head_dim;
    int rc = check_tokens(T);
    if (rc != KDA_OK) return rc;
    if (H < 0 || H > 65535) return set_error(KDA_ERR_INVALID_ARG, "num_heads = %d out of range", H);
    if (D < 1 || D > 8192) return set_error(KDA_ERR_UNSUPPORTED, "head_dim %d outside [1, 8192]", D);
    if (!(eps >= 0.f)) return set_error(KDA_ERR_INVALID_ARG, "eps %g is negative", (double)eps);
    if (activation < KDA_ACT_NONE || activation > KDA_ACT_SILU)
        return set_error(KDA_ERR_UNSUPPORTED, "activation %d not supported", activation);
    if (dtype < KDA_F32 || dtype > KDA_F16)
        return set_error(KDA_ERR_UNSUPPORTED, "dtype %d not supported (0 fp32, 1 bf16, 2 fp16)", dtype);
    if (T == 0 || H == 0) return KDA_OK;
    if (!x || !out) return set_error(KDA_ERR_INVALID_ARG, "x or out is NULL");
    const size_t elt = dtype_size(dtype);
    if (!aligned(x, elt) || !aligned(out, elt) || !aligned(gate, elt) || !aligned(weight, 4))
        return set_error(KDA_ERR_UNSUPPORTED, "a pointer is not aligned to its type");
    rc = check_view("x", T, H, D, x_stride_t, x_stride_h);
    if (rc == KDA_OK && gate) rc = check_view("gate", T, H, D, gate_stride_t, gate_stride_h);
    if (rc == KDA_OK) rc = check_view("out", T, H, D, out_stride_t, out_stride_h);
    if (rc == KDA_OK) rc = check_written("out", T, H, D, out_stride_t, out_stride_h);
    if (rc != KDA_OK) return rc;
    const Rows rx = rows_of(x, T, H, D, x_stride_t, x_stride_h, elt);
    const Rows ro = rows_of(out, T, H, D, out_stride_t, out_stride_h, elt);
    const Span so = view("out", out, T, H, D, out_stride_t, out_stride_h, elt);
    const Span sw = span("weight", weight, (size_t)D * 4);
    if (!same_rows(rx, ro) && may_share(rx, ro)) return set_error(KDA_ERR_INVALID_ARG, "out overlaps x");
    if (gate && may_share(rows_of(gate, T, H, D, gate_stride_t, gate_stride_h, elt), ro))
        return set_error(KDA_ERR_INVALID_ARG, "out overlaps gate");
    if (weight && overlap(so, sw)) return set_error(KDA_ERR_INVALID_ARG, "out overlaps weight");
    const kda::NormParams p{x,           gate,         weight,        out,
                            x_stride_t,  x_stride_h,   gate_stride_t, gate_stride_h,
                            out_stride_t, out_stride_h, T,            H,
                            D,           eps,          activation,    dtype};
    const cudaError_t e = kda::launch_gated_norm(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_error(e, "kda_gated_norm");
}

}  // extern "C"
