// The gated delta rule's walk over a sequence's chunks on the tensor cores (tcgen05,
// accumulators in tensor memory).  For a chunk of C = 64 tokens with incoming state S (V x K),
// with kda_delta_chunk's k, q, T and P:
//
//     X = S [k q]^T                   128 x 128 x 128
//     R = beta (V - c X_k)            in registers
//     U = R T^T,  O = X_q + U P^T     128 x 64 x 64
//     S' = e^{G_C} S + (w U) k        128 x 128 x 64
//
// All products have the value rows as their M: a thread keeps a quarter of a row of S in fp32
// registers, and everything it rounds or scales belongs to that row.  Rows are independent of
// each other but for the keys, so nothing has to be summed across threads.
//
// A CTA walks its share of the (sequence, head) pairs one after the other, its warps in roles:
//   0-15   operands: four warps for each 32 rows
//   16-19  the output rows
//   20     issues the products and the blocks' copies, and says what comes next
//   21-23  turn v over, so that a value row's tokens lie beside each other, and find its
//          largest
// The chain X, R, U, dS, S of one chunk after the other is the bound: 5 K cycles, 2.6 us, of which
// its products are 1.8 K (46 cycles for one of 128 x 64 x 16, 65 for 128 x 128 x 16, A in tensor
// memory) and their three round trips 1.1 K; the rest are the makers' instructions.  The outputs'
// products, about 1.3 K, run meanwhile.  The roles keep all else off the chain, and an SM has one
// CTA, whose registers then let a warp have all its values of a step in flight (two CTAs of half as
// many registers took 10.7 K cycles a chunk).
// An item's begin and end take 7 to 10 us.  12 heads: 16384 tokens in segments take 106 us (first
// pass) and 69, 128 sequences of 117,555 tokens 488 us, the tensor pipe active for 23 and 28 % of the time.
//
// Rounding.  Operands are fp16: k and q exactly, up to their rows' powers of two and but for entries
// below 2^-17 of a row's length; S, R, U, T and P as the sum of two (22 bits; with one, a state would
// be off by 2^-12, and an output, whose terms may cancel, by as much of what the state held).
// S, R and U of a row are scaled by one power of two, from a bound that holds for all three: with
// |v| <= m and beta <= b in the chunk, |R| <= b (m + |S|) and |U| <= b (m + |S| + 64 b m), since
// I - beta k k^T does not lengthen a row for beta in [0, 2] and a token adds at most b m; |S| itself
// is bounded by that of a chunk before and 64 b m of that chunk, so that no thread waits for
// another's maximum.  The bound is up to 2^10 too large; fp16's exponent has room for it: a term
// is kept to 2^-25 of 2^14, the bound.  What is smaller than 2^-29 or so of the most that the
// chunk writes is lost beside it.
//
// Infinities and NaN stay in their value row (in v or the state) or sequence and head (in k)
// from their token on: R's entries that are not finite become zero for the products and their
// rows get NaN afterwards, until a token clears the state.

#include "kda_device.cuh"
#include "kda_f32x2.cuh"
#include "kda_ops.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

using namespace dev;

constexpr int D = kD;
constexpr int C = kC;
constexpr int kThreads = 768;
constexpr int kMakers = 16;  // warps 0 .. 15, four parts of each row
constexpr int kWriters = 4;  // warps 16 .. 19
constexpr int kIssuer = 20;
constexpr int kTurners = 3;  // warps 21 .. 23
constexpr int kKeys = D / 4, kToks = C / 4;  // of a maker

// Shared memory.
constexpr int kTile = C * D * 2;
constexpr int kTiles = kDeltaBlock - kDeltaK;
constexpr int kSmTiles = 0;                      // [2] the tiles of kda_delta_chunk's blocks
constexpr int kSmScalars = kSmTiles + 2 * kTiles; // [4] their scalars, which the output rows read last
constexpr int kSmV = kSmScalars + 4 * kDeltaK;   // v as it comes
constexpr int kSmVT = kSmV + kTile;              // [2][128][64] v by value rows, 16-byte pieces swizzled
constexpr int kSmVMax = kSmVT + 2 * kTile;       // [2][128] largest |v| of a value row
constexpr int kSmSMax = kSmVMax + 2 * D * 4;     // [2][4][128] largest |S| of a quarter of a row
constexpr int kSmBad = kSmSMax + 8 * D * 4;      // [4][128][4] tokens whose R is not finite, 16 bits a maker
constexpr int kSmInv = kSmBad + 4 * D * 8;       // [4][128] the rows' scales undone
constexpr int kSmBar = kSmInv + 4 * D * 4;
enum Bar {
    kFull = 0,              // [2] block there
    kFullV = kFull + 2,
    kXDone,
    kUDone,
    kDDone,
    kODone,                 // [2] by the place of O
    kEnd = kODone + 2,
    kTurned,                // [2] v turned over, its largest found
    kOEmpty = kTurned + 2,  // [2] O read
    kVEmpty = kOEmpty + 2,  // [2] v's rows read
    kSReady = kVEmpty + 2,  // [2] half of each part's keys
    kRReady = kSReady + 2,
    kUReady,
    kPReady,                // U itself there, in R's place
    kMax,                   // an item's first state's largest values there
    kItem,                  // [2] item there
    kItemFree = kItem + 2,  // [2] and done with
    kNumBars = kItemFree + 2
};
constexpr int kSmMisc = kSmBar + kNumBars * 8;   // abort flag, tensor-memory base
// A sequence and head, or a segment of one, to be walked.
struct Item {
    int h, t0, len, chunks;
    bool outputs, values;  // makes outputs; has values (not the rows of a transition)
    const uint8_t* blocks; // of the first chunk
    const void* from;      // the pool's state that it starts from, or nullptr
    const float* begins;   // a segment's
    void* state;           // where its state goes: the pool, or nullptr
    float* plane;          // or the segment's
    float* kept;           // what a transition is to be multiplied by, or nullptr
};
constexpr int kSmItem = kSmMisc + 16;
constexpr int kSmStage = (kSmItem + 2 * (int)sizeof(Item) + 127) / 128 * 128;  // [16][32][64 bytes] for each maker warp
constexpr int kSmemBytes = kSmStage + kMakers * 2048;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
static_assert(kTiles % 1024 == 0 && kDeltaK % 1024 == 0 && kSmV % 1024 == 0 && kSmVT % 1024 == 0 && kSmBar % 8 == 0, "alignment");

// Tensor memory columns.  Operands have, for 16 of their K, 8 columns of the high part and 8
// of the low one.
constexpr uint32_t kTmCols = 512;
constexpr uint32_t kTmS = 0;
constexpr uint32_t kTmR = 128;
constexpr uint32_t kTmU = 192;
constexpr uint32_t kTmX = 256;    // X_k; then, with U's place, dS
constexpr uint32_t kTmUAcc = 320;
constexpr uint32_t kTmDS = 256;
constexpr uint32_t kTmO = 384;    // [2]

constexpr uint32_t kIdescKK = mma_idesc(0, 0, 0, 128, 64);  // B K-major
constexpr uint32_t kIdescHalf = mma_idesc(0, 0, 0, 128, 32);
constexpr uint32_t kIdescKM = mma_idesc(0, 0, 1, 128, 128); // B MN-major

extern __shared__ __align__(1024) uint8_t smem[];

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Sixteen of K, from 16 s on, of a lower triangle's columns: of the right half the lower rows alone.
__device__ __forceinline__ void mma_lower(uint32_t d, uint32_t a, uint64_t b, int s, uint32_t accumulate) {
    if (s < 2)
        mma_f16_ts(d, a, b + 2 * s, kIdescKK, accumulate);
    else
        mma_f16_ts(d + C / 2, a, b + 2 * s + (C / 2 * 128 >> 4), kIdescHalf, accumulate);
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint64_t* bar(int i) { return reinterpret_cast<uint64_t*>(smem + kSmBar) + i; }
__device__ __forceinline__ volatile int& abort_flag() { return *reinterpret_cast<volatile int*>(smem + kSmMisc); }

// Sixteen columns of this thread's lane, there on return.
__device__ __forceinline__ void load16(uint32_t a, f2 (&v)[8]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(a)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
__device__ __forceinline__ void load32(uint32_t a, f2 (&v)[16]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Sixteen values as the sum of two fp16 each, as an operand's columns.
__device__ __forceinline__ void store_split(uint32_t a, const f2 (&x)[8]) {
    uint32_t r[16];
    const f2 minus = pack2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = unpack2(x[i]);
        const __half2 hi = __floats2half2_rn(f.x, f.y);
        r[i] = reinterpret_cast<const uint32_t&>(hi);
        const float2 h = __half22float2(hi);
        const float2 lo = unpack2(fma2(pack2(h.x, h.y), minus, x[i]));
        r[8 + i] = pack_half2(lo.x, lo.y);
    }
    tmem_st16(a, r);
}

// max(m, |a|, |b|), NaN if one is.
__device__ __forceinline__ float max_abs(float m, f2 x) {
    const float2 f = unpack2(x);
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(f.x), "f"(f.y));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// 2^(14 - e) for a bound below 2^e, and its inverse.
__device__ __forceinline__ float scale_of(float bound, float& inverse) {
    const int e = max(14, min(254, (int)(__float_as_uint(bound) >> 23)));
    inverse = __uint_as_float((uint32_t)(e - 13) << 23);
    return __uint_as_float((uint32_t)(267 - e) << 23);
}

// Waits for a phase; gives up after about a second, or once another warp has.  A whole
// warp goes on or leaves together.
__device__ __forceinline__ bool wait(int b, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar(b), parity & 1))) return true;
        if (__any_sync(0xffffffffu, abort_flag())) return false;
    }
    abort_flag() = 1;
    return false;
}
// One arrival of a whole warp, its tensor-memory accesses before it.
__device__ __forceinline__ void arrive_warp(int b, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
}
__device__ __forceinline__ uint8_t* tiles(int c) { return smem + kSmTiles + (c & 1) * kTiles; }
__device__ __forceinline__ uint8_t* scalars_at(int c) { return smem + kSmScalars + (c & 3) * kDeltaK; }
__device__ __forceinline__ const DeltaScalars* scalars(int c) { return reinterpret_cast<const DeltaScalars*>(scalars_at(c)); }
__device__ __forceinline__ volatile float* vmax(int c) { return reinterpret_cast<volatile float*>(smem + kSmVMax) + (c & 1) * D; }
__device__ __forceinline__ volatile float* smax_of(int c, int part) {
    return reinterpret_cast<volatile float*>(smem + kSmSMax) + ((c & 1) * 4 + part) * D;
}
__device__ __forceinline__ volatile uint2* bad_of(int c, int row) {
    return reinterpret_cast<volatile uint2*>(smem + kSmBad) + (c & 3) * D + row;
}
__device__ __forceinline__ volatile float* inv_of(int c) { return reinterpret_cast<volatile float*>(smem + kSmInv) + (c & 3) * D; }

__device__ __forceinline__ volatile const Item& ring(int k) { return *(reinterpret_cast<const Item*>(smem + kSmItem) + (k & 1)); }

// This CTA's items: the list, longest first, dealt out in turns of alternating direction.
__device__ __forceinline__ int item_of(int k) {
    const int g = gridDim.x, b = blockIdx.x;
    return k * g + (k & 1 ? g - 1 - b : b);
}
__device__ __forceinline__ bool next_item(int k, int total) { return item_of(k) < total && wait(kItem + (k & 1), k >> 1); }
__device__ __forceinline__ void done_with(int k, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kItemFree + (k & 1)));
}

// Item i of the walk over all sequences, or (local) of the segments' first pass: all of a cut
// sequence but its last segment from zero, then all but its first and last from the identity.
template <class S>
__device__ __forceinline__ Item item_at(const DeltaParams& p, const LinCuts& cuts, bool local, int i) {
    Item w;
    const int after = p.n_seg - p.n_cut;  // segments that are not their sequence's first
    w.h = i % p.H;
    i /= p.H;
    w.values = !local || i < after;
    bool first = true, last = true;
    int n, at = 0, plane = 0, r = 0;
    if (i < after || local) {
        const int skip = w.values ? 1 : 2;  // segments of each sequence that have no such item
        if (!w.values) i -= after;
        while (i >= cuts.first[r + 1] - skip * (r + 1)) ++r;
        const int g = i - (cuts.first[r] - skip * r) + (local && w.values ? 0 : 1);
        n = cuts.seq[r];
        w.t0 = cuts.t0[r] + g * p.seg_len;
        w.len = min(p.seg_len, cuts.len[r] - g * p.seg_len);
        at = g * (p.seg_len / C);
        first = g == 0;
        last = g + 1 == cuts.first[r + 1] - cuts.first[r];
        plane = ((cuts.first[r] + g) * p.H + w.h) * 2;
    } else {
        n = p.long_list[p.n_cut + i - after];
        w.t0 = p.cu[n];
        w.len = p.cu[n + 1] - w.t0;
    }
    w.outputs = first || !local;
    w.chunks = (w.len + C - 1) / C;
    w.blocks = p.blocks + (((int64_t)p.seq_off[n] + at) * p.H + w.h) * kDeltaBlock;
    const int slot = p.idx[n];
    S* const state = slot >= 0 && slot < p.num_slots
                         ? static_cast<S*>(p.pool) + (size_t)slot * p.stride0 + (size_t)w.h * D * D : nullptr;
    w.from = first && state && p.has_init[n] != 0 ? state : nullptr;
    w.begins = first || local ? nullptr : p.planes + (size_t)(plane - 2 * p.H) * D * D;
    w.state = last && !local ? state : nullptr;
    w.plane = local ? p.planes + (size_t)(plane + !w.values) * D * D : nullptr;
    w.kept = w.values ? nullptr : p.kept + plane / 2;
    return w;
}

// Warp 20: items, products, and the copies of the chunks' blocks.  Chunks are counted over all
// items here as elsewhere: n.
template <class S>
struct Issuer {
    const DeltaParams& p;
    const LinCuts& cuts;
    const bool local, lead;
    const int total;
    int loads = 0, at_item = 0, at_chunk = 0, outs = 0;

    __device__ __forceinline__ void publish(int k) {
        if (item_of(k) >= total) return;
        if (lead) {
            const Item w = item_at<S>(p, cuts, local, item_of(k));
            *(reinterpret_cast<Item*>(smem + kSmItem) + (k & 1)) = w;
            if (w.from) {
                const char* from = static_cast<const char*>(w.from);
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(D * D * sizeof(S))) : "memory");
            }
            mbar_arrive(bar(kItem + (k & 1)));
        }
        __syncwarp();
    }
    // The next chunk's block, if its item is known.
    __device__ __forceinline__ void load(int known) {
        if (at_item > known || item_of(at_item) >= total) return;
        if (lead) {
            const volatile Item& w = ring(at_item);
            const uint32_t bytes = w.outputs ? kDeltaBlock : kDeltaQ;
            mbar_arrive_expect_tx(bar(kFull + (loads & 1)), bytes);
            const uint8_t* from = w.blocks + (int64_t)at_chunk * p.H * kDeltaBlock;
            bulk_g2s(scalars_at(loads), from, kDeltaK, bar(kFull + (loads & 1)));
            bulk_g2s(tiles(loads), from + kDeltaK, bytes - kDeltaK, bar(kFull + (loads & 1)));
        }
        __syncwarp();
        ++loads;
        if (++at_chunk == ring(at_item).chunks) at_chunk = 0, ++at_item;
    }
    __device__ __forceinline__ bool go(uint32_t tm) {
        constexpr uint64_t kHalf = kTile / 2 >> 4;  // descriptors' addresses count 16 bytes
        publish(0);
        grid_dep_wait();                            // the blocks are written
        load(0);
        load(0);
        int n = 0;
#pragma unroll 1
        for (int k = 0; item_of(k) < total; ++k) {
            const int chunks = ring(k).chunks;
            const bool outputs = ring(k).outputs;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, ++n) {
                const uint32_t at = smem_u32(tiles(n)), o = tm + kTmO + (outs & 1) * C;
                if (!wait(kFull + (n & 1), n >> 1)) return false;
                // each maker's first 16 keys, then its others
                const uint64_t kd = sw128_desc(at, 0, 1024);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (!wait(kSReady + b, n)) return false;
                    tc_fence_after();
                    if (lead) {
#pragma unroll
                        for (int s = b; s < 8; s += 2)
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                mma_f16_ts(tm + kTmX, tm + kTmS + 16 * s + 8 * part, kd + (s >> 2) * kHalf + (s & 3) * 2, kIdescKK,
                                           s > 0 || part > 0);
                        if (b == 1) mma_commit(bar(kXDone));
                    }
                    __syncwarp();
                }
                // the chunk before's products are over (without outputs they were with dS)
                if (outs > 0 && !wait(kODone + ((outs - 1) & 1), (outs - 1) >> 1)) return false;
                if (c == 0) {
                    if (k > 0 && item_of(k + 1) < total && !wait(kItemFree + ((k - 1) & 1), (k - 1) >> 1)) return false;
                    publish(k + 1);
                }
                if (loads < n + 2) load(k + 1);
                // (the outputs' products fill the pipe's pauses: X_q here, while R is made, P U behind dS; with
                // half of X_q behind U 128 sequences' walk took 589 us instead of 584)
                constexpr uint64_t kNext = C * C * 2 >> 4;
                const uint64_t qd = sw128_desc(at + kDeltaQ - kDeltaK, 0, 1024), pd = sw128_desc(at + kDeltaP - kDeltaK, 0, 1024);
                const uint64_t td = sw128_desc(at + kDeltaT - kDeltaK, 0, 1024);
                // The outputs of the chunk before last are read: O's place is free, and of the rings of four no
                // place is written that a chunk of which outputs are still to be read has.
                const int read = outputs ? outs - 1 : outs;
                if (read > 0 && !wait(kOEmpty + ((read - 1) & 1), (read - 1) >> 1)) return false;
                if (outputs) {
                    tc_fence_after();
                    if (lead) {
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int s = 0; s < 8; ++s)
                                mma_f16_ts(o, tm + kTmS + 16 * s + 8 * part, qd + (s >> 2) * kHalf + (s & 3) * 2, kIdescKK,
                                           s > 0 || part > 0);
                    }
                    __syncwarp();
                }
                if (!wait(kRReady, n)) return false;
                tc_fence_after();
                if (lead) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        mma_lower(tm + kTmUAcc, tm + kTmR + 16 * s, td + kNext, s, s > 0);
                        mma_lower(tm + kTmUAcc, tm + kTmR + 16 * s + 8, td, s, 1);
                        mma_lower(tm + kTmUAcc, tm + kTmR + 16 * s, td, s, 1);
                    }
                    mma_commit(bar(kUDone));
                }
                __syncwarp();
                if (!wait(kUReady, n)) return false;
                tc_fence_after();
                if (lead) {
                    const uint64_t km = sw128_desc(at, kTile / 2, 1024);
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint64_t b = km + s * (2048 >> 4);
                        mma_f16_ts(tm + kTmDS, tm + kTmU + 16 * s + 8, b, kIdescKM, s > 0);
                        mma_f16_ts(tm + kTmDS, tm + kTmU + 16 * s, b, kIdescKM, 1);
                    }
                    mma_commit(bar(kDDone));
                }
                __syncwarp();
                if (outputs) {
                    if (!wait(kPReady, outs)) return false;
                    tc_fence_after();
                    if (lead) {
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const uint64_t right = 2 * (2 + s);
                            mma_f16_ts(o, tm + kTmR + 16 * s, td + right, kIdescHalf, 1);
                            mma_f16_ts(o + C / 2, tm + kTmR + 16 * s, td + kNext + right, kIdescHalf, 1);
                            mma_f16_ts(o + C / 2, tm + kTmR + 16 * (2 + s), pd + right, kIdescHalf, 1);
                        }
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            mma_lower(o, tm + kTmR + 16 * s + 8, pd, s, 1);
                            mma_lower(o, tm + kTmR + 16 * s, pd, s, 1);
                        }
                        mma_commit(bar(kODone + (outs & 1)));
                    }
                    __syncwarp();
                    ++outs;
                }
            }
        }
        return true;
    }
    // Its copies and products in flight end before the CTA does.
    __device__ __forceinline__ void finish() {
        if (lead) mma_commit(bar(kEnd));
        __syncwarp();
        bool ok = mbar_wait(bar(kEnd), 0);
        for (int i = 0; i < 2; ++i) {
            const int n = (loads + 1 - i) / 2;  // loads of slot i
            if (n > 0) ok = mbar_wait(bar(kFull + i), (n - 1) & 1) && ok;
        }
        if (!ok) abort_flag() = 1;
    }
};

// Warps 21-23: v by value rows, and each row's largest finite |v|.  Tokens past the sequence's
// end are zeros.
struct Turner {
    const CUtensorMap* map;
    const int total, which, lane;
    int loads = 0;

    __device__ __forceinline__ void load_v(const volatile Item& w, int c) {
        if (lane == 0) {
            const int h = w.h, t = w.t0 + c * C;
            mbar_arrive_expect_tx(bar(kFullV), kTile);
            tma_load_3d(smem + kSmV, map, bar(kFullV), 0, h, t);
            tma_load_3d(smem + kSmV + kTile / 2, map, bar(kFullV), 64, h, t);
        }
        __syncwarp();
        ++loads;
    }
    __device__ __forceinline__ bool go() {
        int n = 0;
#pragma unroll 1
        for (int k = 0; item_of(k) < total; ++k) {
            if (!wait(kItem + (k & 1), k >> 1)) return false;
            const volatile Item& w = ring(k);
            const int chunks = w.values ? w.chunks : 0, len = w.len;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, ++n) {
                if (which == 0 && loads == n) load_v(w, c);
                if (!wait(kFullV, n) || (n > 1 && !wait(kVEmpty + (n & 1), (n >> 1) - 1))) return false;
                const int live = len - c * C;
                const uint32_t from = smem_u32(smem + kSmV), to = smem_u32(smem + kSmVT) + (n & 1) * kTile;
#pragma unroll 1
                for (int g = which; g < D / 8; g += kTurners) {
                    uint32_t r[8];
                    const int piece = ((g & 7) ^ (lane & 7)) << 4;
                    const uint32_t a = from + (g >> 3) * (kTile / 2) + lane * 128 + piece;
                    ldsm_x4_t(a, r[0], r[1], r[2], r[3]);
                    ldsm_x4_t(a + 32 * 128, r[4], r[5], r[6], r[7]);
                    const int t = 2 * (lane & 3);
                    if (live < C) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (8 * i + t >= live) r[i] &= 0xFFFF0000u;
                            if (8 * i + t + 1 >= live) r[i] &= 0x0000FFFFu;
                        }
                    }
                    const int row = 8 * g + (lane & 7);
                    const uint32_t b = to + row * 128;
                    stsm_x4(b + (((lane >> 3) ^ (lane & 7)) << 4), r[0], r[1], r[2], r[3]);
                    stsm_x4(b + (((4 + (lane >> 3)) ^ (lane & 7)) << 4), r[4], r[5], r[6], r[7]);
                    __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = __hmax2_nan(m, __habs2(reinterpret_cast<const __nv_bfloat162&>(r[i])));
                    float f = max_nan(__low2float(m), __high2float(m));
                    if (__any_sync(0xffffffffu, !finite(f))) {
                        f = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float x = fabsf(__uint_as_float(r[i] << 16)), y = fabsf(__uint_as_float(r[i] & 0xFFFF0000u));
                            f = fmaxf(f, finite(x) ? x : 0.f);
                            f = fmaxf(f, finite(y) ? y : 0.f);
                        }
                    }
                    f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 1));
                    f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 2));
                    if ((lane & 3) == 0) vmax(n)[8 * g + (lane >> 2)] = f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kTurned + (n & 1)));
                if (which == 0) {
                    // all have read v: the next chunk's, of this item or the one after
                    if (!wait(kTurned + (n & 1), n >> 1)) return false;
                    if (c + 1 < chunks) {
                        load_v(w, c + 1);
                    } else if (item_of(k + 1) < total) {
                        if (!wait(kItem + ((k + 1) & 1), (k + 1) >> 1)) return false;
                        if (ring(k + 1).values) load_v(ring(k + 1), 0);
                    }
                }
            }
            done_with(k, lane);
        }
        return true;
    }
    __device__ __forceinline__ void finish() {
        if (loads > 0 && !mbar_wait(bar(kFullV), (loads - 1) & 1)) abort_flag() = 1;
    }
};

// Whether tokens up to i leave a row without a finite value: bit i of the result.  `bad` are
// the tokens that bring one in, `clears` those that clear the state.
__device__ __noinline__ uint2 poisoned(uint2 bad, uint2 clears) {
    uint2 r = make_uint2(0, 0);
    bool on = false;
    for (int i = 0; i < C; ++i) {
        const unsigned bit = 1u << (i & 31);
        if ((i < 32 ? clears.x : clears.y) & bit) on = false;
        if ((i < 32 ? bad.x : bad.y) & bit) on = true;
        if (on) (i < 32 ? r.x : r.y) |= bit;
    }
    return r;
}

// Warps 16-19: a thread has an output row's 64 tokens.  n counts the chunks with outputs, all
// the chunks of all items.
__device__ __forceinline__ bool write(const DeltaParams& p, int total, uint32_t base, int warp, int lane) {
    const int row = 32 * (warp & 3) + lane;
    const uint32_t tm = base + ((uint32_t)(32 * (warp & 3)) << 16) + kTmO;
    const int64_t st = (int64_t)p.H * D;
    int n = 0, all = 0;
#pragma unroll 1
    for (int k = 0; item_of(k) < total; ++k) {
        if (!wait(kItem + (k & 1), k >> 1)) return false;
        const int h = ring(k).h, t0 = ring(k).t0, len = ring(k).len, chunks = ring(k).chunks;
        const bool outputs = ring(k).outputs;
        done_with(k, lane);
        if (!outputs) {
            all += chunks;
            continue;
        }
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, ++n, ++all) {
            if (!wait(kODone + (n & 1), n >> 1)) return false;
            tc_fence_after();
            const DeltaScalars* sc = scalars(all);
            uint2 spoils = make_uint2(bad_of(all, row)->x, bad_of(all, row)->y);
            const bool spoilt = __any_sync(0xffffffffu, (spoils.x | spoils.y) != 0);
            if (spoilt) spoils = poisoned(spoils, make_uint2(sc->clears[0], sc->clears[1]));
            const int live = len - c * C;
            const bool plain = !spoilt && live >= C;
            const float f = inv_of(all)[row] * p.scale;
            __nv_bfloat16* o = p.out + ((int64_t)(t0 + c * C) * p.H + h) * D + row;
#pragma unroll 1
            for (int b = 0; b < C; b += 16) {
                f2 x[8];
                load16(tm + (n & 1) * C + b, x);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 d = *reinterpret_cast<const float4*>(sc->down + b + 2 * i);
                    x[i] = mul2(mul2(x[i], pack2(d.x, d.y)), pack2(f, f));
                    x[i + 1] = mul2(mul2(x[i + 1], pack2(d.z, d.w)), pack2(f, f));
                }
                if (plain) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 y = unpack2(x[i]);
                        o[0] = __float2bfloat16_rn(y.x);
                        o[st] = __float2bfloat16_rn(y.y);
                        o += 2 * st;
                    }
                    continue;
                }
                const unsigned lost = (b < 32 ? spoils.x : spoils.y) >> (b & 31);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 y = unpack2(x[i]);
                    if (b + 2 * i < live) o[0] = __float2bfloat16_rn(lost >> (2 * i) & 1 ? NAN : y.x);
                    if (b + 2 * i + 1 < live) o[st] = __float2bfloat16_rn(lost >> (2 * i + 1) & 1 ? NAN : y.y);
                    o += 2 * st;
                }
            }
            arrive_warp(kOEmpty + (n & 1), lane);
        }
    }
    return true;
}

// Where a segment's state has an entry: a thread's 32 keys by fours, those of all threads beside
// each other.
__host__ __device__ constexpr int state_at(int row, int key) { return ((key % kKeys / 4) * 4 * D + key / kKeys * D + row) * 4 + key % 4; }
// And a transition: row j's fours in another order, so that the chain's fragments, of eight
// columns and rows two apart, lie in different banks.
__host__ __device__ constexpr int phi_at(int j, int k) { return state_at(j ^ (k / 4 & 1), k); }

// 32 rows' keys of a warp between its threads, a row each, and the pool: 64 bytes of a row by
// four lanes (by threads, an access has 32 lines: 2 us each way).
__device__ __forceinline__ uint8_t* staged(int warp, int row, int piece) {
    return smem + kSmStage + warp * 2048 + row * 64 + ((piece ^ (row >> 1 & 3)) << 4);
}
template <class S>
__device__ __forceinline__ void load_state(const S* from, int warp, int lane, f2 (&s)[kKeys / 2]) {
    constexpr int N = 16 / sizeof(S), H = 4 * N;  // values of a piece, of 64 bytes
    from += (32 * (warp & 3) + (lane >> 2)) * D + (warp >> 2) * kKeys + (lane & 3) * N;
    uint4 x[kKeys / H][4];
#pragma unroll
    for (int b = 0; b < kKeys / H; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[b][i] = *reinterpret_cast<const uint4*>(from + 8 * i * D + b * H);
#pragma unroll
    for (int b = 0; b < kKeys / H; ++b) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(staged(warp, 8 * i + (lane >> 2), lane & 3)) = x[b][i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[N];
            rows::load<S, N>(reinterpret_cast<const S*>(staged(warp, lane, i))).get(f);
#pragma unroll
            for (int j = 0; j < N; j += 2) s[(b * H + i * N + j) / 2] = pack2(f[j], f[j + 1]);
        }
    }
}
template <class S>
__device__ __forceinline__ void store_state(S* to, int warp, int lane, const f2 (&s)[kKeys / 2]) {
    constexpr int N = 16 / sizeof(S), H = 4 * N;
    to += (32 * (warp & 3) + (lane >> 2)) * D + (warp >> 2) * kKeys + (lane & 3) * N;
#pragma unroll
    for (int b = 0; b < kKeys / H; ++b) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[N];
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const float2 y = unpack2(s[(b * H + i * N + j) / 2]);
                f[j] = y.x, f[j + 1] = y.y;
            }
            rows::Piece<S, N> x;
            x.set(f);
            rows::store<S, N>(reinterpret_cast<S*>(staged(warp, lane, i)), x);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(to + 8 * i * D + b * H) = *reinterpret_cast<const uint4*>(staged(warp, 8 * i + (lane >> 2), lane & 3));
    }
}

// Warps 0-15: a thread has a quarter of value row `row`: 32 keys, 16 of a chunk's tokens.
// Walks an item, the CTA's chunks n on and its chunks with values nv on, and leaves the state
// in s, whether a token cleared it and the decay over all.
template <class S>
__device__ __forceinline__ bool make(const DeltaParams& p, int k, int& n, int& nv, uint32_t base, int warp, int lane,
                                     f2 (&s)[kKeys / 2], bool& cleared, float& decay) {
    const int chunks = ring(k).chunks;
    const bool values = ring(k).values, outputs = ring(k).outputs;
    const int part = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t tm = base + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll
    for (int i = 0; i < kKeys / 2; ++i) s[i] = 0;
    const S* const from = static_cast<const S*>(ring(k).from);
    const float* const begins = ring(k).begins;
    if (from) {
        load_state(from, warp, lane, s);
    } else if (begins) {
        grid_dep_wait();
#pragma unroll
        for (int i = 0; i < kKeys; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(begins + state_at(row, part * kKeys + i));
            s[i / 2] = pack2(f.x, f.y), s[i / 2 + 1] = pack2(f.z, f.w);
        }
    } else if (!values) {
#pragma unroll
        for (int i = 0; i < kKeys; i += 2) {
            const int key = part * kKeys + i;
            s[i / 2] = pack2(key == row ? 1.f : 0.f, key + 1 == row ? 1.f : 0.f);
        }
    }
    cleared = false;
    decay = 1.f;
    float smax = 0.f;
#pragma unroll
    for (int i = 0; i < kKeys / 2; ++i) smax = max_abs(smax, s[i]);
    smax_of(n, part)[row] = smax;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kMax));
    if (!wait(kMax, k)) return false;
    // the largest |S| of the row a chunk ago; what a chunk adds to |S| at most
    auto of_row = [&](int c) {
        return max_nan(max_nan(smax_of(c, 0)[row], smax_of(c, 1)[row]), max_nan(smax_of(c, 2)[row], smax_of(c, 3)[row]));
    };
    float was = of_row(n), adds, scale, inv;
    auto rescale = [&](int at, int at_v, float grown) {
        const float l = 11.32f * (finite(was) ? was : 0.f) + grown;  // |S| <= sqrt(128) max
        const float b = scalars(at)->strongest, m = values ? vmax(at_v)[row] : 0.f;
        adds = 64.f * b * m;
        // (v itself has to stay finite when it is scaled)
        scale = scale_of(fmaxf(fmaxf(l, b * (m + l + adds)), 0x1p-60f * m), inv);
    };
    // 16 keys of S's operand; of a row with infinities or NaN as zeros
    auto store_s = [&](int b, bool live) {
        f2 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = live ? mul2(s[8 * b + i], pack2(scale, scale)) : 0;
        store_split(tm + kTmS + kKeys * part + 16 * b, x);
    };
    if ((values && !wait(kTurned + (nv & 1), nv >> 1)) || !wait(kFull + (n & 1), n >> 1)) return false;
    rescale(n, nv, 0.f);
    // (the whole row's: with one entry that is not finite, the scale bounds none of the others)
    store_s(0, finite(was));
    store_s(1, finite(was));
    tmem_wait_st();
    arrive_warp(kSReady, lane);
    arrive_warp(kSReady + 1, lane);

#pragma unroll 1
    for (int c = 0; c < chunks; ++c, ++n) {
        const DeltaScalars* sc = scalars(n);
        // R
        const int clear = sc->first_clear;
        cleared = cleared || clear < C;
        // y0 + bc X, made of all but X while its products run
        f2 y0[8], bc[8];
        {
            uint4 v[2] = {};
            if (values) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    v[j] = *reinterpret_cast<const uint4*>(smem + kSmVT + (nv & 1) * kTile + row * 128 + (((2 * part + j) ^ (row & 7)) << 4));
            }
            const uint32_t vw[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float4 ci = *reinterpret_cast<const float4*>(sc->c + kToks * part + 2 * i);
                const float4 bi = *reinterpret_cast<const float4*>(sc->beta + kToks * part + 2 * i);
                const f2 cc[2] = {pack2(-ci.x, -ci.y), pack2(-ci.z, -ci.w)};
                const f2 bb[2] = {pack2(bi.x, bi.y), pack2(bi.z, bi.w)};
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const f2 vv = pack2(__uint_as_float(vw[i + u] << 16), __uint_as_float(vw[i + u] & 0xFFFF0000u));
                    y0[i + u] = mul2(bb[u], mul2(vv, pack2(scale, scale)));
                    bc[i + u] = mul2(bb[u], cc[u]);
                }
            }
        }
        if (!wait(kXDone, n)) return false;
        tc_fence_after();
        {
            f2 x[8];
            if (c > 0) was = of_row(n);
            load16(tm + kTmX + kToks * part, x);
            const bool dead = !finite(was);
            const int mine = clear - kToks * part;  // among this thread's tokens
            if (mine < kToks) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = unpack2(x[i]);
                    x[i] = pack2(2 * i < mine ? f.x : 0.f, 2 * i + 1 < mine ? f.y : 0.f);
                }
            }
            f2 check = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = fma2(bc[i], x[i], y0[i]);
                check = fma2(x[i], 0, check);
            }
            unsigned bad = 0;
            const float2 ch = unpack2(check);
            if (__any_sync(0xffffffffu, ch.x + ch.y != 0.f || dead)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float2 f = unpack2(x[i]);
                    if (!finite(f.x) || (dead && 2 * i < mine)) bad |= 1u << (2 * i), f.x = 0.f;
                    if (!finite(f.y) || (dead && 2 * i + 1 < mine)) bad |= 2u << (2 * i), f.y = 0.f;
                    x[i] = pack2(f.x, f.y);
                }
            }
            store_split(tm + kTmR + kToks * part, x);
            reinterpret_cast<volatile uint16_t*>(bad_of(n, row))[part] = (uint16_t)bad;
            if (part == 0) inv_of(n)[row] = inv;
        }
        tmem_wait_st();
        arrive_warp(kRReady, lane);
        if (values) {
            if (lane == 0) mbar_arrive(bar(kVEmpty + (nv & 1)));
            ++nv;
        }
        // U
        if (!wait(kUDone, n)) return false;
        tc_fence_after();
        {
            f2 x[8], y[8];
            load16(tm + kTmUAcc + kToks * part, x);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float4 wi = *reinterpret_cast<const float4*>(sc->w + kToks * part + 2 * i);
                y[i] = mul2(x[i], pack2(wi.x, wi.y));
                y[i + 1] = mul2(x[i + 1], pack2(wi.z, wi.w));
            }
            store_split(tm + kTmU + kToks * part, y);
            tmem_wait_st();
            arrive_warp(kUReady, lane);
            // for the outputs U itself, in R's place, on its way while dS's products run
            if (outputs) store_split(tm + kTmR + kToks * part, x);
        }
        // S
        const bool more = c + 1 < chunks;
        decay *= sc->gamma;
        const f2 gamma = pack2(sc->gamma, sc->gamma), back = pack2(2.f * inv, 2.f * inv);
        if (clear < C) {
#pragma unroll
            for (int i = 0; i < kKeys / 2; ++i) s[i] = 0;
        }
        bool lost = false;
        {
            const uint2 bad = make_uint2(bad_of(n, row)->x, bad_of(n, row)->y);
            if (__any_sync(0xffffffffu, (bad.x | bad.y) != 0)) lost = poisoned(bad, make_uint2(sc->clears[0], sc->clears[1])).y >> 31;
        }
        if (more) {
            if ((values && !wait(kTurned + (nv & 1), nv >> 1)) || !wait(kFull + ((n + 1) & 1), (n + 1) >> 1)) return false;
            rescale(n + 1, nv, adds);
        }
        if (outputs) {
            tmem_wait_st();
            arrive_warp(kPReady, lane);
        }
        if (!wait(kDDone, n)) return false;
        tc_fence_after();
        smax = 0.f;
        {
            f2 x[16];
            load32(tm + kTmDS + kKeys * part, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[i] = fma2(gamma, s[i], mul2(x[i], back));
                smax = max_abs(smax, s[i]);
            }
        }
        if (lost) smax = NAN;
        // (rare, and before the operand is given away: rows with infinities or NaN)
        const bool strange = __any_sync(0xffffffffu, !finite(smax));
        if (lost) {
#pragma unroll
            for (int i = 0; i < kKeys / 2; ++i) s[i] = pack2(NAN, NAN);
        }
        if (more) {
            smax_of(n + 1, part)[row] = smax;
            if (!strange) {
                store_s(0, true);
                tmem_wait_st();
                arrive_warp(kSReady, lane);
                store_s(1, true);
            } else {
                store_s(0, finite(smax));
                tmem_wait_st();
                arrive_warp(kSReady, lane);
                store_s(1, finite(smax));
            }
            tmem_wait_st();
            arrive_warp(kSReady + 1, lane);
        }
    }
    return true;
}

template <class S>
__global__ void __launch_bounds__(kThreads, 1)
kda_delta_walk(const __grid_constant__ DeltaParams p, const __grid_constant__ CUtensorMap v_map,
               const __grid_constant__ LinCuts cuts, bool local, int total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* const base = reinterpret_cast<uint32_t*>(smem + kSmMisc + 8);
    if (threadIdx.x == 0) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        for (int i = 0; i < kNumBars; ++i)
            mbar_init(bar(i), i >= kItemFree ? kMakers + kWriters + kTurners : i >= kItem ? 1 : i >= kVEmpty ? kMakers
                              : i >= kOEmpty ? kWriters : i >= kTurned ? kTurners : 1);
        abort_flag() = 0;
        fence_mbar_init();
    }
    if (warp == kIssuer) tmem_alloc(base, kTmCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *base;
    // registers: 512 x 96 + 128 x 64 + 128 x 32 of the launch's 768 x 80
    if (warp < kMakers) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
        int n = 0, nv = 0;
#pragma unroll 1
        for (int k = 0; next_item(k, total); ++k) {
            f2 s[kKeys / 2];
            bool cleared;
            float decay;
            if (!make<S>(p, k, n, nv, tm, warp, lane, s, cleared, decay)) break;
            S* const state = static_cast<S*>(ring(k).state);
            float *const plane = ring(k).plane, *const kept = ring(k).kept;
            const int row = 32 * (warp & 3) + lane, keys = (warp >> 2) * kKeys;
            if (plane && !kept) {
#pragma unroll
                for (int j = 0; j < kKeys / 2; j += 2) {
                    const float2 a = unpack2(s[j]), b = unpack2(s[j + 1]);
                    *reinterpret_cast<float4*>(plane + state_at(row, keys + 2 * j)) = make_float4(a.x, a.y, b.x, b.y);
                }
            } else if (plane) {
                // a transition, its entries at most the decay: for the chain as sums of two fp16
                float undo;
                const float up = scale_of(fminf(decay, 1.f), undo);
#pragma unroll
                for (int i = 0; i < kKeys; i += 4) {
                    uint32_t e[4];
#pragma unroll
                    for (int u = 0; u < 4; u += 2) {
                        const float2 a = unpack2(s[(i + u) / 2]);
                        const float x = a.x * up, y = a.y * up;
                        const __half2 hi = __floats2half2_rn(x, y);
                        const float2 f = __half22float2(hi);
                        const uint32_t h = reinterpret_cast<const uint32_t&>(hi), l = pack_half2(x - f.x, y - f.y);
                        e[u] = __byte_perm(h, l, 0x5410);
                        e[u + 1] = __byte_perm(h, l, 0x7632);
                    }
                    *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(plane) + phi_at(row, keys + i)) =
                        make_uint4(e[0], e[1], e[2], e[3]);
                }
                if (threadIdx.x == 0) *kept = cleared ? -1.f : undo;
            } else if (state) {
                store_state(state, warp, lane, s);
            }
            done_with(k, lane);
        }
        tmem_wait_st();  // (of an item that was left)
        tc_fence_before();
        __syncthreads();
    } else if (warp < kIssuer) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        write(p, total, tm, warp, lane);
        tc_fence_before();
        __syncthreads();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
        if (warp == kIssuer) {
            Issuer<S> issuer{p, cuts, local, elect_one(), total};
            issuer.go(tm);
            issuer.finish();
        } else {
            Turner t{&v_map, total, warp - kIssuer - 1, lane};
            t.go();
            t.finish();
        }
        __syncthreads();
        __syncwarp();
        if (warp == kIssuer) {
            tc_fence_after();
            if (abort_flag() && lane == 0) atomicOr(p.status, 1);
            tmem_dealloc(tm, kTmCols);
        }
    }
}

// The states that the segments of a cut sequence start from: with a segment's N and Phi,
// S <- S Phi + N, from its first one's end on.  A CTA has 16 value rows of a (sequence, head), a
// warp 16 of the keys.  S and Phi are sums of two fp16, S's rows scaled by a power of two,
// Phi by one for all, from its largest possible entry, the decay over the segment.
// Transitions come by bulk copies, two at a time, N a step ahead.
// Bound by the chain, about 1 us a segment; with fp32 products it took 2.7, the FMA units' rate
// being half of that.
constexpr int kChainThreads = 256;
constexpr int kChainRows = 16;
constexpr int kChainPlane = D * D * 4;
constexpr int kChainTile = kChainRows * D * 2;
constexpr int kChainS = 2 * kChainPlane;                    // S, high and low part
constexpr int kChainMax = kChainS + 2 * kChainTile;         // [8][16] largest of a row, by warp
constexpr int kChainBar = kChainMax + 8 * kChainRows * 4;
constexpr int kChainSmem = kChainBar + 16;
__global__ void __launch_bounds__(kChainThreads, 1)
kda_delta_chain(const __grid_constant__ DeltaParams p, const __grid_constant__ LinCuts cuts) {
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t* const phi = reinterpret_cast<const uint32_t*>(smem);
    uint8_t* const tile = smem + kChainS;
    float* const most = reinterpret_cast<float*>(smem + kChainMax);
    uint64_t* const full = reinterpret_cast<uint64_t*>(smem + kChainBar);
    const int r = blockIdx.x / p.H, h = blockIdx.x % p.H, row0 = blockIdx.y * kChainRows;
    const int first = cuts.first[r], steps = cuts.first[r + 1] - first - 2;
    auto plane = [&](int g) { return p.planes + ((size_t)(first + g) * p.H + h) * 2 * D * D; };
    if (threadIdx.x == 0) {
        mbar_init(full, 1);
        mbar_init(full + 1, 1);
        fence_mbar_init();
    }
    __syncthreads();
    grid_dep_wait();
    auto fetch = [&](int g) {
        mbar_arrive_expect_tx(full + (g & 1), kChainPlane);
        bulk_g2s(smem + (g & 1) * kChainPlane, plane(g) + D * D, kChainPlane, full + (g & 1));
    };
    if (threadIdx.x == 0) {
        if (steps >= 1) fetch(1);
        if (steps >= 2) fetch(2);
    }
    // a thread has rows `row` and row + 8 at keys col, col + 1, col + 8, col + 9: s[8's][row][key]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane >> 2, col = warp * 16 + (lane & 3) * 2;
    auto at = [&](int t, int u) { return state_at(row0 + row + 8 * u, col + 8 * t); };
    float2 s[2][2], next[2][2];
    float kept = 0.f, scale[2], inv[2];
    auto fetch_n = [&](int g) {
        if (g > steps) return;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) next[t][u] = *reinterpret_cast<const float2*>(plane(g) + at(t, u));
        kept = p.kept[(size_t)(first + g) * p.H + h];
    };
    // S's rows' scales and operand; all have the state of a step behind them
    auto keep = [&]() {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float m = fmaxf(fmaxf(fabsf(s[0][u].x), fabsf(s[0][u].y)), fmaxf(fabsf(s[1][u].x), fabsf(s[1][u].y)));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            if ((lane & 3) == 0) most[warp * kChainRows + row + 8 * u] = m;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, most[i * kChainRows + row + 8 * u]);
            scale[u] = scale_of(m, inv[u]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t to = sw128_off(row + 8 * u, col + 8 * t, kChainRows);
                const float x = s[t][u].x * scale[u], y = s[t][u].y * scale[u];
                const __half2 hi = __floats2half2_rn(x, y);
                const float2 f = __half22float2(hi);
                *reinterpret_cast<__half2*>(tile + to) = hi;
                *reinterpret_cast<uint32_t*>(tile + kChainTile + to) = pack_half2(x - f.x, y - f.y);
            }
        }
    };
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) s[t][u] = *reinterpret_cast<const float2*>(plane(0) + at(t, u));
    fetch_n(1);
    keep();
    for (int g = 1; g <= steps; ++g) {
        if (!__syncthreads_and(mbar_wait(full + (g & 1), ((g - 1) >> 1) & 1))) {
            // report, and let the copies in flight land
            if (threadIdx.x == 0) {
                atomicOr(p.status, 1);
                mbar_wait(full + (g & 1), ((g - 1) >> 1) & 1);
                if (g < steps) mbar_wait(full + ((g + 1) & 1), (g >> 1) & 1);
            }
            return;
        }
        float d[2][4] = {};
        const uint32_t* f = phi + (g & 1) * D * D;
        const uint32_t ta = smem_u32(tile) + sw128_off(lane & 15, 0, kChainRows);
        const int swap = lane & 7;
#pragma unroll
        for (int ks = 0; ks < D; ks += 16) {
            uint32_t hi[4], lo[4];
            const uint32_t o = (ks >> 6) * (kChainRows * 128) + ((((ks & 63) / 8 + (lane >> 4)) ^ swap) << 4) - (swap << 4);
            ldsm_x4(ta + o, hi[0], hi[1], hi[2], hi[3]);
            ldsm_x4(ta + kChainTile + o, lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int j = ks + (lane & 3) * 2, k = warp * 16 + 8 * t + row;
                uint32_t bh[2], bl[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t x = f[phi_at(j + 8 * u, k)], y = f[phi_at(j + 8 * u + 1, k)];
                    bh[u] = __byte_perm(x, y, 0x5410);
                    bl[u] = __byte_perm(x, y, 0x7632);
                }
                mma_f16(d[t], lo, bh[0], bh[1]);
                mma_f16(d[t], hi, bl[0], bl[1]);
                mma_f16(d[t], hi, bh[0], bh[1]);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float back = kept * inv[u];
                float2 y = next[t][u];
                if (kept >= 0.f) y.x = fmaf(d[t][2 * u], back, y.x), y.y = fmaf(d[t][2 * u + 1], back, y.y);
                s[t][u] = y;
                *reinterpret_cast<float2*>(plane(g) + at(t, u)) = y;
            }
        fetch_n(g + 1);
        keep();  // (its barrier: all are done with the operand and the transition)
        if (threadIdx.x == 0 && g + 2 <= steps) {
            fence_proxy_async();
            fetch(g + 2);
        }
    }
}

// A [T][H][128] view of bf16 in boxes of 64 values x 1 head x 64 tokens, swizzled; tokens past
// the end read as zeros.
bool make_v_map(CUtensorMap* m, const DeltaParams& p) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<Encode>(f) : nullptr;
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {D, (cuuint64_t)p.H, (cuuint64_t)p.T};
    // a dimension of one entry never steps: any stride that encodes will do
    const cuuint64_t strides[2] = {(cuuint64_t)(p.H == 1 ? D : p.v_sh) * 2, (cuuint64_t)(p.T == 1 ? D : p.v_st) * 2};
    const cuuint32_t box[3] = {64, 1, C}, step[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.v), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches with programmatic stream serialization: set up while the last CTAs of the kernel
// before still run.
template <class... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, size_t bytes, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class S>
cudaError_t launch(const DeltaParams& p, const LinCuts& cuts, const CUtensorMap& v_map, cudaStream_t s) {
    static unsigned configured = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 32 || !(configured & (1u << dev))) {
        e = cudaFuncSetAttribute(kda_delta_walk<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kda_delta_chain, cudaFuncAttributeMaxDynamicSharedMemorySize, kChainSmem);
        if (e != cudaSuccess) return e;
        if (dev < 32) configured |= 1u << dev;
    }
    const auto walk = [&](bool local, int segments) {
        const int items = segments * p.H, sms = num_sms();
        return launch_after(kda_delta_walk<S>, dim3((unsigned)(items < sms ? items : sms)), kThreads, kSmemBytes, s, p, v_map, cuts,
                            local, items);
    };
    if (p.n_cut > 0) {
        e = walk(true, 2 * p.n_seg - 3 * p.n_cut);
        if (e == cudaSuccess)
            e = launch_after(kda_delta_chain, dim3((unsigned)(p.n_cut * p.H), D / kChainRows), kChainThreads, kChainSmem, s, p, cuts);
        if (e != cudaSuccess) return e;
    }
    return walk(false, p.n_seg - 2 * p.n_cut + p.n_long);
}

// How the longest sequences are cut, from the long sequences' lengths (longest first).  In
// units of a chunk's time in the walk: uncut it takes as long as its longest sequence.  Cut into
// k segments, the first pass walks all but the last one twice (but for the first), the
// second all but the first; the chain between them takes half a unit a segment, and the two
// more launches about four.  `single` is the time of the single tokens, on all SMs: they run beside
// the last walk on the SMs that it leaves, and then on all.
struct Cut {
    int seg = 0, n_cut = 0, n_seg = 0;
};
Cut cut_rule(const int32_t* lens, int n, int H, int sms, int64_t planes, float single) {
    Cut best;
    if (n <= 0 || (int64_t)n * H > sms) return best;  // a wave of whole sequences fills the GPU
    auto chunks_of = [](int len) { return (len + C - 1) / C; };
    const auto left = [&](int64_t items, int length) {  // of the single tokens, after the walk
        const float beside = items < sms ? (float)length * (float)(sms - items) / (float)sms : 0.f;
        return single > beside ? single - beside : 0.f;
    };
    const int longest = chunks_of(lens[0]);
    float least = (float)longest + left((int64_t)n * H, longest);
    for (int k = 2; k <= 32; ++k) {
        const int seg = (longest + k - 1) / k;
        if (seg < kDeltaMinSeg) break;
        Cut c;
        c.seg = seg;
        int64_t local = 0, rest = 0;
        int most = 0;
        for (int i = 0; i < n; ++i) {
            const int m = (chunks_of(lens[i]) + seg - 1) / seg;
            if (m < 2) {
                rest += H;
                continue;
            }
            ++c.n_cut, c.n_seg += m;
            local += (int64_t)(2 * (m - 1) - 1) * H;
            rest += (int64_t)(m - 1) * H;
            most = m > most ? m : most;
        }
        if (c.n_cut > kLinCuts || (int64_t)c.n_seg * H > planes) break;
        const auto waves = [&](int64_t items) { return (float)((items + sms - 1) / sms); };
        const float time = (waves(local) + waves(rest)) * (float)seg + 0.5f * (float)(most - 2) + 4.f + left(rest, seg);
        if (time < least) least = time, best = c;
    }
    return best;
}

}  // namespace

void delta_cut(DeltaParams& p, LinCuts& cuts, const SeqTables& t) {
    // a single token's state of a head goes there and back at 6.6 TB/s (5.9 if of 2 bytes), a
    // chunk takes 2.6 us; a sequence of more tokens takes some 30 ns more for a head
    const float state = p.st_dtype == KDA_STATE_F32 ? 0.0077f : 0.0042f;
    const float single = state * (float)p.n_short + 0.012f * (float)p.n_mid;
    const Cut c = cut_rule(t.long_lens, p.n_long, p.H, num_sms(), delta_planes(p.T, p.H), single * (float)p.H);
    p.seg_len = c.seg * C;
    p.n_cut = c.n_cut;
    p.n_seg = c.n_seg;
    cuts.first[0] = 0;
    for (int r = 0; r < c.n_cut; ++r) {
        cuts.seq[r] = t.long_seqs[r];
        cuts.t0[r] = t.bounds[t.long_seqs[r]];
        cuts.len[r] = t.long_lens[r];
        cuts.first[r + 1] = cuts.first[r] + (t.long_lens[r] + p.seg_len - 1) / p.seg_len;
    }
}

cudaError_t launch_delta_walk(const DeltaParams& p, const LinCuts& cuts, cudaStream_t s) {
    if (p.n_long <= 0) return cudaSuccess;
    if ((int64_t)p.n_long * p.H > INT32_MAX / 4) return cudaErrorInvalidValue;
    CUtensorMap v_map;
    if (!make_v_map(&v_map, p)) return cudaErrorInvalidValue;
    if (p.st_dtype == KDA_STATE_F32) return launch<float>(p, cuts, v_map, s);
    if (p.st_dtype == KDA_STATE_BF16) return launch<__nv_bfloat16>(p, cuts, v_map, s);
    return launch<__half>(p, cuts, v_map, s);
}

}  // namespace kda
