// Linear attention with a decay for each head, chunk by chunk on the tensor
// cores (tcgen05, accumulators in tensor memory).  For a chunk of C = 128 tokens
// with incoming state S (V x K), prefix sums G of the log decays, suffix sums R:
//
//     X = q k^T                    P_ij = X_ij e^{G_i - G_j}   (j <= i, else 0)
//     O = e^{G_i} (q S^T) + P v    out = scale O
//     dS = (e^{R_j} v_j)^T k       S' = e^{G_C} S + dS
//
// One CTA walks one (sequence, head) at a time; its warps have roles:
//   0-7   state: weighted v (W) into tensor memory, S in registers, S as the
//         q S^T product's operand in shared memory
//   8-11  scores: X to P in place, the e^{G_i} on q S^T, the output rows
//   12    issues the MMAs     13  issues the TMA loads
//   14    claims items and makes the decays
//
// Rounding.  Operands are bf16.  q, k and v are; P and S are carried as a sum of
// two bf16 (16 bits: with one, a rounding as large as out's own would be added
// to it), W as a sum of three (24 bits, the state is fp32).  dS starts from zero
// every chunk and S' is formed in fp32 registers, so that S is rounded once a
// chunk however the tensor cores round their partial sums.
//
// Infinities and NaN.  A masked score is a zero by selection, but a zero times an
// infinite v is NaN: P v would carry it to the chunk's earlier tokens.  The state
// warps, which read all of v for W, therefore clear such values in the tile (W
// keeps them: the state holds them from the chunk's end on), and the score warps
// put a NaN into their columns from their token on.

#include <type_traits>

#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

using namespace dev;

constexpr int D = kD;
constexpr int C = 128;
constexpr int kThreads = 15 * 32;
constexpr int kTile = C * D * 2;  // bytes of a q, k or v tile
constexpr int kSlots = 5;         // tiles in flight or in use
constexpr int kItems = 4;         // items the claims run ahead

// Shared memory.  Tiles are two halves of 64 columns, 128-byte swizzled.
constexpr int kSmS = 0;                        // S as bf16: high part, then low part
constexpr int kSmTile = 2 * kTile;
constexpr int kSmG = kSmTile + kSlots * kTile; // [2][G, prefix sums in log2; e^R]
constexpr int kSmItem = kSmG + 2 * 2 * C * 4;
struct Item {
    int t0, len, h, n, slot, flags;
    float pad[2];
};
enum { kInit = 1, kStore = 2, kEnd = 4 };
constexpr int kSmBar = kSmItem + kItems * (int)sizeof(Item);

enum Bar {
    kFull = 0,                  // [5] tile loaded
    kEmpty = kFull + kSlots,    // [5] tile consumed
    kDecFull = kEmpty + kSlots, // [2] decays of a chunk made
    kDecEmpty = kDecFull + 2,   // [2] and read
    kItemFull = kDecEmpty + 2,  // [4] item claimed
    kItemEmpty = kItemFull + kItems,
    kXFull = kItemEmpty + kItems,  // q k^T in X
    kPFull,                     // P in X
    kQSFull,                    // q S^T in O; S's operand read
    kQSScaled,                  // e^{G_i} applied
    kOFull,                     // the chunk's O complete
    kOEmpty,                    // and read
    kWFull,                     // [2] two K steps of W written
    kWEmpty = kWFull + 2,       // [2] and read
    kDSFull = kWEmpty + 2,      // dS complete
    kDSEmpty,                   // and read
    kSFull,                     // S's operand written
    kCleared,                   // rows past a sequence's end cleared
    kDone,                      // everything issued has completed
    kNumBars
};
constexpr int kSmGamma = kSmBar + kNumBars * 8;  // [2] e^{G_C}
constexpr int kSmBad = kSmGamma + 8;             // [2][8] value columns with infinities or NaN
constexpr int kSmMisc = kSmBad + 64;             // tensor-memory base, abort flag
constexpr int kSmemBytes = kSmMisc + 8;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

// Tensor memory columns.
constexpr uint32_t kTmX = 0;    // X; then P: per 32 tokens 16 columns high part, 16 low
constexpr uint32_t kTmO = 128;
constexpr uint32_t kTmDS = 256;
constexpr uint32_t kTmW = 384;  // [2] buffers of 2 K steps x (high, middle, low) x 8 columns
constexpr uint32_t kTmCols = 512;

constexpr uint32_t kIdescKK = mma_idesc(1, 0, 0, 128, 128);  // B K-major
constexpr uint32_t kIdescKM = mma_idesc(1, 0, 1, 128, 128);  // B MN-major

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
        "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31]), "r"(a)
        : "memory");
}
// 16 lanes x 8 columns: r0 holds lane t/4, column t%4; r1 lane t/4 + 8; r2, r3 the
// same four columns on.  The layout of ldmatrix fragments.
__device__ __forceinline__ void tmem_st_16x8(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2,
                                             uint32_t r3) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r0),
                 "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

__device__ __forceinline__ void store32(void* p, const uint32_t* r, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

struct Maps {
    CUtensorMap q, k, v;
};

// What every role needs.
struct Ctx {
    uint8_t* smem;
    uint64_t* bar;
    volatile int* abort;
    uint32_t tmem;
    int lane;

    // Waits for a barrier's phase; gives up after about a second, or once another
    // role has (the callers then leave their loops).
    __device__ __forceinline__ bool wait(int b, uint32_t parity) const {
        for (uint32_t i = 0; i < kWaitLimit; ++i) {
            if (mbar_try_wait(bar + b, parity)) return true;
            if (*abort) return false;
        }
        *abort = 1;
        return false;
    }
    // The same for a whole warp, which goes on or leaves together.
    __device__ __forceinline__ bool wait_all(int b, uint32_t parity) const {
        return __all_sync(0xffffffffu, wait(b, parity));
    }
    __device__ __forceinline__ void arrive(int b) const { mbar_arrive(bar + b); }
    __device__ __forceinline__ uint8_t* tile(int i) const { return smem + kSmTile + (i % kSlots) * kTile; }
    // Barrier and phase of tile i's load.
    static __device__ __forceinline__ int full(int i) { return kFull + i % kSlots; }
    static __device__ __forceinline__ uint32_t full_phase(int i) { return (i / kSlots) & 1; }
    __device__ __forceinline__ const float* decays(int c) const {
        return reinterpret_cast<const float*>(smem + kSmG) + (c & 1) * 2 * C;
    }
    __device__ __forceinline__ float gamma(int c) const {
        return reinterpret_cast<const float*>(smem + kSmGamma)[c & 1];
    }
    // The role's it-th item; false when there is none (or on abort).
    __device__ __forceinline__ bool item(int it, Item* out, bool whole_warp) const {
        const int b = kItemFull + it % kItems, phase = (it / kItems) & 1;
        if (whole_warp ? !wait_all(b, phase) : !wait(b, phase)) return false;
        *out = reinterpret_cast<const Item*>(smem + kSmItem)[it % kItems];
        if (whole_warp) __syncwarp();
        if (!whole_warp || lane == 0) arrive(kItemEmpty + it % kItems);
        return !(out->flags & kEnd);
    }
};
__device__ __forceinline__ int chunks(int len) { return (len + C - 1) / C; }

// ---- warp 14: items and decays ------------------------------------------------
__device__ __forceinline__ void decay_role(const LinParams& p, const Ctx& x) {
    const int n_items = p.n_long * p.H;
    int c = 0;
    for (int it = 0;; ++it) {
        if (it >= kItems && !x.wait_all(kItemEmpty + it % kItems, ((it / kItems) + 1) & 1)) return;
        int i = 0;
        if (x.lane == 0) i = atomicAdd(reinterpret_cast<int*>(reinterpret_cast<char*>(p.status) + kWsQueueOff), 1);
        i = __shfl_sync(0xffffffffu, i, 0);
        Item item{};
        if (i < n_items) {
            item.n = p.long_list[i / p.H];
            item.h = i % p.H;
            item.t0 = p.cu[item.n];
            item.len = p.cu[item.n + 1] - item.t0;
            item.slot = p.idx[item.n];
            const bool ok = item.slot >= 0 && item.slot < p.num_slots;
            if (!ok && x.lane == 0) atomicOr(p.status, 4);
            item.flags = (ok ? kStore : 0) | (ok && p.has_init[item.n] ? kInit : 0);
        } else {
            item.flags = kEnd;
        }
        if (x.lane == 0) {
            reinterpret_cast<Item*>(x.smem + kSmItem)[it % kItems] = item;
            x.arrive(kItemFull + it % kItems);  // releases the write
        }
        if (item.flags & kEnd) return;
        const float* g = p.g + item.h;
        for (int j = 0; j < chunks(item.len); ++j, ++c) {
            // four tokens a lane; tokens past the end decay nothing
            float a[4], pre[4], suf[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = j * C + 4 * x.lane + e;
                float v = 0.f;
                if (t < item.len) v = g[(int64_t)(item.t0 + t) * p.g_st];
                a[e] = v < kMinDecay ? kMinDecay : v;
            }
            pre[0] = a[0];
#pragma unroll
            for (int e = 1; e < 4; ++e) pre[e] = pre[e - 1] + a[e];
            suf[3] = 0.f;
#pragma unroll
            for (int e = 2; e >= 0; --e) suf[e] = suf[e + 1] + a[e + 1];
            float up = pre[3], down = pre[3];  // sums over the lanes up to here, from here on
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, up, w);
                const float d = __shfl_down_sync(0xffffffffu, down, w);
                if (x.lane >= w) up += u;
                if (x.lane + w < 32) down += d;
            }
            const float total = __shfl_sync(0xffffffffu, up, 31);
            float before = __shfl_up_sync(0xffffffffu, up, 1);
            float after = __shfl_down_sync(0xffffffffu, down, 1);
            if (x.lane == 0) before = 0.f;
            if (x.lane == 31) after = 0.f;
            if (c >= 2 && !x.wait_all(kDecEmpty + (c & 1), ((c >> 1) + 1) & 1)) return;
            float* dst = const_cast<float*>(x.decays(c));
            constexpr float kLog2e = 1.4426950408889634f;
            float4 G, w;
            G.x = (before + pre[0]) * kLog2e, G.y = (before + pre[1]) * kLog2e;
            G.z = (before + pre[2]) * kLog2e, G.w = (before + pre[3]) * kLog2e;
            w.x = expf(after + suf[0]), w.y = expf(after + suf[1]);
            w.z = expf(after + suf[2]), w.w = expf(after + suf[3]);
            reinterpret_cast<float4*>(dst)[x.lane] = G;
            reinterpret_cast<float4*>(dst + C)[x.lane] = w;
            if (x.lane == 0) reinterpret_cast<float*>(x.smem + kSmGamma)[c & 1] = expf(total);
            __syncwarp();
            if (x.lane == 0) x.arrive(kDecFull + (c & 1));
        }
    }
}

// ---- warp 13, one lane: loads -------------------------------------------------
// Returns the number of tiles issued.
__device__ __forceinline__ int load_role(const Maps& maps, const LinParams& p, const Ctx& x) {
    int tile = 0;
    Item item;
    for (int it = 0; x.item(it, &item, false); ++it) {
        for (int j = 0; j < chunks(item.len); ++j) {
            const int t = item.t0 + j * C;
#pragma unroll
            for (int m = 0; m < 3; ++m, ++tile) {  // k, q, v
                if (tile >= kSlots && !x.wait(kEmpty + tile % kSlots, ((tile / kSlots) + 1) & 1)) return tile;
                const CUtensorMap* map = m == 0 ? &maps.k : m == 1 ? &maps.q : &maps.v;
                const int h = m == 2 ? item.h : item.h / p.rep;
                uint64_t* bar = x.bar + kFull + tile % kSlots;
                uint8_t* dst = x.tile(tile);
                mbar_arrive_expect_tx(bar, kTile);
                tma_load_3d(dst, map, bar, 0, h, t);
                tma_load_3d(dst + kTile / 2, map, bar, 64, h, t);
            }
        }
    }
    return tile;
}

// ---- warp 12, one lane: products ------------------------------------------------
__device__ __forceinline__ void mma_role(const Ctx& x) {
    const uint32_t base = smem_u32(x.smem);
    auto kmaj = [&](uint32_t a, int ks) {  // K-major: 16 columns on
        return sw128_desc(a + (ks >> 2) * (kTile / 2) + (ks & 3) * 32, 16, 1024);
    };
    auto mnmaj = [&](uint32_t a, int ks) {  // MN-major: 16 rows on
        return sw128_desc(a + ks * 2048, kTile / 2, 1024);
    };
    int tile = 0, c = 0, with_s = 0, wb = 0;
    Item item;
    for (int it = 0; x.item(it, &item, false); ++it) {
        const int nc = chunks(item.len);
        for (int j = 0; j < nc; ++j, ++c, tile += 3) {
            const bool has_s = j > 0 || (item.flags & kInit);
            const uint32_t k = smem_u32(x.tile(tile)), q = smem_u32(x.tile(tile + 1)),
                           v = smem_u32(x.tile(tile + 2));
            if (!x.wait(x.full(tile), x.full_phase(tile)) || !x.wait(x.full(tile + 1), x.full_phase(tile + 1)))
                return;
            // X is free once the previous chunk's P v has read it
            if (c > 0 && !x.wait(kOFull, (c + 1) & 1)) return;
            tc_fence_after();
            for (int ks = 0; ks < 8; ++ks)
                mma_f16_ss(x.tmem + kTmX, kmaj(q, ks), kmaj(k, ks), kIdescKK, ks > 0);
            mma_commit(x.bar + kXFull);
            // O is free once the previous chunk's rows have been read
            if (c > 0 && !x.wait(kOEmpty, (c + 1) & 1)) return;
            if (has_s) {
                if (!x.wait(kSFull, with_s & 1)) return;
                tc_fence_after();
                for (int part = 1; part >= 0; --part)  // low part first
                    for (int ks = 0; ks < 8; ++ks)
                        mma_f16_ss(x.tmem + kTmO, kmaj(q, ks), kmaj(base + kSmS + part * kTile, ks), kIdescKK,
                                   part == 0 || ks > 0);
                mma_commit(x.bar + kQSFull);
            }
            mma_commit(x.bar + kEmpty + (tile + 1) % kSlots);
            if (c > 0 && !x.wait(kDSEmpty, (c + 1) & 1)) return;
            for (int half = 0; half < 4; ++half, ++wb) {  // 32 tokens each
                if (!x.wait(kWFull + (wb & 1), (wb >> 1) & 1)) return;
                tc_fence_after();
                const uint32_t w = x.tmem + kTmW + (wb & 1) * 48;
                for (int s = 0; s < 2; ++s)
                    for (int part = 2; part >= 0; --part)
                        mma_f16_ts(x.tmem + kTmDS, w + s * 24 + part * 8, mnmaj(k, 2 * half + s), kIdescKM,
                                   half > 0 || s > 0 || part < 2);
                mma_commit(x.bar + kWEmpty + (wb & 1));
            }
            mma_commit(x.bar + kDSFull);
            mma_commit(x.bar + kEmpty + tile % kSlots);
            if (!x.wait(kPFull, c & 1)) return;
            if (has_s && !x.wait(kQSScaled, with_s & 1)) return;
            tc_fence_after();
            for (int ks = 0; ks < 8; ++ks)
                for (int part = 1; part >= 0; --part)
                    mma_f16_ts(x.tmem + kTmO, x.tmem + kTmX + 32 * (ks >> 1) + 16 * part + 8 * (ks & 1),
                               mnmaj(v, ks), kIdescKM, has_s || ks > 0 || part == 0);
            mma_commit(x.bar + kOFull);
            mma_commit(x.bar + kEmpty + (tile + 2) % kSlots);
            with_s += has_s;
        }
    }
}

// Bit e: v holds an infinity or NaN in column col + e between tokens t0 and t1 of
// the item, for the columns in `cols`.
__device__ __noinline__ uint32_t nonfinite_up_to(const LinParams& p, const Item& item, int t0, int t1,
                                                 int col, uint32_t cols) {
    const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v) + (int64_t)item.h * p.v_sh + col;
    uint32_t hit = 0;
    for (int t = t0; t <= t1; ++t)
        for (uint32_t m = cols & ~hit; m; m &= m - 1) {
            const int e = __ffs(m) - 1;
            if ((v[(int64_t)(item.t0 + t) * p.v_st + e] & 0x7F80) == 0x7F80) hit |= 1u << e;
        }
    return hit;
}

// ---- warps 8-11: scores and output rows; thread = chunk row ----------------------
__device__ __forceinline__ void score_role(const LinParams& p, const Ctx& x, int w) {
    const int row = 32 * w + x.lane;
    const uint32_t tm = x.tmem + ((uint32_t)(32 * w) << 16);
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    int c = 0, with_s = 0;
    Item item;
    for (int it = 0; x.item(it, &item, true); ++it) {
        for (int j = 0; j < chunks(item.len); ++j, ++c) {
            const bool has_s = j > 0 || (item.flags & kInit);
            if (!x.wait_all(kDecFull + (c & 1), (c >> 1) & 1)) return;
            const float* G = x.decays(c);
            const float gi = G[row];
            if (!x.wait_all(kXFull, c & 1)) return;
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                uint32_t r[32], o[32];
                if (b <= w) {
                    tmem_ld32(tm + kTmX + 32 * b, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 gj = *reinterpret_cast<const float4*>(G + 32 * b + e);
                        float v[4] = {__uint_as_float(r[e]) * ex2(gi - gj.x),
                                      __uint_as_float(r[e + 1]) * ex2(gi - gj.y),
                                      __uint_as_float(r[e + 2]) * ex2(gi - gj.z),
                                      __uint_as_float(r[e + 3]) * ex2(gi - gj.w)};
                        if (b == w) {
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                if (e + u > x.lane) v[u] = 0.f;
                        }
#pragma unroll
                        for (int u = 0; u < 4; u += 2) {
                            const uint32_t hi = pack_bf162(v[u], v[u + 1]);
                            o[(e + u) / 2] = hi;
                            o[16 + (e + u) / 2] = pack_bf162(v[u] - bf_lo(hi), v[u + 1] - bf_hi(hi));
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                tmem_st32(tm + kTmX + 32 * b, o);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (x.lane == 0) {
                x.arrive(kPFull);
                x.arrive(kDecEmpty + (c & 1));
            }
            if (has_s) {
                if (!x.wait_all(kQSFull, with_s & 1)) return;
                tc_fence_after();
                const float f = ex2(gi);
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tm + kTmO + 32 * b, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(f * __uint_as_float(r[e]));
                    tmem_st32(tm + kTmO + 32 * b, r);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (x.lane == 0) x.arrive(kQSScaled);
                ++with_s;
            }
            if (!x.wait_all(kOFull, c & 1)) return;
            tc_fence_after();
            const uint32_t* bad = reinterpret_cast<const uint32_t*>(x.smem + kSmBad) + 8 * (c & 1);
            const int t = j * C + row;
            __nv_bfloat16* out = p.out + ((size_t)(item.t0 + t) * p.H + item.h) * D;
            uint32_t y[64];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t r[32];
                tmem_ld32(tm + kTmO + 32 * b, r);
                tmem_wait_ld();
                if (const uint32_t cols = bad[b] | bad[4 + b]) {
                    const uint32_t hit = nonfinite_up_to(p, item, j * C, min(t, item.len - 1), 32 * b, cols);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (hit >> e & 1) r[e] = 0x7FFFFFFFu;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    y[16 * b + e / 2] = pack_bf162(p.scale * __uint_as_float(r[e]), p.scale * __uint_as_float(r[e + 1]));
            }
            tc_fence_before();
            __syncwarp();
            if (x.lane == 0) x.arrive(kOEmpty);
            if (t < item.len) {
#pragma unroll
                for (int b = 0; b < 8; ++b) store32(out + 16 * b, y + 8 * b, wide);
            }
        }
    }
}

// ---- warps 0-7: weighted v and the state ------------------------------------------
// Thread: value row 32 (warp % 4) + lane, key columns 64 (warp / 4) .. + 63.
template <class S>
__device__ __forceinline__ float4 load4(const S* s);
template <>
__device__ __forceinline__ float4 load4(const float* s) {
    return *reinterpret_cast<const float4*>(s);
}
template <>
__device__ __forceinline__ float4 load4(const __nv_bfloat16* s) {
    const uint2 r = *reinterpret_cast<const uint2*>(s);
    return make_float4(bf_lo(r.x), bf_hi(r.x), bf_lo(r.y), bf_hi(r.y));
}
template <>
__device__ __forceinline__ float4 load4(const __half* s) {
    const uint2 r = *reinterpret_cast<const uint2*>(s);
    const float2 a = __half22float2(reinterpret_cast<const __half2&>(r.x));
    const float2 b = __half22float2(reinterpret_cast<const __half2&>(r.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float* s, float4 v) { *reinterpret_cast<float4*>(s) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* s, float4 v) {
    *reinterpret_cast<uint2*>(s) = make_uint2(pack_bf162(v.x, v.y), pack_bf162(v.z, v.w));
}
__device__ __forceinline__ void store4(__half* s, float4 v) {
    *reinterpret_cast<uint2*>(s) = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
}

// Clears infinities and NaN in a lane's column of the warp's tokens (16 of every
// 32); returns the warp's columns that had any.
__device__ __noinline__ uint32_t clear_nonfinite(uint8_t* vt, int col, int sg) {
    bool any = false;
    for (int i = 0; i < 64; ++i) {
        const int tok = 32 * (i >> 4) + 16 * sg + (i & 15);
        uint16_t* at = reinterpret_cast<uint16_t*>(vt + sw128_off(tok, col, C));
        if ((*at & 0x7F80) == 0x7F80) {
            *at = 0;
            any = true;
        }
    }
    fence_proxy_async();
    return __ballot_sync(0xffffffffu, any);
}

template <class P>
__device__ __forceinline__ void state_role(const LinParams& p, const Ctx& x, int warp) {
    const int sg = warp >> 2;
    const int row = 32 * (warp & 3) + x.lane;
    const uint32_t tm = x.tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    int tile = 0, c = 0, with_s = 0, wb = 0, cleared = 0;
    float S[64];
    // S as the product's operand: row `row`, columns 64 sg .. + 63
    auto write_operand = [&]() {
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                hi[u] = pack_bf162(S[e + 2 * u], S[e + 2 * u + 1]);
                lo[u] = pack_bf162(S[e + 2 * u] - bf_lo(hi[u]), S[e + 2 * u + 1] - bf_hi(hi[u]));
            }
            uint8_t* at = x.smem + kSmS + sw128_off(row, 64 * sg + e, C);
            *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(at + kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async();
        __syncwarp();
        if (x.lane == 0) x.arrive(kSFull);
    };
    Item item;
    for (int it = 0; x.item(it, &item, true); ++it) {
        const int nc = chunks(item.len);
        P* pool = static_cast<P*>(p.pool) +
                  (item.flags & kStore ? (size_t)item.slot * p.stride0 : 0) +
                  ((size_t)item.h * D + row) * D + 64 * sg;
        if (item.flags & kInit) {
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                const float4 v = load4<P>(pool + e);
                S[e] = v.x, S[e + 1] = v.y, S[e + 2] = v.z, S[e + 3] = v.w;
            }
            // the last q S^T that read the operand
            if (with_s > 0 && !x.wait_all(kQSFull, (with_s + 1) & 1)) return;
            write_operand();
            ++with_s;
        } else {
#pragma unroll
            for (int e = 0; e < 64; ++e) S[e] = 0.f;
        }
        for (int j = 0; j < nc; ++j, ++c, tile += 3) {
            const int live = min(C, item.len - j * C);
            uint8_t* vt = x.tile(tile + 2);
            if (!x.wait_all(x.full(tile + 2), x.full_phase(tile + 2))) return;
            if (live < C) {
                // rows past the sequence's end belong to others: they weigh nothing,
                // and may hold anything, so they are cleared
                if (!x.wait_all(x.full(tile), x.full_phase(tile))) return;
                uint8_t* kt = x.tile(tile);
                for (int i = (warp * 32 + x.lane); i < (C - live) * 16; i += 256) {
                    const uint32_t at = (i & 8 ? kTile / 2 : 0) + (live + (i >> 4)) * 128 + (i & 7) * 16;
                    *reinterpret_cast<uint4*>(kt + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(vt + at) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
                if (x.lane == 0) x.arrive(kCleared);
                if (!x.wait_all(kCleared, cleared & 1)) return;
                ++cleared;
            }
            if (!x.wait_all(kDecFull + (c & 1), (c >> 1) & 1)) return;
            const float* wt = x.decays(c) + C;
            const float gamma = x.gamma(c);
            const uint32_t vs = smem_u32(vt);
            uint32_t top = 0;  // largest magnitudes, as bits
#pragma unroll 1
            for (int half = 0; half < 4; ++half, ++wb) {
                const int ks = 2 * half + sg;  // this warp's 16 tokens
                const float2 wa = *reinterpret_cast<const float2*>(wt + 16 * ks + 2 * (x.lane & 3));
                const float2 wc = *reinterpret_cast<const float2*>(wt + 16 * ks + 8 + 2 * (x.lane & 3));
                if (wb >= 2 && !x.wait_all(kWEmpty + (wb & 1), ((wb >> 1) + 1) & 1)) return;
                tc_fence_after();
#pragma unroll
                for (int u = 0; u < 2; ++u) {  // 16 value rows each
                    // matrices: tokens 0-7 and 8-15, value rows 0-7 and 8-15
                    const int tok = 16 * ks + (x.lane & 7) + ((x.lane >> 4) << 3);
                    const int col = 32 * (warp & 3) + 16 * u + (((x.lane >> 3) & 1) << 3);
                    uint32_t r[4], hi[4], mi[4], lo[4];
                    ldsm_x4_t(vs + sw128_off(tok, col, C), r[0], r[1], r[2], r[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        top = __vmaxu2(top, r[e] & 0x7FFF7FFFu);
                        const float2 w = e < 2 ? wa : wc;
                        float a = w.x * bf_lo(r[e]), b = w.y * bf_hi(r[e]);
                        hi[e] = pack_bf162(a, b);
                        a -= bf_lo(hi[e]), b -= bf_hi(hi[e]);
                        mi[e] = pack_bf162(a, b);
                        a -= bf_lo(mi[e]), b -= bf_hi(mi[e]);
                        lo[e] = pack_bf162(a, b);
                    }
                    const uint32_t at = tm + ((uint32_t)(16 * u) << 16) + kTmW + (wb & 1) * 48 + sg * 24;
                    tmem_st_16x8(at, hi[0], hi[1], hi[2], hi[3]);
                    tmem_st_16x8(at + 8, mi[0], mi[1], mi[2], mi[3]);
                    tmem_st_16x8(at + 16, lo[0], lo[1], lo[2], lo[3]);
                }
                tmem_wait_st();
                tc_fence_before();
                if (half == 3) {
                    const bool any = (top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u;
                    uint32_t cols = 0;
                    if (__any_sync(0xffffffffu, any)) cols = clear_nonfinite(vt, 32 * (warp & 3) + x.lane, sg);
                    if (x.lane == 0) reinterpret_cast<uint32_t*>(x.smem + kSmBad)[8 * (c & 1) + warp] = cols;
                }
                __syncwarp();
                if (x.lane == 0) x.arrive(kWFull + (wb & 1));
            }
            if (x.lane == 0) x.arrive(kDecEmpty + (c & 1));
            if (!x.wait_all(kDSFull, c & 1)) return;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t r[32];
                tmem_ld32(tm + kTmDS + 64 * sg + 32 * b, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    S[32 * b + e] = fmaf(gamma, S[32 * b + e], __uint_as_float(r[e]));
            }
            tc_fence_before();
            __syncwarp();
            if (x.lane == 0) x.arrive(kDSEmpty);
            if (j + 1 < nc) {
                if (with_s > 0 && !x.wait_all(kQSFull, (with_s + 1) & 1)) return;
                write_operand();
                ++with_s;
            }
        }
        if (item.flags & kStore) {
#pragma unroll
            for (int e = 0; e < 64; e += 4) store4(pool + e, make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]));
        }
    }
}

template <class P>
__global__ void __launch_bounds__(kThreads, 1) kda_lin_walk(const __grid_constant__ Maps maps, LinParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    Ctx x;
    x.smem = smem;
    x.bar = reinterpret_cast<uint64_t*>(smem + kSmBar);
    x.lane = threadIdx.x & 31;
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kSmMisc);
    x.abort = reinterpret_cast<volatile int*>(smem + kSmMisc + 4);
    if ((smem_u32(smem) & 1023) != 0) {  // swizzled tiles need 1 KB alignment
        if (threadIdx.x == 0) atomicOr(p.status, 2);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            int n = 1;
            if (i == kDecEmpty || i == kDecEmpty + 1) n = 12;
            if (i >= kItemEmpty && i < kItemEmpty + kItems) n = 14;
            if (i == kPFull || i == kQSScaled || i == kOEmpty) n = 4;
            if (i == kWFull || i == kWFull + 1 || i == kDSEmpty || i == kSFull || i == kCleared) n = 8;
            mbar_init(x.bar + i, n);
        }
        *x.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.q);
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    if (warp == 12) tmem_alloc(slot, kTmCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    x.tmem = *slot;

    int issued = 0;
    if (warp < 8) {
        state_role<P>(p, x, warp);
    } else if (warp < 12) {
        score_role(p, x, warp - 8);
    } else if (warp == 12) {
        if (x.lane == 0) {
            mma_role(x);
            mma_commit(x.bar + kDone);
        }
    } else if (warp == 13) {
        if (x.lane == 0) issued = load_role(maps, p, x);
    } else {
        decay_role(p, x);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*x.abort) {
        // a wait gave up: let the copies and products in flight end before their memory goes
        if (threadIdx.x == 0) atomicOr(p.status, 1);
        if (warp == 13 && x.lane == 0)
            for (int i = max(0, issued - kSlots); i < issued; ++i)
                mbar_wait(x.bar + kFull + i % kSlots, (i / kSlots) & 1);
    }
    if (warp == 12) {
        mbar_wait(x.bar + kDone, 0);
        tc_fence_after();
    }
    __syncthreads();
    if (warp == 12) tmem_dealloc(x.tmem, kTmCols);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                         cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
    }();
    return fn;
}

// Boxes of 64 values x 1 head x C tokens of a [T][H][128] view; tokens past the
// end read as zeros.
bool make_map(CUtensorMap* m, const void* base, int64_t T, int H, int64_t st, int64_t sh) {
    if (!encode_fn()) return false;
    // a dimension of one entry never steps: any stride that encodes will do
    if (T == 1) st = D;
    if (H == 1) sh = D;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)C};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                       box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class P>
cudaError_t launch(const Maps& maps, const LinParams& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kda_lin_walk<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)p.n_long * p.H;
    const int grid = (int)(items < num_sms() ? items : num_sms());
    kda_lin_walk<P><<<grid, kThreads, kSmemBytes, s>>>(maps, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_walk(const LinParams& p, cudaStream_t s) {
    if (p.n_long <= 0) return cudaSuccess;
    if ((int64_t)p.n_long * p.H > INT32_MAX - 65536) return cudaErrorInvalidValue;
    Maps maps;
    if (!make_map(&maps.q, p.q, p.T, p.H / p.rep, p.q_st, p.q_sh) ||
        !make_map(&maps.k, p.k, p.T, p.H / p.rep, p.k_st, p.k_sh) ||
        !make_map(&maps.v, p.v, p.T, p.H, p.v_st, p.v_sh))
        return cudaErrorInvalidValue;
    if (p.st_dtype == KDA_STATE_F32) return launch<float>(maps, p, s);
    if (p.st_dtype == KDA_STATE_BF16) return launch<__nv_bfloat16>(maps, p, s);
    return launch<__half>(maps, p, s);
}

}  // namespace kda
