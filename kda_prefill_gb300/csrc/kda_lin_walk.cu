// Linear attention with a decay for each head, chunk by chunk on the tensor
// cores (tcgen05, accumulators in tensor memory).  For a chunk of C = 128 tokens
// with incoming state S (V x K), prefix sums G of the log decays, suffix sums R:
//
//     X = q k^T                    P_ij = X_ij e^{G_i - G_j}   (j <= i, else 0)
//     O = e^{G_i} (q S^T) + P v    out = scale O
//     dS = (e^{R_j} v_j)^T k       S' = e^{G_C} S + dS
//
// One CTA walks one (sequence, head) at a time; its warps have roles:
//   0-7   S in registers, and as the q S^T product's operand in shared memory
//   8-15  W, the weighted v, into tensor memory
//   16-23 X to P, in place
//   24-27 the e^{G_i} on q S^T, the output rows
//   28    issues the MMAs     29  issues the TMA loads
//   30    claims items and makes the decays
// A chunk's products are issued as a quarter of dS, X, another, q S^T, the rest of dS, P v:
// what a role needs time for (P after X, S after dS, e^{G_i} after q S^T, the rows after
// P v) has products beside it that do not wait for it.
//
// The products are the bound: 72 of 128 x 128 x 16, 64 cycles each, 4.6 K cycles a chunk,
// of which the tensor pipe reaches about three quarters while it shares shared and tensor
// memory with the operands' makers (6.3 K cycles a chunk; 128 sequences of 117,555 tokens
// x 12 heads: 340 to 343 us, tensor pipe active 61 % of the time, 48 % of a copy's rate).
// Chunks of 128 fill the products' M: with 64, q S^T would run at half rate, and S would
// be read, rounded and written as an operand twice as often.
//
// A few long sequences would leave most SMs idle.  They are cut into segments: a first
// launch makes each segment's state from zero (Local), kda_lin_chain the states that the
// segments start from, and the walk takes them as items.  1 x 16384 tokens x 12 heads:
// 80 to 81 us (27 Local, 53 the walk), 418 us uncut.
//
// Rounding.  Operands are bf16.  q, k and v are; P and S are carried as a sum of
// two bf16 (16 bits: with one, a rounding as large as out's own would be added
// to it).  W has to keep 24 bits, the state being fp32: with the weight as a sum
// of three bf16, w = w1 + w2 + w3, it is the four bf16 a = v w1, its remainder
// v w1 - a (exact, one fused product), b = v w2 and the remainder v w2 - b + v w3.
// Five operations on pairs of bf16 make them; the shortest sum, of three, would
// take thirteen in fp32.  dS starts from zero
// every chunk and S' is formed in fp32 registers, so that S is rounded once a
// chunk however the tensor cores round their partial sums.
//
// Decays of scores.  G_i - G_j is a sum of the decays between the two and is made as one:
// a difference of sums over the chunk would lose the bits of weak decays behind strong
// ones (32 tokens of -0.01 behind 96 of -inf: off by 1.4e-3).  In the 32 x 32 blocks on
// the diagonal the sum grows token by token from the row to the left.  Left of them
// e^{G_i - G_j} is e^{G_i - G_b} e^{G_b - G_j}, b the last token of column j's block: both
// factors are at most one, the first is one a row and block and the second one a token,
// so neither overflows and few exponentials are left; G_i - G_b is the row's sum within
// its block and whole blocks' sums.
//
// Infinities and NaN.  A masked score is a zero by selection, but a zero times an
// infinite v is NaN: P v would carry it to the chunk's earlier tokens.  The W
// warps, which read all of v, therefore clear such values in the tile (W keeps
// them: the state holds them from the chunk's end on), and the output warps put a
// NaN into their columns from their token on.
//
// Clearing.  A decay below kMinDecay clears the state whatever it held, so nothing from
// before it may be multiplied by its zero: the scores of a row with columns before its last
// clearing token, q S^T of the rows from a chunk's first one on and S at the chunk's end
// are zero by selection.  dS can take a NaN from a token before the last clearing one, its
// weight being zero: where a cleared chunk's dS is not finite, the state warps sum the
// tokens from that one on themselves.  Chunks without a clearing token only look at a flag,
// and the rare work is out of line: inline it took registers of all (16384 tokens x 12
// heads 96 us instead of 80 to 81).

#include <type_traits>

#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

using namespace dev;

constexpr int D = kD;
constexpr int C = 128;
constexpr int kThreads = 32 * 32;
constexpr int kTile = C * D * 2;  // bytes of a q, k or v tile
// Tiles in flight or in use: q's, and two of v and of k, used by turns.  A chunk's q is
// free after q S^T, its v after P v, its k after dS and once the chunk's output rows,
// which pass through it, have left; so the next v is on its way a chunk ahead and the next
// q and k half a chunk (in one ring for all, v's loads would wait for the rows).
// Local has S's place too: four of v and three of k, whose loads then cover their latency.
constexpr int kSlots = 5, kLocalSlots = 7;
constexpr int kItems = 3;         // items the claims run ahead

// Shared memory.  Tiles are two halves of 64 columns, 128-byte swizzled.
constexpr int kSmS = 0;                        // S as bf16: high part, then low part
constexpr int kSmTile = 2 * kTile;
constexpr int kSmW = kSmTile + kSlots * kTile;  // [2][64] e^R of token pairs, each in three parts
constexpr int kSmA = kSmW + 2 * (C / 2) * 12;   // [128] decays in log2
constexpr int kSmT = kSmA + C * 4;              // [4] their sums over each 32 tokens
constexpr int kSmM = kSmT + 16;                 // [4] which of each 32 tokens clear the state
constexpr int kSmCf = kSmM + 16;                // [96] e^{G_b - G_j}
struct Item {
    int t0, len, h, n, flags;
    int plane;  // of the workspace: the segment's state
};
constexpr int kSmItem = kSmCf + 96 * 4;
enum { kInit = 1, kStore = 2, kEnd = 4, kPlane = 8 };
constexpr int kSmBar = kSmItem + kItems * (int)sizeof(Item);
static_assert(kSmBar % 8 == 0, "barriers are 8-byte aligned");

enum Bar {
    kFull = 0,                       // [7] tile loaded
    kEmpty = kFull + kLocalSlots,    // [7] tile consumed
    kDecFull = kEmpty + kLocalSlots, // [2] weights and e^{G_C} of a chunk made
    kDecEmpty = kDecFull + 2,   // [2] and read
    kGFull = kDecEmpty + 2,     // decays, their sums and the factors of score columns made
    kGEmpty,                    // and read
    kItemFull,                  // [3] item claimed
    kItemEmpty = kItemFull + kItems,
    kXFull = kItemEmpty + kItems,  // q k^T in X
    kPFull,                     // P in X
    kQSFull,                    // q S^T in O; S's operand read
    kQSScaled,                  // e^{G_i} applied
    kOFull,                     // the chunk's O complete
    kOEmpty,                    // and read
    kWFull,                     // [4] 32 tokens of W written, by buffer (two; Local: four)
    kWEmpty = kWFull + 4,       // [4] and read
    kDSFull = kWEmpty + 4,      // [2] dS complete (Local has two, by turns)
    kDSEmpty = kDSFull + 2,     // [2] and read
    kSFull = kDSEmpty + 2,      // S's operand written
    kCleared,                   // rows past a sequence's end cleared
    kDone,                      // everything issued has completed
    kNumBars
};
constexpr int kSmGamma = kSmBar + kNumBars * 8;  // [2] e^{G_C}, or kClearing
constexpr int kSmBad = (kSmGamma + 8 + 15) & ~15;  // [2][8] value columns with infinities or NaN
constexpr int kSmMisc = kSmBad + 64;             // tensor-memory base, abort flag
constexpr int kSmRows = kSmMisc + 8;             // warps done with a chunk's output rows
constexpr int kSmemBytes = kSmRows + 8;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
static_assert(kSmA % 16 == 0 && kSmT % 16 == 0 && kSmM % 16 == 0 && kSmCf % 16 == 0 && kSmBad % 16 == 0, "read by 16 bytes");
static_assert(kSmGamma % 8 == 0 && kSmMisc % 8 == 0 && kSmRows % 8 == 0, "words");

// Tensor memory columns.
constexpr uint32_t kTmX = 0;    // X; then P: per 16 tokens 8 columns high part, 8 low
constexpr uint32_t kTmO = 128;
constexpr uint32_t kTmDS = 256;
// W's buffers of 32 tokens: two K steps x four parts x 8 columns, two of them; Local has
// four, X's and O's places being free.
constexpr uint32_t kTmW = 384;
__host__ __device__ constexpr uint32_t w_column(bool local, int n) {
    return local && n >= 2 ? 64 * (n - 2) : kTmW + 64 * (n & 1);
}
constexpr uint32_t kTmCols = 512;
// dS's place, barrier and phase for chunk c.  Local has two, the other in O's place: with
// one, a chunk's products waited for the chunk before to be read (16384 tokens x 12 heads: 80.6 us
// instead of 82.0).
template <bool Local> __device__ __forceinline__ uint32_t ds_column(int c) { return Local && (c & 1) ? kTmO : kTmDS; }
template <bool Local> __device__ __forceinline__ int ds_bar(int c) { return Local ? c & 1 : 0; }
template <bool Local> __device__ __forceinline__ uint32_t ds_phase(int c) { return (Local ? c >> 1 : c) & 1; }

// In place of a decay over tokens of which one clears the state.
constexpr float kClearing = -1.f;

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

// 32 or 16 columns of this thread's lane.
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
__device__ __forceinline__ void tmem_ld16u(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
        : "memory");
}
// 16 lanes x 32 columns: per four columns two registers, of lane t/4 and lane t/4 + 8,
// column t%4.  The layout of ldmatrix fragments.  (A store of 8 columns takes as long as
// one of 32; with this one and seven slots 16384 tokens x 12 heads went from 83.6 to 82.4 us.)
__device__ __forceinline__ void tmem_st_16x32(uint32_t a, const uint32_t (&r)[4][4]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15};" ::"r"(r[0][0]),
        "r"(r[0][1]), "r"(r[0][2]), "r"(r[0][3]), "r"(r[1][0]), "r"(r[1][1]), "r"(r[1][2]), "r"(r[1][3]),
        "r"(r[2][0]), "r"(r[2][1]), "r"(r[2][2]), "r"(r[2][3]), "r"(r[3][0]), "r"(r[3][1]), "r"(r[3][2]),
        "r"(r[3][3]), "r"(a)
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

// Two fp32 values in one 64-bit register.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 from_bf(uint32_t x) { return pack2(bf_lo(x), bf_hi(x)); }
// The next bf16 part of a pair: returns it and leaves the exact remainder in a.
__device__ __forceinline__ uint32_t take_bf(f2& a) {
    const float2 v = unpack2(a);
    const uint32_t hi = pack_bf162(v.x, v.y);
    a = fma2(from_bf(hi), pack2(-1.f, -1.f), a);
    return hi;
}
__device__ __forceinline__ uint32_t last_bf(f2 a) {
    const float2 v = unpack2(a);
    return pack_bf162(v.x, v.y);
}
// Pairs of bf16.
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_bf2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t neg_bf2(uint32_t a) {
    uint32_t r;
    asm("neg.bf16x2 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Slots of a chunk's tiles, and the phase of their barriers.
constexpr int kQ = 0;
template <bool Local> __device__ __forceinline__ uint8_t* tile(int slot) {
    extern __shared__ __align__(1024) uint8_t smem[];
    return smem + (Local ? kSmS : kSmTile) + slot * kTile;
}
__device__ __forceinline__ uint32_t q_phase(int c) { return c & 1; }
template <bool Local> constexpr int kVs = Local ? 4 : 2;  // slots of v, and of k
template <bool Local> constexpr int kKs = Local ? 3 : 2;
template <bool Local> __device__ __forceinline__ int v_slot(int c) { return (Local ? 0 : 1) + c % kVs<Local>; }
template <bool Local> __device__ __forceinline__ int k_slot(int c) { return (Local ? 4 : 3) + c % kKs<Local>; }
template <bool Local> __device__ __forceinline__ uint32_t v_phase(int c) { return (c / kVs<Local>) & 1; }
template <bool Local> __device__ __forceinline__ uint32_t k_phase(int c) { return (c / kKs<Local>) & 1; }
static_assert(kSmS + kLocalSlots * kTile == kSmTile + kSlots * kTile, "the same room");

struct Maps {
    CUtensorMap q, k, v, out;
    CUtensorMap pool;  // boxes of 128 bytes of 32 rows
    int store_states;  // the pool has a map
};

// What every role needs.
struct Ctx {
    uint8_t* smem;
    uint64_t* bar;
    volatile int* abort;
    uint32_t tmem;
    int lane;

    // Waits for phases of barriers; gives up after about a second, or once another role
    // has (the callers then leave their loops).  A whole warp goes on or leaves together.
    // Waiting for several at once overlaps the looks at them, over a hundred cycles each
    // even when the phase is over.  A role must have seen a barrier's phase before last
    // to be over when it waits for one: parities alone do not tell them apart.
    __device__ __forceinline__ uint32_t at(int b) const { return smem_u32(smem) + kSmBar + 8 * b; }
#define KDA_WAIT_END                               \
    "@p bra DONE;\n\t"                             \
    "ld.volatile.shared.u32 f, [%1];\n\t"          \
    "setp.ne.u32 p, f, 0;\n\t"                     \
    "@p bra OUT;\n\t"                              \
    "sub.u32 n, n, 1;\n\t"                         \
    "setp.ne.u32 p, n, 0;\n\t"                     \
    "@p bra AGAIN;\n\t"                            \
    "st.volatile.shared.u32 [%1], 1;\n\t"          \
    "OUT:\n\tmov.u32 %0, 0;\n\tbra END;\n\t"      \
    "DONE:\n\tmov.u32 %0, 1;\n\tEND:\n\t}"
    __device__ __forceinline__ bool wait(int b, uint32_t parity) const {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .u32 n, f;\n\tmov.u32 n, %2;\n\tAGAIN:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%3], %4;\n\t" KDA_WAIT_END
            : "=r"(ok)
            : "r"(smem_u32(smem) + kSmMisc + 4), "n"(kWaitLimit), "r"(at(b)), "r"(parity)
            : "memory");
        return ok != 0;
    }
    __device__ __forceinline__ bool wait_all(int b, uint32_t parity) const {
        return __all_sync(0xffffffffu, wait(b, parity));
    }
    __device__ __forceinline__ bool wait_all(int b0, uint32_t p0, int b1, uint32_t p1) const {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 n, f;\n\tmov.u32 n, %2;\n\tAGAIN:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%3], %4;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 q, [%5], %6;\n\tand.pred p, p, q;\n\t" KDA_WAIT_END
            : "=r"(ok)
            : "r"(smem_u32(smem) + kSmMisc + 4), "n"(kWaitLimit), "r"(at(b0)), "r"(p0), "r"(at(b1)), "r"(p1)
            : "memory");
        return __all_sync(0xffffffffu, ok != 0);
    }
    __device__ __forceinline__ bool wait_all(int b0, uint32_t p0, int b1, uint32_t p1, int b2, uint32_t p2) const {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 n, f;\n\tmov.u32 n, %2;\n\tAGAIN:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%3], %4;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 q, [%5], %6;\n\tand.pred p, p, q;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 q, [%7], %8;\n\tand.pred p, p, q;\n\t" KDA_WAIT_END
            : "=r"(ok)
            : "r"(smem_u32(smem) + kSmMisc + 4), "n"(kWaitLimit), "r"(at(b0)), "r"(p0), "r"(at(b1)), "r"(p1),
              "r"(at(b2)), "r"(p2)
            : "memory");
        return __all_sync(0xffffffffu, ok != 0);
    }
#undef KDA_WAIT_END
    __device__ __forceinline__ void arrive(int b) const { mbar_arrive(bar + b); }
    // Parts of the weights of the token pairs of chunk c.
    __device__ __forceinline__ const uint32_t* weights(int c) const {
        return reinterpret_cast<const uint32_t*>(smem + kSmW) + (c & 1) * 3 * (C / 2);
    }
    // Whether the chunk whose decays are there has a clearing token.
    __device__ __forceinline__ bool clears() const {
        const uint4 m = *reinterpret_cast<const uint4*>(smem + kSmM);
        return (m.x | m.y | m.z | m.w) != 0;
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
// The last clearing token up to a row of the chunk, or -1.
__device__ __forceinline__ int last_clearing(const uint4 m, int row) {
    const uint32_t words[4] = {m.x, m.y, m.z, m.w};
    int at = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t up_to = row < 32 * i ? 0u : row >= 32 * i + 31 ? ~0u : (2u << (row - 32 * i)) - 1u;
        if (words[i] & up_to) at = 32 * i + 31 - __clz(words[i] & up_to);
    }
    return at;
}

// ---- warp 30: items and decays ------------------------------------------------
// Item i of the call.  The cut sequences' segments come first; Local: all but their last.
template <bool Local>
__device__ __forceinline__ Item make_item(const LinParams& p, const LinCuts& cuts, int i, int lane) {
    Item item{};
    const int k = i / p.H;
    item.h = i - k * p.H;
    const int n_seg = Local ? p.n_seg - p.n_cut : p.n_seg;
    bool last = true;
    if (k < n_seg) {
        int r = 0;
        for (;; r += 32) {  // the sequence whose segments k is among
            const int m = r + lane;
            const uint32_t past = __ballot_sync(0xffffffffu, m < p.n_cut && cuts.first[m + 1] - (Local ? m + 1 : 0) > k);
            if (past || r + 32 >= p.n_cut) {
                r += past ? __ffs(past) - 1 : 0;
                break;
            }
        }
        const int s = k - (cuts.first[r] - (Local ? r : 0));
        item.n = cuts.seq[r];
        item.t0 = cuts.t0[r] + s * p.seg_len;
        item.len = min(p.seg_len, cuts.len[r] - s * p.seg_len);
        item.plane = (cuts.first[r] + s) * p.H + item.h;
        item.flags = kPlane;
        last = cuts.first[r] + s + 1 == cuts.first[r + 1];
    } else {
        item.n = p.long_list[p.n_cut + k - n_seg];
        item.t0 = p.cu[item.n];
        item.len = p.cu[item.n + 1] - item.t0;
    }
    if (Local) return item;
    if (last) item.flags |= kStore;
    // a segment's initial state is in the workspace, and the state warps look its slot up
    if (k >= n_seg) {
        const int slot = p.idx[item.n];
        if (p.has_init[item.n] && slot >= 0 && slot < p.num_slots) {
            item.flags |= kInit;
            // into the L2 cache: the state warps get there when the item before is done
            const int bytes = D * D * (p.st_dtype == KDA_STATE_F32 ? 4 : 2);
            const char* from = static_cast<const char*>(p.pool) +
                               ((size_t)slot * p.stride0 + (size_t)item.h * D * D) * (bytes / (D * D));
            if (lane == 0)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
        }
    }
    return item;
}

template <bool Local>
__device__ __forceinline__ void decay_role(const LinParams& p, const LinCuts& cuts, const Ctx& x) {
    const int n_items = (Local ? p.n_seg - p.n_cut : p.n_seg + p.n_long - p.n_cut) * p.H;
    int* queue = reinterpret_cast<int*>(reinterpret_cast<char*>(p.status) + (Local ? kWsDecodeOff : kWsQueueOff));
    int c = 0;
    for (int it = 0;; ++it) {
        if (it >= kItems && !x.wait_all(kItemEmpty + it % kItems, ((it / kItems) + 1) & 1)) return;
        int i = blockIdx.x;  // the first item by place, the others in the order of their claims
        if (it > 0 && n_items <= (int)gridDim.x) {
            i = n_items;
        } else if (it > 0) {
            if (x.lane == 0) i = gridDim.x + atomicAdd(queue, 1);
            i = __shfl_sync(0xffffffffu, i, 0);
        }
        Item item{};
        if (i < n_items)
            item = make_item<Local>(p, cuts, i, x.lane);
        else
            item.flags = kEnd;
        if (x.lane == 0) {
            reinterpret_cast<Item*>(x.smem + kSmItem)[it % kItems] = item;
            x.arrive(kItemFull + it % kItems);  // releases the write
        }
        if (item.flags & kEnd) return;
        const float* g = p.g + item.h;
        for (int j = 0; j < chunks(item.len); ++j, ++c) {
            // four tokens a lane; tokens past the end decay nothing
            float a[4], suf[4];
            uint32_t clear = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = j * C + 4 * x.lane + e;
                float v = 0.f;
                if (t < item.len) v = g[(int64_t)(item.t0 + t) * p.g_st];
                a[e] = v < kMinDecay ? kMinDecay : v;
                clear |= v < kMinDecay ? 1u << e : 0u;
            }
            suf[3] = 0.f;
#pragma unroll
            for (int e = 2; e >= 0; --e) suf[e] = suf[e + 1] + a[e + 1];
            const float sum = suf[0] + a[0];
            float down = sum;  // over the lanes from here on
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const float d = __shfl_down_sync(0xffffffffu, down, w);
                if (x.lane + w < 32) down += d;
            }
            const float total = __shfl_sync(0xffffffffu, down, 0);
            float after = __shfl_down_sync(0xffffffffu, down, 1);
            if (x.lane == 31) after = 0.f;
            if (c >= 2 && !x.wait_all(kDecEmpty + (c & 1), ((c >> 1) + 1) & 1)) return;
            uint32_t* w = const_cast<uint32_t*>(x.weights(c)) + 6 * x.lane;
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                f2 v = pack2(expf(after + (u ? suf[2] : suf[0])), expf(after + (u ? suf[3] : suf[1])));
                w[3 * u] = take_bf(v);
                w[3 * u + 1] = take_bf(v);
                w[3 * u + 2] = last_bf(v);
            }
            const bool clears = __any_sync(0xffffffffu, clear != 0);
            if (x.lane == 0)
                reinterpret_cast<float*>(x.smem + kSmGamma)[c & 1] = clears ? kClearing : expf(total);
            __syncwarp();
            if (x.lane == 0) x.arrive(kDecFull + (c & 1));
            if (Local) continue;
            // the sums from here to the end of each 32 tokens (eight lanes)
            float rest = sum;
#pragma unroll
            for (int w = 1; w < 8; w <<= 1) {
                const float d = __shfl_down_sync(0xffffffffu, rest, w, 8);
                if ((x.lane & 7) + w < 8) rest += d;
            }
            const float sum32 = rest;  // of the eight lanes, in their first one
            uint32_t clear32 = clear << (4 * (x.lane & 7));
            if (clears) {
#pragma unroll
                for (int w = 1; w < 8; w <<= 1) clear32 |= __shfl_xor_sync(0xffffffffu, clear32, w);
            }
            rest = __shfl_down_sync(0xffffffffu, rest, 1, 8);
            if ((x.lane & 7) == 7) rest = 0.f;
            if (c > 0 && !x.wait_all(kGEmpty, (c + 1) & 1)) return;
            constexpr float kLog2e = 1.4426950408889634f;
            reinterpret_cast<float4*>(x.smem + kSmA)[x.lane] =
                make_float4(a[0] * kLog2e, a[1] * kLog2e, a[2] * kLog2e, a[3] * kLog2e);
            if ((x.lane & 7) == 0) {
                reinterpret_cast<float*>(x.smem + kSmT)[x.lane >> 3] = sum32 * kLog2e;
                reinterpret_cast<uint32_t*>(x.smem + kSmM)[x.lane >> 3] = clear32;
            }
            if (x.lane < 24)
                reinterpret_cast<float4*>(x.smem + kSmCf)[x.lane] =
                    make_float4(expf(rest + suf[0]), expf(rest + suf[1]), expf(rest + suf[2]), expf(rest + suf[3]));
            __syncwarp();
            if (x.lane == 0) x.arrive(kGFull);
        }
    }
}

// ---- warp 29, one lane: loads -------------------------------------------------
// Returns the numbers of q, v and k tiles issued.
template <bool Local>
__device__ __forceinline__ int3 load_role(const Maps& maps, const LinParams& p, const Ctx& x) {
    int c = 0;
    auto load = [&](int slot, const CUtensorMap* map, int h, int t) {
        uint64_t* bar = x.bar + kFull + slot;
        uint8_t* dst = tile<Local>(slot);
        mbar_arrive_expect_tx(bar, kTile);
        tma_load_3d(dst, map, bar, 0, h, t);
        tma_load_3d(dst + kTile / 2, map, bar, 64, h, t);
    };
    Item item;
    for (int it = 0; x.item(it, &item, false); ++it) {
        for (int j = 0; j < chunks(item.len); ++j, ++c) {
            const int t = item.t0 + j * C;
            if (c >= kVs<Local> && !x.wait(kEmpty + v_slot<Local>(c), v_phase<Local>(c) ^ 1)) return make_int3(c, c, c);
            load(v_slot<Local>(c), &maps.v, item.h, t);
            if constexpr (!Local) {
                if (c >= 1 && !x.wait(kEmpty + kQ, q_phase(c) ^ 1)) return make_int3(c, c + 1, c);
                load(kQ, &maps.q, item.h / p.rep, t);
            }
            if (c >= kKs<Local> && !x.wait(kEmpty + k_slot<Local>(c), k_phase<Local>(c) ^ 1)) return make_int3(c + 1, c + 1, c);
            load(k_slot<Local>(c), &maps.k, item.h / p.rep, t);
        }
    }
    return make_int3(c, c, c);
}

// ---- warp 28: products ----------------------------------------------------------
// The warp runs as one (descriptors stay in uniform registers); one elected lane
// issues.
template <bool Local>
__device__ __forceinline__ void mma_role(const Ctx& x) {
    const uint32_t base = smem_u32(x.smem);
    // descriptors of a tile read K-major (16 columns a step) and MN-major (16 rows)
    auto kdesc = [&](uint32_t a) { return sw128_desc(a, 16, 1024); };
    auto mdesc = [&](uint32_t a) { return sw128_desc(a, kTile / 2, 1024); };
    constexpr auto kstep = [](int ks) { return (uint64_t)(((ks >> 2) * (kTile / 2) + (ks & 3) * 32) >> 4); };
    constexpr auto mstep = [](int ks) { return (uint64_t)((ks * 2048) >> 4); };
    const uint64_t s_hi = kdesc(base + kSmS), s_lo = kdesc(base + kSmS + kTile);
    const bool lead = elect_one();
    int c = 0, with_s = 0;
    Item item;
    for (int it = 0; x.item(it, &item, true); ++it) {
        const int nc = chunks(item.len);
        for (int j = 0; j < nc; ++j, ++c) {
            const bool has_s = j > 0 || (item.flags & (kInit | kPlane));
            const uint32_t qa = smem_u32(tile<Local>(kQ)), va = smem_u32(tile<Local>(v_slot<Local>(c))),
                           ka = smem_u32(tile<Local>(k_slot<Local>(c)));
            const uint64_t k = kdesc(ka), q = kdesc(qa), km = mdesc(ka), vm = mdesc(va);
            auto add_tokens = [&](int n) {  // dS over tokens 32 n .. 32 n + 31
                tc_fence_after();
                if (lead) {
#pragma unroll 1
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int part = 3; part >= 0; --part)  // the smallest first
                            mma_f16_ts(x.tmem + ds_column<Local>(c), x.tmem + w_column(Local, n) + 32 * s + 8 * part,
                                       km + mstep(2 * n + s), kIdescKM, n > 0 || s > 0 || part < 3);
                    mma_commit(x.bar + kWEmpty + (Local ? n : n & 1));
                }
                __syncwarp();
            };
            if constexpr (Local) {
                if (c < 2 ? !x.wait_all(kFull + k_slot<Local>(c), k_phase<Local>(c))
                          : !x.wait_all(kFull + k_slot<Local>(c), k_phase<Local>(c),
                                        kDSEmpty + ds_bar<Local>(c), ds_phase<Local>(c) ^ 1)) return;
#pragma unroll 1
                for (int n = 0; n < 4; ++n) {
                    if (!x.wait_all(kWFull + n, c & 1)) return;
                    add_tokens(n);
                }
                if (lead) {
                    x.arrive(kEmpty + v_slot<Local>(c));  // read by the W warps alone
                    mma_commit(x.bar + kDSFull + ds_bar<Local>(c));
                    mma_commit(x.bar + kEmpty + k_slot<Local>(c));
                }
                __syncwarp();
                continue;
            }
            if (c == 0 ? !x.wait_all(kFull + k_slot<Local>(c), k_phase<Local>(c), kWFull, 0)
                       : !x.wait_all(kFull + k_slot<Local>(c), k_phase<Local>(c), kWFull, 0, kDSEmpty, (c + 1) & 1)) return;
            add_tokens(0);
            // X is free once the previous chunk's P v has read it
            if (c == 0 ? !x.wait_all(kFull + kQ, q_phase(c))
                       : !x.wait_all(kFull + kQ, q_phase(c), kOFull, (c + 1) & 1)) return;
            tc_fence_after();
            if (lead) {
#pragma unroll 2
                for (int ks = 0; ks < 8; ++ks)
                    mma_f16_ss(x.tmem + kTmX, q + kstep(ks), k + kstep(ks), kIdescKK, ks > 0);
                mma_commit(x.bar + kXFull);
                if (!has_s) mma_commit(x.bar + kEmpty + kQ);
            }
            __syncwarp();
            if (!x.wait_all(kWFull + 1, 0)) return;
            add_tokens(1);
            // O is free once the previous chunk's rows have been read
            if (has_s) {
                if (c == 0 ? !x.wait_all(kSFull, with_s & 1) : !x.wait_all(kSFull, with_s & 1, kOEmpty, (c + 1) & 1)) return;
                tc_fence_after();
                if (lead) {
#pragma unroll 2
                    for (int ks = 0; ks < 16; ++ks)  // the low part first
                        mma_f16_ss(x.tmem + kTmO, q + kstep(ks & 7), (ks < 8 ? s_lo : s_hi) + kstep(ks & 7), kIdescKK, ks > 0);
                    mma_commit(x.bar + kQSFull);
                    mma_commit(x.bar + kEmpty + kQ);
                }
                __syncwarp();
            }
            if (!x.wait_all(kWFull, 1)) return;
            add_tokens(2);
            if (!x.wait_all(kWFull + 1, 1)) return;
            add_tokens(3);
            if (lead) mma_commit(x.bar + kDSFull);
            __syncwarp();
            if (has_s ? !x.wait_all(kPFull, c & 1, kQSScaled, with_s & 1)
                      : c == 0 ? !x.wait_all(kPFull, 0) : !x.wait_all(kPFull, c & 1, kOEmpty, (c + 1) & 1)) return;
            tc_fence_after();
            if (lead) {
#pragma unroll 1
                for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (int part = 1; part >= 0; --part)
                        mma_f16_ts(x.tmem + kTmO, x.tmem + kTmX + 16 * ks + 8 * part,
                                   vm + mstep(ks), kIdescKM, has_s || ks > 0 || part == 0);
                mma_commit(x.bar + kOFull);  // k's tile takes the output rows now
                mma_commit(x.bar + kEmpty + v_slot<Local>(c));
            }
            __syncwarp();
            with_s += has_s;
        }
    }
}

// Puts a NaN into the row's columns, of those in `cols`, where v holds an infinity or
// NaN between tokens t0 and t1 of the item, from the last clearing one on.
__device__ __noinline__ void put_nonfinite(const LinParams& p, const Item& item, int t0, int t1, int row,
                                           uint4 cols, uint8_t* tile) {
    const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v) + (int64_t)item.h * p.v_sh;
#pragma unroll 1
    for (int t = t1; t > t0; --t)
        if (p.g[(int64_t)(item.t0 + t) * p.g_st + item.h] < kMinDecay) t0 = t;
#pragma unroll 1
    for (int g = 0; g < 4; ++g)
#pragma unroll 1
        for (uint32_t m = g == 0 ? cols.x : g == 1 ? cols.y : g == 2 ? cols.z : cols.w; m; m &= m - 1) {
            const int col = 32 * g + __ffs(m) - 1;
#pragma unroll 1
            for (int t = t0; t <= t1; ++t)
                if ((v[(int64_t)(item.t0 + t) * p.v_st + col] & 0x7F80) == 0x7F80) {
                    *reinterpret_cast<uint16_t*>(tile + sw128_off(row, col, C)) = 0x7FFF;
                    break;
                }
        }
}

// Zeroes the scores of columns before the row's last clearing token, which may be NaN.
__device__ __noinline__ void drop_scores(uint32_t tm, int warp) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int w = warp & 3, n = last_clearing(*reinterpret_cast<const uint4*>(smem + kSmM), 32 * w + (threadIdx.x & 31)) - 16 * (warp >> 2);
#pragma unroll 1
    for (int b = 0; b <= w; ++b) {
        uint32_t r[16];
        tmem_ld16u(tm + 32 * b, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (32 * b + e < n) r[e] = 0u;
        tmem_st16(tm + 32 * b, r);
    }
    tmem_wait_st();
}

// ---- warps 16-23: scores; thread = chunk row ------------------------------------
// Warps 16-19 take the even groups of 16 columns, warps 20-23 the odd ones.
__device__ __forceinline__ void score_role(const LinParams& p, const Ctx& x, int w8) {
    const int w = w8 & 3, odd = w8 >> 2;
    const int row = 32 * w + x.lane;
    const uint32_t tm = x.tmem + ((uint32_t)(32 * w) << 16) + kTmX + 16 * odd;
    const float* A = reinterpret_cast<const float*>(x.smem + kSmA);
    const float* T = reinterpret_cast<const float*>(x.smem + kSmT);
    const float2* cf = reinterpret_cast<const float2*>(x.smem + kSmCf) + 8 * odd;
    int c = 0;
    Item item;
    for (int it = 0; x.item(it, &item, true); ++it) {
        for (int j = 0; j < chunks(item.len); ++j, ++c) {
            // The decays are there long before the scores.  Their sums up to this row from the
            // first token of its 16, and from that of its 32.
            if (!x.wait_all(kGFull, c & 1)) return;
            float from16 = A[row];
#pragma unroll
            for (int u = 1; u < 16; u <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, from16, u, 16);
                if ((x.lane & 15) >= u) from16 += up;
            }
            const float first16 = __shfl_sync(0xffffffffu, from16, 15);
            float left = x.lane & 16 ? first16 + from16 : from16;
            const bool clears = x.clears();
            if (!x.wait_all(kXFull, c & 1)) return;
            tc_fence_after();
            if (clears) drop_scores(tm, w8);
            // Sixteen scores become eight pairs of high parts and eight of low parts, in place,
            // the last columns first.
            uint32_t r[16];
            auto split_and_store = [&](int b, auto factor) {
                uint32_t o[16];
#pragma unroll
                for (int e = 14; e >= 0; e -= 2) {
                    f2 v = mul2(pack2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), factor(e));
                    o[e / 2] = take_bf(v);
                    o[8 + e / 2] = last_bf(v);
                }
                tmem_st16(tm + 32 * b, o);
            };
#pragma unroll 1
            for (int b = w - 1; b >= 0; --b) {
                tmem_ld16u(tm + 32 * b, r);
                const float f = ex2(left);
                left += T[b];
                const f2 ff = pack2(f, f);
                tmem_wait_ld();
                split_and_store(b, [&](int e) {
                    const float2 u = cf[16 * b + e / 2];
                    return mul2(ff, pack2(u.x, u.y));
                });
            }
            tmem_ld16u(tm + 32 * w, r);
            const float2* Aw = reinterpret_cast<const float2*>(A + 32 * w + 16 * odd);
            const int last = x.lane - 16 * odd;  // of this row, in the group
            float d = last > 15 ? from16 : 0.f;
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e > last) r[e] = 0u;
            split_and_store(w, [&](int e) {
                const float2 u = Aw[e / 2];
                const float f1 = ex2(d);
                if (e + 1 <= last) d += u.y;
                const float f0 = ex2(d);
                if (e <= last) d += u.x;
                return pack2(f0, f1);
            });
            const uint32_t zero[16] = {};
#pragma unroll 1
            for (int b = w + 1; b < 4; ++b) tmem_st16(tm + 32 * b, zero);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (x.lane == 0) {
                x.arrive(kPFull);
                x.arrive(kGEmpty);
            }
        }
    }
}

// ---- warps 24-27: output rows; thread = chunk row --------------------------------
__device__ __forceinline__ void out_role(const Maps& maps, const LinParams& p, const Ctx& x, int w) {
    const int row = 32 * w + x.lane;
    const uint32_t tm = x.tmem + ((uint32_t)(32 * w) << 16) + kTmO;
    const f2 scale = pack2(p.scale, p.scale);
    int c = 0, with_s = 0;
    Item item;
    for (int it = 0; x.item(it, &item, true); ++it) {
        for (int j = 0; j < chunks(item.len); ++j, ++c) {
            const bool has_s = j > 0 || (item.flags & (kInit | kPlane));
            if (!x.wait_all(kGFull, c & 1)) return;
            float sum = reinterpret_cast<const float*>(x.smem + kSmA)[row];  // from the chunk's start on
#pragma unroll
            for (int u = 1; u < 32; u <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, sum, u);
                if (x.lane >= u) sum += up;
            }
            const float4 T = *reinterpret_cast<const float4*>(x.smem + kSmT);
            if (w > 2) sum += T.z;
            if (w > 1) sum += T.y;
            if (w > 0) sum += T.x;
            float f = ex2(sum);
            if (x.clears() && last_clearing(*reinterpret_cast<const uint4*>(x.smem + kSmM), row) >= 0) f = kClearing;
            __syncwarp();
            if (x.lane == 0) x.arrive(kGEmpty);
            if (has_s) {
                if (!x.wait_all(kQSFull, with_s & 1)) return;
                tc_fence_after();
                const f2 ff = pack2(f, f);
                const bool dead = f == kClearing, some = __any_sync(0xffffffffu, dead);
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tm + 32 * b, r);
                    tmem_wait_ld();
                    if (some) {  // may be NaN
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = dead ? 0u : r[e];
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 v = unpack2(mul2(ff, pack2(__uint_as_float(r[e]), __uint_as_float(r[e + 1]))));
                        r[e] = __float_as_uint(v.x), r[e + 1] = __float_as_uint(v.y);
                    }
                    tmem_st32(tm + 32 * b, r);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (x.lane == 0) x.arrive(kQSScaled);
                ++with_s;
            }
            if (!x.wait_all(kOFull, c & 1)) return;
            tc_fence_after();
            // The rows go through k's tile, which has been read, so that whole rows
            // are written to memory: lanes that each store a row of their own fill
            // the load/store unit with single sectors and hold up everything else.
            uint8_t* kt = tile<false>(k_slot<false>(c));
            const uint4* bad = reinterpret_cast<const uint4*>(x.smem + kSmBad) + 2 * (c & 1);
            uint4 cols = bad[0];
            cols.x |= bad[1].x, cols.y |= bad[1].y, cols.z |= bad[1].z, cols.w |= bad[1].w;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                uint32_t r[32];
                tmem_ld32(tm + 32 * b, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t y[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        y[u] = last_bf(mul2(scale, pack2(__uint_as_float(r[e + 2 * u]), __uint_as_float(r[e + 2 * u + 1]))));
                    *reinterpret_cast<uint4*>(kt + sw128_off(row, 32 * b + e, C)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (x.lane == 0) x.arrive(kOEmpty);
            if (cols.x | cols.y | cols.z | cols.w)
                put_nonfinite(p, item, j * C, min(j * C + row, item.len - 1), row, cols, kt);
            const int live = item.len - j * C - 32 * w;  // rows of this warp's 32
            const int t = item.t0 + j * C + 32 * w;
            fence_proxy_async();
            __syncwarp();
            if (live >= 32) {
                if (x.lane == 0) {
                    tma_store_3d(&maps.out, kt + 32 * w * 128, 0, item.h, t);
                    tma_store_3d(&maps.out, kt + kTile / 2 + 32 * w * 128, 64, item.h, t);
                    bulk_commit();
                    bulk_wait_read_all();
                }
            } else {
                // two rows at a time, 16 bytes a lane
                const int half = x.lane >> 4, l16 = x.lane & 15;
                __nv_bfloat16* out = p.out + ((int64_t)t * p.H + item.h) * D + 8 * l16;
#pragma unroll 1
                for (int r = half; r < live; r += 2)
                    *reinterpret_cast<uint4*>(out + (int64_t)r * p.H * D) =
                        *reinterpret_cast<const uint4*>(kt + sw128_off(32 * w + r, 8 * l16, C));
                fence_proxy_async();
            }
            // the last of the four warps frees the tile
            __syncwarp();
            if (x.lane == 0) {
                __threadfence_block();
                if ((atomicAdd(reinterpret_cast<int*>(x.smem + kSmRows), 1) & 3) == 3)
                    x.arrive(kEmpty + k_slot<false>(c));
            }
        }
    }
}

// Clears infinities and NaN in a lane's column, in every other 32 tokens from `odd` on;
// returns the warp's columns that had any.
__device__ __noinline__ uint32_t clear_nonfinite(uint8_t* vt, int col, int odd) {
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        const int tok = 64 * (i >> 5) + 32 * odd + (i & 31);
        uint16_t* at = reinterpret_cast<uint16_t*>(vt + sw128_off(tok, col, C));
        if ((*at & 0x7F80) == 0x7F80) {
            *at = 0;
            any = true;
        }
    }
    fence_proxy_async();
    return __ballot_sync(0xffffffffu, any);
}

// ---- warps 8-15: weighted v ---------------------------------------------------------
// A warp makes 32 value rows of 32 tokens at a time: warps 8-11 of the first and third 32,
// warps 12-15 of the others; Local: each four warps of warps 8-23 of one 32.
template <bool Local>
__device__ __forceinline__ void weight_role(const LinParams& p, const Ctx& x, int w8) {
    const int w4 = w8 & 3, group = w8 >> 2;
    const uint32_t tm = x.tmem + ((uint32_t)(32 * w4) << 16);
    // a lane's place in four 8 x 8 matrices: tokens 0-7 and 8-15, value rows 0-7 and 8-15
    const int tok = (x.lane & 7) + ((x.lane >> 4) << 3);
    const int col = 32 * w4 + (((x.lane >> 3) & 1) << 3);
    int c = 0, cleared = 0;
    Item item;
    for (int it = 0; x.item(it, &item, true); ++it) {
        const int nc = chunks(item.len);
        for (int j = 0; j < nc; ++j, ++c) {
            const int live = min(C, item.len - j * C);
            uint8_t* vt = tile<Local>(v_slot<Local>(c));
            if (!x.wait_all(kFull + v_slot<Local>(c), v_phase<Local>(c))) return;
            if (!Local && live < C) {  // (a segment but the last is full)
                // rows past the sequence's end belong to others: they weigh nothing,
                // and may hold anything, so they are cleared
                if (!x.wait_all(kFull + k_slot<Local>(c), k_phase<Local>(c))) return;
                uint8_t* kt = tile<Local>(k_slot<Local>(c));
#pragma unroll 1
                for (int i = 32 * w8 + x.lane; i < (C - live) * 16; i += 256) {
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
            const uint32_t* wt = x.weights(c) + 3 * (x.lane & 3);
            const uint32_t vs = smem_u32(vt);
            uint32_t nan2 = 0;  // becomes NaN with any part that is one
#pragma unroll 1
            for (int n = group; n < 4; n += Local ? 4 : 2) {
                const int b = Local ? n : group, t0 = 32 * n;
                const uint32_t column = w_column(Local, n);
                // the buffer's last steps have been read
                if (Local ? c > 0 && !x.wait_all(kWEmpty + b, (c + 1) & 1)
                          : (c > 0 || n >= 2) && !x.wait_all(kWEmpty + b, n < 2)) return;
                tc_fence_after();
#pragma unroll 1
                for (int s = 0; s < 2; ++s) {  // 16 tokens
                    uint32_t w[2][3];  // the weights' parts, of tokens 2 (lane % 4) .. + 1 and those 8 on
#pragma unroll
                    for (int u = 0; u < 3; ++u) {
                        w[0][u] = wt[3 * (t0 / 2 + 8 * s) + u];
                        w[1][u] = wt[3 * (t0 / 2 + 8 * s + 4) + u];
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {  // 16 value rows
                        uint32_t r[4], t[4][4];
                        ldsm_x4_t(vs + sw128_off(t0 + 16 * s + tok, col + 16 * i, C), r[0], r[1], r[2], r[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t* u = w[e >> 1];
                            t[0][e] = mul_bf2(r[e], u[0]);
                            t[1][e] = fma_bf2(r[e], u[0], neg_bf2(t[0][e]));  // exact
                            t[2][e] = mul_bf2(r[e], u[1]);
                            t[3][e] = fma_bf2(r[e], u[2], fma_bf2(r[e], u[1], neg_bf2(t[2][e])));
                            nan2 = fma_bf2(t[1][e], 0u, nan2);  // an infinite or NaN value leaves a NaN
                        }
                        const uint32_t at = tm + ((uint32_t)(16 * i) << 16) + column + 32 * s;
                        tmem_st_16x32(at, t);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                if (!Local && n >= 2) {
                    uint32_t cols = 0;
                    if (__any_sync(0xffffffffu, (nan2 & 0x7FFF7FFFu) != 0))
                        cols = clear_nonfinite(vt, 32 * w4 + x.lane, group);
                    if (x.lane == 0) reinterpret_cast<uint32_t*>(x.smem + kSmBad)[8 * (c & 1) + w8] = cols;
                }
                __syncwarp();
                if (x.lane == 0) x.arrive(kWFull + b);
            }
            if (x.lane == 0) x.arrive(kDecEmpty + (c & 1));
        }
    }
}

// ---- warps 0-7: the state ----------------------------------------------------------
// Thread: value row 32 (warp % 4) + lane, key columns 64 (warp / 4) .. + 63.
template <class P>
__device__ __forceinline__ float4 load4(const P* s);
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

// Where this warp's part of the dS of a cleared chunk (`live` tokens from t0 on) is not
// finite, makes it anew in place: sums the tokens from the last clearing one on.
__device__ __noinline__ void mend_ds(const LinParams& p, int t0, int live, int h, uint32_t tm, int row, int col) {
    uint32_t r[16];
    float nan = 0.f;
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
        tmem_ld16u(tm + 16 * b, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) nan = fmaf(__uint_as_float(r[e]), 0.f, nan);
    }
    if (!__any_sync(0xffffffffu, nan != 0.f)) return;
    const __nv_bfloat16* v = p.v + (int64_t)h * p.v_sh + row;
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
        const __nv_bfloat16* k = p.k + (int64_t)(h / p.rep) * p.k_sh + col + 16 * b;
        float decay = 0.f;  // after token t
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = 0u;
#pragma unroll 1
        for (int t = t0 + live - 1; t >= t0; --t) {
            const float w = expf(decay) * __bfloat162float(v[(int64_t)t * p.v_st]);
            const uint4* kt = reinterpret_cast<const uint4*>(k + (int64_t)t * p.k_st);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 u = kt[i];
                const uint32_t pair[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t* at = r + 8 * i + 2 * e;
                    at[0] = __float_as_uint(fmaf(w, bf_lo(pair[e]), __uint_as_float(at[0])));
                    at[1] = __float_as_uint(fmaf(w, bf_hi(pair[e]), __uint_as_float(at[1])));
                }
            }
            const float g = p.g[(int64_t)t * p.g_st + h];
            if (g < kMinDecay) break;
            decay += g;
        }
        tmem_st16(tm + 16 * b, r);
    }
    tmem_wait_st();
}

template <class P, bool Local>
__device__ __forceinline__ void state_role(const Maps& maps, const LinParams& p, const Ctx& x, int warp) {
    const int sg = warp >> 2;
    const int row = 32 * (warp & 3) + x.lane;
    const uint32_t tm = x.tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 64 * sg;
    int c = 0;
    f2 S[32];
    // S as the product's operand: row `row`, columns 64 sg .. + 63
    auto write_operand = [&]() {
        uint8_t* at = x.smem + kSmS + sg * (kTile / 2) + row * 128;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                f2 a = S[4 * e + u];
                hi[u] = take_bf(a);
                lo[u] = last_bf(a);
            }
            const uint32_t chunk = (e ^ (row & 7)) << 4;
            *reinterpret_cast<uint4*>(at + chunk) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(at + kTile + chunk) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async();
        __syncwarp();
        if (x.lane == 0) x.arrive(kSFull);
    };
    // The warp's 32 x 64 fp32 values of S in the shared memory of its part of the
    // operand (4 KB of the high, 4 KB of the low part): row r, values 4 e .. 4 e + 3.
    // Pool rows pass through it so that memory sees whole rows, not one a lane.
    auto staged = [&](int r, int e) {
        return reinterpret_cast<float4*>(x.smem + kSmS + (e >> 3) * kTile + sg * (kTile / 2) +
                                         (32 * (warp & 3) + r) * 128 + (((e & 7) ^ (r & 7)) << 4));
    };
    const int l16 = x.lane & 15, half = x.lane >> 4;
    bool leaving = false;  // a state on its way from the operand's place to the pool
    auto place_free = [&]() {
        if (leaving) {
            if (x.lane == 0) bulk_wait_read_all();
            __syncwarp();
            leaving = false;
        }
    };
    Item item;
    for (int it = 0; x.item(it, &item, true); ++it) {
        const int nc = chunks(item.len);
        // this lane's 4 columns of the warp's rows half, half + 2, ...
        const int slot = Local ? 0 : p.idx[item.n];
        const bool ok = slot >= 0 && slot < p.num_slots;
        P* pool = static_cast<P*>(p.pool) + (ok ? (size_t)slot * p.stride0 : 0) +
                  ((size_t)item.h * D + 32 * (warp & 3) + half) * D + 64 * sg + 4 * l16;
        // a segment's state in the workspace: this thread's 4 columns 4 e .. every 256 x 4 values
        float4* plane = reinterpret_cast<float4*>(p.planes) + (size_t)item.plane * (D * D / 4) + 32 * warp + x.lane;
        float kept = 1.f;  // Local: what is left of the state after the segment, or kClearing
        if (!Local && (item.flags & kPlane)) {
            grid_dep_wait();  // the chain kernel may still run
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float4 v = plane[256 * e];
                S[2 * e] = pack2(v.x, v.y), S[2 * e + 1] = pack2(v.z, v.w);
            }
            place_free();
            write_operand();
        } else if (!Local && (item.flags & kInit)) {
            float4 rows[16];  // all in flight at once
#pragma unroll
            for (int r = 0; r < 16; ++r) rows[r] = load4<P>(pool + 2 * r * D);
            place_free();
            // the last q S^T has read the operand: it was issued before the last dS
#pragma unroll
            for (int r = 0; r < 16; ++r) *staged(2 * r + half, l16) = rows[r];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float4 v = *staged(x.lane, e);
                S[2 * e] = pack2(v.x, v.y), S[2 * e + 1] = pack2(v.z, v.w);
            }
            __syncwarp();
            write_operand();
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) S[e] = 0ull;
        }
        for (int j = 0; j < nc; ++j, ++c) {
            if (!x.wait_all(kDecFull + (c & 1), (c >> 1) & 1)) return;
            const float gamma = x.gamma(c);
            __syncwarp();
            if (x.lane == 0) x.arrive(kDecEmpty + (c & 1));
            if (!x.wait_all(kDSFull + ds_bar<Local>(c), ds_phase<Local>(c))) return;
            tc_fence_after();
            const f2 g2 = pack2(gamma, gamma);
            const bool clears = gamma == kClearing;
            if (clears) {
                mend_ds(p, item.t0 + j * C, min(C, item.len - j * C), item.h, tm + ds_column<Local>(c), row, 64 * sg);
#pragma unroll
                for (int e = 0; e < 32; ++e) S[e] = 0ull;
            }
            if (Local) kept = clears || kept == kClearing ? kClearing : kept * gamma;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t r[16];
                tmem_ld16u(tm + ds_column<Local>(c) + 16 * b, r);
                tmem_wait_ld();
                if (b == 3) {
                    tc_fence_before();
                    __syncwarp();
                    if (x.lane == 0) x.arrive(kDSEmpty + ds_bar<Local>(c));
                }
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    S[8 * b + e / 2] = fma2(g2, S[8 * b + e / 2],
                                             pack2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])));
            }
            if (!Local && j + 1 < nc) {
                place_free();
                write_operand();
            }
        }
        if (Local) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 a = unpack2(S[2 * e]), b = unpack2(S[2 * e + 1]);
                plane[256 * e] = make_float4(a.x, a.y, b.x, b.y);
            }
            if (threadIdx.x == 0) p.kept[item.plane] = kept;
        } else if (ok && (item.flags & kStore)) {  // the chunk's q S^T, issued before dS, has read the operand
            place_free();
            if (maps.store_states) {
                // as the pool's type in rows of 128 bytes, swizzled as its map's boxes are:
                // fp32 columns 0-31 in the high part's place, 32-63 in the low part's
                uint8_t* mine = x.smem + kSmS + sg * (kTile / 2) + 32 * (warp & 3) * 128;
                if constexpr (sizeof(P) == 4) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 a = unpack2(S[2 * e]), b = unpack2(S[2 * e + 1]);
                        *staged(x.lane, e) = make_float4(a.x, a.y, b.x, b.y);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint2 u[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 a = unpack2(S[4 * e + 2 * i]), b = unpack2(S[4 * e + 2 * i + 1]);
                            store4(reinterpret_cast<P*>(&u[i]), make_float4(a.x, a.y, b.x, b.y));
                        }
                        *reinterpret_cast<uint4*>(mine + x.lane * 128 + ((e ^ (x.lane & 7)) << 4)) =
                            make_uint4(u[0].x, u[0].y, u[1].x, u[1].y);
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (x.lane == 0) {
                    const int y = item.h * D + 32 * (warp & 3);
                    tma_store_3d(&maps.pool, mine, 64 * sg, y, slot);
                    if (sizeof(P) == 4) tma_store_3d(&maps.pool, mine + kTile, 64 * sg + 32, y, slot);
                    bulk_commit();
                }
                leaving = true;
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 a = unpack2(S[2 * e]), b = unpack2(S[2 * e + 1]);
                    *staged(x.lane, e) = make_float4(a.x, a.y, b.x, b.y);
                }
                __syncwarp();
#pragma unroll 4
                for (int r = 0; r < 32; r += 2) store4(pool + r * D, *staged(r + half, l16));
                __syncwarp();
            }
        }
    }
}

// Local: the segments' states from zero, nothing else (the q, score and output parts idle).
template <class P, bool Local>
__global__ void __launch_bounds__(kThreads, 1) kda_lin_walk(const __grid_constant__ Maps maps, const __grid_constant__ LinParams p,
                                                             const __grid_constant__ LinCuts cuts) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    Ctx x;
    x.smem = smem;
    x.bar = reinterpret_cast<uint64_t*>(smem + kSmBar);
    x.lane = threadIdx.x & 31;
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kSmMisc);
    x.abort = reinterpret_cast<volatile int*>(smem + kSmMisc + 4);
    if ((smem_u32(smem) & 1023) != 0) {  // swizzled tiles need 1 KB alignment
        if (threadIdx.x == 0) *p.status = 2;
        return;
    }
    if (threadIdx.x < kNumBars) {
        const int i = threadIdx.x;
        int n = 1;
        if (i == kDecEmpty || i == kDecEmpty + 1) n = Local ? 24 : 16;
        if (i == kGEmpty) n = 12;
        if (i >= kItemEmpty && i < kItemEmpty + kItems) n = Local ? 26 : 30;
        if (i == kQSScaled || i == kOEmpty) n = 4;
        if (i >= kWFull && i < kWFull + 4) n = 4;
        if (i == kDSEmpty || i == kDSEmpty + 1 || i == kSFull || i == kCleared || i == kPFull) n = 8;
        mbar_init(x.bar + i, n);
        fence_mbar_init();
    } else if (threadIdx.x == 64) {
        *x.abort = 0;
        *reinterpret_cast<int*>(smem + kSmRows) = 0;
    } else if (threadIdx.x >= 96 && threadIdx.x < 100) {
        prefetch_tmap(threadIdx.x == 96 ? &maps.v : threadIdx.x == 97 ? &maps.q : threadIdx.x == 98 ? &maps.k : &maps.out);
    }
    if (warp == 28) tmem_alloc(slot, kTmCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    x.tmem = *slot;

    // what follows in the stream may be set up; it waits for this grid where it has to
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // registers: the launch's 1024 x 64 = 256 x 104 + 256 x 56 + 256 x 48 + 128 x 56 + 128 x 40,
    // Local: 256 x 104 + 512 x 56 + 256 x 40
    int3 issued = make_int3(0, 0, 0);
    if (warp < 8) {
        more_registers<104>();
        state_role<P, Local>(maps, p, x, warp);
        // a state may be on its way to the pool, also where a wait gave up
        if (x.lane == 0) bulk_wait_all();
    } else if (warp < 16) {
        fewer_registers<56>();
        weight_role<Local>(p, x, warp - 8);
    } else if (warp < 24) {
        fewer_registers<Local ? 56 : 48>();
        if constexpr (Local)
            weight_role<Local>(p, x, warp - 8);
        else
            score_role(p, x, warp - 16);
    } else if (warp < 28) {
        fewer_registers<Local ? 40 : 56>();
        if constexpr (!Local) out_role(maps, p, x, warp - 24);
    } else {
        fewer_registers<40>();
        if (warp == 28) {
            mma_role<Local>(x);
            if (elect_one()) mma_commit(x.bar + kDone);  // the lane that issued
        } else if (warp == 29) {
            if (x.lane == 0) issued = load_role<Local>(maps, p, x);
        } else if (warp == 30) {
            decay_role<Local>(p, cuts, x);
        } else if (blockIdx.x == 0 && (Local || p.n_cut == 0)) {
            write_status(p, x.lane);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*x.abort) {
        // a wait gave up: let the loads and products in flight end, too, before their memory goes
        if (threadIdx.x == 0) atomicOr(p.status, 1);
        if (warp == 29 && x.lane == 0) {
            if (!Local && issued.x > 0) mbar_wait(x.bar + kFull + kQ, q_phase(issued.x - 1));
            for (int i = max(0, issued.y - kVs<Local>); i < issued.y; ++i)
                mbar_wait(x.bar + kFull + v_slot<Local>(i), v_phase<Local>(i));
            for (int i = max(0, issued.z - kKs<Local>); i < issued.z; ++i)
                mbar_wait(x.bar + kFull + k_slot<Local>(i), k_phase<Local>(i));
        }
    }
    if (warp == 28) {
        mbar_wait(x.bar + kDone, 0);
        tc_fence_after();
    }
    __syncthreads();
    if (warp == 28) tmem_dealloc(x.tmem, kTmCols);
}

// From the states that segments make from zero to the states they start from, in place:
// with S the sequence's initial state, plane s takes S and S becomes kept_s S + (what
// plane s held).  The first segment's is taken from the pool here, too: the last
// segment's walk writes the pool, perhaps before the first one's has started.
//
// Bound by the reads' latency, so they all go out at once: a thread has four columns of a
// row in up to AHEAD segments, threads side by side (in y) have the segments that follow,
// and the states between their runs are handed on through shared memory.
constexpr int kChainAhead = 8, kChainRuns = 20;  // 160 segments at most
template <class P, int AHEAD, int X, int RUNS>
__global__ void __launch_bounds__(X* RUNS) kda_lin_chain(const __grid_constant__ LinParams p,
                                                         const __grid_constant__ LinCuts cuts) {
    __shared__ float4 sum[RUNS][X];
    __shared__ float left[RUNS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int r = blockIdx.y / p.H, h = blockIdx.y % p.H;
    const int first = cuts.first[r], segs = cuts.first[r + 1] - first;
    const int n = cuts.seq[r], slot = p.idx[n];
    const int at = blockIdx.x * X + threadIdx.x;  // as the state warps hold it: e, warp, lane
    const int e = at >> 8, warp = (at >> 5) & 7;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (slot >= 0 && slot < p.num_slots && p.has_init[n])
        S = load4<P>(static_cast<const P*>(p.pool) + (size_t)slot * p.stride0 +
                     ((size_t)h * D + 32 * (warp & 3) + (at & 31)) * D + 64 * (warp >> 2) + 4 * e);
    const size_t step = (size_t)p.H * (D * D / 4);
    const int s0 = threadIdx.y * AHEAD, run = min(AHEAD, segs - s0);  // this thread's segments
    float4* plane = reinterpret_cast<float4*>(p.planes) + (size_t)h * (D * D / 4) + at + (first + s0) * step;
    const float* kept = p.kept + (size_t)(first + s0) * p.H + h;
    auto next = [](float4 a, float k, float4 v) {
        if (k == kClearing) a = make_float4(0.f, 0.f, 0.f, 0.f);
        return make_float4(fmaf(k, a.x, v.x), fmaf(k, a.y, v.y), fmaf(k, a.z, v.z), fmaf(k, a.w, v.w));
    };
    grid_dep_wait();  // the segments' states are made
    float4 v[AHEAD];
    float k[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f), k[i] = 1.f;
        if (i < run && s0 + i < segs - 1) v[i] = plane[i * step], k[i] = kept[(size_t)i * p.H];
    }
    if (RUNS > 1) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        float all = 1.f;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            t = next(t, k[i], v[i]), all = all == kClearing || k[i] == kClearing ? kClearing : all * k[i];
        sum[threadIdx.y][threadIdx.x] = t;
        if (threadIdx.x == 0) left[threadIdx.y] = all;
        __syncthreads();
        for (int i = 0; i < threadIdx.y; ++i) S = next(S, left[i], sum[i][threadIdx.x]);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (i < run) {
            plane[i * step] = S;
            S = next(S, k[i], v[i]);
        }
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

// Boxes of 128 bytes x 1 x `rows` of a 3-D tensor, 128-byte swizzled; rows past the end
// read as zeros.  The middle dimension's boxes are one wide, or with rows_in_middle the
// last one's.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, int elt, const void* base, const int64_t (&dim)[3],
              const int64_t (&stride)[2], int rows, bool rows_in_middle) {
    if (!encode_fn()) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim[0], (cuuint64_t)dim[1], (cuuint64_t)dim[2]};
    const cuuint64_t strides[2] = {(cuuint64_t)stride[0] * elt, (cuuint64_t)stride[1] * elt};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / elt), rows_in_middle ? (cuuint32_t)rows : 1,
                               rows_in_middle ? 1 : (cuuint32_t)rows};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode_fn()(m, type, 3, const_cast<void*>(base), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A [T][H][128] view of bf16.
bool make_rows_map(CUtensorMap* m, const void* base, int64_t T, int H, int64_t st, int64_t sh, int rows) {
    // a dimension of one entry never steps: any stride that encodes will do
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, {D, H, T}, {H == 1 ? D : sh, T == 1 ? D : st}, rows,
                    false);
}

// Launches with programmatic stream serialization where `early`: set up while the kernel
// before still runs, whose results it then waits for.
template <class... A>
cudaError_t launch_after(bool early, void (*kernel)(A...), dim3 grid, dim3 threads, size_t smem, cudaStream_t s,
                         const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class P, bool Local>
cudaError_t launch_one(bool early, const Maps& maps, const LinParams& p, const LinCuts& cuts, int64_t items,
                       cudaStream_t s) {
    static bool ready[32] = {};  // per device: the shared memory is allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 32 || !ready[dev]) {
        e = cudaFuncSetAttribute(kda_lin_walk<P, Local>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 32) ready[dev] = true;
    }
    const int grid = (int)(items < num_sms() ? items : num_sms());
    return launch_after(early, kda_lin_walk<P, Local>, dim3(grid), dim3(kThreads), kSmemBytes, s, maps, p, cuts);
}

template <class P>
cudaError_t launch_chain(const LinParams& p, const LinCuts& cuts, cudaStream_t s) {
    int most = 0;
    for (int r = 0; r < p.n_cut; ++r) most = max(most, cuts.first[r + 1] - cuts.first[r]);
    // Runs of 8: 152 segments are one trip to memory (a prompt of 16384 x 2 heads 33.8 us;
    // one thread's run of all of them, 16 at a time, 37.8 us).  Up to four segments need no
    // joining: 119.1 us instead of 122.1 for four prompts of 2048 beside 512 of one token.
    const unsigned y = (unsigned)(p.n_cut * p.H), columns = D * D / 4;
    if (most <= 4)
        return launch_after(true, kda_lin_chain<P, 4, 128, 1>, dim3(columns / 128, y), dim3(128), 0, s, p, cuts);
    return launch_after(true, kda_lin_chain<P, kChainAhead, 32, kChainRuns>, dim3(columns / 32, y),
                        dim3(32, (most + kChainAhead - 1) / kChainAhead), 0, s, p, cuts);
}

template <class P>
cudaError_t launch(const Maps& maps, const LinParams& p, const LinCuts& cuts, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const bool cut = p.n_cut > 0;
    const int64_t items = (int64_t)(p.n_seg + p.n_long - p.n_cut) * p.H;  // Local has fewer
    if (items > num_sms()) e = cudaMemsetAsync(p.status, 0, kWsClearBytes, s);  // the queues
    if (cut && e == cudaSuccess) {
        // the segments' states do not depend on the pool's type
        e = launch_one<float, true>(false, maps, p, cuts, (int64_t)(p.n_seg - p.n_cut) * p.H, s);
        if (e == cudaSuccess)
            e = launch_chain<P>(p, cuts, s);
    }
    if (e == cudaSuccess)
        e = launch_one<P, false>(cut, maps, p, cuts, items, s);
    return e;
}

// How the longest sequences are cut, from the long sequences' lengths (longest first).
// Uncut, the walk takes as long as its longest sequence or as all chunks shared out,
// whichever is more.  Cut, a segment's walk has to wait for the states of those before it,
// which are made first from k and v alone, in about half of a walk's time; `start` chunks'
// time goes into the two more launches and the states' way through memory, more of it the
// more states there are: none for up to three (sequence, head) pairs, and from there on one
// more chunk for every sixteen, up to four.  That is a fit to the times below, no more.  The
// segments are as long as lets one wave of CTAs take all items, or, where there are more
// sequences than that, as an even share of the chunks.
// Cut and uncut, 12 heads: 22.6 and 26.7 us for 640 tokens, 22.6 and 32.8 us for 896, 28.7
// and 61.5 us for 2048, 37.1 and 116 us for 4097, 80.1 and 418 us for 16384; 26.7 and 32.8
// us for two of 896; 128.3 and 131.2 us for four of 2048 beside 512 of one token (all from
// their states).  Two heads: 18.5 and 22.6 us for 512 tokens.  Left uncut, 12 heads: 384
// tokens (20.5 us, cut 22.4), three of 768 (30.1 us, cut 28.7), four of 640 (26.7 us, cut
// 31.1), four of 1024 (36.9 us, cut 37.4), six of 900 to 1600 (51.3 us, cut 53.1).  Only the
// longest sequence is compared: where all are alike and just exceed one wave of CTAs (13
// prompts of 2048: 123.8 us, 12 of them 74.3), nothing is cut.
struct Cut {
    int seg_len = 0, n_cut = 0, n_seg = 0;
};
Cut cut_rule(const int32_t* lens, int n, int H, int sms) {
    auto chunks_of = [](int len) { return (len + C - 1) / C; };
    Cut cut;
    if (n <= 0) return cut;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) total += chunks_of(lens[i]);
    const int longest = chunks_of(lens[0]);
    const int64_t share = (total * H + sms - 1) / sms;
    int seg = (int)(share < longest ? share : longest);
    auto items = [&](int L) {
        int64_t m = 0;
        for (int i = 0; i < n; ++i) m += (chunks_of(lens[i]) + L - 1) / L;
        return m * H;
    };
    if ((int64_t)n * H <= sms) {  // the shortest segments that fit
        int hi = longest;
        while (seg < hi) {
            const int mid = seg + (hi - seg) / 2;
            if (items(mid) <= sms) hi = mid; else seg = mid + 1;
        }
    }
    const int64_t pairs = (int64_t)n * H, start = pairs < 52 ? (pairs + 12) / 16 : 4;
    if (longest < kLinMinCut || longest <= seg + (seg + 1) / 2 + start) return cut;
    cut.seg_len = seg * C;
    for (; cut.n_cut < n && chunks_of(lens[cut.n_cut]) > seg; ++cut.n_cut)
        cut.n_seg += (chunks_of(lens[cut.n_cut]) + seg - 1) / seg;
    if (cut.n_cut > kLinCuts || (int64_t)cut.n_seg * H > kLinPlanes ||
        (longest + seg - 1) / seg > kChainAhead * kChainRuns) return Cut();
    return cut;
}

}  // namespace

void lin_cut(LinParams& p, LinCuts& cuts, const SeqTables& t) {
    const Cut c = cut_rule(t.long_lens, p.n_long, p.H, num_sms());
    p.seg_len = c.seg_len;
    p.n_cut = c.n_cut;
    p.n_seg = c.n_seg;
    cuts.first[0] = 0;
    for (int r = 0; r < c.n_cut; ++r) {
        cuts.seq[r] = t.long_seqs[r];
        cuts.t0[r] = t.bounds[t.long_seqs[r]];
        cuts.len[r] = t.long_lens[r];
        cuts.first[r + 1] = cuts.first[r] + (t.long_lens[r] + c.seg_len - 1) / c.seg_len;
    }
}

cudaError_t launch_lin_walk(const LinParams& p, const LinCuts& cuts, cudaStream_t s) {
    if (p.n_long <= 0) return cudaSuccess;
    if ((int64_t)p.n_long * p.H > INT32_MAX - 65536) return cudaErrorInvalidValue;
    Maps maps;
    if (!make_rows_map(&maps.q, p.q, p.T, p.H / p.rep, p.q_st, p.q_sh, C) ||
        !make_rows_map(&maps.k, p.k, p.T, p.H / p.rep, p.k_st, p.k_sh, C) ||
        !make_rows_map(&maps.v, p.v, p.T, p.H, p.v_st, p.v_sh, C) ||
        !make_rows_map(&maps.out, p.out, p.T, p.H, (int64_t)p.H * D, D, 32))
        return cudaErrorInvalidValue;
    // the pool as [slots][H x 128][128]; one too large for a map is written without
    const bool wide = p.st_dtype == KDA_STATE_F32;
    maps.store_states = make_map(&maps.pool, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                                 wide ? 4 : 2, p.pool, {D, (int64_t)p.H * D, p.num_slots}, {D, p.stride0}, 32, true);
    if (p.st_dtype == KDA_STATE_F32) return launch<float>(maps, p, cuts, s);
    if (p.st_dtype == KDA_STATE_BF16) return launch<__nv_bfloat16>(maps, p, cuts, s);
    return launch<__half>(maps, p, cuts, s);
}

}  // namespace kda
