// Attention of a chunk of new tokens over the paged cache and over the chunk
// itself (include/kivi.h, kivi_paged_chunk_attn).
//
//   o_i = sum_t softmax_t(f(q_i . k_t)) v_t      over t <= c + i (and t > c + i - window),
//
// c cached tokens, f(x) = scale x, capped: cap tanh(scale x / cap), plus
// slope_h (t - (c + i)).  The query heads of a kv head are rows beside each
// other, so that they share its keys.
//
// The two products run on the fifth-generation tensor cores: a tile is 128 rows
// by 128 keys, S = Q K^T and O += P V, operands in shared memory (128-byte
// swizzle, the contracted index contiguous), P in tensor memory over S, sums
// in tensor memory.  A CTA (one per SM) holds up to 256 rows as two tiles A and
// B that take turns: while one's softmax runs, the other's products do.  With
// at most 128 rows A and B are the same rows and take alternate key tiles,
// joined at the end.
//
// Roles (warps):
//   0-3, 4-7   tile A / B: softmax, a row a lane (logits from tensor memory, running maximum,
//              exponentials, probabilities back as fp16), then one lane issues the tile's
//              next MMAs; epilogue
//   8-15       four the keys, 32 tokens of a tile each, from codes to fp16 in shared memory;
//              the next tile's bytes are loaded into registers while this one waits its
//              turn; four the values, the same, transposed ([channel][token])
//   16         finds the spans of items that the CTA works on, ahead of the others (17-19: idle,
//              they fill their warpgroup for the redistribution of registers)
// A warp of its own for the MMAs was slower: its code, some 250 instructions a turn, is run
// once in a thousand cycles and has left the instruction cache each time (a turn took 2000
// cycles with nothing to wait for).  For the same reason the loops are kept small.
//
// Dequantization: a code pair masked in place and OR-ed with fp16 1024 is
// 1024 + code * 2^pos, exact; one FMA makes it the code, a second one
// fp16(code * step + zero), rounded once.  The cache's tiles are fragments of
// 8x8 matrices, so stmatrix puts them where the MMA's swizzle wants them.
// Rows that are still fp16 (residual and chunk) are copied; values of tiles
// that hold nothing else stay token by token (the MMA takes both orders).
//
// Bound by the chain of a tile's steps (S, the walk over its logits, the four warps' meeting, P V and the next S), of which
// two tiles overlap: no pipe is full.  A tile of 128 keys by 256 rows takes some 4400 cycles, its 32 MMAs 2050 of them, the
// instructions 2650 issue slots a scheduler; over 512 new tokens of each of 8 sequences over 4096 (32 heads of 128, 2
// bits) ncu shows issue active 45%, the tensor pipe 40%, exponentials 21%: 330 us, 883 TFLOP/s; a prompt of 8192
// tokens, with nothing to dequantize, 538 us, 1020.
//
// Roundings: keys and values to fp16 (half a step of 2^-10), probabilities to
// fp16, scaled so that 2^4 at least stands for the row's largest: what falls below fp16's
// range is under 2^-29 of it.  Everything else is fp32.  The keys' rounding is what shows: outputs are off by some 1e-3
// of their size where channels are outliers, by 2.4e-4 if keys alone were exact, 2e-4 being the outputs' own rounding.  Exact
// keys are a second operand (what is left of each number) in the same product: S twice, 64 KB more of shared memory than
// there is beside two stages.
// The reference is the
// maximum of some tile so far, raised (and the sums in tensor memory scaled) when the
// weights of 64 keys reach 2^15 together, which leaves the result the same.
//
// A value that is not finite would reach rows that do not see it
// through the product (0 * inf): it is taken as zero and noted, and the rows that
// see it become NaN at the end.  A dequantized number beyond fp16's range whose step and zero
// are finite is held as the largest fp16 number: off by 2^-10 of it at most, since a block's
// extremes are fp16 numbers and its step is off by 2^-11.
#pragma once

#include <math.h>
#include <stddef.h>

#include <atomic>

#include "kivi_dequant.cuh"

namespace kivi {
namespace chunk_detail {

using namespace mma_detail;

constexpr int kChunkWarps = 20, kChunkThreads = 32 * kChunkWarps;
// Registers a thread: the launch's, and what the five warpgroups (A, B, keys, values, the rest) make of them.  2 bits:
// none of the roles that repeat spills; 4 bits: one value of the filling warps; 8 bits, whose words of a unit alone take
// 32: a few.
constexpr int kRegs = 96;
template <int BITS>
struct Regs {
    static constexpr int SOFTMAX = BITS == 8 ? 120 : 128, FILL = BITS == 8 ? 96 : 88, REST = 48;
    static_assert(2 * SOFTMAX + 2 * FILL + REST <= 5 * kRegs, "registers of the launch");
};
constexpr int kSpanRing = 4, kSpanReaders = 16;
constexpr int kNoTile = 0x7fffffff;
constexpr float kLift = 4.f;       // weights are held times 2^4
constexpr float kMostSum = 32768.f;   // of 64 weights: each is in fp16's range then
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int BITS>
struct Shape {
    static constexpr int KCH = D / 8;                     // 8-channel groups of a token
    static constexpr int W = D * BITS / 64;               // words of a lane in a 16-token code tile
    static constexpr int TILE = 2 * D * BITS;             // bytes of a code tile
    static constexpr int Q_BYTES = kHalf * D * 2;         // one tile of queries
    static constexpr int K_BYTES = kTile * D * 2;         // one stage of keys (values: the same)
    static constexpr int OFF_Q = 0, OFF_K = 2 * Q_BYTES, OFF_V = OFF_K + 2 * K_BYTES, OFF_ENT = OFF_V + 2 * K_BYTES;
    static constexpr int OFF_BAR = OFF_ENT + 8 * 4 * D;   // steps and zeros of the unit that each filling warp works on
    static constexpr int OFF_XCH = OFF_BAR + 1024;         // (m, l) of tile B's rows
    static constexpr int BYTES = OFF_XCH + kHalf * 8 + 1024;   // (base aligned to 1024)
    // one CTA per SM, also where less shared memory is needed: it takes all of the SM's tensor memory
    static constexpr int SMEM = BYTES < 117 * 1024 ? 117 * 1024 : BYTES;
    static constexpr int COL_S = 0, COL_O = 256;          // tensor memory columns: S of A and B, O of A and B
    static_assert(SMEM <= 232448, "shared memory");
};

// What the roles know of a span: the tiles [tile0, tile0 + nt) of an item's keys for its rows.
struct Span {
    int more;                   // 0: there is none
    int seq, tok0, n_quant, n_resid;
    int t0, t1, head;           // the item's tokens of the chunk, kv head
    int tile0, nt, na, nb;      // key tiles, of tile A, of tile B
    int both;                   // A and B are different rows (else the same, alternate tiles)
    int first, whole;           // holds the item's first tile, all of them
    int pad;
    __device__ __forceinline__ int tiles(int x) const { return x ? nb : na; }
    __device__ __forceinline__ int tile(int x, int i) const { return both ? i : 2 * i + x; }   // of x's step i
};

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], o_full[2], drained[2];      // of A, B
    uint64_t span_full[kSpanRing], span_empty[kSpanRing];
    uint32_t tmem;
    int failed;         // a wait ran out: the outputs from here on are NaN
    int ended;          // no span comes any more, although none said so
    int busy;           // a tile's MMAs are being issued
    unsigned bad;       // spans with a block-table entry outside the pool: bit number % 32
    int last_odd[2 * kSpanRing];   // of a span (number % 8): the last quantized token whose value is not finite, or -1
    int odd_tile[2][2 * kSpanRing];   // the first and the last tile with an fp16 value that is not finite, or kNoTile and -1
    alignas(16) Span spans[kSpanRing];
};
static_assert(sizeof(Bars) <= 1024, "barriers");
#define BAR(member) (uint32_t) offsetof(Bars, member)     // (barriers are used by their 32-bit shared address)

// ---- tensor memory and tcgen05 ----
__device__ __forceinline__ void tmem_alloc(uint32_t* out) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(out)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(at));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void ld32(uint32_t at, float (&x)[32]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
__device__ __forceinline__ void ld16(uint32_t at, float (&x)[16]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
__device__ __forceinline__ void st32(uint32_t at, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void st32(uint32_t at, const float (&x)[32]) {
    st32(at, reinterpret_cast<const uint32_t*>(x));
}
__device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// (the first eight of x)
__device__ __forceinline__ void st8(uint32_t at, const float (&x)[16]) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Wait for the loads: what they bring passes through, so that no use of it is moved ahead of the wait.
__device__ __forceinline__ void wait_ld(float (&x)[16]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void wait_ld(float (&x)[32]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
                   "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                   "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand, contracted index contiguous, 128-byte swizzle: rows of 128 bytes in
// groups of eight (1024 bytes); the descriptor's fields in 16-byte units.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3fff) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// The same memory as an operand of [64-column blocks][rows][128 bytes] whose rows are the contracted index: rows in
// groups of eight 1024 bytes apart, blocks of 64 columns kTile * 128 bytes.
__device__ __forceinline__ uint64_t operand_rows(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(kTile * 128 / 16) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// fp16 x fp16 -> fp32, M = 128, N columns, the contracted index contiguous in both operands (or, rows: not in B)
__host__ __device__ constexpr uint32_t mma_kind(int n, bool rows = false) {
    return (1u << 4) | ((uint32_t)rows << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}
template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tile_sync(int x) { asm volatile("bar.sync %0, 128;" ::"r"(3 + x) : "memory"); }
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int ID, int N>
__device__ __forceinline__ void named_sync() { asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory"); }

// Wait for an mbarrier's phase, 2^31 cycles (about a second) at most; a wait that runs out marks the CTA,
// and no wait of a marked CTA waits, but a patient one (for MMAs in flight at its end).  Each lane has a result of
// its own: a warp that goes on together takes them together.
template <bool PATIENT = false>
__device__ __forceinline__ bool wait_for(uint32_t bars, uint32_t bar, uint32_t parity) {
    const unsigned t0 = (unsigned)clock();
    while (!mbar_try(bar, parity)) {
        if ((unsigned)clock() - t0 < 1u << 31 && (PATIENT || !lds32(bars + BAR(failed)))) continue;
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(bars + BAR(failed)), "r"(1) : "memory");
        return false;
    }
    return true;
}
// The waits for spans (a span may take long, its tiles' waits do not).  The warps of a role meet at barriers within a
// span, so they have to agree whether there is one: the planner's wait alone runs out (2^36 cycles), it tells them that
// no span comes any more, and a span that is there by then counts.  (Theirs, 2^37 cycles, are for form.)
__device__ __forceinline__ bool wait_place(uint32_t bars, uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (clock64() - t0 < 1ll << 36) continue;
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(bars + BAR(failed)), "r"(1) : "memory");
        __threadfence_block();
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(bars + BAR(ended)), "r"(1) : "memory");
        return false;
    }
    return true;
}
__device__ __forceinline__ bool wait_span(uint32_t bars, uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (lds32(bars + BAR(ended))) return mbar_try(bar, parity);
        if (clock64() - t0 < 1ll << 37) continue;
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(bars + BAR(failed)), "r"(1) : "memory");
        return false;
    }
    return true;
}

// A lane's words of a unit's two code tiles, as loaded.
template <int W>
struct Words {
    uint4 v[2][W < 4 ? 1 : W / 4];
};
template <int W, int TILE>
__device__ __forceinline__ void load_unit(const uint8_t* p, Words<W>& w) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if constexpr (W == 2) {
            const uint2 v = ldg_stream2(p + t * TILE);
            w.v[t][0].x = v.x; w.v[t][0].y = v.y;
        } else {
#pragma unroll
            for (int j = 0; j < W / 4; ++j) w.v[t][j] = ldg_stream(p + t * TILE + 16 * j);
        }
    }
}
// Words J .. J + BITS / 2 - 1 of tile t, from the front of what is left of them (the loops below are kept loops, their
// bodies are small): x[t]; the loaded registers themselves are not touched, so that the next loads need not be waited for.
template <int W>
__device__ __forceinline__ void tile_words(const Words<W>& u, uint32_t (&w)[2][W]) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            const uint4& v = u.v[t][j / 4];
            w[t][j] = j % 4 ? v.z : v.x;
            w[t][j + 1] = j % 4 ? v.w : v.y;
        }
}
template <int BITS, int N>
__device__ __forceinline__ void next_words(uint32_t (&w)[2][N]) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j + BITS / 2 < N; ++j) w[t][j] = w[t][j + BITS / 2];
}
// Keys: fp16(code * step + zero), rows row0 .. row0 + 31 of the operand at dst.  The channel group C's step and
// zero pair of the lane is at ent + 16 C + 4 i (zeros 2 D bytes on); it holds for both code tiles.
template <int D, int BITS, int W>
__device__ __forceinline__ void key_unit(const Words<W>& u, uint32_t ent, uint32_t dst, int row0, int lane) {
    const int r7 = lane & 7;
    const uint32_t rows = dst + (row0 + (lane & 15)) * 128, e0 = ent + 4 * (lane & 3);
    uint32_t x[2][W];
    tile_words(u, x);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {                         // channels 32 c ..
        const uint32_t at = rows + (c >> 1) * (kTile * 128), e = e0 + 64 * c;
        uint32_t s[4], z[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            s[g] = lds32(e + 16 * g);
            z[g] = lds32(e + 16 * g + 2 * D);
        }
        // matrices: (group, tokens 0-7), (group, 8-15), (next group, ...); this lane gives a row's address
        const int chunk = 4 * (c & 1) + (lane >> 4);
        const uint32_t to0 = at + ((chunk ^ r7) << 4), to1 = at + (((chunk + 2) ^ r7) << 4);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            stmatrix4(to0 + t * 2048, hfma2(code_of<BITS, 0, 0>(x[t]), s[0], z[0]), hfma2(code_of<BITS, 0, 1>(x[t]), s[0], z[0]),
                      hfma2(code_of<BITS, 1, 0>(x[t]), s[1], z[1]), hfma2(code_of<BITS, 1, 1>(x[t]), s[1], z[1]));
            stmatrix4(to1 + t * 2048, hfma2(code_of<BITS, 2, 0>(x[t]), s[2], z[2]), hfma2(code_of<BITS, 2, 1>(x[t]), s[2], z[2]),
                      hfma2(code_of<BITS, 3, 0>(x[t]), s[3], z[3]), hfma2(code_of<BITS, 3, 1>(x[t]), s[3], z[3]));
        }
        next_words<BITS>(x);
    }
}
// Values into columns (tokens) tok0 .. tok0 + 31 of the operand [D channels][tokens] at dst.  ent: per code tile the
// steps, channel group j's at 32 j (this lane's four tokens at 8 i), and the zeros.
template <int D, int BITS, int W>
__device__ __forceinline__ void value_unit(const Words<W>& u, uint32_t ent, int lgG, uint32_t dst, int tok0, int lane) {
    const int r7 = lane & 7, ve = 64 * (D >> lgG);
    // (128 tokens a row in two blocks of 64; a unit lies in one)
    const uint32_t rows = dst + (tok0 >> 6) * (D * 128) + (8 * (lane >> 4) + r7) * 128, e0 = ent + 8 * (lane & 3);
    const int chunk0 = ((tok0 >> 3) & 7) + ((lane >> 3) & 1);
    const uint32_t col[2] = {(uint32_t)((chunk0 ^ r7) << 4), (uint32_t)(((chunk0 + 2) ^ r7) << 4)};
    uint32_t x[2][W];
    tile_words(u, x);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        const uint32_t e = e0 + 32 * ((32 * c) >> lgG), at = rows + c * 4096;
        uint2 s[2], z[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = lds64(e + t * ve);
            z[t] = lds64(e + t * ve + ve / 2);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t to = at + col[t];
            stmatrix4(to, hfma2(code_of<BITS, 0, 0>(x[t]), s[t].x, z[t].x), hfma2(code_of<BITS, 0, 1>(x[t]), s[t].y, z[t].y),
                      hfma2(code_of<BITS, 1, 0>(x[t]), s[t].x, z[t].x), hfma2(code_of<BITS, 1, 1>(x[t]), s[t].y, z[t].y));
            stmatrix4(to + 2048, hfma2(code_of<BITS, 2, 0>(x[t]), s[t].x, z[t].x), hfma2(code_of<BITS, 2, 1>(x[t]), s[t].y, z[t].y),
                      hfma2(code_of<BITS, 3, 0>(x[t]), s[t].x, z[t].x), hfma2(code_of<BITS, 3, 1>(x[t]), s[t].y, z[t].y));
        }
        next_words<BITS>(x);
    }
}

__device__ __forceinline__ uint32_t lds16(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)v) : "memory");
}
// Of a unit some of whose steps or zeros are large: numbers beyond fp16's range become the largest one; values whose step
// or zero is not finite become zeros (keys like that stay: they reach their own column of the logits alone).  A token a
// lane; whether its value was one of those.
template <int D>
__device__ __forceinline__ bool mend_unit(bool values, uint32_t ent, int lgG, uint32_t dst, int tok, int lane) {
    const int ve = 64 * (D >> lgG);
    bool odd = false;
#pragma unroll 1
    for (int ch = 0; ch < D; ++ch) {
        const uint32_t at = dst + (values ? operand_at<D>(ch, tok >> 3) + 2 * (tok & 7) : operand_at<kTile>(tok, ch >> 3) + 2 * (ch & 7));
        const uint32_t x = lds16(at);
        if ((x & 0x7c00u) != 0x7c00u) continue;
        const uint32_t s = ent + (values ? (lane >> 4) * ve + 32 * (ch >> lgG) + 8 * ((lane >> 1) & 3) + 4 * ((lane >> 3) & 1) + 2 * (lane & 1)
                                         : 2 * ch);
        if ((lds16(s) & 0x7c00u) != 0x7c00u && (lds16(s + (values ? ve / 2 : 2 * D)) & 0x7c00u) != 0x7c00u) {
            sts16(at, (x & 0x8000u) | 0x7bffu);
        } else if (values) {
            sts16(at, 0u);
            odd = true;
        }
    }
    return odd;
}

// (asm volatile: not moved ahead of the wait for the preceding kernel, as __ldg may be)
__device__ __forceinline__ uint4 ldg_row(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ int ldg_int(const int* p) {
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// (an exponent of ones carries into the sign's place)
__device__ __forceinline__ uint32_t odd_bits(uint32_t v) { return (v & 0x7c007c00u) + 0x04000400u; }
__device__ __forceinline__ bool not_finite(const uint4& v) {
    return ((odd_bits(v.x) | odd_bits(v.y) | odd_bits(v.z) | odd_bits(v.w)) & 0x80008000u) != 0u;
}

// 16 bytes global -> shared, asynchronous; zeros instead where there are none
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Where the fp16 rows of a span are: row f of [residual | chunk].
struct Rows {
    const __half *resid, *chunk;      // kv head's first residual row, its first new token
    long long step;                   // elements between new tokens
    int n_resid, n;                   // residual rows, all rows
    __device__ __forceinline__ const __half* at(int f, int D) const {
        return f < n_resid ? resid + (long long)f * D : chunk + (long long)(f - n_resid) * step;
    }
};
// 32 fp16 rows [f0, f0 + 32) (zeros behind the last) as they lie, token by token: keys, and values of a tile that
// holds nothing but rows.
template <int D>
__device__ __forceinline__ void plain_rows(const Rows& k, int f0, uint32_t dst, int row0, int lane) {
    constexpr int LPR = D / 8, RPI = 32 / LPR;                 // lanes a row, rows an instruction
    const int lr = lane % LPR, sub = lane / LPR;
    const uint32_t to = dst + (uint32_t)((lr >> 3) * (kTile * 128) + (row0 + sub) * 128);
    if (f0 >= k.n_resid && f0 + 32 <= k.n) {                   // all of them new tokens: evenly spaced
        const __half* src = k.chunk + (f0 + sub - k.n_resid) * k.step + 8 * lr;
        const long long step = RPI * k.step;
#pragma unroll 4
        for (int h = 0; h < 32; h += RPI, src += step)
            cp_async16_or_zero(to + h * 128 + (((lr & 7) ^ ((sub + h) & 7)) << 4), src, true);
    } else {
#pragma unroll 1
        for (int h = 0; h < 32; h += RPI) {
            const int f = f0 + h + sub;
            cp_async16_or_zero(to + h * 128 + (((lr & 7) ^ ((sub + h) & 7)) << 4), k.at(f < k.n ? f : 0, D) + 8 * lr, f < k.n);
        }
    }
    cp_async_wait_all();
}
// Of rows that plain_rows has brought: those that are not finite become zeros; whether there was one.
template <int D>
__device__ __forceinline__ bool clear_odd_rows(uint32_t dst, int row0, int lane) {
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const int lr = lane % LPR, sub = lane / LPR;
    const uint32_t at = dst + (uint32_t)((lr >> 3) * (kTile * 128) + (row0 + sub) * 128);
    uint32_t odd = 0;
#pragma unroll 4
    for (int h = 0; h < 32; h += RPI) {
        const uint4 v = lds128(at + h * 128 + (((lr & 7) ^ ((sub + h) & 7)) << 4));
        odd |= odd_bits(v.x) | odd_bits(v.y) | odd_bits(v.z) | odd_bits(v.w);
    }
    if (!__any_sync(kFull, (odd & 0x80008000u) != 0u)) return false;
#pragma unroll 1
    for (int h = 0; h < 32; h += RPI) {
        const uint32_t x = at + h * 128 + (((lr & 7) ^ ((sub + h) & 7)) << 4);
        const unsigned who = __ballot_sync(kFull, not_finite(lds128(x)));
        if (who >> (LPR * sub) & (LPR == 16 ? 0xffffu : 0xffu)) sts128(x, uint4{0, 0, 0, 0});
    }
    return true;
}
// The same rows as values, transposed.  A lane loads 8 channels of a token; as matrices of
// (8 tokens) x (channel pairs of four lanes) they are stored transposed, each row of a matrix to its channel.
// Rows that are not finite become zeros; whether there was one.
template <int D>
__device__ __forceinline__ bool value_rows(const Rows& v, int f0, uint32_t dst, int tok0, int lane) {
    const int g = lane >> 2, i = lane & 3;
    unsigned any = 0;
#pragma unroll 1
    for (int t2 = 0; t2 < 2; ++t2) {
        uint4 x[2][D / 32];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int f = f0 + 16 * t2 + 8 * u + g;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                x[u][j] = uint4{0, 0, 0, 0};
                if (f < v.n) x[u][j] = ldg_row(v.at(f, D) + 8 * (4 * j + i));
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bool odd = false;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) odd |= not_finite(x[u][j]);
            const unsigned who = __ballot_sync(kFull, odd);
            any |= who;
            if (who >> (4 * g) & 15u) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j) x[u][j] = uint4{0, 0, 0, 0};
            }
            // matrix m of an instruction: register m, channels 32 j + 8 (r / 2) + 2 m + r % 2 for its rows r
            const int m = lane >> 3, r = lane & 7;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const int ch = 32 * j + 8 * (r >> 1) + 2 * m + (r & 1);
                stmatrix4_trans(dst + operand_at<D>(ch, (tok0 >> 3) + 2 * t2 + u), x[u][j].x, x[u][j].y, x[u][j].z, x[u][j].w);
            }
        }
    }
    return any != 0;
}

// ---- spans: one warp finds them, the others read them ----
inline __device__ void plan_spans(const ChunkArgs& a, Bars& b, uint32_t bars, int lane) {
    if (lane == 0) {
        ChunkWalk walk;
        walk.start(&a.plan, a.seqs, a.n_seqs, chunk_begin(a.weight, a.n_ctas, blockIdx.x),
                   chunk_begin(a.weight, a.n_ctas, blockIdx.x + 1LL));
        uint32_t n = 0;
        bool more = true;
        while (more) {
            more = walk.next();
            if (n == 0) a.jobs[blockIdx.x] = more ? merge_job(walk, a.weight, a.n_ctas, blockIdx.x) : MergeJob{0, 0, 0, 0};
            const uint32_t slot = n % kSpanRing;
            if (!wait_place(bars, bars + BAR(span_empty) + 8 * slot, ((n / kSpanRing) & 1) ^ 1)) break;
            Span o;
            o.more = more;
            if (more) {
                const ChunkItem& it = walk.s.it;
                const ChunkSeq& q = a.seqs[walk.s.seq];
                o.seq = q.seq;
                o.tok0 = q.tok0;
                o.n_quant = q.n_quant;
                o.n_resid = q.n_resid;
                o.t0 = it.t0;
                o.t1 = it.t1;
                o.head = walk.s.head;
                o.tile0 = it.lo + walk.s.first;
                o.nt = walk.s.last - walk.s.first;
                o.both = it.both;
                o.first = walk.s.first == 0;
                o.whole = walk.s.whole();
                if (it.both) {
                    // tile A's rows end at kHalf: its own last key tile
                    const int ta = last_tile((long long)q.n_quant + q.n_resid, it.t0 + kHalf / a.plan.nq) - o.tile0;
                    o.na = ta < 0 ? 0 : ta < o.nt ? ta : o.nt;
                    o.nb = o.nt;
                } else {
                    o.na = (o.nt + 1) / 2;
                    o.nb = o.nt / 2;
                }
            }
            // (the roles are at spans n - 4 to n: a mark of 24 spans ago is nobody's)
            atomicAnd(&b.bad, ~(1u << ((n + 8) % 32)));
            b.last_odd[n % (2 * kSpanRing)] = b.odd_tile[1][n % (2 * kSpanRing)] = -1;    // (of span n - 8: nobody's)
            b.odd_tile[0][n % (2 * kSpanRing)] = kNoTile;
            b.spans[slot] = o;
            arrive(bars + BAR(span_full) + 8 * (slot));
            ++n;
        }
    }
    __syncwarp();
}
// A warp's view of them: next() gives the next span, which stays in place until the one after is asked for.
struct SpanReader {
    const Bars& b;
    uint32_t bars;
    uint32_t n;                 // of spans read; the present one is number n - 1
    __device__ __forceinline__ unsigned mark() const { return 1u << ((n - 1) % 32); }
    __device__ __forceinline__ uint32_t place() const { return (n - 1) % (2 * kSpanRing); }
    __device__ __forceinline__ SpanReader(const Bars& data, uint32_t at) : b(data), bars(at), n(0) {}
    __device__ __forceinline__ void release() const { arrive(bars + BAR(span_empty) + 8 * ((n - 1) % kSpanRing)); }
    __device__ __forceinline__ const Span* next(int lane) {      // a whole warp
        if (n) {
            __syncwarp();
            if (lane == 0) release();
        }
        const uint32_t slot = n % kSpanRing;
        const bool ok = __all_sync(kFull, wait_span(bars, bars + BAR(span_full) + 8 * slot, (n / kSpanRing) & 1));
        ++n;
        const Span* s = &b.spans[slot];
        return ok && s->more ? s : nullptr;
    }
};

// ---- producers: warp w of 4 fills tokens 32 w .. 32 w + 31 of each tile, keys or values ----
// (one body for both: the instruction cache)
template <int D, int BITS>
__device__ void fill_tiles(const ChunkArgs& a, Bars& b, uint32_t bars, uint32_t smem, bool values, int w, int lane) {
    using S = Shape<D, BITS>;
    constexpr int W = S::W, TILE = S::TILE;
    const uint32_t full = bars + (values ? BAR(v_full) : BAR(k_full));
    constexpr uint32_t kEmpty = BAR(k_empty) - BAR(k_full);
    static_assert(kEmpty == BAR(v_empty) - BAR(v_full), "the same for both");
    const uint32_t ent = smem + S::OFF_ENT + (4 * values + w) * (4 * D);
    const uint32_t stages = smem + (values ? S::OFF_V : S::OFF_K);
    const int lgG = a.lgG, ve = 64 * (D >> lgG);               // bytes of value entries of a code tile
    const int last_ent = (values ? 2 * ve / 16 : 4 * D / 16) - 1;   // 16-byte groups of a unit's steps and zeros, less one
    // A step of 2^(15 - BITS) or a zero of 2^15 and more (a bit 15 after the addition), without which no number of a unit
    // is beyond fp16's range.
    const int run = values ? ve / 16 : 4 * D / 16;             // 16-byte groups: half of them steps, half zeros, ..
    const bool steps_lane = min(lane, last_ent) % run < run / 2;
    SpanReader reader(b, bars);
    // the unit ahead: its bytes where it is quantized
    const Span* sp = nullptr;
    int t = 0, t_end = 0;                                      // (of the span the rest is read again: registers)
    bool quantized = false;
    int have = 0, entry = 0;                                   // table entries of tiles have .. have + 31, one a lane
    Words<W> words;
    uint4 ents{};
    auto ahead = [&]() {
        bool fresh = false;
        if (++t >= t_end) {
            sp = reader.next(lane);
            if (!sp) return;
            t = sp->tile0;
            t_end = t + sp->nt;
            fresh = true;
        }
        const int key0 = t * kTile + 32 * w, n_quant = sp->n_quant;
        quantized = key0 < n_quant;
        if (!quantized) return;
        if (fresh || t >= have + 32) {
            have = t;
            const int key = (t + lane) * kTile + 32 * w;
            entry = key < n_quant ? ldg_int(a.table + (long long)sp->seq * a.max_blocks + (key >> lgG)) : 0;
        }
        int page = __shfl_sync(kFull, entry, t - have);
        if ((unsigned)page >= (unsigned)a.n_pages) {           // an entry outside the pool: the span's outputs are NaN
            page = 0;
            if (lane == 0) atomicOr(&b.bad, reader.mark());
        }
        const uint8_t* part = a.buf + (unsigned long long)(unsigned)page * (unsigned)a.page_bytes +   // (a page: under 2^32 bytes)
                              (unsigned)(2 * sp->head + values) * (unsigned)a.part_bytes;
        const int tile = (key0 & ((1 << lgG) - 1)) >> 4;
        ents = ldg_stream(part + (TILE << (lgG - 4)) + (values ? tile * ve : 0) + 16 * min(lane, last_ent));
        load_unit<W, TILE>(part + tile * TILE + lane * (4 * W), words);
    };
    ahead();
    for (uint32_t tc = 0; sp; ++tc) {
        const uint32_t stage = tc & 1, ph = (tc >> 1) & 1;
        const uint32_t dst = stages + stage * S::K_BYTES;
        const bool ok = __all_sync(kFull, wait_for(bars, full + kEmpty + 8 * stage, ph ^ 1));
        if (quantized) {
            const uint32_t large = steps_lane ? (0x0800u + BITS * 0x0400u) * 0x00010001u : 0x08000800u;
            auto over = [&](uint32_t v) { return (v & 0x7fff7fffu) + large; };
            const bool mend = __any_sync(kFull, ((over(ents.x) | over(ents.y) | over(ents.z) | over(ents.w)) & 0x80008000u) != 0u);
            if (lane <= last_ent) sts128(ent + 16 * lane, ents);
            __syncwarp();
            if (values) value_unit<D, BITS>(words, ent, lgG, dst, 32 * w, lane);
            else key_unit<D, BITS>(words, ent, dst, 32 * w, lane);
            if (mend) {
                __syncwarp();
                const unsigned who = __ballot_sync(kFull, mend_unit<D>(values, ent, lgG, dst, 32 * w + lane, lane));
                if (who && lane == 0) atomicMax(&b.last_odd[reader.place()], t * kTile + 32 * w + 31 - __clz(who));
            }
        } else if (ok) {
            const long long resid = values ? a.v_resid_off : a.k_resid_off;
            const long long step = values ? a.v_stride[0] : a.k_stride[0], per_head = values ? a.v_stride[1] : a.k_stride[1];
            const Rows r{reinterpret_cast<const __half*>(a.buf + resid) + ((long long)sp->seq * a.plan.Hkv + sp->head) * a.R * D,
                         (values ? a.v : a.k) + sp->tok0 * step + sp->head * per_head, step, sp->n_resid, sp->n_resid + sp->t1};
            const int n_quant = sp->n_quant, f0 = t * kTile + 32 * w - n_quant;
            bool odd = false;
            if (!values || t * kTile >= n_quant) {
                plain_rows<D>(r, f0, dst, 32 * w, lane);
                if (values) odd = clear_odd_rows<D>(dst, 32 * w, lane);
            } else {
                odd = value_rows<D>(r, f0, dst, 32 * w, lane);
            }
            if (odd && lane == 0) {
                atomicMin(&b.odd_tile[0][reader.place()], t);
                atomicMax(&b.odd_tile[1][reader.place()], t);
            }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive(full + 8 * stage);
        ahead();
    }
}

// The tensor core takes MMAs in the order of their issue and makes the thread that issues wait.  A tile's run of
// them is kept together: mixed with the other tile's, both would be done when the second one is (in step, A and B took
// 5000 cycles a tile).
__device__ __forceinline__ void take_turn(uint32_t bars) {
    const uint32_t at = bars + BAR(busy);
    const unsigned t0 = (unsigned)clock();
    while (true) {
        uint32_t old;
        asm volatile("atom.shared.cas.b32 %0, [%1], 0, 1;" : "=r"(old) : "r"(at) : "memory");
        if (!old || (unsigned)clock() - t0 >= 1u << 31) return;   // (a lost turn costs time only)
    }
}
__device__ __forceinline__ void pass_turn(uint32_t bars) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(bars + BAR(busy)), "r"(0) : "memory");
}

// ---- MMAs of tile X, by one warp: it runs as one (descriptors stay in uniform registers), one lane issues ----
// The product P V of tile number cv (of the CTA) and then S of tile number ck, over the P that the product
// reads: one thread's MMAs run in the order of their issue.  A stage is free when both tiles have said so
// (`times`: a tile that the other one has no use for is let go twice).
template <int D, int BITS>
__device__ __forceinline__ void issue_mmas(uint32_t bars, uint32_t smem, uint32_t tmem, int x, int q_tile, bool product, bool add,
                                           bool rows, uint32_t cv, int times_v, bool next, uint32_t ck, int times_k) {
    using S = Shape<D, BITS>;
    bool ok = true;
    if (product) ok = wait_for(bars, bars + BAR(v_full) + 8 * (cv & 1), (cv >> 1) & 1);
    if (next) ok = wait_for(bars, bars + BAR(k_full) + 8 * (ck & 1), (ck >> 1) & 1) && ok;
    ok = __all_sync(kFull, ok);
    fence_after();
    if (!ok || !elect_one()) return;
    const uint32_t s_at = tmem + S::COL_S + x * kTile;
    take_turn(bars);
    if (product) {                                           // O_x += P_x V_t
        const uint32_t v_at = smem + S::OFF_V + (cv & 1) * S::K_BYTES;
        if (rows) {                                          // values token by token
            const uint64_t va = operand_rows(v_at);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                mma_ts(tmem + S::COL_O + x * D, s_at + 8 * k, va + k * (16 * 128 / 16), mma_kind(D, true), k > 0 || add);
        } else {
            const uint64_t va = operand(v_at);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                mma_ts(tmem + S::COL_O + x * D, s_at + 8 * k, va + (((k >> 2) * (D * 128) + (k & 3) * 32) >> 4), mma_kind(D),
                       k > 0 || add);
        }
        for (int j = 0; j < times_v; ++j) commit(bars + BAR(v_empty) + 8 * (cv & 1));
    }
    if (next) {                                              // S_x = Q_x K_t^T
        const uint64_t qa = operand(smem + S::OFF_Q + q_tile * S::Q_BYTES);
        const uint64_t ka = operand(smem + S::OFF_K + (ck & 1) * S::K_BYTES);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4;
            mma_ss(s_at, qa + off, ka + off, mma_kind(kTile), k > 0);
        }
        commit(bars + BAR(s_full) + 8 * x);
        pass_turn(bars);
        for (int j = 0; j < times_k; ++j) commit(bars + BAR(k_empty) + 8 * (ck & 1));
    } else {
        commit(bars + BAR(o_full) + 8 * x);
        pass_turn(bars);
    }
}

// ---- tile X: softmax (four warps, a row a lane), and the issue of its MMAs ----
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Weights 2^(mul v - ref) of 16 columns as fp16 pairs, their sums (mul and -ref twice each).
__device__ __forceinline__ void weights16(uint32_t* p, const float* v, uint64_t mul, uint64_t ref, uint64_t (&sum)[2]) {
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        float2 y = unpair(fma2(pair(v[j], v[j + 1]), mul, ref));
        y.x = exp2_ftz(y.x);
        y.y = exp2_ftz(y.y);
        sum[(j / 2) & 1] = add2(sum[(j / 2) & 1], pair(y.x, y.y));
        p[j / 2] = pack_f16x2(y.x, y.y);
    }
}
__device__ __forceinline__ float max16(float m, const float (&v)[16]) {
    float n = fmaxf(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < 16; j += 4) {
        m = fmaxf(fmaxf(m, v[j]), v[j + 1]);
        if (j + 2 < 16) n = fmaxf(fmaxf(n, v[j + 2]), v[j + 3]);
    }
    return fmaxf(m, n);
}

// The weights of half a tile at `from` whose largest is beyond fp16's range by the present reference: of logits whose neighbours
// in fp32 are several apart (from 2^24 on) the largest may be far above its rounded value.  Its weight stays 2^15.
// Stored at `to`; their sum.  (A call, not a part of the loop: inlined, a prompt of 8192 tokens took 540 us, so 535.)
static __device__ __noinline__ float clamped_half(uint32_t from, uint32_t to, float mul, float ref) {
    float l = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        float v[16], p[16];
        ld16(from + 16 * c, v);
        wait_ld(v);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float y0 = fmaf(v[j], mul, -ref), y1 = fmaf(v[j + 1], mul, -ref);
            y0 = exp2_ftz(y0 > 15.f ? 15.f : y0);      // (NaN stays)
            y1 = exp2_ftz(y1 > 15.f ? 15.f : y1);
            l += y0 + y1;
            p[j / 2] = __uint_as_float(pack_f16x2(y0, y1));
        }
        st8(to + 8 * c, p);                            // (over logits that have been read)
    }
    return l;
}

// Base-2 logit of a capped score of s = q . k: cap tanh(y) log2(e), y = scale s / cap, tanh(y) = 1 - 2 / (exp(2 y) + 1), which is
// off by 2^-20 at most.  Up to a cap of kSmallCap that moves a logit by 2^-14, an eighth of what a weight's rounding to fp16
// does.  With larger caps it would lose the scores in the one: there, where |y| is below 1/4, it is y times the series of
// tanh(y) / y up to y^6 (the next term is 62/2835 y^8: 2^-21.5 at 1/4), and the logit is off by 2^-19 of itself, whatever the
// cap; one beyond all scores leaves them as they are.  (Chosen by the call: 512 tokens of each of 8 sequences over 4096, 32
// heads, take 533 us with the first form and 594 with the second.)
constexpr float kSmallCap = 64.f;
__device__ __forceinline__ float capped(float s, float exp_mul, float cap_out) {
    return fmaf(-2.f * cap_out, rcp_ftz(exp2_ftz(s * exp_mul) + 1.f), cap_out);
}
__device__ __forceinline__ float capped_wide(float s, float y_mul, float scale_log2, float cap_out) {
    const float y = s * y_mul, y2 = y * y;
    const float series = fmaf(fmaf(fmaf(-17.f / 315.f, y2, 2.f / 15.f), y2, -1.f / 3.f), y2, 1.f);
    const float far = capped(y, 2.f * kLog2e, cap_out);
    return fabsf(y) < 0.25f ? s * scale_log2 * series : far;
}

template <int D, int BITS, bool MOD>
__device__ void softmax_rows(const ChunkArgs& a, Bars& b, uint32_t bars, uint32_t smem, float2* xch, uint32_t tmem, int x, int warp, int lane) {
    using S = Shape<D, BITS>;
    const int row = 32 * (warp & 3) + lane;                    // of tile X
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t ts = lanes + S::COL_S + x * kTile, to = lanes + S::COL_O + x * D;
    const int lgq = a.plan.nq >> 1;                            // log2 of 1, 2 or 4 query heads
    uint32_t sc = 0, oc = 0, tc = 0;                           // S, last products and key tiles so far
    SpanReader reader(b, bars);
    while (const Span* sp = reader.next(lane)) {
        const bool both = sp->both;
        const int r = both ? x * kHalf + row : row;            // row of the item
        const int n_rows = (sp->t1 - sp->t0) << lgq;
        const int steps = sp->tiles(x), tile0 = sp->tile0;
        // queries into the operand (the same rows: A loads them, for both)
        if (both || x == 0) {
            constexpr int LPR = D / 8, RPI = 32 / LPR;         // lanes a row, rows an instruction
            const int lr = lane % LPR, sub = lane / LPR;
            const __half* first = a.q + (long long)(sp->tok0 + sp->t0) * a.q_stride[0] + (sp->head << lgq) * a.q_stride[1] + 8 * lr;
            const uint32_t dst = smem + S::OFF_Q + x * S::Q_BYTES;
#pragma unroll 4
            for (int h = 0; h < 32; h += RPI) {
                const int to_row = row - lane + h + sub, from = r - lane + h + sub;
                const long long at = (long long)(from >> lgq) * a.q_stride[0] + (from & ((1 << lgq) - 1)) * a.q_stride[1];
                cp_async16_or_zero(dst + operand_at<kHalf>(to_row, lr), first + (from < n_rows ? at : 0), from < n_rows);
            }
            cp_async_wait_all();
            fence_proxy_async();
        }
        if (both) tile_sync(x);
        else named_sync<1, 256>();
        // the tile of step i, by its number in the CTA; how often it is let go
        auto tile = [&](int i) { return tc + (both ? i : 2 * i + x); };
        auto times = [&](int i) { return both && i < sp->na ? 1 : 2; };
        if ((warp & 3) == 0 && steps) issue_mmas<D, BITS>(bars, smem, tmem, x, both ? x : 0, false, false, false, 0, 0, true, tile(0),
                                                     times(0));
        // A row's position is p0 + (r >> lgq): the last key that it sees.  Of the warp's rows the first one sees
        // least, the last one starts last.
        const int p0 = sp->n_quant + sp->n_resid + sp->t0, r0 = r - lane;
        const int w_hi = p0 + (r0 >> lgq), w_lo = a.plan.window ? p0 + ((r0 + 31) >> lgq) - a.plan.window + 1 : 0;
        const bool any = r0 < n_rows;
        const float slope = MOD && a.slopes && r < n_rows
                                ? __ldg(a.slopes + (sp->head << lgq) + (r & ((1 << lgq) - 1))) * kLog2e : 0.f;
        // (without a cap: not used)
        const float cap_in = fminf(a.scale * (a.cap <= kSmallCap ? 2.f * kLog2e : 1.f) / a.cap, 0x1.fffffep127f), cap_out = a.cap * kLog2e;
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < steps; ++i) {
            const int key0 = (tile0 + (both ? i : 2 * i + x)) * kTile;
            const bool ok = __all_sync(kFull, wait_for(bars, bars + BAR(s_full) + 8 * (x), sc & 1));
            float mul = a.scale_log2;
            ++sc;
            fence_after();
            if (ok && any) {
                // (loops over a tile's columns stay loops: unrolled, the roles' code misses the instruction cache)
                const bool cut = key0 + kTile - 1 > w_hi || key0 < w_lo;
                if (MOD || cut) {                              // logits other than mul * S, hidden ones: written back as such
                    const int hi = p0 + (r >> lgq), lo = a.plan.window ? hi - a.plan.window + 1 : 0;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float v[32];
                        if (!MOD && key0 + 32 * c + 31 <= w_hi && key0 + 32 * c >= w_lo) continue;   // (all rows see all)
                        ld32(ts + 32 * c, v);
                        wait_ld(v);
                        const int d = key0 + 32 * c - hi;      // key less position of the first column
                        if (MOD && a.cap > kSmallCap) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = capped_wide(v[j], cap_in, a.scale_log2, cap_out);
                        } else if (MOD && a.cap > 0.f) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = capped(v[j], cap_in, cap_out);
                        } else if (MOD) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] *= a.scale_log2;
                        }
                        if (MOD && a.slopes) {
                            const float first = slope * (float)d;
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = fmaf(slope, (float)j, v[j] + first);
                        }
                        if (cut) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j > -d || j < lo - hi - d) v[j] = -INFINITY;
                        }
                        st32(ts + 32 * c, v);
                    }
                    wait_st();
                    if (MOD) mul = 1.f;
                }
                // Half a tile at a time: the weights by the present reference are kept in registers until their sum
                // has shown that each is in range (64 of 2^5 are 2^11); a reference that is
                // too low, or none yet, is raised and the half taken again.
                const uint64_t mul2 = pair(mul, mul);
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const uint32_t from = ts + 64 * h;
                    bool again = true;
                    while (true) {
                        const float ref = m == -INFINITY ? 0.f : m - kLift;
                        const uint64_t ref2 = pair(-ref, -ref);
                        uint64_t sum[2] = {0, 0};
                        uint32_t p[32];
                        float v[16], u[16];
                        ld16(from, v);
#pragma unroll
                        for (int c = 0; c < 4; c += 2) {
                            wait_ld(v);
                            ld16(from + 16 * c + 16, u);
                            weights16(p + 8 * c, v, mul2, ref2, sum);
                            wait_ld(u);
                            if (c < 2) ld16(from + 32, v);
                            weights16(p + 8 * c + 8, u, mul2, ref2, sum);
                        }
                        const float2 total = unpair(add2(sum[0], sum[1]));
                        const float all = total.x + total.y;
                        if (!__any_sync(kFull, all >= kMostSum || (again && m == -INFINITY))) {
                            st32(ts + 32 * h, p);
                            l += all;
                            break;
                        }
                        if (!again) {
                            l += clamped_half(from, ts + 32 * h, mul, ref);
                            break;
                        }
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            ld16(from + 16 * c, v);
                            wait_ld(v);
                            mx = max16(mx, v);
                        }
                        // (down: the largest weight is 2^4 at least, and under 2^5 where fp32 tells such logits apart)
                        mx = __fmul_rd(mx, mul);
                        again = false;                         // (the weights by the maximum fit, if there is one)
                        // raised by a whole number, so that scaling what is there (sums, the first half's weights) is exact;
                        // after a jump beyond fp32's exponents nothing is left of it
                        const float rise = mx - m;
                        const float top = m == -INFINITY || rise > 1000.f ? mx : m + fmaxf(0.f, floorf(rise));
                        const float f = m == -INFINITY ? 0.f : exp2_ftz(m - top);
                        m = top;
                        l *= f;
                        if (h) {
                            wait_st();
                            // (two factors: weights of up to 2^15 outlast a factor that fp16 does not hold)
                            const float g1 = fmaxf(f, 0x1p-15f), g2 = fminf(f * 0x1p15f, 1.f);
                            const uint32_t f1 = pack_f16x2(g1, g1), f2 = pack_f16x2(g2, g2);
                            float y[32];
                            ld32(ts, y);
                            wait_ld(y);
#pragma unroll
                            for (int j = 0; j < 32; ++j) p[j] = hmul2(hmul2(__float_as_uint(y[j]), f1), f2);
                            st32(ts, p);
                        }
                        if (i > 0) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                ld32(to + 32 * c, o);
                                wait_ld(o);
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] *= f;
                                st32(to + 32 * c, o);
                            }
                        }
                    }
                }
                wait_st();
            }
            fence_before();
            tile_sync(x);
            if ((warp & 3) == 0)
                issue_mmas<D, BITS>(bars, smem, tmem, x, both ? x : 0, true, i > 0, key0 >= sp->n_quant, tile(i), times(i), i + 1 < steps, tile(i + 1),
                                    times(i + 1));
        }
        tc += sp->nt;
        // ---- epilogue ----
        bool fine = true;
        if (steps) {
            fine = __all_sync(kFull, wait_for(bars, bars + BAR(o_full) + 8 * (x), oc & 1));
            ++oc;
        }
        fence_after();
        float wa = 1.f, wb = 0.f;                              // weights of A's and B's sums
        const bool join = !both && sp->nb > 0;
        if (!both) {
            if (x == 1) {
                xch[row] = make_float2(m, l);
                fence_before();
                named_sync<1, 256>();
                named_sync<2, 256>();                          // A has read B's sums
                continue;
            }
            named_sync<1, 256>();
            fence_after();
            if (join) {
                const float2 o = xch[row];
                const float top = fmaxf(m, o.x);
                const float base = top == -INFINITY ? 0.f : top;
                wa = exp2_ftz(m - base);
                wb = exp2_ftz(o.x - base);
                l = l * wa + o.y * wb;
                m = top;
            }
        }
        if (!fine || *(volatile int*)&b.failed || (*(volatile unsigned*)&b.bad & reader.mark())) m = l = NAN;
        const bool valid = r < n_rows;
        // (all rows are behind the quantized tokens)
        if (const int t = *(volatile int*)&b.last_odd[reader.place()]; t >= 0 && (!a.plan.window || t > p0 + (r >> lgq) - a.plan.window))
            m = l = NAN;
        const int odd0 = *(volatile int*)&b.odd_tile[0][reader.place()], odd1 = *(volatile int*)&b.odd_tile[1][reader.place()];
        if (__any_sync(kFull, odd0 != kNoTile && odd1 >= 0)) {
            // fp16 values that are not finite, in these two tiles at least: a row is NaN if it sees one.  The warp looks for them
            // again, token by token: the first one hides from no row that sees the end of its tile, unless there is a window.
            constexpr int LPR = D / 8, RPI = 32 / LPR;         // lanes a row, rows an instruction
            const Rows v{reinterpret_cast<const __half*>(a.buf + a.v_resid_off) +
                             ((long long)sp->seq * a.plan.Hkv + sp->head) * a.R * D,
                         a.v + sp->tok0 * a.v_stride[0] + sp->head * a.v_stride[1], a.v_stride[0], sp->n_resid, 0};
            const int hi = p0 + (r >> lgq), lo = a.plan.window ? hi - a.plan.window + 1 : 0;
            const int end = min((a.plan.window ? odd1 : odd0) * kTile + kTile, p0 + (min(r0 + 31, n_rows - 1) >> lgq) + 1);
            int t = max(max(odd0 * kTile, sp->n_quant), a.plan.window ? p0 + (r0 >> lgq) - a.plan.window + 1 : 0);
            if (valid && !a.plan.window && hi >= odd0 * kTile + kTile - 1) m = l = NAN;
#pragma unroll 1
            for (; t < end && __any_sync(kFull, valid && l == l); t += RPI) {
                const int at = t + lane / LPR;
                unsigned who = __ballot_sync(kFull, at < end && not_finite(ldg_row(v.at(min(at, end - 1) - sp->n_quant, D) + 8 * (lane % LPR))));
                for (; who; who &= who - 1) {
                    const int x = t + (__ffs(who) - 1) / LPR;
                    if (x >= lo && x <= hi) m = l = NAN;
                }
            }
        }
        __syncwarp();
        const bool whole = sp->whole;
        float* part = a.ws + (((long long)blockIdx.x * 2 + sp->first) * kRows + r) * chunk_partial_stride(D);
        __half* out = a.out + (long long)(sp->tok0 + sp->t0 + (r >> lgq)) * a.out_stride[0] +
                      ((sp->head << lgq) + (r & ((1 << lgq) - 1))) * a.out_stride[1];
        const float inv = 1.f / l;
        if (any) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                __syncwarp();
                if (steps) {
                    ld32(to + 32 * c, o);
                    wait_ld(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0.f;
                }
                if (join) {
                    float p[32];
                    ld32(lanes + S::COL_O + D + 32 * c, p);
                    wait_ld(p);
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = o[j] * wa + p[j] * wb;
                }
                if (valid && whole) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        uint4 v;
                        v.x = pack_out(o[j] * inv, o[j + 1] * inv);
                        v.y = pack_out(o[j + 2] * inv, o[j + 3] * inv);
                        v.z = pack_out(o[j + 4] * inv, o[j + 5] * inv);
                        v.w = pack_out(o[j + 6] * inv, o[j + 7] * inv);
                        *reinterpret_cast<uint4*>(out + 32 * c + j) = v;
                    }
                } else if (valid) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4*>(part + 32 * c + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
            }
            if (valid && !whole) *reinterpret_cast<float2*>(part + D) = make_float2(m, l);
        }
        if (!both) {
            fence_before();
            named_sync<2, 256>();
        }
    }
    if ((warp & 3) == 0) {         // no MMA is in flight when the CTA ends (after a wait that ran out; else none is)
        if (elect_one()) commit(bars + BAR(drained) + 8 * x);
        __syncwarp();
        wait_for<true>(bars, bars + BAR(drained) + 8 * x, 0);
    }
}

template <int D, int BITS, bool MOD>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkArgs a) {
    using S = Shape<D, BITS>;
    extern __shared__ uint8_t raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem = smem_u32(base), bars = smem + S::OFF_BAR;
    Bars& b = *reinterpret_cast<Bars*>(base + S::OFF_BAR);
    float2* xch = reinterpret_cast<float2*>(base + S::OFF_XCH);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int j = 0; j < 2; ++j) {
            mbar_init(&b.k_full[j], 4);
            mbar_init(&b.v_full[j], 4);
            mbar_init(&b.k_empty[j], 2);
            mbar_init(&b.v_empty[j], 2);
            mbar_init(&b.s_full[j], 1);
            mbar_init(&b.o_full[j], 1);
            mbar_init(&b.drained[j], 1);
        }
        for (int j = 0; j < kSpanRing; ++j) {
            mbar_init(&b.span_full[j], 1);
            mbar_init(&b.span_empty[j], kSpanReaders);
        }
        b.failed = b.ended = b.busy = 0;
        b.bad = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&b.tmem);
    fence_before();
    __syncthreads();
    fence_after();
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const uint32_t tmem = b.tmem;
    if (warp < 8) {
        more_regs<Regs<BITS>::SOFTMAX>();
        softmax_rows<D, BITS, MOD>(a, b, bars, smem, xch, tmem, warp >> 2, warp, lane);
    } else if (warp < 16) {
        fewer_regs<Regs<BITS>::FILL>();
        // keys on two of the SM's four schedulers, values on the others: each has the code of one to hold
        fill_tiles<D, BITS>(a, b, bars, smem, warp & 2, (warp & 1) + 2 * (warp >= 12), lane);
    } else {
        fewer_regs<Regs<BITS>::REST>();
        if (warp == 16) plan_spans(a, b, bars, lane);
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0) tmem_free(tmem);
}

template <int D, int BITS, bool MOD>
cudaError_t launch_chunk(const ChunkArgs& a, cudaStream_t st) {
    using S = Shape<D, BITS>;
    auto kernel = chunk_attn_kernel<D, BITS, MOD>;
    // the opt-in to its shared memory is a property of the kernel on a device: made once for each
    static std::atomic<unsigned long long> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev > 63 || !(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        if (dev <= 63) ready.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)a.n_ctas);
    lc.blockDim = dim3(kChunkThreads);
    lc.dynamicSmemBytes = S::SMEM;
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, a);
}
template <int D>
cudaError_t launch_chunk_bits(const ChunkArgs& a, int bits, cudaStream_t st) {
    const bool mod = a.cap > 0.f || a.slopes;
#define KIVI_C(B) \
    if (bits == B) return mod ? launch_chunk<D, B, true>(a, st) : launch_chunk<D, B, false>(a, st);
    KIVI_C(2) KIVI_C(4) KIVI_C(8)
#undef KIVI_C
    return cudaErrorInvalidValue;
}

}  // namespace chunk_detail
}  // namespace kivi
