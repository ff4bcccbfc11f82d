// Internal declarations of the calls that bring several tokens of a sequence at
// once to the paged cache: attention of a chunk, its append, branches, reading back.
#pragma once

#include "kivi_blocks.cuh"

namespace kivi {

// ---- attention of a chunk (kivi.h, kivi_paged_chunk_attn) ----
//
// Work of a call.  Per (sequence, kv head) the queries of the chunk are rows,
// row = token * nq + query head of the group, in items of kRows rows; an item
// reads its keys in tiles of kTile tokens, from the first one that any of its
// rows sees to the last.  An item of more than kHalf rows does the MMAs of two halves a
// tile, one of fewer rows of one; both dequantize it, so their tiles weigh 4 and 3 (with 2
// and 1, of a chunk of 5 whole items and 52 rows over 131072 tokens of 8 heads the CTAs that
// held the 52 rows took twice as long as the others: 929 us, 798 with 4 and 3).  An item's
// tiles come after a lead of weight 14, for what a CTA does once for it (queries in, outputs
// out; a prompt of 8192 tokens of 32 heads over 8: 618 us with a lead of 8, 556 with 11, 533 with 14, 534 with 16, 535 with
// 19; chunks of 777 tokens of 16 heads at most, 64 channels: 96, 99, 98, 98, 106).  Items are in the order sequence, item of the chunk, kv head; CTA c of n takes
// the tiles that start in weights [c W / n, (c + 1) W / n).  A CTA that holds all of an item's
// tiles writes its outputs, others partial results, which a merge joins.
constexpr int kRows = 256, kHalf = 128, kTile = 128;
constexpr int kBothWeight = 4, kHalfWeight = 3, kItemLead = 14;
constexpr int kMaxChunkCtas = 192;       // most CTAs of a call (one per SM)

struct ChunkSeq {
    long long start;    // weight of the sequences before it
    int seq;            // sequence slot: residual rows and block-table row
    int n;              // new tokens
    int tok0;           // its first new token in the packed inputs
    int n_quant;        // quantized tokens
    int n_resid;        // residual rows
    int pad;
};

struct ChunkPlan {
    int nq, Hkv;        // query heads per kv head, kv heads
    int window;         // 0: none
};

__host__ __device__ inline long long floor_div64(long long x) { return x >> 6; }

// Tokens an item's rows cover: kRows / nq, 64 w4.
__host__ __device__ inline int item_tokens(const ChunkPlan& p) { return kRows / p.nq; }
__host__ __device__ inline int item_count(const ChunkPlan& p, int n) {
    return (int)(((long long)n * p.nq + kRows - 1) / kRows);
}
// first and one-past-last key tile of the tokens [t0, t1) of a chunk after c cached tokens
__host__ __device__ inline int first_tile(const ChunkPlan& p, long long c, long long t0) {
    const long long x = c + t0 - p.window + 1;
    return p.window && x > 0 ? (int)(x / kTile) : 0;
}
__host__ __device__ inline int last_tile(long long c, long long t1) { return (int)((c + t1 + kTile - 1) / kTile); }

// One item: its rows, tiles and weight.
struct ChunkItem {
    int t0, t1;         // its tokens of the chunk
    int lo, hi;         // key tiles
    int both;           // more than kHalf rows
    __host__ __device__ int weight() const { return both ? kBothWeight : kHalfWeight; }
    __host__ __device__ long long start(int tile) const { return kItemLead + (long long)weight() * tile; }
    __host__ __device__ long long total() const { return start(hi - lo); }
    // the first tile that starts at weight x or behind it
    __host__ __device__ int tile_at(long long x) const {
        return x <= kItemLead ? 0 : (int)((x - kItemLead + weight() - 1) / weight());
    }
};
__host__ __device__ inline ChunkItem chunk_item(const ChunkPlan& p, const ChunkSeq& s, int m) {
    ChunkItem it;
    const int tpm = item_tokens(p);
    const long long c = (long long)s.n_quant + s.n_resid;
    it.t0 = m * tpm;
    it.t1 = s.n - it.t0 < tpm ? s.n : it.t0 + tpm;
    it.lo = first_tile(p, c, it.t0);
    it.hi = last_tile(c, it.t1);
    it.both = (it.t1 - it.t0) * p.nq > kHalf;
    return it;
}

// Tiles of the first m items of a chunk after c tokens, all of them whole: the sum
// over j < m of ceil((c + (j + 1) T) / 128) less the first tiles, T = 64 w.
__host__ __device__ inline long long whole_tiles(const ChunkPlan& p, long long c, long long m) {
    const long long w = item_tokens(p) / 64;
    const long long a = (c + 63) / 64;
    // sum over j of ceil((a + (j + 1) w) / 2)
    long long sum;
    auto F = [](long long x) { return (x + 1) * (x + 1) / 4; };       // ceil(1/2) + ... + ceil(x/2)
    auto H = [](long long x) { return x * x / 4; };                   // floor(1/2) + ... + floor(x/2), x >= -1
    if (w == 1) sum = F(a + m) - F(a);
    else sum = m * ((a + 1) / 2) + (w / 2) * (m * (m + 1) / 2);
    if (p.window) {
        const long long b = floor_div64(c - p.window + 1);            // floor
        const long long m0 = b >= 0 ? 0 : (-b + w - 1) / w;           // first item whose first key is not below 0
        if (m > m0) {
            const long long b0 = b + w * m0, n = m - m0;
            if (w == 1) sum -= H(b0 + n - 1) - (b0 > 0 ? H(b0 - 1) : 0);
            else sum -= n * (b0 / 2) + (w / 2) * (n * (n - 1) / 2);
        }
    }
    return sum;
}
// weight of the items before item m of a sequence (all heads); m == item_count: the sequence's
__host__ __device__ inline long long items_weight(const ChunkPlan& p, const ChunkSeq& s, int m) {
    const int n = item_count(p, s.n);
    const long long c = (long long)s.n_quant + s.n_resid;
    const int whole = m < n ? m : n - 1;
    long long w = kBothWeight * whole_tiles(p, c, whole) + (long long)kItemLead * whole;
    if (m == n) w += chunk_item(p, s, n - 1).total();
    return w * p.Hkv;
}

// The tiles [first, last) of item (seq, m, head) that a CTA takes.
struct ChunkSpan {
    int seq, m, head;
    ChunkItem it;
    int first, last;    // relative to it.lo
    __host__ __device__ bool whole() const { return first == 0 && last == it.hi - it.lo; }
};
// Walks over a CTA's spans.
struct ChunkWalk {
    const ChunkPlan* p;
    const ChunkSeq* seqs;
    int n_seqs;
    long long x, end;   // weights left to take
    ChunkSpan s;
    long long item0;    // weight where the present item starts
    // Start at weight x0; the item that holds it (an item's tiles that start below x0 are skipped).
    __host__ __device__ void start(const ChunkPlan* plan, const ChunkSeq* sq, int n, long long x0, long long x1) {
        p = plan;
        seqs = sq;
        n_seqs = n;
        x = x0;
        end = x1;
        int lo = 0, hi = n - 1;
        while (lo < hi) {                       // the last sequence that starts at or below x0
            const int mid = (lo + hi + 1) / 2;
            if (sq[mid].start <= x0) lo = mid; else hi = mid - 1;
        }
        s.seq = lo;
        const long long off = x0 - sq[lo].start;
        int ml = 0, mh = item_count(*p, sq[lo].n) - 1;
        while (ml < mh) {
            const int mid = (ml + mh + 1) / 2;
            if (items_weight(*p, sq[lo], mid) <= off) ml = mid; else mh = mid - 1;
        }
        s.m = ml;
        s.it = chunk_item(*p, sq[lo], ml);
        const long long in = off - items_weight(*p, sq[lo], ml);
        s.head = (int)(in / s.it.total());
        item0 = x0 - in % s.it.total();
    }
    // The next span with a tile; false when the range is used up.
    __host__ __device__ bool next() {
        while (x < end) {
            const long long tot = s.it.total();
            s.first = s.it.tile_at(x - item0);
            s.last = s.it.tile_at(end - item0 < tot ? end - item0 : tot);
            x = item0 + tot;                    // (beyond end: the loop ends with the next call)
            if (s.first < s.last) return true;
            advance();
        }
        return false;
    }
    __host__ __device__ void advance() {
        item0 += s.it.total();
        if (++s.head == p->Hkv) {
            s.head = 0;
            if (++s.m == item_count(*p, seqs[s.seq].n)) {
                s.m = 0;
                if (++s.seq == n_seqs) { x = end; s.seq = 0; return; }
            }
            s.it = chunk_item(*p, seqs[s.seq], s.m);
        }
    }
};

struct ChunkArgs {
    const uint8_t* buf;
    const int* table;
    const __half *q, *k, *v;
    __half* out;
    long long q_stride[2], k_stride[2], v_stride[2], out_stride[2];   // token, head (elements)
    long long page_bytes, part_bytes, k_resid_off, v_resid_off;
    int R, lgG, Hq, max_blocks, n_pages, n_seqs, n_ctas;   // lgG: log2 of the group size
    float scale_log2;   // scores to base-2 logits
    float cap;          // > 0: scores are capped at it
    float scale;        // softmax_scale
    const float* slopes;
    ChunkPlan plan;
    long long weight;   // of the whole call
    float* ws;          // partial results: [n_ctas][2][kRows][chunk_partial_stride(D)]
    struct MergeJob* jobs;   // [n_ctas]: what each CTA's first span leaves to be joined
    ChunkSeq seqs[kMaxCallSeqs];
};
// An item whose first tiles CTA c - 1 did and whose others CTAs c .. c + parts - 2 did, written by CTA c
// (parts 0: its first span continues no item, or CTA c - 1 did not begin it).
struct MergeJob {
    int parts, rows;    // rows of the item
    int tok, head;      // its first new token in the packed tensors, kv head
};
// CTAs of a call whose items are `items` (of all heads): a whole tile's weight for each at least, leads not counted.
__host__ __device__ inline int chunk_ctas(long long weight, long long items, int most) {
    const long long n = (weight - kItemLead * items) / kBothWeight;
    return (int)(n < 1 ? 1 : n < most ? n : most);
}
// The weights [x0, x1) of CTA c.
__host__ __device__ inline long long chunk_begin(long long weight, int n_ctas, long long c) { return c * weight / n_ctas; }
constexpr int chunk_partial_stride(int D) { return D + 4; }      // o[D], m, l of a row (16-byte aligned)

// (the first span that the walk gives; called after next())
__host__ __device__ inline MergeJob merge_job(const ChunkWalk& w, long long weight, int n_ctas, int c) {
    MergeJob j{0, 0, 0, 0};
    if (w.s.first == 0 || chunk_begin(weight, n_ctas, c - 1LL) > w.item0 + w.s.it.start(0)) return j;
    const long long last = w.item0 + w.s.it.start(w.s.it.hi - w.s.it.lo - 1);
    j.parts = 2;
    while (c - 1 + j.parts < n_ctas && chunk_begin(weight, n_ctas, c - 1LL + j.parts) <= last) ++j.parts;
    j.rows = (w.s.it.t1 - w.s.it.t0) * w.p->nq;
    j.tok = w.seqs[w.s.seq].tok0 + w.s.it.t0;
    j.head = w.s.head;
    return j;
}

// Outputs: finite weights of finite values, which the weights' own roundings may take past the largest fp16 number (by
// 2^-11 of it): such a one is the largest.  NaN stays.
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
    uint32_t v;
    asm("{\n .reg .b32 t;\n cvt.rn.f16x2.f32 t, %2, %1;\n min.NaN.f16x2 t, t, %3;\n max.NaN.f16x2 %0, t, %4;\n}"
        : "=r"(v) : "f"(lo), "f"(hi), "r"(0x7bff7bffu), "r"(0xfbfffbffu));
    return v;
}

cudaError_t launch_chunk_attn_d64(const ChunkArgs& a, int bits, cudaStream_t st);
cudaError_t launch_chunk_attn_d128(const ChunkArgs& a, int bits, cudaStream_t st);
cudaError_t launch_chunk_merge(const ChunkArgs& a, int D, cudaStream_t st);

// Sequences with few rows (new tokens x query heads per kv head) that see all
// cached tokens: up to kGroupRows rows of a kv head are taken as the query heads
// of a single-token call, whose decode kernel reads the cache for them; the merge adds
// the new tokens.  A sequence of more rows makes several groups, each reads the cache again.
// By groups and by the wide kernel (us a call; 2 bits but where said):
//   rows of a kv head                            4           8           12          16          24
//   8 sequences of 512-7680, 32 heads            51 / 102    87 / 102    123 / 103   159 / 103   236 / 104
//   the same with 4 bits                         58 / 118    93 / 119    131 / 119   171 / 119   253 / 119
//   the same, 32 heads over 8                    20 / 35     31 / 35     39 / 36     48 / 36     65 / 36
//   16 sequences to 15872, 32 over 8, 4 bits     44 / 116    69 / 117    95 / 117    119 / 117   172 / 117
//   64 sequences of 1000, 32 over 8              32 / 65     56 / 65     -           99 / 65     -
// To 8 rows groups are faster; to 16 they cost up to half as much again and keep the decode kernel's accuracy (exact
// dequantized operands), which a verified proposal then shares with the token that is decoded alone; beyond, they would
// cost twice and more.
constexpr int kGroupRows = 4, kFewRows = 16;
struct ChunkGroup {
    int tok0;           // the sequence's first new token in the packed inputs
    int row0, rows;     // its rows of each kv head
};
struct GroupArgs {
    const __half *q, *k, *v;
    __half *out, *gathered;                                           // gathered: [groups][Hkv][nv][D]
    long long q_stride[2], k_stride[2], v_stride[2], out_stride[2];
    const float* ws;    // partial results of the decode kernel
    float scale_log2;
    int Hkv, nq, nv, n; // query heads per kv head, rows per group, groups
    WorkMap wm;
    PagedSeq seqs[kMaxCallSeqs];
    ChunkGroup groups[kMaxCallSeqs];
};
cudaError_t launch_gather_rows(const GroupArgs& a, int D, cudaStream_t st);
cudaError_t launch_group_merge(const GroupArgs& a, int D, cudaStream_t st);

// ---- append of a chunk, branches, reading back (kivi_pages.cu) ----

// A new block of a chunk: rows [row0, row0 + G) of the sequence's virtual rows
// (its residual rows, then its new tokens) quantized into page.
struct ChunkJob {
    int seq, row0, n_resid, tok0;
    int page, tbl_idx;
};
constexpr int kMaxChunkJobs = 1024;      // per launch
cudaError_t launch_quantize_chunk(const PagedGeometry& pg, uint8_t* buf, const __half* k, const long long* k_stride,
                                  const __half* v, const long long* v_stride, const ChunkJob* jobs, int n,
                                  cudaStream_t st, int* launches);

// The residual after a chunk: virtual rows [shift, shift + keep) become residual rows [0, keep).
struct ChunkTail {
    int seq, n_resid, tok0, shift, keep;
};
cudaError_t launch_store_tail(const PagedGeometry& pg, uint8_t* buf, const __half* k, const long long* k_stride,
                              const __half* v, const long long* v_stride, const ChunkTail* tails, int n,
                              cudaStream_t st);

// Branch i: sequence slot to[i] gets the first n_blocks[i] table entries and n_resid[i] residual rows of from[i].
struct ForkJob {
    int from, to, n_blocks, n_resid;
};
cudaError_t launch_fork(const PagedGeometry& pg, uint8_t* buf, const ForkJob* jobs, int n, cudaStream_t st, int* launches);

// Tokens [first, first + count) of each sequence as fp16 [n][Hkv][count][D].
cudaError_t launch_read(const PagedGeometry& pg, const uint8_t* buf, const RowSeq* seqs, int n, long long first,
                        long long count, __half* k, __half* v, cudaStream_t st);

}  // namespace kivi
