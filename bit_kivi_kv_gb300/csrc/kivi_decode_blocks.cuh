// Decode attention over a list of blocks per (query row, kv head) and the fp16
// residual.
//
//   o = sum_t softmax_t(scale * q . k_hat_t) * v_hat_t,   t in the listed
//   blocks' tokens and the residual rows,
//
// with the key and value arithmetic of the dense decode kernel
// (kivi_decode_mma.cuh: codes as fp16 subnormals in mma.sync, steps folded into
// the query and the probabilities, zero points on the side, online softmax in
// the log2 domain, everything summed in fp32).
//
// What differs is the shape of the work: a list has tens of blocks, so a call
// reads little and its latency counts.  One CTA, or a thread-block cluster of
// them, takes one row; its warps split the row's residual tiles (16 rows) and
// tile pairs (32 tokens) by weight, stage their partial results (m, l, o) in
// shared memory, and merge them there (a cluster through distributed shared
// memory): one launch, no workspace, no second kernel.  The blocks' addresses come from the list (paged: through the block
// table), which each warp turns into byte offsets in shared memory, a part of
// the list at a time.
#pragma once

#include "kivi_blocks.cuh"
#include "kivi_decode_mma.cuh"

namespace kivi {
namespace blocks_detail {

using namespace mma_detail;

constexpr int kListCache = 32;      // list entries a warp keeps as byte offsets, one a lane
constexpr int kMaxCluster = 8;      // CTAs that share a row, at most (the portable cluster size)
constexpr int kMaxRowWarps = 16;    // warps of a CTA, at most: two partials each, one a lane in the merge

// Registers a thread may have: 128 (16 warps an SM), and at head_dim 128 with
// four query heads per kv head 168 (12 warps an SM).
template <int D, int NQ>
constexpr int kCtaWarps = (D == 128 && NQ == 4) ? 12 : kMaxRowWarps;

struct Args {
    const uint8_t* cache;
    const __half* q;
    __half* out;
    const int* list;                // [rows][n_list] block numbers; negative: no block
    long long NB, part_bytes, slot_bytes, tile_bytes, k_resid_off, v_resid_off;
    int R, Hq, Hkv;
    int n_list;
    int n_blocks, n_resid;          // dense: quantized blocks and residual rows of every row
    int wq, wr;                     // weights of a tile pair and of a residual tile
    float scale_log2;
    int stall_bytes;                // failure-detection test hook, as in the dense decode kernel
};

struct PagedArgs : Args {
    const int* table;
    int max_blocks, n_pages;
    RowSeq seqs[kMaxCallSeqs];
};

template <bool PAGED>
struct ArgsOf { using type = Args; };
template <>
struct ArgsOf<true> { using type = PagedArgs; };

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// the address of this CTA's shared variable at `a` in the cluster's CTA `rank`
__device__ __forceinline__ uint32_t cluster_map(uint32_t a, uint32_t rank) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
    return d;
}
__device__ __forceinline__ void stc128(uint32_t a, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void stc32(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_u32(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The MMAs of 16-token tiles, A fragments from the lane's words w, B fragments
// from bfrag(t): a key tile sums every k-step into acc, a value tile m-tile t
// into acc[t].
template <int BITS, int W, int KS, typename B>
__device__ __forceinline__ void key_mma(const uint32_t (&w)[W], const B& bfrag, float (&acc)[4]) {
#pragma unroll
    for (int t = 0; t < KS; ++t) {
        uint32_t fa[4];
        a_frag_inline<BITS, false, W>(w, t, fa);
        const uint2 bq = bfrag(t);
        mma16816(acc, fa, bq.x, bq.y);
    }
}
template <int BITS, int W, int KS, typename B>
__device__ __forceinline__ void key_mma2(const uint32_t (&w)[W], const uint32_t (&v)[W], const B& bfrag,
                                         float (&acc)[4], float (&acc2)[4]) {
    uint32_t w8[W], v8[W];
#pragma unroll
    for (int x = 0; x < W; ++x) { w8[x] = w[x] >> 8; v8[x] = v[x] >> 8; }
#pragma unroll
    for (int t = 0; t < KS; ++t) {
        uint32_t fa[4], fb[4];
        a_frag<BITS, false, W>(w, w8, t, fa);
        a_frag<BITS, false, W>(v, v8, t, fb);
        const uint2 bq = bfrag(t);
        mma16816(acc, fa, bq.x, bq.y);
        mma16816(acc2, fb, bq.x, bq.y);
    }
}
template <int BITS, int W, int KS, typename B>
__device__ __forceinline__ void value_mma(const uint32_t (&w)[W], const B& bfrag, float (&acc)[KS][4]) {
    uint32_t w8[W];
    if constexpr (BITS != 8) {
#pragma unroll
        for (int x = 0; x < W; ++x) w8[x] = w[x] >> 8;
    }
#pragma unroll
    for (int t = 0; t < KS; ++t) {
        uint32_t fa[4];
        if constexpr (BITS == 8) a_frag_inline<BITS, true, W>(w, t, fa);
        else a_frag<BITS, true, W>(w, w8, t, fa);
        const uint2 bq = bfrag(t);
        mma16816(acc[t], fa, bq.x, bq.y);
    }
}

// Dynamic shared memory of a CTA: per warp its copy ring (which later takes the
// listed blocks' value sums [NQ][D] fp32), the key fragment table, the list's
// offsets; the residual tiles' value sums [NQ][D] fp32 take the table's place.
template <int D, int BITS, int NQ, int G>
struct Smem {
    using C = Cfg<D, BITS, NQ, G>;
    static constexpr int RING = C::STAGES * C::STAGE_BYTES;
    static constexpr int ROWS = NQ > 1 ? 32 : 8 * NQ + 1;      // rows of the key fragment table
    static constexpr int FRAG = RING, OFFS = FRAG + ROWS * C::QSTRIDE * 4, END = OFFS + kListCache * 8;
    static constexpr int SUMS = FRAG;
    static constexpr int WARP = (END + 127) / 128 * 128;
    static_assert(NQ * D * 4 <= RING, "the value sums reuse the copy ring");
    static_assert(NQ * D * 4 <= ROWS * C::QSTRIDE * 4, "the tiles' sums reuse the table");
};

template <int D, int BITS, int NQ, int G, bool PAGED>
__global__ void __launch_bounds__(32 * kCtaWarps<D, NQ>, 1)
    decode_blocks_kernel(const __grid_constant__ typename ArgsOf<PAGED>::type a) {
    using C = Cfg<D, BITS, NQ, G>;
    using S = Smem<D, BITS, NQ, G>;
    constexpr int KS = C::KSTEPS, W = C::W, NGRP = C::NGRP, GB = C::GB, NBF = C::NBF;
    constexpr int PPB = C::TPB / 2;                   // tile pairs per block
    // the row's scaled query times 2^query_exponent (fp32), and the fp16 hi / lo parts
    // of it times the code scale 2^-(BITS*pos), shared by the CTA's warps
    __shared__ __align__(16) float qf[NQ][D];
    __shared__ uint32_t qhc_s[NQ][D / 2], qlc_s[NQ][D / 2];
    __shared__ float qunit_s[NQ];                 // 2^-query_exponent
    __shared__ __align__(8) uint64_t full_bar[kMaxRowWarps][C::STAGES];
    // the residual's query: fp16 hi and lo parts of each head, a padded row each
    __shared__ __align__(16) __half qres[2 * NQ][D + 8];
    // partial results: (m, l, status) per query head of each warp's residual
    // tiles and of its listed blocks
    __shared__ __align__(16) float4 head_s[2 * kMaxRowWarps][NQ];
    // from the cluster's CTAs: their value sums of this CTA's outputs, and their heads
    __shared__ __align__(16) float recv_s[NQ * D];
    __shared__ __align__(16) float4 recv_head[kMaxCluster][NQ];
    extern __shared__ __align__(128) uint8_t dyn_smem[];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, i = lane & 3;
    const int warps = blockDim.x >> 5;
    const uint32_t crank = cluster_rank(), csize = cluster_size();
    const int cshift = 31 - __clz((int)csize);    // (a power of two)
    const unsigned row32 = blockIdx.x >> cshift;  // (rows are at most 65535)
    const int b = (int)(row32 / (unsigned)a.Hkv), hk = (int)(row32 % (unsigned)a.Hkv);
    const long long row = row32;
    uint8_t* ring = dyn_smem + warp * S::WARP;
    uint32_t* qfrag = reinterpret_cast<uint32_t*>(ring + S::FRAG);
    long long* offs = reinterpret_cast<long long*>(ring + S::OFFS);
    uint64_t* bars = full_bar[warp];
    // B columns from 2 NQ on are zero: with the fragments in registers each lane
    // has its row of the table, else those lanes share the row behind the others'
    for (int idx = 8 * NQ * C::QSTRIDE + lane; idx < S::ROWS * C::QSTRIDE; idx += 32) qfrag[idx] = 0u;
    if (lane == 0) {
#pragma unroll
        for (int st = 0; st < C::STAGES; ++st) mbar_init(&bars[st], 1);
        if (a.stall_bytes && blockIdx.x == 0 && warp == 0) mbar_expect_tx_only(smem_u32(&bars[0]), (uint32_t)a.stall_bytes);
        fence_mbar_init();
    }
    __syncwarp();
    if (csize > 1) cluster_arrive();              // waited for before the merge writes to the other CTAs
    int qoff[D / 64];     // this lane's Qt table offsets (channel pairs (D/64)*lane + j)
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const int cp = (D / 64) * lane + j, cc = (2 * cp) & 15;
        qoff[j] = ((cc & 7) >> 1) * C::QSTRIDE + 2 * (cp >> 3) + (cc >> 3);
    }
    const uint32_t ring_u32 = smem_u32(ring), bars_u32 = smem_u32(bars);
    const long long vdelta = PAGED ? a.part_bytes : a.NB * a.part_bytes;   // key part -> value part of a block
    const int colP = g >> 1, hP = colP / GB, jP = colP % GB;   // this lane's B column for the values
    const bool lo_col = (g & 1) != 0;
    const bool col_ok = hP < NQ;
    const int hO = i / GB, jO = i % GB;                        // this lane's output columns (2i, 2i+1)
    const uint32_t eoff = 32u * jP + 8u * i;
    const long long tiles_bytes = (long long)C::TPB * a.tile_bytes;

    // ---- this warp's share of the row by weight: residual tiles (16 rows), then listed pairs ----
    int nblk, n_res;
    long long rslot;
    if constexpr (PAGED) {
        const RowSeq& sq = a.seqs[b];
        nblk = sq.n_blocks;
        n_res = sq.n_resid;
        rslot = (long long)sq.seq * a.Hkv + hk;
    } else {
        nblk = a.n_blocks;
        n_res = a.n_resid;
        rslot = row;
    }
    // Every worker (a warp) gets its share of the tiles, and pairs up to its
    // share of the weight: tiles from w T / n on, pairs from the largest count on
    // that the weight position of a worker up to w leaves beside the tiles
    // before it.
    const int P = min(a.n_list, nblk) * PPB, T = (n_res + 15) / 16;
    const int workers = (int)csize * warps, worker = (int)crank * warps + warp;
    // (Every warp has to find the same bounds: separately rounded operations
    // give the same fp32 values wherever the expression is compiled.)
    const float per_one = __frcp_rn((float)workers), inv_wq = __frcp_rn((float)a.wq);
    const float per_worker =
        __fmul_rn(__fadd_rn(__fmul_rn((float)T, (float)a.wr), __fmul_rn((float)P, (float)a.wq)), per_one);
    const float per_tile = __fmul_rn((float)T, per_one);
    auto tiles_at = [&](int v) { return floorf(__fmaf_rn((float)v, per_tile, 0.02f)); };   // (whole counts stay whole)
    const int tb = (int)tiles_at(worker), te = worker + 1 == workers ? T : (int)tiles_at(worker + 1);
    auto pairs_at = [&](int v) {                  // pairs that fit before worker v beside the tiles before it
        const float left = __fsub_rn(__fmul_rn((float)v, per_worker), __fmul_rn(tiles_at(v), (float)a.wr));
        return min(P, max(0, (int)ceilf(__fmaf_rn(left, inv_wq, -0.02f))));
    };
    int wb = 0;
    for (int v = lane; v <= worker; v += 32) wb = max(wb, pairs_at(v));
    wb = worker == 0 ? 0 : __reduce_max_sync(kFull, wb);
    int we = worker + 1 == workers ? P : max(wb, pairs_at(worker + 1));
    // A list with more places than the row has blocks (mostly a short sequence's in a
    // ragged call: its blocks, then -1) is dealt out place by place, so that every
    // warp gets its part of the blocks wherever they stand.
    const bool dealt = a.n_list > nblk;
    if (dealt) {
        wb = 0;
        we = nblk > 0 && a.n_list > worker ? ((a.n_list - worker - 1) / workers + 1) * PPB : 0;
    }

    // everything below reads what earlier kernels on the stream may have written
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();

    // a residual tile's rows: lane (g, i) holds channels 32 j + 8 i .. + 7 of rows g, g + 8
    constexpr int DJ = D / 32;
    const __half* kr = reinterpret_cast<const __half*>(a.cache + a.k_resid_off) + rslot * a.R * D;
    const __half* vr = reinterpret_cast<const __half*>(a.cache + a.v_resid_off) + rslot * a.R * D;
    uint4 kx[2][DJ], vx[2][DJ];
    auto load_rows = [&](int tile) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = 16 * tile + g + 8 * s;
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
                kx[s][j] = vx[s][j] = make_uint4(0, 0, 0, 0);
                if (r < n_res) {
                    kx[s][j] = ldg_stream(kr + (long long)r * D + 32 * j + 8 * i);
                    vx[s][j] = ldg_stream(vr + (long long)r * D + 32 * j + 8 * i);
                }
            }
        }
    };
    const int* list = a.list + row * a.n_list;
    uint32_t status = 0;       // 1: a bulk copy did not complete in time; 2: an entry outside the cache
    // entry j of the warp's, none past the n-th
    auto list_entry = [&](int j, int n) {
        int e = -1;                               // (volatile: not moved behind the loads that follow it)
        const bool ok = j < n;
        if (dealt) j = worker + j * workers;
        if (ok) asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(e) : "l"(list + j));
        return e;
    };
    // entry e as the byte offset of its block's key part; -1: no block
    auto offset_of = [&](int e) {
        long long off = -1;
        if (e >= nblk) {
            status |= 2u;
        } else if (e >= 0) {
            if constexpr (PAGED) {
                const int pg = __ldg(a.table + (long long)a.seqs[b].seq * a.max_blocks + e);
                if ((unsigned)pg < (unsigned)a.n_pages)
                    off = ((long long)pg * a.Hkv + hk) * 2 * a.part_bytes;
                else
                    status |= 2u;
            } else {
                off = row * a.slot_bytes + (long long)e * a.part_bytes;
            }
        }
        return off;
    };
    int k = wb;                // next pair to process
    int j0 = 0, kend = wb;     // the part of the list in offs: entries from j0, pairs below kend
    uint32_t item = 0;         // ring item of pair k
    auto issue = [&](int kk, uint32_t it) {       // one lane: pair kk -> ring stage of item it
        const uint32_t st = it % C::STAGES;
        const uint32_t dst = ring_u32 + st * C::STAGE_BYTES, bar = bars_u32 + 8 * st;
        const long long off = offs[kk / PPB - j0];
        if (off < 0) {                            // no block: nothing to wait for
            mbar_arrive_u32(bar);
            return;
        }
        const uint8_t* kp = a.cache + off;
        const uint8_t* vp = kp + vdelta;
        if constexpr (C::WHOLE) {
            mbar_expect_tx_u32(bar, C::STAGE_BYTES);
            tma_1d_u32(dst + C::KT, kp, 2 * C::TILE + C::KSZ, bar);
            tma_1d_u32(dst + C::VT, vp, 2 * C::TILE + 2 * C::ENT, bar);
        } else {
            const int t = 2 * (kk % PPB);         // the pair's first tile in the block
            const bool kz = t == 0 || kk == wb;
            mbar_expect_tx_u32(bar, 4 * C::TILE + 2 * C::ENT + (kz ? C::KSZ : 0));
            tma_1d_u32(dst + C::KT, kp + t * C::TILE, 2 * C::TILE, bar);
            if (kz) tma_1d_u32(dst + C::KE, kp + tiles_bytes, C::KSZ, bar);
            tma_1d_u32(dst + C::VT, vp + t * C::TILE, 2 * C::TILE, bar);
            tma_1d_u32(dst + C::VE, vp + tiles_bytes + t * C::ENT, 2 * C::ENT, bar);
        }
    };
    // the part of the list from pair k on: its entries, ...
    static_assert(kListCache == 32, "one entry a lane");
    int entry = -1;
    auto read_part = [&]() {
        j0 = k / PPB;
        const int end = min((we - 1) / PPB + 1, j0 + kListCache);
        kend = min(we, end * PPB);
        entry = list_entry(j0 + lane, end);
    };
    // ... then their offsets, and the part's first copies.  The part ends behind its last
    // block; entries without one from there on are read again, or passed over if
    // the part has none.
    auto begin_part = [&]() {
        const uint32_t some = __ballot_sync(kFull, entry >= 0);
        if (some == 0u) k = kend;
        kend = min(kend, (j0 + 32 - __clz(some)) * PPB);
        offs[lane] = offset_of(entry);
        __syncwarp();
        if (lane < C::STAGES && k + lane < kend) {   // the part's first copies, a lane each
            fence_proxy_async();
            issue(k + lane, item + lane);
        }
        __syncwarp();
    };
    // a lane's channel pairs (D / 64 of them) of query head j, one warp a head
    // (volatile: on its way while the list is read)
    const __half* qp = a.q + ((long long)b * a.Hq + hk * NQ) * D;
    constexpr int CPL = D / 64;
    auto query = [&](int j, uint32_t (&x)[CPL]) {
        const __half* p = qp + j * D + 2 * CPL * lane;
        if constexpr (CPL == 2) asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[CPL - 1]) : "l"(p));
        else asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(x[0]) : "l"(p));
    };
    uint32_t qv[CPL] = {};
    if (warp < NQ) query(warp, qv);
    if (k < we) {
        read_part();
        begin_part();
    }
    for (int j = warp; j < NQ; j += warps) {
        if (j != warp) query(j, qv);
        const uint32_t most = max(abs_max_f16x2(qv[0]), abs_max_f16x2(qv[CPL - 1]));
        const int ex = query_exponent(unpack_f16x2(__reduce_max_sync(kFull, most)).x * a.scale_log2);
        if (lane == 0) qunit_s[j] = pow2i(-ex);
#pragma unroll
        for (int u = 0; u < CPL; ++u) {
            const int cp = CPL * lane + u;
            const float2 f = unpack_f16x2(qv[u]);
            const float x0 = f.x * a.scale_log2 * pow2i(ex), x1 = f.y * a.scale_log2 * pow2i(ex);
            qf[j][2 * cp] = x0;
            qf[j][2 * cp + 1] = x1;
            const uint32_t hi = pack_f16x2(x0, x1);
            const float2 hf = unpack_f16x2(hi);
            *reinterpret_cast<uint32_t*>(&qres[2 * j][2 * cp]) = hi;
            *reinterpret_cast<uint32_t*>(&qres[2 * j + 1][2 * cp]) = pack_f16x2(x0 - hf.x, x1 - hf.y);
            // channels 2cp, 2cp+1 have class cp / 4: their codes read as code * 2^(BITS*pos - 24)
            const float cs = pow2i(-BITS * ((cp >> 2) % (8 / BITS)));
            const float y0 = x0 * cs, y1 = x1 * cs;
            const uint32_t hic = pack_f16x2(y0, y1);
            const float2 hcf = unpack_f16x2(hic);
            qhc_s[j][cp] = hic;
            qlc_s[j][cp] = pack_f16x2(y0 - hcf.x, y1 - hcf.y);
        }
    }
    __syncthreads();

    // this lane's head: the logits' unit of the fp16 rows, and of the block at hand
    const float qunit = qunit_s[i < NQ ? i : 0];
    float unit = 0.f;
    float m = -INFINITY, l = 0.f;
    bool fresh = true;                            // no tile counted yet
    float o[KS][4];
    float zeta[NBF];
#pragma unroll
    for (int t = 0; t < KS; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
#pragma unroll
    for (int f = 0; f < NBF; ++f) zeta[f] = 0.f;
    constexpr bool QB_REGS = NQ > 1;
    uint32_t qb[2 * KS] = {};
    auto qbk = [&](const int kk) -> uint2 {       // the key B fragment of k-step kk (see build_q_frags)
        if constexpr (QB_REGS)
            return make_uint2(qb[2 * kk], qb[2 * kk + 1]);
        else
            return *reinterpret_cast<const uint2*>(qfrag + min(lane, 8 * NQ) * C::QSTRIDE + 2 * kk);
    };
    float beta = 0.f;

    ValueRange range;
    KeyRange krange;
    const int ao_lane = (lane & ~3) | (hO < NQ ? hO : 0), az_lane = col_ok ? hP : 0;
    auto softmax = [&](const float (&sc)[4], float (&p)[4], float unit, uint32_t steps) {
        softmax_pair(sc, p, unit, steps, range, m, l, fresh, o, zeta, ao_lane, az_lane);
    };
    // probabilities of tokens 2i, 2i+1, 2i+8, 2i+9 of head hP, and their fp16 hi / lo parts
    auto gather = [&](float p0, float p1, float (&pr)[4]) {
        const int src = 8 * i + (col_ok ? hP : 0);
        pr[0] = __shfl_sync(kFull, p0, src);
        pr[1] = __shfl_sync(kFull, p0, src + 4);
        pr[2] = __shfl_sync(kFull, p1, src);
        pr[3] = __shfl_sync(kFull, p1, src + 4);
        if (!col_ok) pr[0] = pr[1] = pr[2] = pr[3] = 0.f;
    };
    auto split_p = [&](const float (&pr)[4], uint32_t& ph01, uint32_t& ph89, uint32_t& pl01, uint32_t& pl89) {
        ph01 = pack_f16x2(pr[0], pr[1]);
        ph89 = pack_f16x2(pr[2], pr[3]);
        const float2 f01 = unpack_f16x2(ph01), f89 = unpack_f16x2(ph89);
        pl01 = pack_f16x2(pr[0] - f01.x, pr[1] - f01.y);
        pl89 = pack_f16x2(pr[2] - f89.x, pr[3] - f89.y);
    };
    const uint32_t lane_words = (uint32_t)(lane * W * 4);
    auto lds_words = [&](uint32_t src, uint32_t (&w)[W]) {   // this lane's words of a tile at src
        if constexpr (W % 4 == 0) {
#pragma unroll
            for (int v = 0; v < W / 4; ++v) {
                const uint4 x = lds128(src + lane_words + 16 * v);
                w[4 * v] = x.x; w[4 * v + 1] = x.y; w[4 * v + 2] = x.z; w[4 * v + 3] = x.w;
            }
        } else {
            const uint2 x = lds64(src + lane_words);
            w[0] = x.x; w[1] = x.y;
        }
    };
    auto sum_l = [&]() {                          // l over the lanes of a head
        float lt = l;
        lt += __shfl_xor_sync(kFull, lt, 4);
        lt += __shfl_xor_sync(kFull, lt, 8);
        lt += __shfl_xor_sync(kFull, lt, 16);
        return lt;
    };
    // a value tile of the stage at stage_u32: the probabilities of its tokens g
    // and g + 8, its words
    auto value_tile = [&](uint32_t stage_u32, int t, float p0, float p1, const uint32_t (&wv)[W]) {
        float prb[4];
        gather(p0, p1, prb);
        uint32_t ph01, ph89, pl01, pl89;
        split_p(prb, ph01, ph89, pl01, pl89);
        const uint32_t ve = stage_u32 + C::VE + t * C::ENT + eoff;
        uint32_t pb[NBF][2];
#pragma unroll
        for (int f = 0; f < NBF; ++f) {            // B fragments of p * step, and p . zero
            const uint2 sv = lds64(ve + 32u * GB * f), zv = lds64(ve + 32u * (NGRP + GB * f));
            uint32_t h01, h89, l01, l89;
            product_parts(ph01, pl01, sv.x, range.grid, h01, l01);
            product_parts(ph89, pl89, sv.y, range.grid, h89, l89);
            pb[f][0] = lo_col ? l01 : h01;
            pb[f][1] = lo_col ? l89 : h89;
            const float2 z01 = unpack_f16x2(zv.x), z89 = unpack_f16x2(zv.y);
            zeta[f] = fmaf(prb[0], z01.x, fmaf(prb[1], z01.y, fmaf(prb[2], z89.x, fmaf(prb[3], z89.y, zeta[f]))));
        }
        auto pbk = [&](int mt) { return make_uint2(pb[(16 * mt / G) / GB][0], pb[(16 * mt / G) / GB][1]); };
        value_mma<BITS, W, KS>(wv, pbk, o);
    };
    // ---- the listed blocks ----
    while (k < we) {
        if (k >= kend) {
            read_part();
            begin_part();
        }
        bool failed = false;
        bool skip = false;
        for (; k < kend; ++k, ++item) {
            const uint32_t st = item % C::STAGES;
            if (!__all_sync(kFull, mbar_wait(&bars[st], (item / C::STAGES) & 1u))) { failed = true; break; }
            const uint8_t* stage = ring + st * C::STAGE_BYTES;
            const uint32_t stage_u32 = ring_u32 + st * C::STAGE_BYTES;
            const bool first_of_block = k % PPB == 0 || k == wb;
            if (first_of_block) skip = offs[k / PPB - j0] < 0;
            if (!skip) {
                if (first_of_block)
                    build_q_frags<C, D, NQ, QB_REGS>(stage + C::KE, qf, qhc_s, qlc_s, qoff, qfrag, lane, qb, beta,
                                                     &qunit, krange, unit, fresh);
                float ca[4] = {0.f, 0.f, 0.f, 0.f}, cb[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t wa[W], wc[W];
                lds_words(stage_u32 + C::KT, wa);
                if constexpr (BITS == 8) {                     // one tile at a time: the words of two do not fit
                    key_mma<BITS, W, KS>(wa, qbk, ca);
                    lds_words(stage_u32 + C::KT + C::TILE, wc);
                    key_mma<BITS, W, KS>(wc, qbk, cb);
                } else {                                       // two chains of sums side by side
                    lds_words(stage_u32 + C::KT + C::TILE, wc);
                    key_mma2<BITS, W, KS>(wa, wc, qbk, ca, cb);
                }
                const float sc[4] = {ca[0] + (ca[1] + beta), ca[2] + (ca[3] + beta), cb[0] + (cb[1] + beta),
                                     cb[2] + (cb[3] + beta)};
                constexpr bool HOIST = BITS != 8 && W <= 4;   // as in the dense kernel
                uint32_t wvh[2][W];
                if constexpr (HOIST) {
                    lds_words(stage_u32 + C::VT, wvh[0]);
                    lds_words(stage_u32 + C::VT + C::TILE, wvh[1]);
                }
                float p[4];
                softmax(sc, p, unit, pair_steps<C, NGRP>(stage_u32, lane));
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t wv[W];
                    if constexpr (HOIST) {
#pragma unroll
                        for (int x = 0; x < W; ++x) wv[x] = wvh[t][x];
                    } else {
                        lds_words(stage_u32 + C::VT + t * C::TILE, wv);
                    }
                    value_tile(stage_u32, t, p[2 * t], p[2 * t + 1], wv);
                }
            }
            __syncwarp();                                      // every lane is done with this stage
            if (lane == 0 && k + C::STAGES < kend) issue(k + C::STAGES, item + C::STAGES);
        }
        if (failed) {
            // a copy timed out: wait (bounded) for the copies in flight, issue no more
            status |= 1u;
            for (int u = 0; u < C::STAGES && k + u < kend; ++u)
                mbar_wait(&bars[(item + u) % C::STAGES], ((item + u) / C::STAGES) & 1u);
            break;
        }
    }
    // ---- the listed blocks' partial result ----
#pragma unroll
    for (int f = 0; f < NBF; ++f) {
        zeta[f] += __shfl_xor_sync(kFull, zeta[f], 1);
        zeta[f] += __shfl_xor_sync(kFull, zeta[f], 2);
    }
    float zo[NBF];
#pragma unroll
    for (int f = 0; f < NBF; ++f) zo[f] = __shfl_sync(kFull, zeta[f], 8 * i);
    float* sums = reinterpret_cast<float*>(ring);
    if (hO < NQ) {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
            const int gr = 16 * mt / G;
            if (gr % GB == jO) {
                // the sums are in units of 2^(BITS*pos - 24), pos = (channel / 8) % (8 / BITS):
                // rows g and g+8 of m-tile mt have classes 2mt and 2mt+1
                const float u0 = pow2i(24 - BITS * ((2 * mt) % (8 / BITS)));
                const float u1 = pow2i(24 - BITS * ((2 * mt + 1) % (8 / BITS)));
                const float z = zo[gr / GB];
                sums[hO * D + 16 * mt + g] = fmaf(o[mt][0] + o[mt][1], u0, z);
                sums[hO * D + 16 * mt + g + 8] = fmaf(o[mt][2] + o[mt][3], u1, z);
            }
        }
    }
    {
        const uint32_t st_all = __reduce_or_sync(kFull, status);
        const float lt = sum_l();
        if (g == 0 && i < NQ) head_s[warps + warp][i] = make_float4(m, lt, (float)st_all, 0.f);
    }

    // ---- the residual tiles: 16 fp16 rows each, straight from memory.  The
    // 16-byte loads hand lane i eight consecutive channels, so the MMAs' k
    // (keys) and m (values) indices run over the channels in another order than
    // the tiles': k-steps 2j, 2j+1 hold channels 32 j + 8 i + 0..3, + 4..7, and
    // m-tile 2j+u has row g at channel 32 j + 8 (g / 2) + 4 u + g % 2, row g + 8
    // two further.  Their partial result is kept apart from the blocks'. ----
    float* rsum = reinterpret_cast<float*>(ring + S::SUMS);
    if (tb < te) {
        m = -INFINITY;
        l = 0.f;
        fresh = true;
        range = ValueRange{};
#pragma unroll
        for (int t = 0; t < KS; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
        // (Prefetching the rows into L2 at the start of the call, or a few pairs
        // ahead, took the bandwidth that the first copies wait for: 7B 12.3 and 11.9
        // us against 11.6; spread over the pairs, 512 rows of four heads: 42.9 against
        // 41.8.  Odd warps taking their tiles first: 44.1.)
        for (int tile = tb; tile < te; ++tile) {
            load_rows(tile);
            const bool okg = 16 * tile + g < n_res, okg8 = 16 * tile + g + 8 < n_res;
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
                uint4 bq = make_uint4(0, 0, 0, 0);
                if (g < 2 * NQ) bq = *reinterpret_cast<const uint4*>(&qres[g < 2 * NQ ? g : 0][32 * j + 8 * i]);
                const uint32_t f0[4] = {kx[0][j].x, kx[1][j].x, kx[0][j].y, kx[1][j].y};
                const uint32_t f1[4] = {kx[0][j].z, kx[1][j].z, kx[0][j].w, kx[1][j].w};
                mma16816(c, f0, bq.x, bq.y);
                mma16816(c, f1, bq.z, bq.w);
            }
            const float sc[4] = {okg ? c[0] + c[1] : -INFINITY, okg8 ? c[2] + c[3] : -INFINITY, -INFINITY, -INFINITY};
            float p[4];
            softmax(sc, p, qunit, 0u);
            float prb[4];
            gather(p[0], p[1], prb);
            uint32_t ph01, ph89, pl01, pl89;
            split_p(prb, ph01, ph89, pl01, pl89);
            const uint32_t pb0 = lo_col ? pl01 : ph01, pb1 = lo_col ? pl89 : ph89;
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
                const uint32_t f0[4] = {movmatrix_trans(vx[0][j].x), movmatrix_trans(vx[0][j].y),
                                        movmatrix_trans(vx[1][j].x), movmatrix_trans(vx[1][j].y)};
                mma16816(o[2 * j], f0, pb0, pb1);
                const uint32_t f1[4] = {movmatrix_trans(vx[0][j].z), movmatrix_trans(vx[0][j].w),
                                        movmatrix_trans(vx[1][j].z), movmatrix_trans(vx[1][j].w)};
                mma16816(o[2 * j + 1], f1, pb0, pb1);
            }
        }
        const float lt = sum_l();
        if (g == 0 && i < NQ) head_s[warp][i] = make_float4(m, lt, 0.f, 0.f);
        if (hO < NQ) {                            // every group slot's columns hold the same sums: each writes some
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                if (mt % GB != jO) continue;
                const int ch = 32 * (mt / 2) + 8 * (g / 2) + 4 * (mt % 2) + g % 2;
                rsum[hO * D + ch] = o[mt][0] + o[mt][1];
                rsum[hO * D + ch + 2] = o[mt][2] + o[mt][3];
            }
        }
    } else {                                      // no tiles: no weight, zero sums
        if (lane < NQ) head_s[warp][lane] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
        for (int idx = 4 * lane; idx < NQ * D; idx += 128)
            *reinterpret_cast<float4*>(rsum + idx) = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    // ---- the log-sum-exp merge: the CTA's partials, then the cluster's CTAs ----
    // Every warp weighs the partials of its outputs' head for itself, one a
    // lane, and hands the weights round by shuffles.
    constexpr int kOutShift = NQ * D == 64 ? 6 : NQ * D == 128 ? 7 : NQ * D == 256 ? 8 : 9;
    static_assert(NQ * D == 1 << kOutShift, "outputs of a row");
    const int span = NQ * D >> cshift;            // the outputs a CTA of the cluster writes
    __half* out = a.out + ((long long)b * a.Hq + hk * NQ) * D;
    __syncwarp();                                 // (the cluster's barrier wants whole warps)
    if (csize > 1) cluster_wait();                // (every CTA has started: its shared memory may be written)
    __syncthreads();
    for (int base = 32 * warp; base < NQ * D; base += blockDim.x) {
        const int idx = base + lane, h = base / D;
        const float4 x = lane < 2 * warps ? head_s[lane][h] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        float M = x.x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, s));
        const float e = x.x == -INFINITY ? 0.f : fast_exp2(x.x - M);   // (a partial without tokens: weight 0)
        float L = x.y * e, sum = 0.f;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) L += __shfl_xor_sync(kFull, L, s);
        const bool bad = __any_sync(kFull, x.z != 0.f);
#pragma unroll 4
        for (int j = 0; j < warps; ++j) {
            const float* mine = reinterpret_cast<const float*>(dyn_smem + j * S::WARP) + idx;
            const float er = __shfl_sync(kFull, e, j), eb = __shfl_sync(kFull, e, warps + j);
            sum = fmaf(mine[S::SUMS / 4], er, fmaf(mine[0], eb, sum));
        }
        if (csize > 1) {
            stc32(cluster_map(smem_u32(&recv_s[(int)crank * span + (idx & (span - 1))]), (unsigned)idx >> (kOutShift - cshift)), sum);
            if (idx % D < (int)csize)             // (csize <= 8 < D) the head's (M, L, status) to each CTA
                stc128(cluster_map(smem_u32(&recv_head[crank][h]), idx % D), make_float4(M, L, bad ? 1.f : 0.f, 0.f));
        } else {
            out[idx] = __float2half_rn(bad ? NAN : sum / L);
        }
    }
    if (csize == 1) return;
    // each CTA has sent the owner of every output its sum, and all of them its
    // heads; nothing is read from afar, so a CTA may leave first
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (int at = tid; at < span; at += blockDim.x) {
        const int idx = (int)crank * span + at, h = idx / D;
        float M = -INFINITY, L = 0.f, s = 0.f, bad = 0.f;
        for (int j = 0; j < (int)csize; ++j) M = fmaxf(M, recv_head[j][h].x);
        for (int j = 0; j < (int)csize; ++j) {
            const float4 x = recv_head[j][h];
            const float e = x.x == -INFINITY ? 0.f : fast_exp2(x.x - M);
            L = fmaf(x.y, e, L);
            s = e == 0.f ? s : fmaf(recv_s[j * span + at], e, s);
            bad += x.z;
        }
        out[idx] = __float2half_rn(bad != 0.f ? NAN : s / L);
    }
}

}  // namespace blocks_detail
}  // namespace kivi
