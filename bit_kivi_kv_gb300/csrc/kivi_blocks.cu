// Decode over chosen blocks (include/kivi.h): the block scores, the selection,
// the launch of attention over the listed blocks, and the dense cache's calls.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <mutex>

#include "kivi_decode_blocks.cuh"

namespace kivi {

cudaError_t launch_decode_blocks_d128(const blocks_detail::Args& a, int bits, int nq, int G, long long rows,
                                      long long units, int num_sms, cudaStream_t st);
cudaError_t launch_decode_blocks_d64(const blocks_detail::Args& a, int bits, int nq, int G, long long rows,
                                     long long units, int num_sms, cudaStream_t st);
cudaError_t launch_decode_blocks_d128p(const blocks_detail::PagedArgs& a, int bits, int nq, int G, long long rows,
                                       long long units, int num_sms, cudaStream_t st);
cudaError_t launch_decode_blocks_d64p(const blocks_detail::PagedArgs& a, int bits, int nq, int G, long long rows,
                                      long long units, int num_sms, cudaStream_t st);

namespace {

using mma_detail::griddepcontrol_launch_dependents;
using mma_detail::griddepcontrol_wait;
using mma_detail::kFull;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

kivi_status failf(kivi_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
kivi_status failf(kivi_status st, const char* fmt, ...) {
    char msg[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return report_error(st, msg);
}

kivi_status launched(cudaError_t e, const char* what) {
    if (e != cudaSuccess) return failf(KIVI_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
    count_launches(1);
    return report_error(KIVI_OK, "");
}

// ---- block scores ----
//
// A key block's entries give, per channel, its least dequantized key z_c and
// its largest z_c + L s_c (L = 2^b - 1), so
//
//   u = sum_c q_c z_c + L sum_c max(q_c, 0) s_c
//
// is at least every logit q . k_hat_t of the block.  A lane holds 8 channels'
// steps or 8 channels' zeros of a block (one 16-byte load) and multiplies them
// with its 8 coefficients, L scale max(q_c, 0) or scale q_c, held in registers
// for the whole row; D / 4 lanes share a block.  Eight loads are in flight per
// lane, and the eight sums are reduced together by halving: each step adds
// the half of the sums that the partner lane drops.
constexpr int kScoreWarps = 8;
constexpr int kScoreLoads = 8;       // 16-byte loads in flight per lane

struct ScoreArgs {
    const uint8_t* cache;
    const __half* q;
    float* scores;
    long long ld, part_bytes, slot_bytes, entries_off;
    int Hq, Hkv, n_blocks;
    int iters;                       // groups of blocks a warp takes
    float scale, levels;
};
struct PagedScoreArgs : ScoreArgs {
    const int* table;
    int max_blocks, n_pages;
    RowSeq seqs[kMaxCallSeqs];
};
template <bool PAGED>
struct ScoreArgsOf { using type = ScoreArgs; };
template <>
struct ScoreArgsOf<true> { using type = PagedScoreArgs; };

template <int D, int NQ, bool PAGED>
__global__ void __launch_bounds__(32 * kScoreWarps)
    block_scores_kernel(const __grid_constant__ typename ScoreArgsOf<PAGED>::type a) {
    constexpr int LPB = D / 4;                // lanes per block
    constexpr int BPL = 32 / LPB;             // blocks a warp-wide load covers
    constexpr int BPI = kScoreLoads * BPL;    // blocks per iteration
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lb = lane % LPB, sub = lane / LPB;
    const long long row = blockIdx.y;
    const int b = (int)blockIdx.y / a.Hkv, hk = (int)blockIdx.y % a.Hkv;
    int nblk = a.n_blocks;
    if constexpr (PAGED) nblk = a.seqs[b].n_blocks;
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    float* out = a.scores + row * a.ld;
    const long long n0 = ((long long)blockIdx.x * kScoreWarps + warp) * a.iters * BPI;
    // a group's loads; a page outside the pool is read as page 0 and marked
    uint4 x[kScoreLoads];
    uint32_t bad = 0u;
    auto load_group = [&](long long first) {
        bad = 0u;
#pragma unroll
        for (int u = 0; u < kScoreLoads; ++u) {
            const long long n = first + u * BPL + sub;
            x[u] = make_uint4(0, 0, 0, 0);
            if (n < nblk) {
                const uint8_t* kp;
                if constexpr (PAGED) {
                    const int pg = __ldg(a.table + (long long)a.seqs[b].seq * a.max_blocks + n);
                    const bool out_of_pool = (unsigned)pg >= (unsigned)a.n_pages;
                    if (out_of_pool) bad |= 1u << u;
                    kp = a.cache + ((long long)(out_of_pool ? 0 : pg) * a.Hkv + hk) * 2 * a.part_bytes;
                } else {
                    kp = a.cache + row * a.slot_bytes + n * a.part_bytes;
                }
                x[u] = mma_detail::ldg_stream(kp + a.entries_off + 16 * lb);
            }
        }
    };
    if (n0 < a.ld) load_group(n0);           // on its way before the query
    // the lane's coefficients: channels 8 (lb % (D/8)) .. of steps (first half of the lanes) or zeros
    const bool steps = lb < LPB / 2;
    float coef[NQ][8];
#pragma unroll
    for (int h = 0; h < NQ; ++h) {
        const uint4 qx = *reinterpret_cast<const uint4*>(a.q + ((long long)b * a.Hq + hk * NQ + h) * D + 8 * (lb % (D / 8)));
        const uint32_t w[4] = {qx.x, qx.y, qx.z, qx.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = mma_detail::unpack_f16x2(w[j]);
            coef[h][2 * j] = steps ? fmaxf(f.x, 0.f) * a.levels * a.scale : f.x * a.scale;
            coef[h][2 * j + 1] = steps ? fmaxf(f.y, 0.f) * a.levels * a.scale : f.y * a.scale;
        }
    }
    for (int it = 0; it < a.iters; ++it) {
        const long long first = n0 + (long long)it * BPI;
        if (first >= a.ld) break;
        if (it) load_group(first);
        float best = -INFINITY;
#pragma unroll
        for (int h = 0; h < NQ; ++h) {
            float s[kScoreLoads];
#pragma unroll
            for (int u = 0; u < kScoreLoads; ++u) {
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                float t = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = mma_detail::unpack_f16x2(w[j]);
                    t = fmaf(coef[h][2 * j], f.x, fmaf(coef[h][2 * j + 1], f.y, t));
                }
                s[u] = PAGED && (bad >> u & 1u) ? NAN : t;
            }
            // sums over the block's LPB lanes; lane bits LPB/2, LPB/4, LPB/8 pick the load
#pragma unroll
            for (int n = kScoreLoads / 2, o = LPB / 2; n >= 1; n /= 2, o /= 2) {
                const bool up = (lane & o) != 0;
#pragma unroll
                for (int u = 0; u < n; ++u) {
                    const float keep = up ? s[u + n] : s[u], give = up ? s[u] : s[u + n];
                    s[u] = keep + __shfl_xor_sync(kFull, give, o);
                }
            }
#pragma unroll
            for (int o = LPB / 16; o >= 1; o /= 2) s[0] += __shfl_xor_sync(kFull, s[0], o);
            best = s[0] != s[0] || best != best ? NAN : fmaxf(best, s[0]);
        }
        const int u = lb / (LPB / 8);
        const long long n = first + u * BPL + sub;
        if (lb % (LPB / 8) == 0 && n < a.ld) out[n] = n < nblk ? best : -INFINITY;
    }
}

template <int D, int NQ, bool PAGED>
cudaError_t launch_scores_t(typename ScoreArgsOf<PAGED>::type& a, long long rows, int num_sms, cudaStream_t st) {
    constexpr int BPI = kScoreLoads * 128 / D;
    // a warp's coefficients cost about one group of blocks: two groups a warp
    // where the grid still gives every SM eight CTAs (131k tokens: 2 groups 21.5
    // us, 4 groups 22.2)
    const long long groups = (a.ld + (long long)kScoreWarps * BPI - 1) / (kScoreWarps * BPI);
    long long iters = groups * rows / (8LL * (num_sms > 0 ? num_sms : 1));
    iters = iters < 1 ? 1 : iters > 2 ? 2 : iters;
    a.iters = (int)iters;
    const long long ctas = (groups + iters - 1) / iters;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_dependent(block_scores_kernel<D, NQ, PAGED>, dim3((unsigned)ctas, (unsigned)rows), 32 * kScoreWarps,
                            st, a);
}

template <bool PAGED>
cudaError_t launch_scores(typename ScoreArgsOf<PAGED>::type& a, const BlockRows& r, cudaStream_t st) {
    const int nq = r.g->Hq / r.g->Hkv;
    const long long rows = (long long)r.n * r.g->Hkv;
#define KIVI_S(DD, NN) \
    if (r.g->D == DD && nq == NN) return launch_scores_t<DD, NN, PAGED>(a, rows, r.num_sms, st);
    KIVI_S(128, 1) KIVI_S(128, 2) KIVI_S(128, 4) KIVI_S(64, 1) KIVI_S(64, 2) KIVI_S(64, 4)
#undef KIVI_S
    return cudaErrorInvalidValue;
}

// ---- selection ----
//
// A score as an unsigned key in the same order: 0 for -inf and NaN (never
// chosen), all ones for a column that is always kept.  -0 and +0 are equal.
__device__ __forceinline__ uint32_t score_key(float x, bool always) {
    if (!(x > -INFINITY)) return 0u;
    if (always) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);   // -FLT_MAX -> 0x00800000 > 0; +inf -> 0xff800000
}

struct SelectArgs {
    const float* scores;
    long long rows, cols, ld;
    int n_keep, keep_first;
    int* blocks;
};

// In both kernels: t is the least key taken, `take` the number of columns
// taken; every key above t is taken, and of those equal to t the first ones in
// index order.  A chosen column's place is the number of chosen ones before it.

// Rows of up to 256 columns, and many of up to 1024: one warp each, its keys in
// registers, no barriers.  t is found by bisection on its bits, highest first,
// each step one count over the warp, until as many keys as wanted are at least t.
constexpr int kWarpRows = 4;         // rows (warps) per CTA

template <int kWarpItems>            // keys a lane
__global__ void __launch_bounds__(32 * kWarpRows) select_blocks_warp_kernel(const SelectArgs a) {
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * kWarpRows + (threadIdx.x >> 5);
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    if (r >= a.rows) return;
    const float* row = a.scores + r * a.ld;
    int* out = a.blocks + r * a.n_keep;
    const int cols = (int)a.cols, K = a.n_keep;
    float x[kWarpItems];
#pragma unroll
    for (int j = 0; j < kWarpItems; ++j) x[j] = 32 * j + lane < cols ? row[32 * j + lane] : -INFINITY;
    uint32_t key[kWarpItems];
#pragma unroll
    for (int j = 0; j < kWarpItems; ++j) key[j] = score_key(x[j], 32 * j + lane < a.keep_first);
    auto count = [&](uint32_t t) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < kWarpItems; ++j) n += key[j] >= t;
        return __reduce_add_sync(kFull, n);
    };
    const int valid = count(1u);
    uint32_t t = 1u;
    if (valid > K) {
        uint32_t most = 0u, least = 0xffffffffu;
#pragma unroll
        for (int j = 0; j < kWarpItems; ++j) {
            most = max(most, key[j]);
            least = key[j] ? min(least, key[j]) : least;
        }
        most = __reduce_max_sync(kFull, most);
        least = __reduce_min_sync(kFull, least);
        // the bits above the highest one in which two keys differ are common to all
        const int top = 31 - __clz(most ^ least);               // -1: all equal
        t = top < 0 ? most : top == 31 ? 0u : most & ~((2u << top) - 1u);
        for (int bit = top; bit >= 0; --bit) {
            const uint32_t c = t | (1u << bit);
            const int n = count(c);
            if (n >= K) t = c;
            if (n == K) break;
        }
    }
    const int take = min(valid, K);
    int above = 0;
#pragma unroll
    for (int j = 0; j < kWarpItems; ++j) above += key[j] > t;
    const int ties = take - __reduce_add_sync(kFull, above);
    const uint32_t below = (1u << lane) - 1u;
    int before_a = 0, before_e = 0;
#pragma unroll
    for (int j = 0; j < kWarpItems; ++j) {
        const uint32_t k = key[j];
        const uint32_t ma = __ballot_sync(kFull, k > t), me = __ballot_sync(kFull, k == t);
        const int ra = before_a + __popc(ma & below), re = before_e + __popc(me & below);
        if (k > t || (k == t && re < ties)) out[ra + min(re, ties)] = 32 * j + lane;
        before_a += __popc(ma);
        before_e += __popc(me);
    }
    for (int j = take + lane; j < K; j += 32) out[j] = -1;
}

// Longer rows: one CTA each.  The keys between two bounds that hold the wanted
// one are counted in 2048 equal bins of the range that they span; the bin of
// the wanted key is the next range, and once it holds few keys each of them is
// ranked against the others.  One round for ordinary scores, three at most; a
// row of equal scores needs none (64 x 4092: rounds alone 8.0 us, so 6.7).  The columns
// that are always kept stay out of the range.  Keys stay in shared memory (in
// registers every pass over them has to be unrolled, and code that runs once
// costs its way into the instruction cache), or are read again
// each time in rows of more than 49152 columns.  Warps own consecutive columns.
constexpr int kHeldKeys = 49152;
constexpr int kPlainKeys = 8192;     // 32 KB, beside 9 KB of counts: no opt-in to more shared memory
constexpr int kBins = 2048;
constexpr int kRanked = 128;         // keys of a bin that are ranked, at most: four a lane

template <int THREADS>
__global__ void __launch_bounds__(THREADS) select_blocks_kernel(const SelectArgs a) {
    constexpr int kW = THREADS / 32;
    constexpr int kBinsPerThread = kBins / THREADS;
    __shared__ int hist[kBins];
    __shared__ uint32_t lo_s[kW], hi_s[kW];
    __shared__ int n_s[kW], m_s[kW];
    __shared__ __align__(16) uint32_t list[kRanked];
    __shared__ uint32_t found_bin, found_key;
    __shared__ int a_s[kW], e_s[kW];
    __shared__ int found_above, found_count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const float* row = a.scores + (long long)blockIdx.x * a.ld;
    int* out = a.blocks + (long long)blockIdx.x * a.n_keep;
    const int cols = (int)a.cols, K = a.n_keep;
    const int items = (cols + THREADS - 1) / THREADS;      // per thread, 32 apart
    const long long c0 = (long long)warp * items * 32 + lane;
    const bool held = cols <= kHeldKeys;
    extern __shared__ uint32_t keys[];                     // [items * THREADS] if held; a thread reads its own
    auto load = [&](long long c) { return c < cols ? score_key(row[c], c < a.keep_first) : 0u; };
    if (held) {
        for (int j0 = 0; j0 < items; j0 += 8) {            // eight loads in flight
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (int)c0 + 32 * (j0 + j);
                x[j] = j0 + j < items && c < cols ? row[c] : -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (int)c0 + 32 * (j0 + j);
                if (j0 + j < items) keys[c] = score_key(x[j], c < a.keep_first);
            }
        }
    }
    auto each = [&](auto f) {                              // f(key, column) of this thread's columns, in order
        if (held) {
#pragma unroll 4
            for (int j = 0; j < items; ++j) f(keys[(int)c0 + 32 * j], (int)c0 + 32 * j);
        } else {
            for (int j = 0; j < items; ++j) f(load(c0 + 32LL * j), (int)(c0 + 32LL * j));
        }
    };
    // the wanted key is among those in [lo, hi]: `above` keys are greater than hi
    uint32_t lo = 1u, hi = 0xfffffffeu;
    int above = 0, valid = 0;
    uint32_t t = 1u;
    if (tid < kRanked) list[tid] = 0u;
    for (int round = 0;; ++round) {
        // the span of the keys left, and (first round) how many there are
        uint32_t least = 0xffffffffu, most = 0u;
        int n = 0, always = 0;
        each([&](uint32_t k, int) {
            if (k >= lo && k <= hi) {
                least = min(least, k);
                most = max(most, k);
                ++n;
            }
            always += k == 0xffffffffu;
        });
        least = __reduce_min_sync(kFull, least);
        most = __reduce_max_sync(kFull, most);
        n = __reduce_add_sync(kFull, n);
        if (round == 0) always = __reduce_add_sync(kFull, always);
        if (lane == 0) {
            lo_s[warp] = least;
            hi_s[warp] = most;
            n_s[warp] = n;
            if (round == 0) m_s[warp] = always;
        }
        for (int j = tid; j < kBins; j += THREADS) hist[j] = 0;
        __syncthreads();
        least = __reduce_min_sync(kFull, lane < kW ? lo_s[lane] : 0xffffffffu);
        most = __reduce_max_sync(kFull, lane < kW ? hi_s[lane] : 0u);
        n = __reduce_add_sync(kFull, lane < kW ? n_s[lane] : 0);
        if (round == 0) {
            above = __reduce_add_sync(kFull, lane < kW ? m_s[lane] : 0);
            valid = n + above;
            if (valid <= K) break;                         // everything that may be taken
            if (above >= K) {                              // the always kept ones fill the places
                t = 0xffffffffu;
                break;
            }
        }
        lo = least;
        hi = most;
        t = lo;
        if (above + n == K || lo == hi) break;             // all of them, or equal ones
        const int shift = max(0, 21 - __clz(hi - lo));     // (hi - lo) >> shift < 2048
        each([&](uint32_t k, int) {
            if (k >= lo && k <= hi) atomicAdd(&hist[(k - lo) >> shift], 1);
        });
        __syncthreads();
        // the bin of the (K - above)-th greatest: counts of the bins above each thread's
        int mine[kBinsPerThread], sum = 0;
#pragma unroll
        for (int j = 0; j < kBinsPerThread; ++j) {
            mine[j] = hist[kBins - 1 - (tid * kBinsPerThread + j)];
            sum += mine[j];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) m_s[warp] = incl;
        __syncthreads();
        int over = above + incl - sum + __reduce_add_sync(kFull, lane < warp ? m_s[lane] : 0);
#pragma unroll
        for (int j = 0; j < kBinsPerThread; ++j) {
            if (over < K && over + mine[j] >= K) {
                found_bin = kBins - 1 - (tid * kBinsPerThread + j);
                found_above = over;
                found_count = mine[j];
            }
            over += mine[j];
        }
        __syncthreads();
        above = found_above;
        hi = lo + min(hi - lo, ((found_bin + 1u) << shift) - 1u);   // (by offsets: lo plus a bin's end may pass 2^32)
        lo = lo + (found_bin << shift);
        t = lo;
        if (shift == 0 || above + found_count == K) break;
        if (found_count <= kRanked) {
            // the bin's keys into a list; each is ranked by a warp, whose lanes hold
            // four of the list's keys each (places past the last hold 0, less than any)
            // (their places from the warps' counts: atomics on one address take turns)
            const int c = found_count;
            int mine_n = 0;
            each([&](uint32_t k, int) { mine_n += k >= lo && k <= hi; });
            mine_n = __reduce_add_sync(kFull, mine_n);
            if (lane == 0) a_s[warp] = mine_n;
            __syncthreads();
            int at = __reduce_add_sync(kFull, lane < warp ? a_s[lane] : 0);
            if (mine_n)
                each([&](uint32_t k, int) {
                    const bool in = k >= lo && k <= hi;
                    const uint32_t m = __ballot_sync(kFull, in);
                    if (in) list[at + __popc(m & ((1u << lane) - 1u))] = k;
                    at += __popc(m);
                });
            __syncthreads();
            const uint4 x = *reinterpret_cast<const uint4*>(&list[4 * lane]);
            for (int j = warp; j < c; j += kW) {
                const uint32_t mine = list[j];
                // greater keys in the low half, equal ones in the high half (both at most 128)
                const int n = (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine) +
                              (((x.x == mine) + (x.y == mine) + (x.z == mine) + (x.w == mine)) << 16);
                const int r = __reduce_add_sync(kFull, n);
                const int greater = above + (r & 0xffff);
                if (lane == 0 && greater < K && greater + (r >> 16) >= K) found_key = mine;
            }
            __syncthreads();
            t = found_key;
            break;
        }
    }
    const int take = min(valid, K);
    int na = 0, ne = 0;
    each([&](uint32_t k, int) {
        na += k > t;
        ne += k == t;
    });
    na = __reduce_add_sync(kFull, na);
    ne = __reduce_add_sync(kFull, ne);
    if (lane == 0) {
        a_s[warp] = na;
        e_s[warp] = ne;
    }
    __syncthreads();
    const int wa = lane < kW ? a_s[lane] : 0, we = lane < kW ? e_s[lane] : 0;
    const int ties = take - __reduce_add_sync(kFull, wa);
    int before_a = __reduce_add_sync(kFull, lane < warp ? wa : 0);
    int before_e = __reduce_add_sync(kFull, lane < warp ? we : 0);
    const uint32_t below = (1u << lane) - 1u;
    each([&](uint32_t k, int c) {
        const uint32_t ma = __ballot_sync(kFull, k > t), me = __ballot_sync(kFull, k == t);
        if ((ma | me) == 0u) return;
        const int ra = before_a + __popc(ma & below), re = before_e + __popc(me & below);
        if (k > t || (k == t && re < ties)) out[ra + min(re, ties)] = c;
        before_a += __popc(ma);
        before_e += __popc(me);
    });
    for (int j = take + tid; j < K; j += THREADS) out[j] = -1;
}

// A token appended to each of n sequences: residual rows of keys and values.
struct AppendArgs {
    uint8_t* buf;
    const __half* k;
    const __half* v;
    long long k_resid_off, v_resid_off;
    int Hkv, R, D;
    AppendRow rows[kMaxCallSeqs];
};
__global__ void __launch_bounds__(128) append_rows_kernel(const __grid_constant__ AppendArgs a) {
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const AppendRow r = a.rows[blockIdx.x];
    const int cpr = a.D / 8;        // 16-byte chunks per row
    const uint4* sk = reinterpret_cast<const uint4*>(a.k) + (long long)blockIdx.x * a.Hkv * cpr;
    const uint4* sv = reinterpret_cast<const uint4*>(a.v) + (long long)blockIdx.x * a.Hkv * cpr;
    uint4* dk = reinterpret_cast<uint4*>(a.buf + a.k_resid_off);
    uint4* dv = reinterpret_cast<uint4*>(a.buf + a.v_resid_off);
    for (int x = threadIdx.x; x < a.Hkv * cpr; x += blockDim.x) {
        const long long at = (((long long)r.seq * a.Hkv + x / cpr) * a.R + r.row) * cpr + x % cpr;
        dk[at] = sk[x];
        dv[at] = sv[x];
    }
}

}  // namespace

cudaError_t launch_block_scores(const BlockRows& r, const __half* q, float scale, float* scores, long long ld,
                                cudaStream_t st) {
    const Geometry& g = *r.g;
    const ScoreArgs base{r.buf, q, scores, ld, g.part_bytes, g.slot_bytes, (g.G / 16) * g.tile_bytes,
                         g.Hq, g.Hkv, r.n_blocks, 1, scale, (float)((1 << g.bits) - 1)};
    if (!r.table) {
        ScoreArgs a = base;
        return launch_scores<false>(a, r, st);
    }
    PagedScoreArgs a;
    static_cast<ScoreArgs&>(a) = base;
    a.table = r.table;
    a.max_blocks = (int)g.NB;
    a.n_pages = (int)r.n_pages;
    for (int i = 0; i < r.n; ++i) a.seqs[i] = r.seqs[i];
    return launch_scores<true>(a, r, st);
}

static cudaError_t launch_select(void (*kernel)(const SelectArgs), int threads, const SelectArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)a.rows);
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = a.cols <= kHeldKeys ? (size_t)((a.cols + threads - 1) / threads) * threads * 4 : 0;
    if (lc.dynamicSmemBytes > 4 * kPlainKeys) {
        // (only the kernel of the longest rows; once per device)
        static std::mutex mu;
        static bool set_up[64];
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (!set_up[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kHeldKeys);
            if (e != cudaSuccess) return e;
            set_up[dev] = true;
        }
    }
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, a);
}

cudaError_t launch_select_blocks(const float* scores, long long rows, long long cols, long long ld, int n_keep,
                                 int keep_first, int* blocks, cudaStream_t st) {
    const SelectArgs a{scores, rows, cols, ld, n_keep, keep_first, blocks};
    const dim3 by_warp((unsigned)((rows + kWarpRows - 1) / kWarpRows));
    if (cols <= 256) return launch_dependent(select_blocks_warp_kernel<8>, by_warp, 32 * kWarpRows, st, a);
    // many rows of up to 1024 columns too: the CTAs of two rows an SM take turns
    // (400 columns, CTA and warp a row: 256 rows 4.5, 5.0 us, 512 rows 8.1, 5.0, 2048
    // rows 16.7, 7.9; 800 columns: 5.6, 8.0 and 10.6, 8.1 and 21.9, 19.1)
    if (rows >= 384 && cols <= 512)
        return launch_dependent(select_blocks_warp_kernel<16>, by_warp, 32 * kWarpRows, st, a);
    if (rows >= 384 && cols <= 1024)
        return launch_dependent(select_blocks_warp_kernel<32>, by_warp, 32 * kWarpRows, st, a);
    // 4 to 8 keys a thread: fewer threads take longer over their keys, more wait
    // longer at the barriers and leave room for fewer rows (64 and 512 rows of 4092:
    // 256 threads 8.6, 19.0 us; 512: 6.7, 15.3; 1024: 6.5, 21.1; 64 x 8000: 512 9.6, 1024 8.1)
    if (cols <= 1024) return launch_select(select_blocks_kernel<256>, 256, a, st);
    if (cols <= 4096) return launch_select(select_blocks_kernel<512>, 512, a, st);
    return launch_select(select_blocks_kernel<1024>, 1024, a, st);
}

cudaError_t launch_decode_blocks(const BlockRows& r, const __half* q, const int* list, int n_list, float scale_log2,
                                 __half* out, cudaStream_t st) {
    const Geometry& g = *r.g;
    const int nq = g.Hq / g.Hkv;
    const long long rows = (long long)r.n * g.Hkv;
    // weights: bytes of a quantized pair / 32; a residual tile, whose loads overlap
    // other warps' work, as 24 of its 64 D bytes (one head of 64 channels, 4 blocks
    // and 2 tiles: 3.15 us, weighted as 40 D bytes 3.7; the 7B layer and 131k
    // tokens do not change between 16 and 64 D)
    const blocks_detail::Args base{r.buf, q, out, list, g.NB, g.part_bytes, g.slot_bytes, g.tile_bytes,
                                   g.k_resid_off, g.v_resid_off, g.R, g.Hq, g.Hkv, n_list, r.n_blocks, r.n_resid,
                                   g.D * g.bits / 4 + 8 * g.D / g.G, 3 * g.D / 4, scale_log2, r.stall_bytes};
    auto units = [&](int nblk, int nres) {
        return (long long)(n_list < nblk ? n_list : nblk) * (g.G / 32) + (nres + 15) / 16;
    };
    if (!r.table) {
        const long long u = units(r.n_blocks, r.n_resid);
        return (g.D == 128 ? launch_decode_blocks_d128 : launch_decode_blocks_d64)(base, g.bits, nq, g.G, rows, u,
                                                                                  r.num_sms, st);
    }
    blocks_detail::PagedArgs a;
    static_cast<blocks_detail::Args&>(a) = base;
    a.table = r.table;
    a.max_blocks = (int)g.NB;
    a.n_pages = (int)r.n_pages;
    long long u = 0;
    for (int i = 0; i < r.n; ++i) {
        a.seqs[i] = r.seqs[i];
        const long long ui = units(r.seqs[i].n_blocks, r.seqs[i].n_resid);
        if (ui > u) u = ui;
    }
    return (g.D == 128 ? launch_decode_blocks_d128p : launch_decode_blocks_d64p)(a, g.bits, nq, g.G, rows, u,
                                                                                r.num_sms, st);
}

cudaError_t launch_append_rows(const Geometry& g, uint8_t* buf, const AppendRow* rows, int n, const __half* new_k,
                               const __half* new_v, cudaStream_t st) {
    AppendArgs a;
    a.buf = buf;
    a.k = new_k;
    a.v = new_v;
    a.k_resid_off = g.k_resid_off;
    a.v_resid_off = g.v_resid_off;
    a.Hkv = g.Hkv;
    a.R = g.R;
    a.D = g.D;
    for (int i = 0; i < n; ++i) a.rows[i] = rows[i];
    return launch_dependent(append_rows_kernel, dim3((unsigned)n), 128, st, a);
}

kivi_status block_scores_call(const BlockRows& r, const void* q, float softmax_scale, float* scores, long long ld,
                              kivi_stream_t stream) {
    const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)r.g->D);
    return launched(launch_block_scores(r, static_cast<const __half*>(q), scale, scores, ld,
                                        reinterpret_cast<cudaStream_t>(stream)), "block scores launch");
}

kivi_status decode_blocks_call(const BlockRows& r, const void* q, const int* blocks, int n_list, void* out,
                               float softmax_scale, kivi_stream_t stream) {
    const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)r.g->D);
    return launched(launch_decode_blocks(r, static_cast<const __half*>(q), blocks, n_list,
                                         scale * 1.4426950408889634f, static_cast<__half*>(out),
                                         reinterpret_cast<cudaStream_t>(stream)), "block decode launch");
}

kivi_status check_scores_args(const void* q, float softmax_scale, const float* scores, long long ld) {
    if (!q || (!scores && ld != 0)) return failf(KIVI_ERR_INVALID_ARG, "null q or scores");
    if (!aligned(q, 16)) return failf(KIVI_ERR_INVALID_ARG, "q must be 16-byte aligned");
    if (!aligned(scores, 4)) return failf(KIVI_ERR_INVALID_ARG, "scores must be 4-byte aligned");
    if (ld < 0) return failf(KIVI_ERR_INVALID_ARG, "negative column count");
    if (!(softmax_scale == softmax_scale) || isinf(softmax_scale))
        return failf(KIVI_ERR_INVALID_ARG, "softmax_scale must be finite");
    return KIVI_OK;
}

kivi_status check_decode_blocks_args(const void* q, const int* blocks, int n_list, const void* out, float softmax_scale) {
    if (!q || !out) return failf(KIVI_ERR_INVALID_ARG, "null q or out");
    if (n_list < 0) return failf(KIVI_ERR_INVALID_ARG, "negative list length");
    if (n_list > (1 << 28)) return failf(KIVI_ERR_UNSUPPORTED, "lists hold at most 2^28 entries");
    if (n_list > 0 && !blocks) return failf(KIVI_ERR_INVALID_ARG, "null block list");
    if (!aligned(q, 16) || !aligned(out, 16)) return failf(KIVI_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
    if (!aligned(blocks, 4)) return failf(KIVI_ERR_INVALID_ARG, "blocks must be 4-byte aligned");
    if (!(softmax_scale == softmax_scale) || isinf(softmax_scale))
        return failf(KIVI_ERR_INVALID_ARG, "softmax_scale must be finite");
    return KIVI_OK;
}

}  // namespace kivi

extern "C" {

kivi_status kivi_block_scores(kivi_cache_t c, const void* q, float softmax_scale, float* scores, long long ld,
                              kivi_stream_t stream) {
    using namespace kivi;
    if (!c) return failf(KIVI_ERR_INVALID_ARG, "null handle");
    const kivi_status sa = check_scores_args(q, softmax_scale, scores, ld);
    if (sa != KIVI_OK) return sa;
    CacheView v = cache_view(c);
    BlockRows r{v.g, v.buf, v.g->B, (int)(v.n_quant / v.g->G), (int)v.n_resid, nullptr, 0, nullptr, 0, 0};
    if (ld < r.n_blocks)
        return failf(KIVI_ERR_CAPACITY, "scores have %lld columns, the cache holds %d blocks", ld, r.n_blocks);
    if (ld == 0) return report_error(KIVI_OK, "");
    const kivi_status sd = cache_device(c);
    if (sd != KIVI_OK) return sd;
    r.num_sms = cache_view(c).num_sms;
    return block_scores_call(r, q, softmax_scale, scores, ld, stream);
}

kivi_status kivi_select_blocks(const float* scores, long long rows, long long cols, long long ld, int n_keep,
                               int keep_first, int* blocks, kivi_stream_t stream) {
    using namespace kivi;
    if (rows < 0 || cols < 0 || n_keep < 0 || keep_first < 0) return failf(KIVI_ERR_INVALID_ARG, "negative size");
    if (ld < cols) return failf(KIVI_ERR_INVALID_ARG, "ld must be at least cols");
    if (keep_first > n_keep) return failf(KIVI_ERR_INVALID_ARG, "keep_first must be at most n_keep");
    if (rows > 0x7fffffffLL || cols > (1LL << 30) || n_keep > (1 << 30))
        return failf(KIVI_ERR_UNSUPPORTED, "rows must be < 2^31, cols and n_keep <= 2^30");
    if (rows == 0 || n_keep == 0) return report_error(KIVI_OK, "");
    if (!blocks || (!scores && cols > 0)) return failf(KIVI_ERR_INVALID_ARG, "null scores or blocks");
    if (!aligned(scores, 4) || !aligned(blocks, 4)) return failf(KIVI_ERR_INVALID_ARG, "scores and blocks must be 4-byte aligned");
    return launched(launch_select_blocks(scores, rows, cols, ld, n_keep, keep_first, blocks,
                                         reinterpret_cast<cudaStream_t>(stream)), "block selection launch");
}

kivi_status kivi_decode_blocks(kivi_cache_t c, const void* q, const int* blocks, int n_list, void* out,
                               float softmax_scale, kivi_stream_t stream) {
    using namespace kivi;
    if (!c) return failf(KIVI_ERR_INVALID_ARG, "null handle");
    const kivi_status sa = check_decode_blocks_args(q, blocks, n_list, out, softmax_scale);
    if (sa != KIVI_OK) return sa;
    CacheView v = cache_view(c);
    if (v.value_queue) return failf(KIVI_ERR_UNSUPPORTED, "the value queue has no decode over chosen blocks");
    if (v.n_quant + v.n_resid == 0) return failf(KIVI_ERR_STATE, "decode on an empty cache");
    const kivi_status sd = cache_device(c);
    if (sd != KIVI_OK) return sd;
    v = cache_view(c);
    const BlockRows r{v.g, v.buf, v.g->B, (int)(v.n_quant / v.g->G), (int)v.n_resid, nullptr, 0, nullptr, v.num_sms,
                      take_stall(c)};
    return decode_blocks_call(r, q, blocks, n_list, out, softmax_scale, stream);
}

}  // extern "C"
