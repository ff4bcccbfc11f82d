// Paged cache: the residual rows after a chunk's append, branches that share
// pages, and tokens read back as fp16 (include/kivi.h, "Chunks of new tokens").
#include "kivi_dequant.cuh"

namespace kivi {
namespace {

using namespace chunk_detail;

struct Resid {
    __half *k, *v;      // [max_seqs][Hkv][R][D]
    int R;
};

// ---- residual rows after a chunk ----
struct TailArgs {
    Resid resid;
    const __half *k, *v;
    long long k_stride[2], v_stride[2];
    ChunkTail tails[kMaxCallSeqs];
};

// CTA (h, i): kv head h of tail i, keys and values.  Rows move towards the front, within
// the rows that are read: all of a step's loads are ahead of its stores.
template <int D>
__global__ void __launch_bounds__(256) store_tail_kernel(const __grid_constant__ TailArgs a) {
    constexpr int LPR = D / 8, RPS = 128 / LPR, AHEAD = 4;    // lanes a row, rows 128 threads take at once
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const ChunkTail& t = a.tails[blockIdx.y];
    const int h = blockIdx.x, values = threadIdx.x >> 7, tid = threadIdx.x & 127;
    const int lr = tid % LPR, sub = tid / LPR;
    __half* resid = (values ? a.resid.v : a.resid.k) + ((long long)t.seq * gridDim.x + h) * a.resid.R * D;
    const long long* stride = values ? a.v_stride : a.k_stride;
    const __half* fresh = (values ? a.v : a.k) + t.tok0 * stride[0] + h * stride[1];
    const int j0 = t.shift ? 0 : min(t.n_resid, t.keep);       // rows that stay where they are
    for (int base = j0; base < t.keep; base += RPS * AHEAD) {
        uint4 x[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int j = base + u * RPS + sub, f = t.shift + j;
            if (j < t.keep) {
                const __half* src = f < t.n_resid ? resid + (long long)f * D : fresh + (f - t.n_resid) * stride[0];
                x[u] = *reinterpret_cast<const uint4*>(src + 8 * lr);
            }
        }
        if (t.shift) __syncthreads();
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int j = base + u * RPS + sub;
            if (j < t.keep) *reinterpret_cast<uint4*>(resid + (long long)j * D + 8 * lr) = x[u];
        }
    }
}

// ---- branches ----
struct ForkArgs {
    Resid resid;
    int* table;
    int max_blocks;
    ForkJob jobs[kMaxCallSeqs];
};

// The block-table entries of branch i, by the CTAs (x, i).  It gives no signal to start its dependent early: the next
// kernel waits until these stores are there.
__global__ void __launch_bounds__(256) fork_table_kernel(const __grid_constant__ ForkArgs a) {
    griddepcontrol_wait();
    const ForkJob& j = a.jobs[blockIdx.y];
    const int* ts = a.table + (long long)j.from * a.max_blocks;
    int* td = a.table + (long long)j.to * a.max_blocks;
    for (int x = blockIdx.x * 256 + threadIdx.x; x < j.n_blocks; x += 256 * gridDim.x) td[x] = ts[x];
}

// CTA (h, i): kv head h of branch i: its residual rows.  A launch of its own, behind the table's: a decode call reads
// the table ahead of its wait for the kernel before it, so that kernel may write residual rows and no table entry.
// (One kernel for both that sends no signal is not enough: a dependent then starts when the CTAs have exited, and
// only its wait makes their stores visible.)
template <int D>
__global__ void __launch_bounds__(256) fork_rows_kernel(const __grid_constant__ ForkArgs a) {
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const ForkJob& j = a.jobs[blockIdx.y];
    const long long rows = (long long)gridDim.x * a.resid.R * D, head = (long long)blockIdx.x * a.resid.R * D;
    const int n = j.n_resid * (D / 8);
    const uint4* sk = reinterpret_cast<const uint4*>(a.resid.k + j.from * rows + head);
    const uint4* sv = reinterpret_cast<const uint4*>(a.resid.v + j.from * rows + head);
    uint4* dk = reinterpret_cast<uint4*>(a.resid.k + j.to * rows + head);
    uint4* dv = reinterpret_cast<uint4*>(a.resid.v + j.to * rows + head);
#pragma unroll 4
    for (int x = threadIdx.x; x < n; x += 256) {
        const uint4 p = sk[x], q = sv[x];
        dk[x] = p;
        dv[x] = q;
    }
}

// ---- reading back ----
struct ReadArgs {
    const uint8_t* buf;
    const int* table;
    const __half *rk, *rv;
    long long page_bytes, part_bytes;
    int Hkv, R, G, max_blocks, n_pages;
    long long first, count;
    __half *k, *v;              // [n][Hkv][count][D]
    RowSeq seqs[kMaxCallSeqs];
};

constexpr int kReadWarps = 4;

// Matrices (group C, tokens 0-7 and 8-15) and (C + 1, ...) of a code tile into rows [16][D] at dst (swizzled as an operand of
// 16 rows): keys as they lie, values (channels x tokens) transposed.  ent: the key steps, or the values' entry tile.
template <int D, int BITS, bool VALUES, int C, int W>
__device__ __forceinline__ void read_groups(const uint32_t (&w)[W], uint32_t ent, int G, uint2 s, uint2 z, uint32_t dst, int lane) {
    if constexpr (C < D / 8) {
        const uint32_t at = dst + operand_at<16>(lane & 15, C + (lane >> 4));
        if constexpr (VALUES) {
            if constexpr (8 * C % 32 == 0) {
                if ((8 * C & (G - 1)) == 0) {
                    s = lds64(ent + 32 * (8 * C / G) + 8 * (lane & 3));
                    z = lds64(ent + 32 * (8 * C / G) + 32 * (D / G) + 8 * (lane & 3));
                }
            }
            stmatrix4_trans(at, hfma2(code_of<BITS, C, 0>(w), s.x, z.x), hfma2(code_of<BITS, C, 1>(w), s.y, z.y),
                            hfma2(code_of<BITS, C + 1, 0>(w), s.x, z.x), hfma2(code_of<BITS, C + 1, 1>(w), s.y, z.y));
        } else {
            const uint32_t e = ent + 16 * C + 4 * (lane & 3);
            const uint32_t s0 = lds32(e), z0 = lds32(e + 2 * D), s1 = lds32(e + 16), z1 = lds32(e + 2 * D + 16);
            stmatrix4(at, hfma2(code_of<BITS, C, 0>(w), s0, z0), hfma2(code_of<BITS, C, 1>(w), s0, z0),
                      hfma2(code_of<BITS, C + 1, 0>(w), s1, z1), hfma2(code_of<BITS, C + 1, 1>(w), s1, z1));
        }
        read_groups<D, BITS, VALUES, C + 2>(w, ent, G, s, z, dst, lane);
    }
}

// A warp per 16 tokens of a (sequence, kv head): values dequantized as matrices in shared memory, then stored
// by rows.  Bound by the stores: 4 D bytes a token written for D bits / 4 + 8 D / G read.
template <int D, int BITS>
__global__ void __launch_bounds__(32 * kReadWarps) read_tokens_kernel(const __grid_constant__ ReadArgs a) {
    constexpr int W = D * BITS / 64, TILE = 2 * D * BITS, LPR = D / 8, RPI = 32 / LPR;
    __shared__ __align__(128) uint8_t rows[kReadWarps][16 * D * 2];
    __shared__ __align__(16) uint8_t entries[kReadWarps][4 * D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const RowSeq q = a.seqs[blockIdx.z];
    const long long tile = a.first / 16 + (long long)blockIdx.x * kReadWarps + warp;
    const long long tok = 16 * tile, end = a.first + a.count;
    if (tok >= end) return;
    const int h = blockIdx.y;
    const long long n_quant = (long long)q.n_blocks * a.G;
    const long long out0 = (((long long)blockIdx.z * a.Hkv + h) * a.count - a.first) * D;     // of token 0
    const int lr = lane % LPR, sub = lane / LPR;
    if (tok >= n_quant) {
        const long long row0 = ((long long)q.seq * a.Hkv + h) * a.R - n_quant;
#pragma unroll
        for (int j = 0; j < 16 / RPI; ++j) {
            const long long t = tok + j * RPI + sub;
            if (t >= a.first && t < end) {
                *reinterpret_cast<uint4*>(a.k + out0 + t * D + 8 * lr) =
                    *reinterpret_cast<const uint4*>(a.rk + (row0 + t) * D + 8 * lr);
                *reinterpret_cast<uint4*>(a.v + out0 + t * D + 8 * lr) =
                    *reinterpret_cast<const uint4*>(a.rv + (row0 + t) * D + 8 * lr);
            }
        }
        return;
    }
    int page = a.table[(long long)q.seq * a.max_blocks + tok / a.G];
    const bool bad = (unsigned)page >= (unsigned)a.n_pages;      // an entry outside the pool: its tokens are NaN
    if (bad) page = 0;
    const int in = (int)(tok % a.G) / 16, tiles = a.G / 16, ve = 64 * (D / a.G);
    const uint8_t* kp = a.buf + page * a.page_bytes + (long long)h * 2 * a.part_bytes;
    const uint8_t* vp = kp + a.part_bytes;
    const uint32_t dst = smem_u32(rows[warp]), ent = smem_u32(entries[warp]);
    auto words = [&](const uint8_t* p, uint32_t (&w)[W]) {
        if constexpr (W == 2) {
            const uint2 v = ldg_stream2(p + 8 * lane);
            w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
            for (int j = 0; j < W / 4; ++j) {
                const uint4 v = ldg_stream(p + 4 * W * lane + 16 * j);
                w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
            }
        }
    };
    uint32_t kw[W], vw[W];
    words(kp + in * TILE, kw);
    words(vp + in * TILE, vw);
    const int n_ve = ve / 16;                                    // 16-byte groups of value entries
    uint4 ke{}, vv{};
    if (lane < 4 * D / 16) ke = ldg_stream(kp + tiles * TILE + 16 * lane);
    if (lane < n_ve) vv = ldg_stream(vp + tiles * TILE + in * ve + 16 * lane);
    auto put = [&](__half* out) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16 / RPI; ++j) {
            const int r = j * RPI + sub;
            uint4 x = lds128(dst + operand_at<16>(r, lr));
            if (bad) x = uint4{0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu};
            if (tok + r >= a.first && tok + r < end) *reinterpret_cast<uint4*>(out + out0 + (tok + r) * D + 8 * lr) = x;
        }
        __syncwarp();
    };
    if (lane < 4 * D / 16) *reinterpret_cast<uint4*>(entries[warp] + 16 * lane) = ke;
    __syncwarp();
    read_groups<D, BITS, false, 0>(kw, ent, a.G, uint2{}, uint2{}, dst, lane);
    put(a.k);
    if (lane < n_ve) *reinterpret_cast<uint4*>(entries[warp] + 16 * lane) = vv;
    __syncwarp();
    read_groups<D, BITS, true, 0>(vw, ent, a.G, uint2{}, uint2{}, dst, lane);
    put(a.v);
}

Resid resid_of(const Geometry& g, uint8_t* buf) {
    return Resid{reinterpret_cast<__half*>(buf + g.k_resid_off), reinterpret_cast<__half*>(buf + g.v_resid_off), g.R};
}

}  // namespace

cudaError_t launch_store_tail(const PagedGeometry& pg, uint8_t* buf, const __half* k, const long long* k_stride,
                              const __half* v, const long long* v_stride, const ChunkTail* tails, int n,
                              cudaStream_t st) {
    const Geometry& g = pg.g;
    TailArgs a;
    a.resid = resid_of(g, buf);
    a.k = k;
    a.v = v;
    for (int j = 0; j < 2; ++j) {
        a.k_stride[j] = k_stride[j];
        a.v_stride[j] = v_stride[j];
    }
    for (int i = 0; i < n; ++i) a.tails[i] = tails[i];
    const dim3 grid((unsigned)g.Hkv, (unsigned)n);
    return g.D == 128 ? launch_dependent(store_tail_kernel<128>, grid, 256, st, a)
                      : launch_dependent(store_tail_kernel<64>, grid, 256, st, a);
}

cudaError_t launch_fork(const PagedGeometry& pg, uint8_t* buf, const ForkJob* jobs, int n, cudaStream_t st, int* launches) {
    const Geometry& g = pg.g;
    ForkArgs a;
    a.resid = resid_of(g, buf);
    a.table = reinterpret_cast<int*>(buf + pg.table_off);
    a.max_blocks = (int)g.NB;
    int most = 0;
    for (int i = 0; i < n; ++i) {
        a.jobs[i] = jobs[i];
        most = jobs[i].n_blocks > most ? jobs[i].n_blocks : most;
    }
    *launches = 0;
    if (most) {
        const int ctas = (most + 255) / 256;
        const cudaError_t e = launch_dependent(fork_table_kernel, dim3((unsigned)(ctas < 16 ? ctas : 16), (unsigned)n), 256, st, a);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    const dim3 grid((unsigned)g.Hkv, (unsigned)n);
    const cudaError_t e = g.D == 128 ? launch_dependent(fork_rows_kernel<128>, grid, 256, st, a)
                                     : launch_dependent(fork_rows_kernel<64>, grid, 256, st, a);
    if (e == cudaSuccess) ++*launches;
    return e;
}

cudaError_t launch_read(const PagedGeometry& pg, const uint8_t* buf, const RowSeq* seqs, int n, long long first,
                        long long count, __half* k, __half* v, cudaStream_t st) {
    const Geometry& g = pg.g;
    ReadArgs a;
    a.buf = buf;
    a.table = reinterpret_cast<const int*>(buf + pg.table_off);
    a.rk = reinterpret_cast<const __half*>(buf + g.k_resid_off);
    a.rv = reinterpret_cast<const __half*>(buf + g.v_resid_off);
    a.page_bytes = pg.page_bytes;
    a.part_bytes = g.part_bytes;
    a.Hkv = g.Hkv;
    a.R = g.R;
    a.G = g.G;
    a.max_blocks = (int)g.NB;
    a.n_pages = (int)pg.n_pages;
    a.first = first;
    a.count = count;
    a.k = k;
    a.v = v;
    for (int i = 0; i < n; ++i) a.seqs[i] = seqs[i];
    const long long tiles = (first + count + 15) / 16 - first / 16;
    const dim3 grid((unsigned)((tiles + kReadWarps - 1) / kReadWarps), (unsigned)g.Hkv, (unsigned)n);
#define KIVI_R(DD, BB) \
    if (g.D == DD && g.bits == BB) return launch_dependent(read_tokens_kernel<DD, BB>, grid, 32 * kReadWarps, st, a);
    KIVI_R(128, 2) KIVI_R(128, 4) KIVI_R(128, 8) KIVI_R(64, 2) KIVI_R(64, 4) KIVI_R(64, 8)
#undef KIVI_R
    return cudaErrorInvalidValue;
}

}  // namespace kivi
