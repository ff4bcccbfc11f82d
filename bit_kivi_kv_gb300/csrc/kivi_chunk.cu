// Chunk attention: the merge of items that several CTAs worked on; the rows of sequences with few of them.
#include "kivi_chunk.cuh"
#include "kivi_decode_mma.cuh"

namespace kivi {
namespace {

using namespace mma_detail;

constexpr int kJoinWarps = 8;
constexpr int kPartRegs = kMaxChunkCtas / 32;

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// Row r of an item that CTAs c - 1 .. worked on, by a warp: o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p over its
// parts, p in order.
template <int D>
__device__ __forceinline__ void merge_row(const ChunkArgs& a, const MergeJob& job, int c, int r, int lane) {
    constexpr int S = chunk_partial_stride(D);
    const int n = job.parts, nq = a.plan.nq;
    auto part = [&](int p) { return a.ws + (((long long)(c - 1 + p) * 2 + (p == 0)) * kRows + r) * S; };
    float w[kPartRegs], top = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < kPartRegs; ++j) {
        const int p = 32 * j + lane;
        w[j] = -INFINITY;
        if (32 * j < n && p < n) w[j] = part(p)[D];
        top = fmaxf(top, w[j]);
    }
    top = warp_max(top);
#pragma unroll
    for (int j = 0; j < kPartRegs; ++j) {
        const int p = 32 * j + lane;
        w[j] = w[j] == -INFINITY ? 0.f : exp2f(w[j] - top);    // (a part that is marked: NaN, and so is the row)
        if (32 * j < n && p < n) l += w[j] * part(p)[D + 1];
    }
    l = warp_sum(l);
    float2 o[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) o[j] = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kPartRegs; ++j) {
        if (32 * j >= n) break;
#pragma unroll 4
        for (int p = 32 * j; p < min(n, 32 * j + 32); ++p) {
            const float f = __shfl_sync(kFull, w[j], p - 32 * j);
            const float* src = part(p);
#pragma unroll
            for (int d = 0; d < D / 64; ++d) {
                const float2 x = *reinterpret_cast<const float2*>(src + 64 * d + 2 * lane);
                o[d].x = fmaf(f, x.x, o[d].x);
                o[d].y = fmaf(f, x.y, o[d].y);
            }
        }
    }
    const float inv = 1.f / l;
    __half* out = a.out + (long long)(job.tok + r / nq) * a.out_stride[0] + (job.head * nq + r % nq) * a.out_stride[1];
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
        *reinterpret_cast<uint32_t*>(out + 64 * d + 2 * lane) = pack_out(o[d].x * inv, o[d].y * inv);
}

// The same for rows r and r + step of an item of kFewParts parts at most, the commonest: everything is loaded at once,
// whatever its weight (three chunks of up to 777 tokens of 16 heads, a call of 108 us: 100).
constexpr int kFewParts = 4;
template <int D>
__device__ __forceinline__ void merge_rows(const ChunkArgs& a, const MergeJob& job, int c, int r0, int step, int lane) {
    constexpr int S = chunk_partial_stride(D);
    const int n = job.parts, nq = a.plan.nq;
    float2 ml[2][kFewParts], x[2][kFewParts][D / 64];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int p = 0; p < kFewParts; ++p) {
            ml[k][p] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int d = 0; d < D / 64; ++d) x[k][p][d] = make_float2(0.f, 0.f);
            const int r = r0 + k * step;
            if (p < n && r < job.rows) {
                const float* src = a.ws + (((long long)(c - 1 + p) * 2 + (p == 0)) * kRows + r) * S;
                ml[k][p] = *reinterpret_cast<const float2*>(src + D);
#pragma unroll
                for (int d = 0; d < D / 64; ++d) x[k][p][d] = *reinterpret_cast<const float2*>(src + 64 * d + 2 * lane);
            }
        }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = r0 + k * step;
        float top = -INFINITY, l = 0.f;
#pragma unroll
        for (int p = 0; p < kFewParts; ++p) top = fmaxf(top, ml[k][p].x);
        float2 o[D / 64];
#pragma unroll
        for (int d = 0; d < D / 64; ++d) o[d] = make_float2(0.f, 0.f);
#pragma unroll
        for (int p = 0; p < kFewParts; ++p) {
            const float w = ml[k][p].x == -INFINITY ? 0.f : exp2f(ml[k][p].x - top);   // (a part that is marked: NaN)
            l = fmaf(w, ml[k][p].y, l);
#pragma unroll
            for (int d = 0; d < D / 64; ++d) {
                o[d].x = fmaf(w, x[k][p][d].x, o[d].x);
                o[d].y = fmaf(w, x[k][p][d].y, o[d].y);
            }
        }
        if (r >= job.rows) return;
        const float inv = 1.f / l;
        __half* out = a.out + (long long)(job.tok + r / nq) * a.out_stride[0] + (job.head * nq + r % nq) * a.out_stride[1];
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
            *reinterpret_cast<uint32_t*>(out + 64 * d + 2 * lane) = pack_out(o[d].x * inv, o[d].y * inv);
    }
}

// Block (x, y): the item that CTA x + 1's first span continues, if CTA x began it; every gridDim.y-th eight of its
// rows.  (The main kernel leaves the jobs: found anew in each block, by division and search, they took 33 us of a call
// of 75.)
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) chunk_merge_kernel(const __grid_constant__ ChunkArgs a) {
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31;
    const MergeJob job = a.jobs[c];
    if (!job.parts) return;
    const int step = gridDim.y * kJoinWarps;
    int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
    if (job.parts <= kFewParts)
        for (; r < job.rows; r += 2 * step) merge_rows<D>(a, job, c, r, step, lane);
    else
        for (; r < job.rows; r += step) merge_row<D>(a, job, c, r, lane);
}

// Rows of the groups as the query heads of a single-token call; rows that a group lacks are zeros.
template <int D>
__global__ void __launch_bounds__(256) gather_rows_kernel(const __grid_constant__ GroupArgs a) {
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
    const int c = (int)(x % (D / 8)), j = (int)(x / (D / 8) % a.nv), h = (int)(x / (D / 8) / a.nv % a.Hkv);
    const long long g = x / (D / 8) / a.nv / a.Hkv;
    if (g >= a.n) return;
    uint4 v{0, 0, 0, 0};
    const ChunkGroup& p = a.groups[g];
    if (j < p.rows) {
        const int r = p.row0 + j;
        const __half* src = a.q + (long long)(p.tok0 + r / a.nq) * a.q_stride[0] + (h * a.nq + r % a.nq) * a.q_stride[1];
        v = *reinterpret_cast<const uint4*>(src + 8 * c);
    }
    reinterpret_cast<uint4*>(a.gathered)[x] = v;
}

template <int C>
__device__ __forceinline__ void load_row(const float* src, float (&x)[C]) {
    if constexpr (C == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        x[0] = v.x; x[1] = v.y;
    }
}

// A warp per row: the partial results over the cached tokens, and the row's new tokens up to its own.
template <int D>
__global__ void __launch_bounds__(128) group_merge_kernel(const __grid_constant__ GroupArgs a) {
    constexpr int S = partial_stride(D), C = D / 32;           // channels a lane holds
    constexpr int kAhead = 8;
    static_assert(S % 4 == 0, "16-byte loads");
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long at = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int j = (int)(at % a.nv), h = (int)(at / a.nv % a.Hkv);
    const long long g = at / a.nv / a.Hkv;
    if (g >= a.n) return;
    const ChunkGroup& p = a.groups[g];
    if (j >= p.rows) return;
    const PagedSeq& sq = a.seqs[g];
    const long long P = sq.P, PR = (sq.n_resid + 31) / 32;
    const long long w0 = sq.start + h * (a.wm.S0 + slot_weight(a.wm, P, 0, PR));
    const long long last = w0 + unit_start_p(a.wm, P, 0, P + PR - 1);
    const int n = (int)(map_owner(a.wm, last) - map_owner(a.wm, w0 + a.wm.S0) + 1);
    const float* base = a.ws + at * kPartialSlots * S;
    const int r = p.row0 + j, tok = r / a.nq, head = h * a.nq + r % a.nq;
    auto widen = [&](const __half* src, float (&x)[C]) {
        if constexpr (C == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(src + 4 * lane);
            const float2 lo = unpack_f16x2(v.x), hi = unpack_f16x2(v.y);
            x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
        } else {
            const float2 v = unpack_f16x2(*reinterpret_cast<const uint32_t*>(src + 2 * lane));
            x[0] = v.x; x[1] = v.y;
        }
    };
    float q[C];
    widen(a.q + (long long)(p.tok0 + tok) * a.q_stride[0] + head * a.q_stride[1], q);
#pragma unroll
    for (int c = 0; c < C; ++c) q[c] *= a.scale_log2;
    // weights of the partials, three a lane
    float w[3], lw[3], top = -INFINITY, l = 0.f;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int i = lane + 32 * k;
        w[k] = -INFINITY;
        lw[k] = 0.f;
        if (i < n) {
            const float4 head = *reinterpret_cast<const float4*>(base + i * S);
            w[k] = head.x;
            lw[k] = head.y;
            bad |= head.z != 0.f;
        }
        top = fmaxf(top, w[k]);
    }
    top = warp_max(top);
#pragma unroll
    for (int k = 0; k < 3; ++k) {                              // (an empty partial: -1)
        w[k] = w[k] == -INFINITY ? -1.f : exp2f(w[k] - top);
        if (!(w[k] < 0.f)) l += w[k] * lw[k];
    }
    l = warp_sum(l);
    float o[C];
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
    for (int i0 = 0; i0 < n; i0 += kAhead) {                   // (loads that wait for no weight)
        float x[kAhead][C];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i0 + u < n) load_row<C>(base + (i0 + u) * S + 4 + C * lane, x[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            if (i >= n) break;
            const float f = __shfl_sync(kFull, i < 32 ? w[0] : i < 64 ? w[1] : w[2], i & 31);
            if (f < 0.f) continue;                             // (an empty partial's values are not written)
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] = fmaf(f, x[u][c], o[c]);
        }
    }
    const __half* kp = a.k + p.tok0 * a.k_stride[0] + h * a.k_stride[1];
    const __half* vp = a.v + p.tok0 * a.v_stride[0] + h * a.v_stride[1];
    for (int t0 = 0; t0 <= tok; t0 += 4) {                     // four new tokens' loads at a time
        float x[4][C], v[4][C];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long t = min(t0 + u, tok);
            widen(kp + t * a.k_stride[0], x[u]);
            widen(vp + t * a.v_stride[0], v[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (t0 + u > tok) break;
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) s = fmaf(q[c], x[u][c], s);
            s = warp_sum(s);
            const float m = fmaxf(top, s), f = exp2f(top - m), e = exp2f(s - m);
            top = m;
            l = l * f + e;
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] = o[c] * f + e * v[u][c];
        }
    }
    // (a token's value that is not finite leaves its channel so, whatever its weight: the row is NaN, as in the wide kernel)
#pragma unroll
    for (int c = 0; c < C; ++c) bad |= !(fabsf(o[c]) < INFINITY);
    const float inv = __any_sync(kFull, bad) ? NAN : 1.f / l;
    __half* out = a.out + (long long)(p.tok0 + tok) * a.out_stride[0] + head * a.out_stride[1] + C * lane;
#pragma unroll
    for (int c = 0; c < C; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack_f16x2(o[c] * inv, o[c + 1] * inv);
}

}  // namespace

cudaError_t launch_chunk_merge(const ChunkArgs& a, int D, cudaStream_t st) {
    int most = 0;
    for (int i = 0; i < a.n_seqs; ++i) most = a.seqs[i].n > most ? a.seqs[i].n : most;
    const long long rows = (long long)most * a.plan.nq < kRows ? (long long)most * a.plan.nq : kRows;
    // (blocks for one wave: eight of 256 threads an SM)
    const long long blocks = (rows + kJoinWarps - 1) / kJoinWarps;
    const dim3 grid((unsigned)(a.n_ctas - 1), (unsigned)(blocks < 8 ? blocks : 8));
    return D == 128 ? launch_dependent(chunk_merge_kernel<128>, grid, 32 * kJoinWarps, st, a)
                    : launch_dependent(chunk_merge_kernel<64>, grid, 32 * kJoinWarps, st, a);
}

cudaError_t launch_gather_rows(const GroupArgs& a, int D, cudaStream_t st) {
    const long long n = (long long)a.n * a.Hkv * a.nv * (D / 8);
    const dim3 grid((unsigned)((n + 255) / 256));
    return D == 128 ? launch_dependent(gather_rows_kernel<128>, grid, 256, st, a)
                    : launch_dependent(gather_rows_kernel<64>, grid, 256, st, a);
}

cudaError_t launch_group_merge(const GroupArgs& a, int D, cudaStream_t st) {
    const dim3 grid((unsigned)(((long long)a.n * a.Hkv * a.nv + 3) / 4));
    return D == 128 ? launch_dependent(group_merge_kernel<128>, grid, 128, st, a)
                    : launch_dependent(group_merge_kernel<64>, grid, 128, st, a);
}

}  // namespace kivi
