// Chunk attention: the merge of items that several CTAs worked on.
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

// Block (c, y): where CTA c + 1's first span continues the item that CTA c began, 8 of that item's rows, a
// warp each: o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p over its parts, p in order.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) chunk_merge_kernel(const __grid_constant__ ChunkArgs a) {
    constexpr int S = chunk_partial_stride(D);
    griddepcontrol_wait();
    griddepcontrol_launch_dependents();
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31;
    ChunkWalk walk;
    walk.start(&a.plan, a.seqs, a.n_seqs, chunk_begin(a.weight, a.n_ctas, c), chunk_begin(a.weight, a.n_ctas, c + 1LL));
    if (!walk.next()) return;
    const ChunkSpan s = walk.s;
    const ChunkSeq& q = a.seqs[s.seq];
    if (s.first == 0 || chunk_begin(a.weight, a.n_ctas, c - 1LL) > walk.item0) return;
    const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), nq = a.plan.nq;
    if (r >= (s.it.t1 - s.it.t0) * nq) return;
    // the parts: CTA c - 1's last span, then the first ones of CTAs c .. c + n - 2
    const long long last = walk.item0 + (long long)(s.it.hi - s.it.lo - 1) * s.it.weight();
    int n = 2;
    while (c - 1 + n < a.n_ctas && chunk_begin(a.weight, a.n_ctas, c - 1LL + n) <= last) ++n;
    auto part = [&](int p) {
        return a.ws + (((long long)(c - 1 + p) * 2 + (p == 0)) * kRows + r) * S;
    };
    float w[kPartRegs], top = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < kPartRegs; ++j) {
        const int p = 32 * j + lane;
        w[j] = -INFINITY;
        if (32 * j < n && p < n) w[j] = part(p)[D];
        top = w[j] != w[j] ? w[j] : fmaxf(top, w[j]);
    }
    const bool bad = __any_sync(kFull, top != top);
    top = warp_max(top);
#pragma unroll
    for (int j = 0; j < kPartRegs; ++j) {
        const int p = 32 * j + lane;
        w[j] = w[j] == -INFINITY ? 0.f : exp2f(w[j] - top);
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
    const float inv = bad ? NAN : 1.f / l;
    const int tok = s.it.t0 + r / nq, head = s.head * nq + r % nq;
    __half* out = a.out + (long long)(q.tok0 + tok) * a.out_stride[0] + head * a.out_stride[1];
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
        *reinterpret_cast<uint32_t*>(out + 64 * d + 2 * lane) = pack_f16x2(o[d].x * inv, o[d].y * inv);
}

}  // namespace

cudaError_t launch_chunk_merge(const ChunkArgs& a, int D, cudaStream_t st) {
    int most = 0;
    for (int i = 0; i < a.n_seqs; ++i) most = a.seqs[i].n > most ? a.seqs[i].n : most;
    const long long rows = (long long)most * a.plan.nq < kRows ? (long long)most * a.plan.nq : kRows;
    const dim3 grid((unsigned)(a.n_ctas - 1), (unsigned)((rows + kJoinWarps - 1) / kJoinWarps));
    return D == 128 ? launch_dependent(chunk_merge_kernel<128>, grid, 32 * kJoinWarps, st, a)
                    : launch_dependent(chunk_merge_kernel<64>, grid, 32 * kJoinWarps, st, a);
}

}  // namespace kivi
