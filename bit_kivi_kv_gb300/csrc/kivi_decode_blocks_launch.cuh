// Launch of one decode_blocks_kernel instance and the dispatch over the
// instances of one head_dim; included by the per-head_dim instantiation files.
#pragma once

#include <mutex>

#include "kivi_decode_blocks.cuh"

namespace kivi {
namespace blocks_launch {

constexpr int kMaxDevices = 64;

// Per-device set-up of one instance: the opt-in to its dynamic shared memory
// and its resident CTAs per SM.
struct InstanceSetup {
    std::mutex mu;
    int per_sm[kMaxDevices] = {};        // 0: not set up on that device yet
};

// CTAs that share a row: the most (a power of two, at most 8) whose whole grid
// is resident at once and whose warps each get a unit of work.
inline int cluster_ctas(long long rows, long long units, long long resident) {
    int c = 1;
    while (c < blocks_detail::kMaxCluster && rows * c * 2 <= resident && 2LL * c * mma_detail::kWarps <= units) c *= 2;
    return c;
}

template <int D, int BB, int NN, int GG, bool PAGED>
cudaError_t launch_one(const typename blocks_detail::ArgsOf<PAGED>::type& a, long long rows, long long units,
                       int num_sms, cudaStream_t st) {
    using namespace blocks_detail;
    using C = Cfg<D, BB, NN, GG>;
    static InstanceSetup setup;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    int per_sm;
    {
        std::lock_guard<std::mutex> lock(setup.mu);
        per_sm = setup.per_sm[dev];
        if (per_sm == 0) {
            e = cudaFuncSetAttribute(decode_blocks_kernel<D, BB, NN, GG, PAGED>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, C::DYN_SMEM);
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                    &per_sm, decode_blocks_kernel<D, BB, NN, GG, PAGED>, kThreads, C::DYN_SMEM);
            if (e != cudaSuccess) return e;
            if (per_sm < 1) per_sm = 1;
            setup.per_sm[dev] = per_sm;
        }
    }
    const int c = cluster_ctas(rows, units, (long long)num_sms * per_sm);
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)(rows * c));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = C::DYN_SMEM;
    lc.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)c;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = c > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, decode_blocks_kernel<D, BB, NN, GG, PAGED>, a);
}

// every (bits, q heads per kv head, G) instance of head_dim D
template <int D, bool PAGED>
cudaError_t dispatch(const typename blocks_detail::ArgsOf<PAGED>::type& a, int bits, int nq, int G, long long rows,
                     long long units, int num_sms, cudaStream_t st) {
#define KIVI_BLK(BB, NN, GG) \
    if (bits == BB && nq == NN && G == GG) return launch_one<D, BB, NN, GG, PAGED>(a, rows, units, num_sms, st);
#define KIVI_BLK_G(BB, NN) KIVI_BLK(BB, NN, 32) KIVI_BLK(BB, NN, 64) if constexpr (D >= 128) { KIVI_BLK(BB, NN, 128) }
    KIVI_BLK_G(2, 1) KIVI_BLK_G(2, 2) KIVI_BLK_G(2, 4)
    KIVI_BLK_G(4, 1) KIVI_BLK_G(4, 2) KIVI_BLK_G(4, 4)
    KIVI_BLK_G(8, 1) KIVI_BLK_G(8, 2) KIVI_BLK_G(8, 4)
#undef KIVI_BLK_G
#undef KIVI_BLK
    return cudaErrorInvalidValue;
}

}  // namespace blocks_launch
}  // namespace kivi
