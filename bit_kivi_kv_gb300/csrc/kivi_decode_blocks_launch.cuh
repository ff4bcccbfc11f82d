// Launch of one decode_blocks_kernel instance and the dispatch over the
// instances of one head_dim; included by the per-head_dim instantiation files.
#pragma once

#include <mutex>

#include "kivi_decode_blocks.cuh"

namespace kivi {
namespace blocks_launch {

constexpr int kMaxDevices = 64;

// Per-device set-up of one instance: the opt-in to its dynamic shared memory
// and what an SM holds of its warps and CTAs.
struct SmRoom {
    int reg_warps = 0;                   // warps by registers; 0: not set up on that device yet
    int sm_bytes = 0, cta_bytes = 0;     // shared memory of an SM; of a CTA, most
    int fixed = 0, per_warp = 0;         // shared memory of a CTA: fixed, and per warp
    // warps of each of n CTAs on one SM
    int warps(long long n) const {
        if (n > reg_warps) return 0;
        const long long by_smem = (min2(sm_bytes / n, cta_bytes + 1024) - 1024 - fixed) / per_warp;
        const long long w = min2(reg_warps / n, by_smem);
        return w < 0 ? 0 : (int)w;
    }
    static long long min2(long long x, long long y) { return x < y ? x : y; }
};
struct InstanceSetup {
    std::mutex mu;
    SmRoom room[kMaxDevices];
};

// A row's CTAs (a power of two, at most 8: a cluster) and their warps, of the
// shapes whose whole grid is resident at once.  Each is charged with the units
// (tile pairs and residual tiles) of a warp, the mean of the busiest one's and
// of an even split, and a cluster with what its merge costs besides: 0.7 unit,
// 0.9 with four query heads, whose merge is larger.  (Of one version of the kernel: 256 rows of 32 blocks: 1 x 8
// warps 11.6 us, 2 x 4 12.9; 192 rows of 128 blocks: 1 x 8 29.5, 2 x 5 25.9; 32
// rows of 16 blocks at head_dim 64: 1 x 16 4.9, 4 x 6 3.9; four query heads, 64
// rows of 2 blocks of 128: 1 x 12 6.2, 2 x 8 7.2.)  Of clusters that cost the
// same, the one with more warps, then the one with smaller CTAs, which spread
// over more SMs (64 rows of 128 blocks: 2 x 16 warps 12.5 us, 4 x 8 11.7).
//
// Small CTAs are placed unevenly while the kernel before still runs, if an SM
// holds more of them than its share: where that leaves a row of 64 KB and more
// two warps, and wherever it leaves one, CTAs of up to four warps in several
// waves (768 rows of 128 blocks: 2 warps 103.4 us, 4 in waves 84.1; with 4 bits
// 127.2 and 97.6, 8 bits at 512 rows 74.8 and 63.7; but 1024 rows of 8 blocks
// 20.1 and 21.8; with three warps, 640 rows, 71.6 and 77.3; no room for more, 8
// bits at 640 rows, 76.0 and 85.8).  A row with nothing to read still has a warp,
// which writes its outputs.
struct Shape { int ctas, warps; };
inline Shape row_shape(long long rows, long long units, int num_sms, const SmRoom& room, int nq,
                       long long row_bytes) {
    Shape best{1, 0};
    long long least = 0;                 // in 1/20 of a unit
    auto share = [&](int c) { return (rows * c + num_sms - 1) / num_sms; };   // CTAs of an SM
    for (int c = 1; c <= blocks_detail::kMaxCluster; c *= 2) {
        long long w = room.warps(share(c));
        if (w * c > units) w = (units + c - 1) / c;
        if (w < 1) continue;
        const long long n = w * c, most = (long long)best.ctas * best.warps;
        const long long t = 10 * ((units + n - 1) / n) + 10 * units / n + (c == 1 ? 0 : nq == 4 ? 18 : 14);
        if (most == 0 || t < least || (t == least && best.ctas > 1 && (n > most || (n == most && w >= 4)))) {
            least = t;
            best = Shape{c, (int)w};
        }
    }
    const bool uneven = row_bytes >= 65536 && room.warps(share(1) + 1) >= best.warps;
    if (best.ctas == 1 && best.warps < (uneven ? 3 : 2)) {
        const long long w = SmRoom::min2(SmRoom::min2(units, 4), room.warps(1));
        best = Shape{1, w < 1 ? 1 : (int)w};
    }
    return best;
}

template <int D, int BB, int NN, int GG, bool PAGED>
cudaError_t launch_one(const typename blocks_detail::ArgsOf<PAGED>::type& a, long long rows, long long units,
                       int num_sms, cudaStream_t st) {
    using namespace blocks_detail;
    static InstanceSetup setup;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    using S = Smem<D, BB, NN, GG>;
    auto kernel = decode_blocks_kernel<D, BB, NN, GG, PAGED>;
    SmRoom room;
    {
        std::lock_guard<std::mutex> lock(setup.mu);
        SmRoom& r = setup.room[dev];
        if (r.reg_warps == 0) {
            SmRoom n;
            cudaFuncAttributes fa;
            e = cudaFuncGetAttributes(&fa, kernel);
            if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n.cta_bytes, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
            if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n.sm_bytes, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
            n.fixed = (int)fa.sharedSizeBytes;
            n.per_warp = S::WARP;
            n.reg_warps = kCtaWarps<D, NN>;
            const int most = n.warps(1);
            if (e == cudaSuccess && most < 1) e = cudaErrorInvalidConfiguration;
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most * S::WARP);
            if (e != cudaSuccess) return e;
            r = n;
        }
        room = r;
    }
    // (bytes as if all units were tile pairs)
    const Shape sh = row_shape(rows, units, num_sms, room, NN, units * 32 * a.wq);
    const int c = sh.ctas;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)(rows * c));
    lc.blockDim = dim3(32 * sh.warps);
    lc.dynamicSmemBytes = sh.warps * S::WARP;
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
    return cudaLaunchKernelEx(&lc, kernel, a);
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
