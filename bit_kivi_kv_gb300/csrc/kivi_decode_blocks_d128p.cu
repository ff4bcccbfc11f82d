// Instantiations of the block-list decode kernel: head_dim 128, paged cache.
#include "kivi_decode_blocks_launch.cuh"

namespace kivi {

cudaError_t launch_decode_blocks_d128p(const blocks_detail::PagedArgs& a, int bits, int nq, int G, long long rows,
                                    long long units, int num_sms, cudaStream_t st) {
    return blocks_launch::dispatch<128, true>(a, bits, nq, G, rows, units, num_sms, st);
}

}  // namespace kivi
