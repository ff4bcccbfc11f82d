// The chunk attention kernel for head_dim 128.
#include "kivi_chunk_attn.cuh"

namespace kivi {
cudaError_t launch_chunk_attn_d128(const ChunkArgs& a, int bits, cudaStream_t st) {
    return chunk_detail::launch_chunk_bits<128>(a, bits, st);
}
}  // namespace kivi
