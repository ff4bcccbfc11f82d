// The chunk attention kernel for head_dim 64.
#include "kivi_chunk_attn.cuh"

namespace kivi {
cudaError_t launch_chunk_attn_d64(const ChunkArgs& a, int bits, cudaStream_t st) {
    return chunk_detail::launch_chunk_bits<64>(a, bits, st);
}
}  // namespace kivi
