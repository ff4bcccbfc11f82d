// Codes of the cache's tiles as fp16 values, and their way into shared memory as
// 8x8 matrices: a lane's code pairs are matrix fragments (kivi.h, "Code tile").
#pragma once

#include "kivi_chunk.cuh"
#include "kivi_decode_mma.cuh"

namespace kivi {
namespace chunk_detail {

using namespace mma_detail;

__device__ __forceinline__ void stmatrix4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
// Byte offset of 16-byte group `chunk` (of 8 elements along the contracted index) of row `row` in an
// operand of ROWS rows: 64 elements side by side per block of 128-byte rows, groups swizzled.
template <int ROWS>
__device__ __forceinline__ uint32_t operand_at(int row, int chunk) {
    return (uint32_t)((chunk >> 3) * (ROWS * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// The code pair at bit POS (0..7) of each half of w, as exact fp16 values.
template <int BITS, int POS>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    constexpr uint32_t mask = ((1u << BITS) - 1u) << POS;
    const uint32_t x = (w & (mask | (mask << 16))) | 0x64006400u;        // 1024 + code 2^POS
    if constexpr (POS == 0) return hsub2(x, 0x64006400u);
    // times 2^-POS, less 1024 * 2^-POS
    constexpr uint32_t m = (uint32_t)(15 - POS) << 10, c = 0x8000u | ((uint32_t)(25 - POS) << 10);
    return hfma2(x, m | (m << 16), c | (c << 16));
}
// the pair of channel group C and order H from a lane's words
template <int BITS, int C, int H, int W>
__device__ __forceinline__ uint32_t code_of(const uint32_t (&w)[W]) {
    constexpr int P = 8 / BITS;
    return code_pair<BITS, BITS * (C % P)>(H ? w[C / P] >> 8 : w[C / P]);
}

}  // namespace chunk_detail
}  // namespace kivi
