// Internal declarations of the decode over chosen blocks, the append without a
// decode and the norm and rotation of queries and keys.
#pragma once

#include "kivi_common.cuh"

namespace kivi {

// ---- decode over chosen blocks (kivi.h, "Decode over chosen blocks") ----

// One sequence of a paged call over blocks.
struct RowSeq {
    int seq;        // sequence slot: residual rows and block-table row
    int n_blocks;   // quantized blocks (Lq / G)
    int n_resid;    // residual rows
};

// Where the blocks of a call's rows are.  Row i * Hkv + h is kv head h of the
// call's query row i.  Dense cache: table null, every row has n_blocks blocks
// and n_resid residual rows.  Paged cache: the rows of seqs[i], their blocks
// in pages through the block table.
struct BlockRows {
    const Geometry* g;
    const uint8_t* buf;
    int n;                      // query rows of the call
    int n_blocks, n_resid;      // dense
    const int* table;           // paged
    long long n_pages;
    const RowSeq* seqs;         // paged: n entries (host memory)
    int num_sms;
    int stall_bytes;            // failure-detection test hook (dense)
};

// scores [n * Hkv][ld]: the bound of each block, -inf from a row's last block on.
cudaError_t launch_block_scores(const BlockRows& r, const __half* q, float scale, float* scores, long long ld,
                                cudaStream_t st);

// list [n * Hkv][n_list] of block numbers -> out [n][Hq][D].
cudaError_t launch_decode_blocks(const BlockRows& r, const __half* q, const int* list, int n_list, float scale_log2,
                                 __half* out, cudaStream_t st);

// The n_keep best of each row's scores (kivi_select_blocks).
cudaError_t launch_select_blocks(const float* scores, long long rows, long long cols, long long ld, int n_keep,
                                 int keep_first, int* blocks, cudaStream_t st);

// Argument checks of kivi_block_scores / kivi_decode_blocks that the dense and the
// paged calls share, and their launches after every check (kivi_blocks.cu).
kivi_status check_scores_args(const void* q, float softmax_scale, const float* scores, long long ld);
kivi_status check_decode_blocks_args(const void* q, const int* blocks, int n_list, const void* out,
                                     float softmax_scale);
kivi_status block_scores_call(const BlockRows& r, const void* q, float softmax_scale, float* scores, long long ld,
                              kivi_stream_t stream);
kivi_status decode_blocks_call(const BlockRows& r, const void* q, const int* blocks, int n_list, void* out,
                               float softmax_scale, kivi_stream_t stream);

// Paged append without decode: token i of new_k / new_v [n][Hkv][D] becomes
// residual row rows[i] of sequence slot seqs[i].
struct AppendRow {
    int seq, row;
};
cudaError_t launch_append_rows(const Geometry& g, uint8_t* buf, const AppendRow* rows, int n, const __half* new_k,
                               const __half* new_v, cudaStream_t st);

// ---- norm and rotation of queries and keys (kivi.h, kivi_qk_norm_rope) ----

// Where the outputs go: slot (batch row, head) j of a tensor at base +
// j * slot_stride, token t of the slot at + t * D elements.
struct QkvDest {
    __half *q, *k, *v;
    long long q_slot, k_slot, v_slot;
};
kivi_status check_qkv(const kivi_qkv* a);
cudaError_t launch_qk_norm_rope(const kivi_qkv& a, const QkvDest& d, cudaStream_t st);

// A launch as a programmatic dependent of the preceding kernel.
template <typename K, typename... A>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = dim3((unsigned)threads);
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, args...);
}

// What the calls outside kivi_api.cu see of a dense cache.
struct CacheView {
    const Geometry* g;
    uint8_t* buf;
    long long n_quant, n_resid;
    int value_queue, num_sms;
};
CacheView cache_view(const struct ::kivi_cache* c);
// The cache's fault for its next decode call (kivi_cache_set_fault), taken: the
// bytes that a copy stage waits for in vain, or 0.
int take_stall(struct ::kivi_cache* c);

}  // namespace kivi
