// pa_masked.h -- interface between the host side (pa_masked_host.cpp) and the kernels of the
// operators around reads of the paged cache that follow a mask of their own: the commit of an
// accepted path of a tree (pa_tree_aux.cu), and decoding over selected blocks -- bounds of the
// blocks' keys, the selection, the attention (pa_blocks.cu).  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace pa {

constexpr int32_t kDevBadSlot = 1, kDevBadBlock = 2, kDevBadLen = 4;   // PA_DEVERR_*

// Mask words of a tree that pa_tree_accept walks (its parents sit in shared memory).
constexpr int32_t kMaxTreeWords = 64;

struct AcceptParams {
    int32_t *accepted, *num_accepted;       // [S][max_accepted], [S]
    int64_t* next_tokens;                   // [S]
    int32_t* new_lens;                      // [S]
    const int64_t *draft, *target;          // [num_tokens]
    const uint32_t* tree_mask;              // [num_tokens][mask_words]
    const int32_t *query_starts, *context_lens;
    int32_t num_seqs, num_tokens, mask_words, max_accepted;
    int32_t* status;
};
cudaError_t launch_tree_accept(const AcceptParams& p, cudaStream_t stream);

constexpr int32_t kMoveTokenLayers = 64;    // layers per launch (kernel parameter space)
struct MoveTokensParams {
    void* key[kMoveTokenLayers];
    void* value[kMoveTokenLayers];
    const int32_t* block_tables;
    const int32_t *new_lens, *accepted, *num_accepted;
    int32_t max_blocks_per_seq, num_seqs, max_accepted, num_layers;
    int32_t num_blocks, num_kv_heads, block_size;
    int32_t row_vecs;                       // 16-byte pieces of a row
    int32_t report;                         // this launch reports bad metadata
    int32_t* status;
};
cudaError_t launch_move_tokens(const MoveTokensParams& p, cudaStream_t stream);

struct BoundsParams {
    int8_t* bounds;                         // [num_blocks][Hkv][2][D]
    float* steps;                           // [num_blocks][Hkv]
    const void* key_cache;
    const int32_t *block_tables, *context_lens, *query_starts;   // query_starts may be null
    int32_t max_blocks_per_seq, num_seqs, num_kv_heads, head_size, block_size, num_blocks;
    int32_t max_new_tokens;
    int32_t slots;                          // blocks that a sequence's new tokens may touch
    int32_t* status;
};
enum class BoundsType { kF16, kBf16, kFp8 };
cudaError_t launch_key_bounds(const BoundsParams& p, BoundsType type, cudaStream_t stream);

struct SelectParams {
    int32_t* selected;                      // [S][q_len][Hkv][num_selected]
    const void* query;                      // [S][q_len][Hq][D]
    const int8_t* bounds;
    const float* steps;
    const int32_t *block_tables, *context_lens;
    int32_t max_blocks_per_seq, num_seqs, q_len, num_q_heads, num_kv_heads, group, head_size;
    int32_t block_size, num_blocks, max_context_len;
    int32_t num_selected, num_first, num_last;
    int32_t max_blocks;                     // blocks of the longest context
    int32_t sms;
    uint32_t* keys;                         // [S * q_len][Hkv][max_blocks] ordered scores
    uint32_t* weights;                      // [S * q_len][Hkv][D / 16][16] pairs of 16-bit weights
    int32_t* status;
};
cudaError_t launch_select_blocks(const SelectParams& p, bool bf16, cudaStream_t stream);
// Blocks that a CTA of the scores takes at a time (their table entries sit in shared memory).
constexpr int32_t kMaxScoreChunk = 512;
// Longest row of blocks that the selection's bitmaps in shared memory hold.
constexpr int32_t kMaxSelectBlocks = 1 << 17;

// The attention over selected blocks.  Every (query token, kv head) is a row: a sequence of one kv
// head, over pools seen as num_blocks * num_kv_heads blocks of one kv head.
struct SparseParams {
    const int32_t *selected, *block_tables, *context_lens;
    int32_t max_blocks_per_seq, num_seqs, q_len, num_kv_heads, block_size, num_blocks, num_selected;
    int32_t cluster;                        // CTAs per row
    int32_t short_ring;                     // less of them on its way per CTA, more CTAs to an SM
    int32_t* status;
};
// List entries of a row, at most (a piece of a list is read up to its own place for every 512 of them).
constexpr int32_t kSparseMaxSelected = 1 << 16;
// List entries that a CTA translates at a time.
constexpr int32_t kSparseEntries = 512;
// A CTA of a cluster takes at least this many tiles of its row.
constexpr int32_t kSparseTiles = 4;
constexpr int32_t kSparseMaxCluster = 16;

// `ctas` CTAs, or, for 0, the CTAs per SM in *per_sm and no launch.
struct DecodeParams;
cudaError_t launch_sparse_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                               const SparseParams& sp, int32_t head_size, int32_t ctas,
                               cudaStream_t stream, int32_t* per_sm);
cudaError_t launch_sparse_f16(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                              const SparseParams& sp, int32_t head_size, int32_t ctas,
                              cudaStream_t stream, int32_t* per_sm);
cudaError_t launch_sparse_fp8(bool q_bf16, const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                              const SparseParams& sp, int32_t ctas, cudaStream_t stream, int32_t* per_sm);

}  // namespace pa
