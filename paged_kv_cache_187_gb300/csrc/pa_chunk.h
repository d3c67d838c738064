// pa_chunk.h -- interface between the host side of the chunk operators (pa_chunk_host.cpp)
// and their kernels: attention of a ragged chunk of new tokens over the paged cache
// (pa_prefill*.cu*), rotary positions fused with the cache write, and block moves
// (pa_chunk_aux.cu).  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace pa {

// Attention tiles: 128 query rows per stream, two streams per work item, 128 tokens.
constexpr int32_t kPfRows = 128;
constexpr int32_t kPfTok = 128;
// The grid never has more CTAs than this (one per SM); the workspace is sized for it.
constexpr int32_t kPfMaxGrid = 160;
// What an item costs beside its tiles (Q, the first scores, the rows' output), in tiles.
constexpr int32_t kPfItemCost = 2;
// What cutting costs a CTA (partial results written, read and joined), in tiles.
constexpr int32_t kPfCutCost = 6;
// Shortest share of the work, in tiles, worth a CTA of its own when contexts are cut.
constexpr int32_t kPfMinShare = 6;

// Calls small enough for one unit per CTA, with contexts too short to be cut, are not
// planned: each CTA finds its own unit from up to 32 sequences' metadata, one per lane.
// (One chunk of 17 tokens over 317: 13.3 us a call with the plan kernel, 9.3 us without.)
constexpr int32_t kPfDirectTokens = 1024;

// Head of the prefill workspace, written by the plan kernel.  A row tile is a run of up to
// 2 * tpt new tokens of a sequence; a unit is a row tile with one kv head, of as many
// 128-token tiles as its last row sees; its cost is its tiles + kPfItemCost.
//   cut 0: whole units, claimed one by one, longest row tiles first (`order`).
//   cut 1: the units' costs laid end to end (row tile by row tile, kv heads innermost) are
//          cut into `shares` equal stretches, one per CTA, so that all finish together.
//          Share b starts at floor(b * cost / shares); a unit belongs to the share in which
//          its cost for beginning ends, and goes on into the next ones.
struct PfHeader {
    uint32_t counter;       // units claimed past the first gridDim.x (cut 0)
    uint32_t total_units;   // row tiles * num_kv_heads
    uint32_t cut;
    uint32_t shares;
    int64_t cost;           // all units'
    uint32_t lines;         // entries of `before`: row tiles, or pairs of them
    uint32_t pairs;         // cut 1, trees: the lines are pairs of row tiles (see prefill_plan_kernel)
    uint32_t pad[56];
};

struct PrefillParams {
    void* out;
    const void* value_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_starts;
    int32_t max_blocks_per_seq;
    int32_t num_tokens, num_seqs, num_q_heads, num_kv_heads, group;
    int32_t num_blocks, block_size, head_size, max_context_len;
    int32_t tpt;               // new tokens per stream: 128 / group
    float scale_log2;          // softmax scale (x k_scale) * log2(e), never 0
    float out_scale;           // v_scale for fp8 caches, else 1
    int32_t grid;              // CTAs of the attention launch
    int32_t max_row_tiles;     // what the workspace has room for
    int32_t direct;            // no plan: CTA b takes unit b (see kPfDirectTokens)
    PfHeader* hdr;
    int4* seqs;                // [num_seqs] (q_start, q_len, len, first row tile)
    int32_t* seq_of;           // [row tiles] the sequence
    int32_t* order;            // [row tiles] longest first; for pairs, the pair's first row tile
    int64_t* before;           // [row tiles + 1] cost of the row tiles (pairs) before, one kv head
    int32_t* arrive;           // [CTAs][2 streams] finished partitions of the unit that a
                               // share leaves unfinished
    float2* part_ml;           // [CTAs][2][2 streams][128] (reference, weight sum): a share
                               // holds the end of a unit begun before it, and the beginning
                               // of one that goes on
    float* part_acc;           // [CTAs][2][2 streams][head_size][128]
    int32_t* status;
    // trees of new tokens (null: causal): bit i of word w of a token's row is set if the token
    // sees new token 32 w + i of its sequence
    const uint32_t* tree_mask; // [num_tokens][mask_words]
    int32_t mask_words;
};

struct PfWorkspace {
    size_t hdr, seqs, seq_of, order, before, arrive, part_ml, part_acc, total;
    int32_t max_row_tiles;
};
PfWorkspace prefill_workspace(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_size, int32_t max_context_len);

cudaError_t launch_prefill_plan(const PrefillParams& p, cudaStream_t stream);
cudaError_t launch_prefill_bf16(const CUtensorMap& qmap, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, const PrefillParams& p, cudaStream_t stream);
cudaError_t launch_prefill_f16(const CUtensorMap& qmap, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, const PrefillParams& p, cudaStream_t stream);
cudaError_t launch_prefill_fp8(bool q_bf16, const CUtensorMap& qmap, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, const PrefillParams& p, cudaStream_t stream);
// The same for trees of new tokens (tree_mask not null).
cudaError_t launch_tree_bf16(const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, const PrefillParams& p, cudaStream_t stream);
cudaError_t launch_tree_f16(const CUtensorMap& qmap, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, const PrefillParams& p, cudaStream_t stream);
cudaError_t launch_tree_fp8(bool q_bf16, const CUtensorMap& qmap, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, const PrefillParams& p, cudaStream_t stream);

constexpr int32_t kMaxRopePairs = 128;
struct RopeParams {
    void* query_out;
    const void *query, *key, *value;
    int64_t q_stride, k_stride, v_stride;     // elements from one token's rows to the next's
    void *key_cache, *value_cache;
    const int32_t* slot_mapping;
    const int64_t* positions;                 // [axes][num_tokens]
    const float* inv_freq;                    // [rot_dim / 2]
    int32_t num_tokens, num_q_heads, num_kv_heads, head_size, rot_dim, block_size, num_blocks;
    int32_t interleaved;
    float k_inv, v_inv;                       // fp8: reciprocal scales
    int32_t* status;
    uint8_t axis[kMaxRopePairs];              // position axis of each rotated pair
};
cudaError_t launch_rope_and_cache(const RopeParams& p, bool bf16, bool kv8, cudaStream_t stream);

constexpr int32_t kMoveLayers = 64;           // layers per launch (kernel parameter space)
struct MoveParams {
    void* key[kMoveLayers];
    void* value[kMoveLayers];
    const int32_t* pairs;                     // [num_pairs][2] (from, to), ascending from
    int32_t* block_tables;                    // null: no tables, or another launch rewrites them
    int64_t num_entries;
    int64_t vecs_per_block;                   // 16-byte pieces of one block of one pool
    int32_t num_layers, num_pairs, num_blocks;
    int32_t report;                           // this launch reports bad pairs
    int32_t* status;
};
cudaError_t launch_move_blocks(const MoveParams& p, cudaStream_t stream);

}  // namespace pa
