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
// Shortest partition of a context, in 128-token tiles.
constexpr int32_t kPfMinPart = 2;

// Head of the prefill workspace, written by the plan kernel.
struct PfHeader {
    uint32_t counter;       // items claimed past the first gridDim.x
    uint32_t total_items;   // list entries * num_kv_heads
    uint32_t pad[62];
};

// One entry of the work list: a partition of the context of one row tile (the query rows
// of up to 2 * tokens_per_stream new tokens of a sequence), for every kv head.
struct alignas(16) PfEntry {
    int32_t seq;       // sequence (block-table row)
    int32_t len;       // context length, clamped
    int32_t q_start;   // first row of the sequence's chunk in query / out
    int32_t q_len;     // new tokens of the sequence
    int32_t tok0;      // first new token of the row tile, counted within the chunk
    int32_t tile0;     // first 128-token tile of the partition
    int32_t tile1;     // one past its last tile
    int32_t nparts;    // partitions of this row tile
    int32_t part;      // which of them
    int32_t slot0;     // first partial-result slot of the row tile (nparts > 1)
    int32_t split;     // index among the row tiles with several partitions
    int32_t pad;
};

struct PrefillParams {
    void* out;
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
    int32_t max_entries;
    int32_t max_slots;
    PfHeader* hdr;
    int4* seqs;                // [num_seqs] (q_start, q_len, len, first row tile)
    PfEntry* list;             // [max_entries]
    int32_t* arrive;           // [split row tiles][num_kv_heads][2 streams]
    float2* part_ml;           // [slot][kv head][stream][128] (reference, weight sum)
    float* part_acc;           // [slot][kv head][stream][head_size][128]
    int32_t* status;
};

struct PfWorkspace {
    size_t hdr, seqs, list, arrive, part_ml, part_acc, total;
    int32_t max_row_tiles, max_entries, max_slots;
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
