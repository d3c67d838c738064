// pa_chunk_device.cuh -- what the plan and the attention kernel of a ragged chunk both read
// from the call's metadata.
#pragma once

#include "pa_chunk.h"

namespace pa {

// Sequence s of the call (nothing for a lane past the last): its rows of query, context
// length and row tiles; metadata out of range is clamped, and reported if asked.
struct PfChunk {
    int32_t start, count, len, row_tiles;
};
__device__ __forceinline__ PfChunk chunk_of(const PrefillParams& p, int32_t s, bool report) {
    PfChunk c = {0, 0, 0, 0};
    if (s >= p.num_seqs) return c;
    const int64_t row_cap = (int64_t)p.max_blocks_per_seq * p.block_size;
    // (2^30 tokens: positions and their tiles stay within 32 bits)
    const int32_t cap = (int32_t)min(min(row_cap, (int64_t)p.max_context_len), (int64_t)1 << 30);
    const int32_t a = p.query_starts[s], b = p.query_starts[s + 1], l = p.context_lens[s];
    c.start = min(max(a, 0), p.num_tokens);
    const int32_t end = min(max(b, c.start), p.num_tokens);
    c.count = end - c.start;
    c.len = min(max(l, 0), cap);
    const bool wide = p.tree_mask && c.count > 32ll * p.mask_words;   // a tree past its masks
    if (report && (c.start != a || end != b || c.len != l || wide) && p.status)
        atomicOr(p.status, 4 /* PA_DEVERR_BAD_LEN */);
    const int32_t span = 2 * p.tpt;
    c.row_tiles = c.count / span + (c.count % span != 0);
    return c;
}

}  // namespace pa
