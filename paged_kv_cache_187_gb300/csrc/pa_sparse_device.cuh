// pa_sparse_device.cuh -- a row's list of selected blocks, as every reader of it takes it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "pa_masked.h"

namespace pa {

struct SparseList {
    int32_t count;      // entries e0 .. e1 - 1 that count
    int32_t tokens;     // tokens in their blocks
};

// Entries e0 .. e1 - 1 of row `row`'s list, by one warp: those that hold tokens which the row sees,
// in order, go to store(place, block), as blocks of the pools with one kv head each (`nowhere` for a
// table entry outside the pool).  The list has to ascend, so only the context's last block can end
// early; entries that do not ascend (entries before e0 count for that), or lie outside the context,
// are left out and flagged.  128 entries at a time, their loads on their way together.
template <class Store>
__device__ __forceinline__ SparseList walk_list(const SparseParams& p, int32_t row, int32_t e0, int32_t e1,
                                                int32_t nowhere, Store&& store) {
    constexpr int kBatch = 4;
    const int32_t lane = threadIdx.x & 31;
    const int32_t h = row % p.num_kv_heads, q = row / p.num_kv_heads, s = q / p.q_len, j = q - s * p.q_len;
    const int32_t* list = p.selected + (size_t)row * p.num_selected;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    const int32_t cap = (int32_t)min((int64_t)p.max_blocks_per_seq * p.block_size, (int64_t)INT32_MAX);
    const int32_t l = p.context_lens[s];
    int32_t seen = 0, blocks = 0, count = 0, top = -1, last = -1;
    bool bad = false;
    for (int32_t i0 = 0; i0 < e1; i0 += 32 * kBatch) {
        int32_t b[kBatch], phys[kBatch];
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
            const int32_t i = i0 + 32 * t + lane;
            b[t] = i < e1 ? list[i] : -1;
        }
        if (i0 == 0) {
            if ((l < 0 || l > cap) && lane == 0 && h == 0 && j == 0 && e0 == 0 && p.status)
                atomicOr(p.status, kDevBadLen);
            seen = max(min(max(l, 0), cap) - p.q_len + j + 1, 0);
            blocks = seen / p.block_size + (seen % p.block_size != 0);
        }
#pragma unroll
        for (int t = 0; t < kBatch; ++t)
            phys[t] = i0 + 32 * t + lane >= e0 && b[t] >= 0 && b[t] < blocks ? table[b[t]] : -1;
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
            if (i0 + 32 * t >= e1) break;
            const bool ours = i0 + 32 * t + lane >= e0;
            // the largest entry up to this one, of those within the context (a running maximum:
            // what a lane shifts in from itself leaves it unchanged)
            int32_t m = b[t] < blocks ? b[t] : -1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) m = max(m, __shfl_up_sync(0xffffffffu, m, o));
            const int32_t below = __shfl_up_sync(0xffffffffu, m, 1);
            const int32_t prev = lane ? max(below, top) : top;
            const bool keep = ours && b[t] >= 0 && b[t] < blocks && b[t] > prev;
            bad |= ours && b[t] >= 0 && !keep;
            const uint32_t kept = __ballot_sync(0xffffffffu, keep);
            if (keep)
                store(count + __popc(kept & ((1u << lane) - 1u)),
                      phys[t] >= 0 && phys[t] < p.num_blocks ? phys[t] * p.num_kv_heads + h : nowhere);
            count += __popc(kept);
            if (kept) last = __shfl_sync(0xffffffffu, b[t], 31 - __clz(kept));
            top = max(top, __shfl_sync(0xffffffffu, m, 31));
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && p.status) atomicOr(p.status, kDevBadBlock);
    SparseList r;
    r.count = count;
    r.tokens = count * p.block_size - (count > 0 && last == blocks - 1 ? blocks * p.block_size - seen : 0);
    return r;
}

}  // namespace pa
