// pa_sparse.cu -- attention over selected blocks of the paged cache.
#include <cstdint>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_masked.h"

namespace pa {

namespace {

constexpr int kTableWarps = 4;

// A warp per (query token, kv head): its selected blocks that hold tokens it sees, in order, as
// blocks of the pools with one kv head each, and the tokens in them.  The list has to ascend, so
// only its last block can end early; entries that do not, or lie outside the context, are left
// out and flagged.
__global__ void __launch_bounds__(32 * kTableWarps) sparse_tables_kernel(const SparseParams p) {
    grid_dependency_wait();
    const int32_t lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kTableWarps + (threadIdx.x >> 5);
    if (row >= (int64_t)p.num_seqs * p.q_len * p.num_kv_heads) return;
    const int32_t h = (int32_t)(row % p.num_kv_heads);
    const int32_t q = (int32_t)(row / p.num_kv_heads), s = q / p.q_len, j = q - s * p.q_len;
    const int64_t cap = min((int64_t)p.max_blocks_per_seq * p.block_size, (int64_t)INT32_MAX);
    const int32_t l = p.context_lens[s];
    if ((l < 0 || l > cap) && lane == 0 && h == 0 && j == 0 && p.status) atomicOr(p.status, kDevBadLen);
    const int32_t seen = max((int32_t)min((int64_t)max(l, 0), cap) - p.q_len + j + 1, 0);
    const int32_t blocks = seen / p.block_size + (seen % p.block_size != 0);
    const int32_t* list = p.selected + row * p.num_selected;
    int32_t* out = p.tables + row * p.num_selected;
    int32_t count = 0, last = -1;
    bool bad = false;
    for (int32_t i0 = 0; i0 < p.num_selected; i0 += 32) {
        const int32_t i = i0 + lane;
        int32_t b = i < p.num_selected ? list[i] : -1;
        // the largest entry before this one, of those within the context (a running maximum:
        // shifted in from below, a lane's own value leaves it unchanged)
        int32_t top = b < blocks ? b : -1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) top = max(top, __shfl_up_sync(0xffffffffu, top, o));
        const int32_t below = __shfl_up_sync(0xffffffffu, top, 1);
        const int32_t prev = lane ? max(below, last) : last;
        const bool keep = b >= 0 && b < blocks && b > prev;
        bad |= b >= 0 && !keep;
        const uint32_t kept = __ballot_sync(0xffffffffu, keep);
        if (keep) {
            const int32_t phys = p.block_tables[(size_t)s * p.max_blocks_per_seq + b];
            out[count + __popc(kept & ((1u << lane) - 1u))] =
                phys >= 0 && phys < p.num_blocks ? phys * p.num_kv_heads + h : -1;
        }
        count += __popc(kept);
        if (kept) last = __shfl_sync(0xffffffffu, b, 31 - __clz(kept));
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && p.status) atomicOr(p.status, kDevBadBlock);
    if (lane == 0)
        p.lens[row] = count == 0 ? 0 : count * p.block_size - (last == blocks - 1 ? blocks * p.block_size - seen : 0);
}

}  // namespace

cudaError_t launch_sparse_tables(const SparseParams& p, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.num_seqs * p.q_len * p.num_kv_heads;
    // An ordinary launch: it writes lengths, which the plan kernel after it reads before it waits.
    sparse_tables_kernel<<<(unsigned)((rows + kTableWarps - 1) / kTableWarps), 32 * kTableWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pa
