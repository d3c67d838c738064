// pa_tree_aux.cu -- what follows the attention of a tree of drafted tokens: the path that the
// model's own choices accept, and its K / V rows moved together in every layer's pools.
#include <cstdint>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_masked.h"

namespace pa {

namespace {

constexpr int kAcceptThreads = 256;
constexpr int kMaxNodes = 32 * kMaxTreeWords;

// One CTA per sequence.  A node's parent is the highest bit of its mask row below itself; the
// node follows its parent if its token is what the model chose there.  Every node walks up to
// see whether it hangs on the root by such steps alone, and the deepest one that does (the
// lowest of those) ends the path.  Bound by latency: a few dependent loads and the walks.
__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const AcceptParams p) {
    __shared__ int16_t parent[kMaxNodes];     // -1: does not follow
    __shared__ uint32_t best;                 // depth << 16 | (0xffff - node)
    grid_dependency_wait();
    const int32_t s = blockIdx.x, tid = threadIdx.x;
    const int32_t a = p.query_starts[s], b = p.query_starts[s + 1], l = p.context_lens[s];
    const int32_t start = min(max(a, 0), p.num_tokens);
    const int32_t end = min(max(b, start), p.num_tokens);
    const int32_t n = min(end - start, 32 * p.mask_words);
    const bool bad = start != a || end != b || n != end - start || l < end - start;
    if (tid == 0) {
        best = 0xffffu;
        if (bad && p.status) atomicOr(p.status, kDevBadLen);
    }
    for (int32_t i = tid; i < n; i += kAcceptThreads) {
        const uint32_t* row = p.tree_mask + (size_t)(start + i) * p.mask_words;
        int32_t up = -1;
        for (int32_t w = i >> 5; w >= 0 && up < 0; --w) {
            uint32_t bits = row[w];
            if (w == i >> 5) bits &= (1u << (i & 31)) - 1u;
            if (bits) up = 32 * w + 31 - __clz(bits);
        }
        if (up >= 0 && p.draft[start + i] != p.target[start + up]) up = -1;
        parent[i] = (int16_t)up;
    }
    __syncthreads();
    for (int32_t i = tid; i < n; i += kAcceptThreads) {
        int32_t at = i;
        uint32_t depth = 0;
        while (at > 0 && parent[at] >= 0) {
            at = parent[at];
            ++depth;
        }
        if (at == 0) atomicMax(&best, depth << 16 | (0xffffu - (uint32_t)i));
    }
    __syncthreads();
    const int32_t depth = (int32_t)(best >> 16);
    const int32_t count = n > 0 ? min(depth + 1, p.max_accepted) : 0;
    int32_t* out = p.accepted + (size_t)s * p.max_accepted;
    for (int32_t j = count + tid; j < p.max_accepted; j += kAcceptThreads) out[j] = -1;
    if (tid == 0) {
        int32_t at = 0xffff - (int32_t)(best & 0xffffu), last = 0;
        for (int32_t j = depth; j >= 0 && count > 0; --j) {
            if (j < count) out[j] = at;
            if (j == count - 1) last = at;
            if (j > 0) at = parent[at];
        }
        p.num_accepted[s] = count;
        p.next_tokens[s] = count > 0 ? p.target[start + last] : -1;
        p.new_lens[s] = max(max(l, 0) - (end - start), 0) + count;
    }
}

constexpr int kMoveThreads = 128;
constexpr int kMoveBatch = 4;        // rows that a thread has on their way
constexpr int kMoveCtas = 12;        // CTAs to an SM
constexpr int kMovePath = 64;        // path entries whose places sit in shared memory at a time
static_assert(kMovePath <= kMoveThreads, "a thread per entry");

// CTA (s, y): sequence s in pool y (2 * layer, + 1 for V).  A thread has one 16-byte column of
// one kv head's rows and takes the path's rows in order, a batch's loads before its stores: a
// row is only ever overwritten after it was read, since path[j] >= j and ascending.  Bound by
// HBM at many layers (a row is 256 bytes per head, at scattered places), else by the chain
// lengths -> tables -> rows.  (64 sequences, 64 pools of 8 heads of 256 bytes: 14.5 us, 4.4 TB/s;
// eight rows at a time, whose registers leave room for 6 CTAs, 17.2; two pools to a CTA 15.8, four
// 18.5.)
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) move_tokens_kernel(const __grid_constant__ MoveTokensParams p) {
    __shared__ int64_t from_s[kMovePath], to_s[kMovePath];   // row of head 0; -1: nothing to move
    grid_dependency_wait();
    const int32_t s = blockIdx.x, tid = threadIdx.x;
    const bool report = p.report && blockIdx.y == 0 && p.status;
    // (the path's first entries are on their way with the lengths)
    const int32_t* path = p.accepted + (size_t)s * p.max_accepted;
    int32_t node = 0, before = -1;
    auto entry = [&](int32_t j) {
        if (j < p.max_accepted) {
            node = path[j];
            if (j > 0) before = path[j - 1];
        }
    };
    if (tid < kMovePath) entry(tid);
    const int32_t n = p.num_accepted[s];
    const int64_t base = (int64_t)p.new_lens[s] - n;
    if (n < 0 || n > p.max_accepted || base < 0) {
        if (report && tid == 0) atomicOr(p.status, kDevBadLen);
        return;
    }
    const int32_t layer = blockIdx.y >> 1;
    const int64_t cap = (int64_t)p.max_blocks_per_seq * p.block_size;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    uint4* const pool = static_cast<uint4*>((blockIdx.y & 1) ? p.value[layer] : p.key[layer]);
    auto row_of = [&](int64_t pos) -> int64_t {
        const int32_t block = table[pos / p.block_size];
        if (block < 0 || block >= p.num_blocks) return -1;
        return (int64_t)block * p.num_kv_heads * p.block_size + pos % p.block_size;
    };
    const int32_t columns = p.num_kv_heads * p.row_vecs;
    for (int32_t j0 = 0; j0 < n; j0 += kMovePath) {
        const int32_t m = min(n - j0, kMovePath);
        if (j0 > 0) __syncthreads();
        if (tid < m) {
            const int32_t i = tid, j = j0 + i;
            if (j0 > 0) entry(j);
            int64_t from = -1, to = -1;
            if (node < j || (j > 0 && before >= node)) {
                if (report) atomicOr(p.status, kDevBadSlot);
            } else if (base + node >= cap) {
                if (report) atomicOr(p.status, kDevBadLen);
            } else if (node != j) {
                from = row_of(base + node);
                to = row_of(base + j);
                if (from < 0 || to < 0) {
                    from = to = -1;
                    if (report) atomicOr(p.status, kDevBadBlock);
                }
            }
            from_s[i] = from;
            to_s[i] = to;
        }
        __syncthreads();
        for (int32_t c = tid; c < columns; c += kMoveThreads) {
            const int32_t h = c / p.row_vecs;
            uint4* const col = pool + ((int64_t)h * p.block_size) * p.row_vecs + (c - h * p.row_vecs);
            for (int32_t i0 = 0; i0 < m; i0 += kMoveBatch) {
                uint4 x[kMoveBatch];
#pragma unroll
                for (int k = 0; k < kMoveBatch; ++k)
                    if (i0 + k < m && from_s[i0 + k] >= 0) x[k] = col[from_s[i0 + k] * p.row_vecs];
#pragma unroll
                for (int k = 0; k < kMoveBatch; ++k)
                    if (i0 + k < m && from_s[i0 + k] >= 0) col[to_s[i0 + k] * p.row_vecs] = x[k];
            }
        }
    }
}

}  // namespace

cudaError_t launch_tree_accept(const AcceptParams& p, cudaStream_t stream) {
    // An ordinary launch: it writes lengths, which a plan kernel may read before it waits.
    tree_accept_kernel<<<p.num_seqs, kAcceptThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_move_tokens(const MoveTokensParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.num_seqs, (unsigned)(2 * p.num_layers));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, move_tokens_kernel, p);
}

}  // namespace pa
