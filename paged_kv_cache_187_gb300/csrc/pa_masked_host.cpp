// pa_masked_host.cpp -- host side of the operators around reads of the cache that follow a mask:
// argument checks, workspaces and launches of pa_tree_accept, pa_move_tokens, pa_key_bounds,
// pa_select_blocks and pa_decode_sparse(_fp8), declared in include/pa.h.  (pa_decode_tree is a
// form of the chunk attention: pa_chunk_host.cpp.)
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/pa.h"
#include "pa_internal.h"
#include "pa_masked.h"

namespace {

pa_status fail(pa_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return (pa_status)pa::set_last_error(st, buf);
}

pa_status ok() { return (pa_status)pa::set_last_error(PA_OK, ""); }

pa_status cuda_fail(cudaError_t e, const char* what) {
    return fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int32_t kMaxGridY = 65535;

// Entries of a list (blocks, an accepted path, a token's row) at most: kernels step past its end in
// 32 bits.
constexpr int32_t kMaxList = 1 << 30;

}  // namespace

extern "C" {

pa_status pa_tree_accept(int32_t* accepted, int32_t max_accepted, int32_t* num_accepted,
                         int64_t* next_tokens, int32_t* new_lens, const int64_t* draft_tokens,
                         const int64_t* target_tokens, const int32_t* tree_mask, int32_t mask_words,
                         const int32_t* query_starts, const int32_t* context_lens, int32_t num_tokens,
                         int32_t num_seqs, int32_t* status_dev, pa_stream stream) {
    if (num_tokens < 0 || num_seqs < 0 || max_accepted <= 0 || mask_words <= 0)
        return fail(PA_ERR_INVALID_ARG, "tree_accept: sizes must be positive (num_tokens, num_seqs >= 0)");
    if (mask_words > pa::kMaxTreeWords)
        return fail(PA_ERR_UNSUPPORTED, "tree_accept: mask_words %d > %d", mask_words, pa::kMaxTreeWords);
    if (max_accepted > kMaxList)
        return fail(PA_ERR_UNSUPPORTED, "tree_accept: max_accepted %d > %d", max_accepted, kMaxList);
    if (num_seqs == 0) return ok();
    if (!accepted || !num_accepted || !next_tokens || !new_lens || !query_starts || !context_lens ||
        (num_tokens > 0 && (!draft_tokens || !target_tokens || !tree_mask)))
        return fail(PA_ERR_INVALID_ARG, "tree_accept: null pointer");
    pa::AcceptParams p;
    std::memset(&p, 0, sizeof(p));
    p.accepted = accepted;
    p.num_accepted = num_accepted;
    p.next_tokens = next_tokens;
    p.new_lens = new_lens;
    p.draft = draft_tokens;
    p.target = target_tokens;
    p.tree_mask = reinterpret_cast<const uint32_t*>(tree_mask);
    p.query_starts = query_starts;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.mask_words = mask_words;
    p.max_accepted = max_accepted;
    p.status = status_dev;
    const cudaError_t e = pa::launch_tree_accept(p, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "tree_accept launch");
    return ok();
}

pa_status pa_move_tokens(void* const* key_caches, void* const* value_caches, int32_t num_layers,
                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                         const int32_t* new_lens, const int32_t* accepted, int32_t max_accepted,
                         const int32_t* num_accepted, int32_t num_seqs, int32_t num_kv_heads,
                         int32_t head_size, int32_t block_size, int32_t num_blocks, pa_dtype dtype,
                         int32_t* status_dev, pa_stream stream) {
    if (num_layers < 0 || num_seqs < 0 || max_blocks_per_seq <= 0 || max_accepted <= 0 ||
        num_kv_heads <= 0 || head_size <= 0 || block_size <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "move_tokens: sizes must be positive (num_layers, num_seqs >= 0)");
    if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_FP8_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "move_tokens: dtype");
    const int64_t row = (int64_t)head_size * (dtype == PA_FP8_E4M3 ? 1 : 2);
    if (row % 16) return fail(PA_ERR_INVALID_ARG, "move_tokens: rows must be 16-byte multiples");
    if (row / 16 * num_kv_heads > kMaxList) return fail(PA_ERR_UNSUPPORTED, "move_tokens: too many heads");
    if (max_accepted > kMaxList)
        return fail(PA_ERR_UNSUPPORTED, "move_tokens: max_accepted %d > %d", max_accepted, kMaxList);
    if (num_seqs == 0 || num_layers == 0) return ok();
    if (!key_caches || !value_caches || !block_tables || !new_lens || !accepted || !num_accepted)
        return fail(PA_ERR_INVALID_ARG, "move_tokens: null pointer");
    for (int32_t l = 0; l < num_layers; ++l) {
        if (!key_caches[l] || !value_caches[l]) return fail(PA_ERR_INVALID_ARG, "move_tokens: null pool");
        if (!aligned16(key_caches[l]) || !aligned16(value_caches[l]))
            return fail(PA_ERR_INVALID_ARG, "move_tokens: pools must be 16-byte aligned");
    }
    pa::MoveTokensParams p;
    std::memset(&p, 0, sizeof(p));
    p.block_tables = block_tables;
    p.new_lens = new_lens;
    p.accepted = accepted;
    p.num_accepted = num_accepted;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.max_accepted = max_accepted;
    p.num_blocks = num_blocks;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.row_vecs = (int32_t)(row / 16);
    p.status = status_dev;
    for (int32_t l0 = 0; l0 < num_layers; l0 += p.num_layers) {
        p.num_layers = std::min(num_layers - l0, pa::kMoveTokenLayers);
        for (int32_t l = 0; l < p.num_layers; ++l) {
            p.key[l] = key_caches[l0 + l];
            p.value[l] = value_caches[l0 + l];
        }
        p.report = l0 == 0;
        const cudaError_t e = pa::launch_move_tokens(p, (cudaStream_t)stream);
        if (e != cudaSuccess) return cuda_fail(e, "move_tokens launch");
    }
    return ok();
}

pa_status pa_key_bounds(int8_t* bounds, float* bound_steps, const void* key_cache,
                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                        const int32_t* context_lens, const int32_t* query_starts,
                        int32_t max_new_tokens, int32_t num_seqs, int32_t num_kv_heads,
                        int32_t head_size, int32_t block_size, int32_t num_blocks, pa_dtype dtype,
                        int32_t* status_dev, pa_stream stream) {
    if (num_seqs < 0 || max_new_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return fail(PA_ERR_INVALID_ARG, "key_bounds: sizes must be positive (num_seqs, max_new_tokens >= 0)");
    if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_FP8_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "key_bounds: dtype");
    if (head_size != 64 && head_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "key_bounds: head_size %d (64 or 128)", head_size);
    if (block_size != 16 && block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "key_bounds: block_size %d (16 or 32)", block_size);
    if (num_seqs == 0 || max_new_tokens == 0) return ok();
    if (!bounds || !bound_steps || !key_cache || !block_tables || !context_lens)
        return fail(PA_ERR_INVALID_ARG, "key_bounds: null pointer");
    if (!aligned16(bounds) || !aligned16(key_cache))
        return fail(PA_ERR_INVALID_ARG, "key_bounds: buffers must be 16-byte aligned");
    pa::BoundsParams p;
    std::memset(&p, 0, sizeof(p));
    p.bounds = bounds;
    p.steps = bound_steps;
    p.key_cache = key_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_starts = query_starts;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.head_size = head_size;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.max_new_tokens = max_new_tokens;
    // n tokens in a row touch (n - 1) / bs + 1 blocks, and one more where they cross an edge
    p.slots = (int32_t)std::min<int64_t>(((int64_t)max_new_tokens + block_size - 2) / block_size + 1,
                                         max_blocks_per_seq);
    p.status = status_dev;
    if ((int64_t)num_seqs * p.slots * num_kv_heads > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "key_bounds: too many blocks");
    const cudaError_t e = pa::launch_key_bounds(p, dtype == PA_FP8_E4M3 ? pa::BoundsType::kFp8
                                                   : dtype == PA_BF16   ? pa::BoundsType::kBf16
                                                                        : pa::BoundsType::kF16,
                                                (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "key_bounds launch");
    return ok();
}

}  // extern "C"

namespace {

// The weights of every row (query token and kv head; head_size 128 at most), then its scores.
struct SelectWorkspace {
    size_t weights, keys, total;
};
SelectWorkspace select_workspace(int64_t rows, int32_t blocks) {
    SelectWorkspace L;
    L.weights = 0;
    L.keys = align256((size_t)rows * 2 * 128 * sizeof(int16_t));
    L.total = L.keys + align256(sizeof(uint32_t) * (size_t)rows * blocks);
    return L;
}

}  // namespace

extern "C" {

size_t pa_select_blocks_workspace_size(int32_t num_seqs, int32_t q_len, int32_t num_kv_heads,
                                       int32_t block_size, int32_t max_context_len) {
    if (num_seqs < 0 || q_len <= 0 || num_kv_heads <= 0 || block_size <= 0 || max_context_len < 0) return 0;
    return select_workspace((int64_t)num_seqs * q_len * num_kv_heads, max_context_len / block_size + 1).total;
}

pa_status pa_select_blocks(int32_t* selected, const void* query, const int8_t* bounds,
                           const float* bound_steps, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t num_seqs,
                           int32_t q_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                           int32_t block_size, int32_t num_blocks, int32_t max_context_len,
                           int32_t num_selected, int32_t num_first, int32_t num_last, pa_dtype dtype,
                           void* workspace, size_t workspace_bytes, int32_t* status_dev,
                           pa_stream stream) {
    if (num_seqs < 0 || q_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || max_context_len < 0 || num_selected <= 0)
        return fail(PA_ERR_INVALID_ARG, "select_blocks: sizes must be positive (num_seqs >= 0)");
    if (num_first < 0 || num_last < 0 || (int64_t)num_first + num_last > num_selected)
        return fail(PA_ERR_INVALID_ARG, "select_blocks: num_first %d and num_last %d of %d blocks", num_first,
                    num_last, num_selected);
    if (num_selected > kMaxList)
        return fail(PA_ERR_UNSUPPORTED, "select_blocks: num_selected %d > %d", num_selected, kMaxList);
    if (dtype != PA_F16 && dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "select_blocks: dtype");
    if (head_size != 64 && head_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "select_blocks: head_size %d (64 or 128)", head_size);
    if (block_size != 16 && block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "select_blocks: block_size %d (16 or 32)", block_size);
    if (num_q_heads % num_kv_heads)
        return fail(PA_ERR_INVALID_ARG, "select_blocks: num_q_heads %% num_kv_heads != 0");
    if (num_q_heads / num_kv_heads > 16)
        return fail(PA_ERR_UNSUPPORTED, "select_blocks: query group %d > 16", num_q_heads / num_kv_heads);
    if (num_kv_heads > kMaxGridY) return fail(PA_ERR_UNSUPPORTED, "select_blocks: too many heads");
    if ((int64_t)num_seqs * q_len > INT32_MAX) return fail(PA_ERR_UNSUPPORTED, "select_blocks: too many rows");
    if ((int64_t)num_blocks * num_kv_heads > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "select_blocks: pool of more than 2^31 blocks of one kv head");
    const int64_t context = std::min<int64_t>(max_context_len, (int64_t)max_blocks_per_seq * block_size);
    const int32_t blocks = (int32_t)((context + block_size - 1) / block_size);
    if (blocks > pa::kMaxSelectBlocks)
        return fail(PA_ERR_UNSUPPORTED, "select_blocks: contexts of %d blocks (at most %d)", blocks,
                    pa::kMaxSelectBlocks);
    if (num_seqs == 0) return ok();
    if (!selected || !query || !bounds || !bound_steps || !block_tables || !context_lens)
        return fail(PA_ERR_INVALID_ARG, "select_blocks: null pointer");
    if (!aligned16(query) || !aligned16(bounds))
        return fail(PA_ERR_INVALID_ARG, "select_blocks: buffers must be 16-byte aligned");
    const SelectWorkspace L = select_workspace((int64_t)num_seqs * q_len * num_kv_heads, blocks);
    if (blocks > num_selected) {
        if (!workspace || workspace_bytes < L.total)
            return fail(PA_ERR_WORKSPACE, "select_blocks: workspace of %zu bytes, need %zu", workspace_bytes, L.total);
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return fail(PA_ERR_INVALID_ARG, "select_blocks: workspace must be 256-byte aligned");
    }
    pa::SelectParams p;
    std::memset(&p, 0, sizeof(p));
    p.selected = selected;
    p.query = query;
    p.bounds = bounds;
    p.steps = bound_steps;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.q_len = q_len;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.head_size = head_size;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.max_context_len = (int32_t)context;
    p.num_selected = num_selected;
    p.num_first = num_first;
    p.num_last = num_last;
    p.max_blocks = blocks;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "select_blocks: device");
    p.sms = sms;
    // One launch, a CTA per row, where an SM has one row of a thousand blocks at most (1 sequence of 200
    // / 1000 / 2000 blocks, 8 kv heads: 7.4 / 10 / 13 us, in three launches 9.6 / 9.9 / 10.4; 19
    // sequences 7.8 / 11.3 / 17.3 and 12.9 / 14 / 18.6; 32, whose rows come in two turns, 14.1 and 13.7
    // at 200; every launch is 2 us of host time too).
    const bool one_launch = blocks <= num_selected ||
                            (blocks <= 1024 && (int64_t)num_seqs * q_len * num_kv_heads <= sms);
    if (!one_launch) {
        p.weights = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + L.weights);
        p.keys = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + L.keys);
    }
    p.status = status_dev;
    e = pa::launch_select_blocks(p, dtype == PA_BF16, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "select_blocks launch");
    return ok();
}

}  // extern "C"

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// A pool as a matrix of rows; a box is 128 bytes of a block's rows.
pa_status encode_pool(CUtensorMap* map, const void* pool, int64_t rows, int32_t head_size, int32_t block_size,
                      bool kv8) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const int32_t elem = kv8 ? 1 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)head_size, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)head_size * elem};
    const cuuint32_t box[2] = {128u / (cuuint32_t)elem, (cuuint32_t)block_size}, ones[2] = {1u, 1u};
    const CUresult r = fn(map, kv8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                          const_cast<void*>(pool), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return PA_OK;
}

struct SparseArgs {
    void* out;
    const void *query, *key_cache, *value_cache;
    const int32_t* block_tables;
    int32_t max_blocks_per_seq;
    const int32_t* context_lens;
    const int32_t* selected;
    int32_t num_selected, num_seqs, q_len, num_q_heads, num_kv_heads, head_size, block_size, num_blocks;
    float scale, k_scale, v_scale;
    pa_dtype dtype;
    bool kv8;
};

pa_status run_sparse(const SparseArgs& a, int32_t* status, cudaStream_t stream) {
    if (a.num_seqs < 0 || a.q_len <= 0 || a.num_q_heads <= 0 || a.num_kv_heads <= 0 || a.num_blocks <= 0 ||
        a.max_blocks_per_seq <= 0 || a.num_selected <= 0)
        return fail(PA_ERR_INVALID_ARG, "decode_sparse: sizes must be positive (num_seqs >= 0)");
    if (a.dtype != PA_F16 && a.dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "decode_sparse: dtype");
    if (a.head_size != 64 && a.head_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "decode_sparse: head_size %d (64 or 128)", a.head_size);
    if (a.kv8 && a.head_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "decode_sparse: an fp8 cache needs head_size 128");
    if (a.kv8 && !(a.k_scale > 0.f && a.v_scale > 0.f))
        return fail(PA_ERR_INVALID_ARG, "decode_sparse: k_scale and v_scale must be positive");
    if (a.block_size != 16 && a.block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "decode_sparse: block_size %d (16 or 32)", a.block_size);
    if (!std::isfinite(a.scale)) return fail(PA_ERR_INVALID_ARG, "decode_sparse: scale must be finite");
    if (a.num_q_heads % a.num_kv_heads)
        return fail(PA_ERR_INVALID_ARG, "decode_sparse: num_q_heads %% num_kv_heads != 0");
    const int32_t group = a.num_q_heads / a.num_kv_heads;
    if (group > 16) return fail(PA_ERR_UNSUPPORTED, "decode_sparse: query group %d > 16", group);
    const int64_t pool_rows = (int64_t)a.num_blocks * a.num_kv_heads * a.block_size;
    if (pool_rows + (int64_t)a.num_kv_heads * a.block_size > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "decode_sparse: pool has more than 2^31 rows");
    const int64_t rows = (int64_t)a.num_seqs * a.q_len * a.num_kv_heads;
    if (rows > (1 << 24)) return fail(PA_ERR_UNSUPPORTED, "decode_sparse: more than 2^24 (token, kv head) rows");
    if (a.num_selected > pa::kSparseMaxSelected)
        return fail(PA_ERR_UNSUPPORTED, "decode_sparse: num_selected %d > %d", a.num_selected, pa::kSparseMaxSelected);
    if (a.num_seqs == 0) return ok();
    if (!a.out || !a.query || !a.key_cache || !a.value_cache || !a.block_tables || !a.context_lens || !a.selected)
        return fail(PA_ERR_INVALID_ARG, "decode_sparse: null pointer");
    if (!aligned16(a.out) || !aligned16(a.query) || !aligned16(a.key_cache) || !aligned16(a.value_cache))
        return fail(PA_ERR_INVALID_ARG, "decode_sparse: device buffers must be 16-byte aligned");
    pa::SparseParams p;
    std::memset(&p, 0, sizeof(p));
    p.selected = a.selected;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.max_blocks_per_seq = a.max_blocks_per_seq;
    p.num_seqs = a.num_seqs;
    p.q_len = a.q_len;
    p.num_kv_heads = a.num_kv_heads;
    p.block_size = a.block_size;
    p.num_blocks = a.num_blocks;
    p.num_selected = a.num_selected;
    p.status = status;
    // the decode's view: a sequence of one kv head per row
    pa::DecodeParams d;
    std::memset(&d, 0, sizeof(d));
    d.out = a.out;
    d.q = a.query;
    d.num_seqs = (int32_t)rows;
    d.num_q_heads = d.group = d.rows = group;
    d.num_kv_heads = 1;
    d.num_blocks = a.num_blocks * a.num_kv_heads;
    d.block_size = a.block_size;
    d.scale_log2 = a.scale * (a.kv8 ? a.k_scale : 1.f) * 1.4426950408889634f;
    d.out_scale = a.kv8 ? a.v_scale : 1.f;
    d.q_len = d.row_chunks = d.row_groups = 1;
    d.status = status;
    CUtensorMap km, vm;
    pa_status st = encode_pool(&km, a.key_cache, pool_rows, a.head_size, a.block_size, a.kv8);
    if (st == PA_OK) st = encode_pool(&vm, a.value_cache, pool_rows, a.head_size, a.block_size, a.kv8);
    if (st != PA_OK) return st;
    const bool bf16 = a.dtype == PA_BF16;
    auto launch = [&](int32_t ctas, int32_t* per_sm) {
        return a.kv8  ? pa::launch_sparse_fp8(bf16, km, vm, d, p, ctas, stream, per_sm)
               : bf16 ? pa::launch_sparse_bf16(km, vm, d, p, a.head_size, ctas, stream, per_sm)
                      : pa::launch_sparse_f16(km, vm, d, p, a.head_size, ctas, stream, per_sm);
    };
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // A cluster per row, as large as leaves every CTA a few tiles and all of them a place: up to 3.4
    // CTAs to an SM, 2.6 in clusters of 16, which need room in one part of the chip.  (us a call, 8 kv
    // heads: 8 rows of 256 blocks 16.1 in clusters of 8 and 12.6 of 16; 32 of 64 blocks 8.7 and 12.2;
    // 64 of 256 blocks 28.8 in clusters of 4 and 26.6 of 8; 152 of 128 30 in twos and 41 in fours.)
    const int64_t tile_blocks = a.kv8 && a.block_size == 16 ? 2 : 1;
    const int64_t tiles = (a.num_selected + tile_blocks - 1) / tile_blocks;
    p.cluster = 1;
    for (int32_t n = 2; n <= pa::kSparseMaxCluster; n *= 2)
        if (10 * rows * n <= (int64_t)(n > 8 ? 26 : 34) * sms && tiles >= (int64_t)n * pa::kSparseTiles) p.cluster = n;
    if (p.cluster == 1) {
        // Whole rows: of the two rings, the one whose CTAs leave fewer places empty in their last turn
        // (640 rows of 128 blocks, bf16: 133 us with the long ring, whose 608 places take two turns,
        // and 99 with the short one; 384 rows 63 and 69; 1024 rows 154 and 168).
        double best = 0.;
        int32_t choice = 0;
        for (int32_t kind = 0; kind < 2 && e == cudaSuccess; ++kind) {
            int32_t per_sm = 0;
            p.short_ring = kind;
            e = launch(0, &per_sm);
            const int64_t places = std::max<int64_t>((int64_t)per_sm * sms, 1), turns = (rows + places - 1) / places;
            const double used = rows <= places ? 1. : (double)rows / (double)(turns * places);
            if (used > best) {
                best = used;
                choice = kind;
            }
        }
        p.short_ring = choice;
    }
    if (e != cudaSuccess) return cuda_fail(e, "decode_sparse: device");
    e = launch((int32_t)(rows * p.cluster), nullptr);
    if (e != cudaSuccess) return cuda_fail(e, "decode_sparse launch");
    return ok();
}

}  // namespace

extern "C" {

// The parts of a row meet in shared memory: no call needs a workspace.
size_t pa_decode_sparse_workspace_size(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) {
    return 0;
}

pa_status pa_decode_sparse(void* out, const void* query, const void* key_cache, const void* value_cache,
                           const int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* context_lens, const int32_t* selected, int32_t num_selected,
                           int32_t num_seqs, int32_t q_len, int32_t num_q_heads, int32_t num_kv_heads,
                           int32_t head_size, int32_t block_size, int32_t num_blocks, float scale,
                           pa_dtype dtype, void* workspace, size_t workspace_bytes, int32_t* status_dev,
                           pa_stream stream) {
    const SparseArgs a{out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens,
                       selected, num_selected, num_seqs, q_len, num_q_heads, num_kv_heads, head_size,
                       block_size, num_blocks, scale, 1.f, 1.f, dtype, false};
    (void)workspace;
    (void)workspace_bytes;
    return run_sparse(a, status_dev, (cudaStream_t)stream);
}

pa_status pa_decode_sparse_fp8(void* out, const void* query, const void* key_cache, const void* value_cache,
                               const int32_t* block_tables, int32_t max_blocks_per_seq,
                               const int32_t* context_lens, const int32_t* selected,
                               int32_t num_selected, int32_t num_seqs, int32_t q_len,
                               int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                               int32_t block_size, int32_t num_blocks, float scale, float k_scale,
                               float v_scale, pa_dtype dtype, void* workspace, size_t workspace_bytes,
                               int32_t* status_dev, pa_stream stream) {
    const SparseArgs a{out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens,
                       selected, num_selected, num_seqs, q_len, num_q_heads, num_kv_heads, head_size,
                       block_size, num_blocks, scale, k_scale, v_scale, dtype, true};
    (void)workspace;
    (void)workspace_bytes;
    return run_sparse(a, status_dev, (cudaStream_t)stream);
}

}  // extern "C"
