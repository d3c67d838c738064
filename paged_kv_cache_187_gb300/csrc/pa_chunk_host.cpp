// pa_chunk_host.cpp -- host side of the chunk operators declared in include/pa.h: argument
// checks, workspace layout, TMA tensor maps and launches of pa_prefill(_fp8),
// pa_rope_and_cache(_fp8) and pa_move_blocks.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/pa.h"
#include "pa_chunk.h"
#include "pa_internal.h"

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

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

pa_status encode(CUtensorMap* map, const void* base, bool bytes, int rank, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint32_t ones[3] = {1u, 1u, 1u};
    const CUresult r =
        fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, (cuuint32_t)rank,
           const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return PA_OK;
}

// Streaming multiprocessors of the current device, asked for once per device.
pa_status sm_count(int* sms) {
    static std::atomic<int> known[256];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    int n = dev >= 0 && dev < 256 ? known[dev].load() : 0;
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        if (dev >= 0 && dev < 256) known[dev].store(n);
    }
    *sms = n;
    return PA_OK;
}

// New tokens per call: row tiles and their scans stay within 32 bits.
constexpr int32_t kMaxTokens = 1 << 24;

struct PrefillArgs {
    void* out;
    const void *query, *key_cache, *value_cache;
    const int32_t* block_tables;
    int32_t max_blocks_per_seq;
    const int32_t *context_lens, *query_starts;
    int32_t num_tokens, num_seqs, num_q_heads, num_kv_heads, head_size, block_size, num_blocks;
    int32_t max_context_len;
    float scale, k_scale, v_scale;
    pa_dtype dtype;
    bool kv8;
};

pa_status run_prefill(const PrefillArgs& a, void* ws, size_t ws_bytes, int32_t* status,
                      cudaStream_t stream) {
    if (a.num_tokens < 0 || a.num_seqs < 0 || a.num_q_heads <= 0 || a.num_kv_heads <= 0 ||
        a.num_blocks <= 0 || a.max_blocks_per_seq <= 0 || a.max_context_len < 0)
        return fail(PA_ERR_INVALID_ARG, "prefill: sizes must be positive (num_tokens, num_seqs >= 0)");
    if (a.num_tokens > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "prefill: num_tokens %d > %d", a.num_tokens, kMaxTokens);
    if (a.dtype != PA_F16 && a.dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "prefill: dtype");
    if (a.head_size != 64 && a.head_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "prefill: head_size %d (64 or 128)", a.head_size);
    if (a.kv8 && a.head_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "prefill: an fp8 cache needs head_size 128");
    if (a.kv8 && !(a.k_scale > 0.f && a.v_scale > 0.f))
        return fail(PA_ERR_INVALID_ARG, "prefill: k_scale and v_scale must be positive");
    if (a.block_size != 16 && a.block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "prefill: block_size %d (16 or 32)", a.block_size);
    if (!std::isfinite(a.scale)) return fail(PA_ERR_INVALID_ARG, "prefill: scale must be finite");
    if (a.num_q_heads % a.num_kv_heads)
        return fail(PA_ERR_INVALID_ARG, "prefill: num_q_heads %% num_kv_heads != 0");
    const int32_t group = a.num_q_heads / a.num_kv_heads;
    if (group > 16) return fail(PA_ERR_UNSUPPORTED, "prefill: query group %d > 16", group);
    const int64_t rows = (int64_t)a.num_blocks * a.num_kv_heads * a.block_size;
    if (rows + (int64_t)a.num_kv_heads * a.block_size > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "prefill: pool has more than 2^31 rows");
    if (a.num_tokens == 0 || a.num_seqs == 0) return ok();
    if (!a.out || !a.query || !a.key_cache || !a.value_cache || !a.block_tables || !a.context_lens ||
        !a.query_starts)
        return fail(PA_ERR_INVALID_ARG, "prefill: null pointer");
    if (!aligned16(a.out) || !aligned16(a.query) || !aligned16(a.key_cache) || !aligned16(a.value_cache))
        return fail(PA_ERR_INVALID_ARG, "prefill: device buffers must be 16-byte aligned");
    const pa::PfWorkspace L = pa::prefill_workspace(a.num_tokens, a.num_seqs, a.num_q_heads,
                                                    a.num_kv_heads, a.head_size, a.max_context_len);
    if ((int64_t)L.max_row_tiles * a.num_kv_heads > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "prefill: too many work items");
    if (!ws || ws_bytes < L.total)
        return fail(PA_ERR_WORKSPACE, "prefill: workspace of %zu bytes, need %zu", ws_bytes, L.total);
    if (reinterpret_cast<uintptr_t>(ws) & 255u)
        return fail(PA_ERR_INVALID_ARG, "prefill: workspace must be 256-byte aligned");
    int sms = 0;
    pa_status st = sm_count(&sms);
    if (st != PA_OK) return st;

    pa::PrefillParams p;
    std::memset(&p, 0, sizeof(p));
    p.out = a.out;
    p.value_cache = a.value_cache;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.query_starts = a.query_starts;
    p.max_blocks_per_seq = a.max_blocks_per_seq;
    p.num_tokens = a.num_tokens;
    p.num_seqs = a.num_seqs;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.group = group;
    p.num_blocks = a.num_blocks;
    p.block_size = a.block_size;
    p.head_size = a.head_size;
    p.max_context_len = a.max_context_len;
    p.tpt = pa::kPfRows / group;
    const float scale = a.scale * (a.kv8 ? a.k_scale : 1.f);
    // never 0: a masked score is infinite, and stays so times any other scale
    p.scale_log2 = scale * 1.4426950408889634f;
    if (std::fabs(p.scale_log2) < 1e-30f) p.scale_log2 = std::copysign(1e-30f, scale);
    p.out_scale = a.kv8 ? a.v_scale : 1.f;
    p.max_row_tiles = L.max_row_tiles;
    // one CTA per SM, but never more than tiles
    const int64_t tiles = (int64_t)L.max_row_tiles * a.num_kv_heads *
                          std::max(1, a.max_context_len / pa::kPfTok + (a.max_context_len % pa::kPfTok != 0));
    p.grid = (int32_t)std::min<int64_t>(std::min(sms, pa::kPfMaxGrid), tiles);
    p.direct = a.num_seqs <= 32 && a.max_context_len <= pa::kPfDirectTokens &&
               (int64_t)L.max_row_tiles * a.num_kv_heads <= std::min(sms, pa::kPfMaxGrid);
    if (p.direct) p.grid = L.max_row_tiles * a.num_kv_heads;
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.hdr = reinterpret_cast<pa::PfHeader*>(w + L.hdr);
    p.seqs = reinterpret_cast<int4*>(w + L.seqs);
    p.seq_of = reinterpret_cast<int32_t*>(w + L.seq_of);
    p.order = reinterpret_cast<int32_t*>(w + L.order);
    p.before = reinterpret_cast<int64_t*>(w + L.before);
    p.arrive = reinterpret_cast<int32_t*>(w + L.arrive);
    p.part_ml = reinterpret_cast<float2*>(w + L.part_ml);
    p.part_acc = reinterpret_cast<float*>(w + L.part_acc);
    p.status = status;

    // query [tokens][heads][dims]: a box is 64 dims (the swizzle span) of one kv head's
    // group and the tokens of a stream; the pools as matrices of rows, a box one block
    CUtensorMap qm, km, vm;
    const int32_t elem = a.kv8 ? 1 : 2;
    const cuuint64_t qdims[3] = {(cuuint64_t)a.head_size, (cuuint64_t)a.num_q_heads, (cuuint64_t)a.num_tokens};
    const cuuint64_t qstr[2] = {(cuuint64_t)a.head_size * 2, (cuuint64_t)a.num_q_heads * a.head_size * 2};
    const cuuint32_t qbox[3] = {64u, (cuuint32_t)group, (cuuint32_t)p.tpt};
    const cuuint64_t dims[2] = {(cuuint64_t)a.head_size, (cuuint64_t)rows};
    const cuuint64_t str[1] = {(cuuint64_t)a.head_size * elem};
    const cuuint32_t box[2] = {128u / (cuuint32_t)elem, (cuuint32_t)a.block_size};
    if ((st = encode(&qm, a.query, false, 3, qdims, qstr, qbox)) != PA_OK) return st;
    if ((st = encode(&km, a.key_cache, a.kv8, 2, dims, str, box)) != PA_OK) return st;
    if ((st = encode(&vm, a.value_cache, a.kv8, 2, dims, str, box)) != PA_OK) return st;

    cudaError_t e = p.direct ? cudaSuccess : pa::launch_prefill_plan(p, stream);
    if (e != cudaSuccess) return cuda_fail(e, "prefill plan launch");
    const bool bf16 = a.dtype == PA_BF16;
    e = a.kv8 ? pa::launch_prefill_fp8(bf16, qm, km, vm, p, stream)
        : bf16 ? pa::launch_prefill_bf16(qm, km, vm, p, stream)
               : pa::launch_prefill_f16(qm, km, vm, p, stream);
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
    return ok();
}

pa_status run_rope(pa::RopeParams& p, const int32_t* pair_axes, int32_t num_axes, pa_dtype dtype,
                   bool kv8, float k_scale, float v_scale, cudaStream_t stream) {
    if (p.num_tokens < 0 || p.num_q_heads <= 0 || p.num_kv_heads <= 0 || p.block_size <= 0 ||
        p.num_blocks <= 0 || p.head_size <= 0)
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: sizes must be positive");
    if (dtype != PA_F16 && dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: dtype");
    if (p.head_size % 16 || p.head_size > 1024)
        return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: head_size %d (a multiple of 16 up to 1024)", p.head_size);
    if (p.rot_dim < 16 || p.rot_dim % 16 || p.rot_dim > p.head_size || p.rot_dim / 2 > pa::kMaxRopePairs)
        return fail(PA_ERR_UNSUPPORTED,
                    "rope_and_cache: rot_dim %d (a multiple of 16 up to head_size and 256)", p.rot_dim);
    if (num_axes < 1 || num_axes > 4)
        return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: num_axes %d (1 .. 4)", num_axes);
    if (num_axes > 1 && !pair_axes)
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: several axes need pair_axes");
    for (int i = 0; i < p.rot_dim / 2; ++i) {
        const int32_t x = pair_axes ? pair_axes[i] : 0;
        if (x < 0 || x >= num_axes)
            return fail(PA_ERR_INVALID_ARG, "rope_and_cache: pair_axes[%d] = %d is not an axis", i, x);
        p.axis[i] = (uint8_t)x;
    }
    const int64_t qrow = (int64_t)p.num_q_heads * p.head_size, krow = (int64_t)p.num_kv_heads * p.head_size;
    if (p.q_stride < qrow || p.k_stride < krow || p.v_stride < krow)
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: a token stride is shorter than a token's rows");
    if (p.q_stride % 8 || p.k_stride % 8 || p.v_stride % 8)
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: token strides must be multiples of 8 elements");
    if (qrow + 2 * krow > (1 << 26))
        return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: too many heads");
    if (kv8 && !(k_scale > 0.f && v_scale > 0.f))
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: scales must be positive");
    if (p.num_tokens == 0) return ok();
    if (!p.query_out || !p.query || !p.key || !p.value || !p.key_cache || !p.value_cache ||
        !p.slot_mapping || !p.positions || !p.inv_freq)
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: null pointer");
    if (!aligned16(p.query_out) || !aligned16(p.query) || !aligned16(p.key) || !aligned16(p.value) ||
        !aligned16(p.key_cache) || !aligned16(p.value_cache))
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: buffers must be 16-byte aligned");
    if (p.query_out == p.query && p.q_stride != qrow)
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: query may be rotated in place only when dense");
    p.k_inv = kv8 ? 1.0f / k_scale : 1.f;
    p.v_inv = kv8 ? 1.0f / v_scale : 1.f;
    cudaError_t e = pa::launch_rope_and_cache(p, dtype == PA_BF16, kv8, stream);
    if (e != cudaSuccess) return cuda_fail(e, "rope_and_cache launch");
    return ok();
}

pa::RopeParams rope_params(void* query_out, const void* query, const void* key, const void* value,
                           int64_t query_stride, int64_t key_stride, int64_t value_stride,
                           void* key_cache, void* value_cache, const int32_t* slot_mapping,
                           const int64_t* positions, const float* inv_freq, int32_t rot_dim,
                           int32_t interleaved, int32_t num_tokens, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_size, int32_t block_size,
                           int32_t num_blocks, int32_t* status) {
    pa::RopeParams p;
    std::memset(&p, 0, sizeof(p));
    p.query_out = query_out;
    p.query = query;
    p.key = key;
    p.value = value;
    p.q_stride = query_stride;
    p.k_stride = key_stride;
    p.v_stride = value_stride;
    p.key_cache = key_cache;
    p.value_cache = value_cache;
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.rot_dim = rot_dim;
    p.interleaved = interleaved ? 1 : 0;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_size = head_size;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.status = status;
    return p;
}

}  // namespace

namespace pa {

// Row tiles: at most one more than full ones per sequence that has tokens.
PfWorkspace prefill_workspace(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_size, int32_t max_context_len) {
    PfWorkspace L;
    const int32_t group = std::max(1, num_q_heads / num_kv_heads);
    const int32_t span = 2 * std::max(1, kPfRows / group);
    L.max_row_tiles = num_tokens / span + std::min(num_seqs, num_tokens);
    // no unit is cut whose context is a single tile
    const size_t parts = max_context_len > kPfTok ? (size_t)kPfMaxGrid * 2 * 2 * kPfRows : 0;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    L.hdr = take(sizeof(PfHeader));
    L.seqs = take(sizeof(int4) * (size_t)num_seqs);
    L.seq_of = take(sizeof(int32_t) * (size_t)L.max_row_tiles);
    L.order = take(sizeof(int32_t) * (size_t)L.max_row_tiles);
    L.before = take(sizeof(int64_t) * ((size_t)L.max_row_tiles + 1));
    L.arrive = take(sizeof(int32_t) * 2 * kPfMaxGrid);
    L.part_ml = take(sizeof(float2) * parts);
    L.part_acc = take(sizeof(float) * parts * head_size);
    L.total = off;
    return L;
}

}  // namespace pa

extern "C" {

size_t pa_prefill_workspace_size(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_size, int32_t max_context_len) {
    if (num_tokens < 0 || num_tokens > kMaxTokens || num_seqs < 0 || num_q_heads <= 0 ||
        num_kv_heads <= 0 || head_size <= 0 || max_context_len < 0)
        return 0;
    return pa::prefill_workspace(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_size,
                                 max_context_len).total;
}

pa_status pa_prefill(void* out, const void* query, const void* key_cache, const void* value_cache,
                     const int32_t* block_tables, int32_t max_blocks_per_seq,
                     const int32_t* context_lens, const int32_t* query_starts, int32_t num_tokens,
                     int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                     int32_t block_size, int32_t num_blocks, int32_t max_context_len, float scale,
                     pa_dtype dtype, void* workspace, size_t workspace_bytes, int32_t* status_dev,
                     pa_stream stream) {
    const PrefillArgs a{out, query, key_cache, value_cache, block_tables, max_blocks_per_seq,
                        context_lens, query_starts, num_tokens, num_seqs, num_q_heads, num_kv_heads,
                        head_size, block_size, num_blocks, max_context_len, scale, 1.f, 1.f, dtype,
                        false};
    return run_prefill(a, workspace, workspace_bytes, status_dev, (cudaStream_t)stream);
}

pa_status pa_prefill_fp8(void* out, const void* query, const void* key_cache,
                         const void* value_cache, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* context_lens,
                         const int32_t* query_starts, int32_t num_tokens, int32_t num_seqs,
                         int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                         int32_t block_size, int32_t num_blocks, int32_t max_context_len,
                         float scale, float k_scale, float v_scale, pa_dtype dtype, void* workspace,
                         size_t workspace_bytes, int32_t* status_dev, pa_stream stream) {
    const PrefillArgs a{out, query, key_cache, value_cache, block_tables, max_blocks_per_seq,
                        context_lens, query_starts, num_tokens, num_seqs, num_q_heads, num_kv_heads,
                        head_size, block_size, num_blocks, max_context_len, scale, k_scale, v_scale,
                        dtype, true};
    return run_prefill(a, workspace, workspace_bytes, status_dev, (cudaStream_t)stream);
}

pa_status pa_rope_and_cache(void* query_out, const void* query, const void* key, const void* value,
                            int64_t query_stride, int64_t key_stride, int64_t value_stride,
                            void* key_cache, void* value_cache, const int32_t* slot_mapping,
                            const int64_t* positions, int32_t num_axes, const int32_t* pair_axes,
                            const float* inv_freq, int32_t rot_dim, int32_t interleaved,
                            int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                            int32_t head_size, int32_t block_size, int32_t num_blocks,
                            pa_dtype dtype, int32_t* status_dev, pa_stream stream) {
    pa::RopeParams p = rope_params(query_out, query, key, value, query_stride, key_stride, value_stride,
                                   key_cache, value_cache, slot_mapping, positions, inv_freq, rot_dim,
                                   interleaved, num_tokens, num_q_heads, num_kv_heads, head_size,
                                   block_size, num_blocks, status_dev);
    return run_rope(p, pair_axes, num_axes, dtype, false, 1.f, 1.f, (cudaStream_t)stream);
}

pa_status pa_rope_and_cache_fp8(void* query_out, const void* query, const void* key,
                                const void* value, int64_t query_stride, int64_t key_stride,
                                int64_t value_stride, void* key_cache, void* value_cache,
                                const int32_t* slot_mapping, const int64_t* positions,
                                int32_t num_axes, const int32_t* pair_axes, const float* inv_freq,
                                int32_t rot_dim, int32_t interleaved, int32_t num_tokens,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                                int32_t block_size, int32_t num_blocks, pa_dtype dtype, float k_scale,
                                float v_scale, int32_t* status_dev, pa_stream stream) {
    pa::RopeParams p = rope_params(query_out, query, key, value, query_stride, key_stride, value_stride,
                                   key_cache, value_cache, slot_mapping, positions, inv_freq, rot_dim,
                                   interleaved, num_tokens, num_q_heads, num_kv_heads, head_size,
                                   block_size, num_blocks, status_dev);
    return run_rope(p, pair_axes, num_axes, dtype, true, k_scale, v_scale, (cudaStream_t)stream);
}

pa_status pa_move_blocks(void* const* key_caches, void* const* value_caches, int32_t num_layers,
                         const int32_t* block_pairs, int32_t num_pairs, int32_t* block_tables,
                         int32_t num_rows, int32_t max_blocks_per_seq, int32_t num_kv_heads,
                         int32_t head_size, int32_t block_size, int32_t num_blocks, pa_dtype dtype,
                         int32_t* status_dev, pa_stream stream) {
    if (num_layers < 0 || num_pairs < 0 || num_kv_heads <= 0 || head_size <= 0 || block_size <= 0 ||
        num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "move_blocks: sizes must be positive");
    if (block_tables && (num_rows < 0 || max_blocks_per_seq <= 0))
        return fail(PA_ERR_INVALID_ARG, "move_blocks: block_tables need num_rows >= 0 and max_blocks_per_seq > 0");
    if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_FP8_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "move_blocks: dtype");
    if (num_pairs > num_blocks)
        return fail(PA_ERR_INVALID_ARG, "move_blocks: %d pairs in a pool of %d blocks", num_pairs, num_blocks);
    if (num_pairs == 0) return ok();
    if (!block_pairs || (num_layers > 0 && (!key_caches || !value_caches)))
        return fail(PA_ERR_INVALID_ARG, "move_blocks: null pointer");
    const int64_t bytes = (int64_t)num_kv_heads * block_size * head_size * (dtype == PA_FP8_E4M3 ? 1 : 2);
    if (bytes % 16) return fail(PA_ERR_INVALID_ARG, "move_blocks: blocks must be 16-byte multiples");
    for (int32_t l = 0; l < num_layers; ++l) {
        if (!key_caches[l] || !value_caches[l]) return fail(PA_ERR_INVALID_ARG, "move_blocks: null pool");
        if (!aligned16(key_caches[l]) || !aligned16(value_caches[l]))
            return fail(PA_ERR_INVALID_ARG, "move_blocks: pools must be 16-byte aligned");
    }
    pa::MoveParams p;
    std::memset(&p, 0, sizeof(p));
    p.pairs = block_pairs;
    p.num_pairs = num_pairs;
    p.num_blocks = num_blocks;
    p.vecs_per_block = bytes / 16;
    p.status = status_dev;
    // the first launch also rewrites the tables and reports bad pairs; without a pool there
    // is still that to do
    int32_t l0 = 0;
    do {
        p.num_layers = std::min(num_layers - l0, pa::kMoveLayers);
        for (int32_t l = 0; l < p.num_layers; ++l) {
            p.key[l] = key_caches[l0 + l];
            p.value[l] = value_caches[l0 + l];
        }
        p.report = l0 == 0;
        p.block_tables = l0 == 0 ? block_tables : nullptr;
        p.num_entries = l0 == 0 && block_tables ? (int64_t)num_rows * max_blocks_per_seq : 0;
        cudaError_t e = pa::launch_move_blocks(p, (cudaStream_t)stream);
        if (e != cudaSuccess) return cuda_fail(e, "move_blocks launch");
        l0 += p.num_layers;
    } while (l0 < num_layers);
    return ok();
}

}  // extern "C"
