// Attention over selected blocks of fp8 E4M3 caches (head_size 128), fp16 or bf16 queries: on the
// tensor cores, two 16-token blocks to a tile, as the decode.
#include "pa_sparse.cuh"

namespace pa {

namespace {

template <bool BF16>
cudaError_t launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p, const SparseParams& sp,
                   int32_t ctas, cudaStream_t stream, int32_t* per_sm) {
    if (sp.block_size == 16)
        return p.group <= 8 ? launch_sparse_one<128, 16, BF16, true, 8, true, 2>(kmap, vmap, p, sp, ctas, stream, per_sm)
                            : launch_sparse_one<128, 16, BF16, true, 16, true, 2>(kmap, vmap, p, sp, ctas, stream, per_sm);
    return p.group <= 8 ? launch_sparse_one<128, 32, BF16, true, 8, true, 1>(kmap, vmap, p, sp, ctas, stream, per_sm)
                        : launch_sparse_one<128, 32, BF16, true, 16, true, 1>(kmap, vmap, p, sp, ctas, stream, per_sm);
}

}  // namespace

cudaError_t launch_sparse_fp8(bool q_bf16, const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                              const SparseParams& sp, int32_t ctas, cudaStream_t stream, int32_t* per_sm) {
    return q_bf16 ? launch<true>(kmap, vmap, p, sp, ctas, stream, per_sm)
                  : launch<false>(kmap, vmap, p, sp, ctas, stream, per_sm);
}

}  // namespace pa
