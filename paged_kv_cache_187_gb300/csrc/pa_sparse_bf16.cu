// Attention over selected blocks of caches of the queries' own type, bf16.
#include "pa_sparse.cuh"

namespace pa {

cudaError_t launch_sparse_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                            const SparseParams& sp, int32_t head_size, int32_t ctas,
                            cudaStream_t stream, int32_t* per_sm) {
    return launch_sparse_16<true>(kmap, vmap, p, sp, head_size, ctas, stream, per_sm);
}

}  // namespace pa
