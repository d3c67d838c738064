// Attention of trees of new tokens over fp8 E4M3 caches (head_size 128), fp16 or bf16 queries.
#include "pa_prefill_launch.cuh"

namespace pa {

cudaError_t launch_tree_fp8(bool q_bf16, const CUtensorMap& qmap, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, const PrefillParams& p, cudaStream_t stream) {
    if (q_bf16)
        return p.block_size == 16
                   ? launch_prefill_one<pf::Cfg<false, true, 128, 16, true, true>>(qmap, kmap, vmap, p, stream)
                   : launch_prefill_one<pf::Cfg<false, true, 128, 32, true, true>>(qmap, kmap, vmap, p, stream);
    return p.block_size == 16
               ? launch_prefill_one<pf::Cfg<false, false, 128, 16, true, true>>(qmap, kmap, vmap, p, stream)
               : launch_prefill_one<pf::Cfg<false, false, 128, 32, true, true>>(qmap, kmap, vmap, p, stream);
}

}  // namespace pa
