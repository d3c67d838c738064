// Chunk attention over caches of the queries' own type, f16.
#include "pa_prefill_launch.cuh"

namespace pa {

cudaError_t launch_prefill_f16(const CUtensorMap& qmap, const CUtensorMap& kmap,
                              const CUtensorMap& vmap, const PrefillParams& p, cudaStream_t stream) {
    if (p.head_size == 128)
        return p.block_size == 16
                   ? launch_prefill_one<pf::Cfg<false, false, 128, 16, false>>(qmap, kmap, vmap, p, stream)
                   : launch_prefill_one<pf::Cfg<false, false, 128, 32, false>>(qmap, kmap, vmap, p, stream);
    return p.block_size == 16
               ? launch_prefill_one<pf::Cfg<false, false, 64, 16, false>>(qmap, kmap, vmap, p, stream)
               : launch_prefill_one<pf::Cfg<false, false, 64, 32, false>>(qmap, kmap, vmap, p, stream);
}

}  // namespace pa
