// Paged decode attention over binary16 caches, of the slots behind a prefix that is
// attended to elsewhere (gemv_attn.cuh).
#include "gemv_attn.cuh"

namespace mbg {

cudaError_t launch_attn_own_f16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s)
{
    return attn::launch<__half, true, true>(a, vec, nt, big, sm_count, s);
}

}  // namespace mbg
