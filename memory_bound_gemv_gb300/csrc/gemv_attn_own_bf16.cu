// Paged decode attention over bfloat16 caches, of the slots behind a prefix that is
// attended to elsewhere (gemv_attn.cuh).
#include "gemv_attn.cuh"

namespace mbg {

cudaError_t launch_attn_own_bf16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s)
{
    return attn::launch<__nv_bfloat16, true, true>(a, vec, nt, big, sm_count, s);
}

}  // namespace mbg
