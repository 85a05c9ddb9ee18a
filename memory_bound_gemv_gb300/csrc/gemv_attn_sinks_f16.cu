// Paged decode attention over binary16 caches, with first slots that stay visible
// (gemv_attn.cuh).
#include "gemv_attn.cuh"

namespace mbg {

cudaError_t launch_attn_sinks_f16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s)
{
    return attn::launch<__half, true, false>(a, vec, nt, big, sm_count, s);
}

}  // namespace mbg
