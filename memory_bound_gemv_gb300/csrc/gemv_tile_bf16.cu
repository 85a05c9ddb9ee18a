// Tiled attention of many tokens over bfloat16 caches (gemv_tile.cuh).
#include "gemv_tile.cuh"

namespace mbg {

cudaError_t launch_tile_bf16(const SpanArgs &a, bool vec, int ctas, cudaStream_t s) { return tile::launch<__nv_bfloat16>(a, vec, ctas, s); }

}  // namespace mbg
