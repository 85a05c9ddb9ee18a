// Tiled attention of many tokens over binary16 caches (gemv_tile.cuh).
#include "gemv_tile.cuh"

namespace mbg {

cudaError_t launch_tile_f16(const SpanArgs &a, bool vec, int ctas, cudaStream_t s) { return tile::launch<__half>(a, vec, ctas, s); }

}  // namespace mbg
