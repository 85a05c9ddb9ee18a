// Paged decode attention over binary16 caches (gemv_attn.cuh), and the
// accumulation of the weights, which does not depend on the cache's type.
#include "gemv_attn.cuh"

namespace mbg {

cudaError_t launch_attn_f16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s)
{
    return attn::launch<__half>(a, vec, nt, big, sm_count, s);
}

// scores_out[b, h, t] = scores_in[b, h, t] + sum over the group's query heads
// of 2^(logit - log2 denominator).  The logits were left by the attention
// kernel (4 bytes per query head and token against the 4 D bytes of K and V);
// recomputing them would read K again.  One thread per token; the sum runs
// over the heads in order.
__global__ void __launch_bounds__(256) mbg_attn_weights_kernel(const __grid_constant__ AttnArgs a, int tile_heads)
{
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.z, h = blockIdx.y;
    const attn::RowSpan span = attn::row_span(a, b);
    const int64_t out_row = (static_cast<int64_t>(b) * a.kv.kv_heads + h) * a.kv.capacity;
    for (int slot = span.first + blockIdx.x * 256 + threadIdx.x; slot < span.len; slot += gridDim.x * 256) {
        float sum = 0.f;
        for (int ht = 0; ht < a.head_tiles; ++ht) {
            const int64_t row = (static_cast<int64_t>(b) * a.kv.kv_heads + h) * a.head_tiles + ht;
            const float *lg = a.logits + (row * a.kv.capacity + slot) * a.logit_heads;
            const float *lse = a.row_lse + row * tile_heads;
            const int heads = min(tile_heads, a.group - ht * tile_heads);
            for (int i = 0; i < heads; i += 2) {
                const float2 x = __ldcg(reinterpret_cast<const float2 *>(lg + i));
                sum += attn::exp2_approx(x.x - __ldg(lse + i));
                if (i + 1 < heads) sum += attn::exp2_approx(x.y - __ldg(lse + i + 1));
            }
        }
        a.scores_out[out_row + slot] = a.scores_in[out_row + slot] + sum;
    }
}

cudaError_t launch_attn_weights(const AttnArgs &a, int nt, cudaStream_t s)
{
    int64_t longest = a.kv.capacity;
    if (a.window > 0 && a.window < longest) longest = a.window;
    int64_t x = (longest + 255) / 256;
    if (x > 512) x = 512;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(x), static_cast<unsigned>(a.kv.kv_heads), static_cast<unsigned>(a.kv.batch));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mbg_attn_weights_kernel, a, 8 * nt);
}

}  // namespace mbg
