// Paged decode attention over binary16 caches (gemv_attn.cuh), and the
// accumulation of the weights, which does not depend on the cache's type.
#include "gemv_attn.cuh"

namespace mbg {

cudaError_t launch_attn_f16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s)
{
    return attn::launch<__half, false, false>(a, vec, nt, big, sm_count, s);
}

// scores_out[b, h, t] = scores_in[b, h, t] + sum over the group's query heads
// of 2^(logit - log2 denominator).  The logits were left by the attention
// kernel (4 bytes per query head and token against the 4 D bytes of K and V);
// recomputing them would read K again.  Bound by latency more than by those
// bytes: a thread takes four tokens of a row, all their logits requested at
// once.  The sum runs over the heads in order.
constexpr int kTokens = 4;

template <int VEC>
__global__ void __launch_bounds__(256) mbg_attn_weights_kernel(const __grid_constant__ AttnArgs a, int tile_heads)
{
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.z, h = blockIdx.y;
    const attn::RowSpan span = attn::row_span<16>(a, b);
    const int64_t out_row = (static_cast<int64_t>(b) * a.kv.kv_heads + h) * a.kv.capacity;
    const int step = gridDim.x * 256 * kTokens;
    // the first blocks take the sinks, and then their share of the others
    for (int s = blockIdx.x * 256 + threadIdx.x; s < span.sinks; s += gridDim.x * 256) {
        float sum = a.scores_in[out_row + s];
        for (int i = 0; i < a.group; ++i) {
            const int64_t row = (static_cast<int64_t>(b) * a.kv.kv_heads + h) * a.head_tiles + i / tile_heads;
            const int k = i % tile_heads;
            sum += attn::exp2_approx(__ldcg(a.logits + (row * a.kv.capacity + s) * a.logit_heads + k) -
                                     __ldg(a.row_lse + row * tile_heads + k));
        }
        a.scores_out[out_row + s] = sum;
    }
    // (a step behind the last slot may lie beyond 2^31)
    for (int64_t s0 = span.first + blockIdx.x * 256 * kTokens + threadIdx.x; s0 < span.len; s0 += step) {
        float sum[kTokens], old[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            sum[k] = 0.f;
            old[k] = s0 + 256 * k < span.len ? a.scores_in[out_row + s0 + 256 * k] : 0.f;
        }
        for (int ht = 0; ht < a.head_tiles; ++ht) {
            const int64_t row = (static_cast<int64_t>(b) * a.kv.kv_heads + h) * a.head_tiles + ht;
            const float *lg = a.logits + (row * a.kv.capacity + s0) * a.logit_heads;
            const float *lse = a.row_lse + row * tile_heads;
            const int heads = min(tile_heads, a.group - ht * tile_heads);
            for (int i = 0; i < heads; i += VEC) {
                float x[kTokens][VEC], d[VEC];
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    if (s0 + 256 * k >= span.len) continue;
                    const float *p = lg + 256 * k * a.logit_heads + i;
                    if (VEC == 4) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p));
                        x[k][0] = v.x, x[k][1] = v.y, x[k][VEC - 2] = v.z, x[k][VEC - 1] = v.w;
                    } else {
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(p));
                        x[k][0] = v.x, x[k][1] = v.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) d[j] = __ldg(lse + i + j);
#pragma unroll
                for (int k = 0; k < kTokens; ++k)
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        if (s0 + 256 * k < span.len && i + j < heads) sum[k] += attn::exp2_approx(x[k][j] - d[j]);
            }
        }
#pragma unroll
        for (int k = 0; k < kTokens; ++k)
            if (s0 + 256 * k < span.len) a.scores_out[out_row + s0 + 256 * k] = old[k] + sum[k];
    }
}

cudaError_t launch_attn_weights(const AttnArgs &a, int nt, cudaStream_t s)
{
    int64_t longest = a.kv.capacity;
    if (a.window > 0 && a.window < longest) longest = a.window;
    int64_t x = (longest + 256 * kTokens - 1) / (256 * kTokens);
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
    return cudaLaunchKernelEx(&cfg, a.logit_heads % 4 == 0 ? mbg_attn_weights_kernel<4> : mbg_attn_weights_kernel<2>, a,
                              8 * nt);
}

}  // namespace mbg
