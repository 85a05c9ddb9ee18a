// Attention of many tokens, row by row: each row (a token's query head) for
// itself, slot by slot, in FP32.
//
// A block takes a row.  Its warps share the slots 32 at a time: a lane forms
// the score of one slot, the warp keeps a running maximum and sum, and adds the
// values weighted; the warps are joined at the end.  Nothing that a row does
// not see is read, so that infinities and NaN there leave no trace.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"
#include "gemv_elem.cuh"
#include "gemv_span.cuh"

namespace mbg {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kMaxDim = 256, kOwn = kMaxDim / 32;
constexpr unsigned kFull = 0xFFFFFFFFu;

struct Shared {
    float q[kMaxDim];
    float o[kWarps][kMaxDim];
    float m[kWarps], l[kWarps];
};

__device__ __forceinline__ float exp2_from(float x, float m)
{
    return exp2f(x - (m == -INFINITY ? 0.f : m));
}

// The sequence that token t belongs to; -1: none.
__device__ int seq_of_token(const SpanArgs &a, int t)
{
    if (a.prefix) return 0;
    int lo = 0, hi = a.kv.batch;  // the last b with starts[b] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (mid < a.kv.batch && __ldg(a.starts + mid) <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <int E>
__device__ void one_row(const SpanArgs &a, Shared &sh, int token, int head)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dim = a.kv.dim;
    if (a.kv.batch == 0) return;
    const span::Seq s = span::seq_of(a, seq_of_token(a, token), false);
    if (token < s.q0 || token >= s.q0 + s.m) return;
    const span::Seen seen = span::seen_by(a, s, token - s.q0);
    const KvView &kv = a.kv;
    const int h = head / a.group;
    for (int d = threadIdx.x; d < dim; d += kThreads)
        sh.q[d] = elem_load1<E>(a.q, token * a.q_st + head * a.q_sh + d);
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) o[i] = 0.f;
    const int sinks = min(a.sinks, min(seen.lo, seen.hi));
    const int64_t count = static_cast<int64_t>(sinks) + max(0, seen.hi - seen.lo);
    const int32_t *table = kv.table + s.b * kv.table_stride;
    for (int64_t i0 = warp * 32; i0 < count; i0 += kThreads) {
        const int64_t i = i0 + lane;
        const int slot = static_cast<int>(i < sinks ? i : seen.lo + (i - sinks));
        int page = -1, off = 0;
        if (i < count) {
            const int idx = slot / kv.page_size;
            off = slot - idx * kv.page_size;
            page = __ldg(table + idx);
            if (page < 0 || page >= kv.num_pages) {
                report_error(a.err, DEVERR_BAD_INDEX);
                page = -1;
            }
        }
        float x = -INFINITY;
        if (page >= 0) {
            const int64_t at = page * kv.ks_page + off * kv.ks_tok + h * kv.ks_head;
            float sum = 0.f;
            for (int d = 0; d < dim; ++d) sum += sh.q[d] * elem_load1<E>(kv.k, at + d);
            x = sum * a.scale_log2;
        }
        float top = x;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, k));
        const float mm = fmaxf(m, top), fix = exp2_from(m, mm), p = exp2_from(x, mm);
        float sum = p;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) sum += __shfl_xor_sync(kFull, sum, k);
        l = l * fix + sum;
        m = mm;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) o[k] *= fix;
        const int n = static_cast<int>(min(static_cast<int64_t>(32), count - i0));
        for (int k = 0; k < n; ++k) {
            const int pg = __shfl_sync(kFull, page, k), of = __shfl_sync(kFull, off, k);
            const float w = __shfl_sync(kFull, p, k);
            if (pg < 0) continue;
            const int64_t at = pg * kv.vs_page + of * kv.vs_tok + h * kv.vs_head;
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
                if (lane + 32 * j < dim) o[j] += w * elem_load1<E>(kv.v, at + lane + 32 * j);
        }
    }
    if (lane == 0) sh.m[warp] = m, sh.l[warp] = l;
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.m[w]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh.l[w] * exp2_from(sh.m[w], top);
    const float fix = exp2_from(m, top);
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        if (lane + 32 * j < dim) sh.o[warp][lane + 32 * j] = o[j] * fix;
    __syncthreads();
    const int64_t row = static_cast<int64_t>(token) * a.q_heads + head;
    for (int d = threadIdx.x; d < dim; d += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sh.o[w][d];
        if (a.pre)
            a.pre[row * (dim + 2) + d] = v;
        else
            elem_store1<E>(a.out, token * a.o_st + head * a.o_sh + d, sum == 0.f ? 0.f : v / sum);
    }
    if (threadIdx.x == 0) {
        if (a.pre) {
            a.pre[row * (dim + 2) + dim] = top;
            a.pre[row * (dim + 2) + dim + 1] = sum;
        } else if (a.lse) {
            a.lse[row] = sum > 0.f || sum != sum ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
        }
    }
    __syncthreads();
}

template <int E>
__global__ void __launch_bounds__(kThreads) mbg_span_rows_kernel(const __grid_constant__ SpanArgs a)
{
    __shared__ Shared sh;
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < (a.prefix ? 1 : a.kv.batch); b += kThreads) span::seq_of(a, b, true);
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        one_row<E>(a, sh, static_cast<int>(r / a.q_heads), static_cast<int>(r % a.q_heads));
}

}  // namespace

cudaError_t launch_span(const SpanArgs &a, bool vec, int elem, int sm_count, cudaStream_t s)
{
    (void)vec;
    cudaLaunchConfig_t cfg = {};
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads;
    const int64_t most = static_cast<int64_t>(sm_count) * 16;
    cfg.gridDim = dim3(static_cast<unsigned>(rows < most ? rows : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, elem == GEMV_ELEM_F16 ? mbg_span_rows_kernel<GEMV_ELEM_F16> : mbg_span_rows_kernel<GEMV_ELEM_BF16>, a);
}

}  // namespace mbg
