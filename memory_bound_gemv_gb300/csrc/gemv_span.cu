// Attention of many tokens: what follows the tiles (gemv_tile.cuh).
//
// Blocks of rows that several CTAs shared are joined from their parts, in the
// order of their slots.  And rows are computed one by one where a tile cannot:
// in the value product a weight of 0 meets the values that other rows of the tile
// see and this one does not, and 0 times an infinite value is NaN.  Rows with a
// NaN are therefore computed again, each for itself, slot by slot, in FP32.
//
// A block takes such a row.  Its warps share the slots 32 at a time: a lane forms
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

// Sixteen rows of a block that was cut: thread (g, r) = (t / 16, t % 16) sums
// every eighth run of four elements of row r.
constexpr int kJoinRows = 16, kJoinGroups = kThreads / kJoinRows;

struct JoinShared {
    int slot[kSpanMaxCtas + 1];
    int count[kWarps];
    float m[kSpanMaxCtas + 1][kJoinRows];
    int bad[kJoinRows];
};

template <int E>
__device__ void join_rows(const SpanArgs &a, Shared &sh, JoinShared &js, int ctas, int c0, int stream, int r16)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, dim = a.kv.dim;
    const SpanInfo first = a.info[2 * c0 + 1];
    if (first.tiles == 0) return;
    const span::Seq s = span::seq_of(a, first.b, false);
    const int row0 = first.row0 + stream * kSpanRows + r16 * kJoinRows;
    const int rows = s.m * a.group;
    if (row0 >= rows || (stream > 0 && row0 >= first.row0 + span_streams(dim) * kSpanRows)) return;
    // the parts behind the first: those of later CTAs that begin with this block
    int parts = 1;
    if (tid == 0) js.slot[0] = 2 * c0 + 1;
    for (int c = c0 + 1; c < ctas; c += kThreads) {
        bool mine = false;
        if (c + tid < ctas) {
            const SpanInfo i = a.info[2 * (c + tid)];
            mine = i.tiles > 0 && i.b == first.b && i.h == first.h && i.row0 == first.row0;
        }
        const unsigned vote = __ballot_sync(kFull, mine);
        __syncthreads();
        if (lane == 0) js.count[warp] = __popc(vote);
        __syncthreads();
        int at = parts;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += js.count[w];
            parts += js.count[w];
        }
        if (mine) js.slot[at + __popc(vote & ((1u << lane) - 1))] = 2 * (c + tid);
    }
    if (tid < kJoinRows) js.bad[tid] = 0;
    __syncthreads();
    const int64_t half = a.part_stride / span_streams(dim);
    const int stat = (dim + 15) / 16 * 16 * kSpanRows, in = r16 * kJoinRows;
    for (int i = tid; i < parts * kJoinRows; i += kThreads) {
        const int p = i / kJoinRows, r = i - p * kJoinRows;
        js.m[p][r] = __ldcg(a.part + js.slot[p] * a.part_stride + stream * half + stat + in + r);
    }
    __syncthreads();
    const int r = tid % kJoinRows, g = tid / kJoinRows, row = row0 + r;
    float top = -INFINITY, sum = 0.f;
    for (int p = 0; p < parts; ++p) top = fmaxf(top, js.m[p][r]);
    for (int p = 0; p < parts; ++p)
        sum += exp2_from(js.m[p][r], top) * __ldcg(a.part + js.slot[p] * a.part_stride + stream * half + stat + kSpanRows + in + r);
    const bool live = row < rows;
    const int token = s.q0 + (live ? row / a.group : 0), head = first.h * a.group + (live ? row % a.group : 0);
    const int64_t index = static_cast<int64_t>(token) * a.q_heads + head;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int d = 4 * g; d < dim; d += 4 * kJoinGroups) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(
                a.part + js.slot[p] * a.part_stride + stream * half + (static_cast<int64_t>(d / 4) * kSpanRows + in + r) * 4));
            const float f = exp2_from(js.m[p][r], top);
            v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
        }
        const float w[4] = {v.x, v.y, v.z, v.w};
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (d + k >= dim) continue;
            if (w[k] != w[k] && sum == sum) js.bad[r] = 1;
            if (a.pre)
                a.pre[index * (dim + 2) + d + k] = w[k];
            else
                elem_store1<E>(a.out, token * a.o_st + head * a.o_sh + d + k, w[k] * inv);
        }
    }
    if (live && g == 0) {
        if (a.pre) {
            a.pre[index * (dim + 2) + dim] = top;
            a.pre[index * (dim + 2) + dim + 1] = sum;
        } else if (a.lse) {
            a.lse[index] = sum > 0.f || sum != sum ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
        }
    }
    __syncthreads();
    for (int i = 0; i < kJoinRows; ++i)
        if (js.bad[i]) one_row<E>(a, sh, s.q0 + (row0 + i) / a.group, first.h * a.group + (row0 + i) % a.group);
    __syncthreads();
}

// The joins of all cut blocks, then the rows to be computed one by one.
template <int E>
__global__ void __launch_bounds__(kThreads) mbg_span_finish_kernel(const __grid_constant__ SpanArgs a, int ctas)
{
    __shared__ Shared sh;
    __shared__ JoinShared js;
    pdl_trigger();
    pdl_wait();
    constexpr int kGroups = kSpanRows / kJoinRows;
    const int streams = span_streams(a.kv.dim), tasks = ctas * streams * kGroups;
    for (int i = blockIdx.x; i < tasks; i += gridDim.x)
        join_rows<E>(a, sh, js, ctas, i / (streams * kGroups), i / kGroups % streams, i % kGroups);
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kThreads; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * kThreads) {
        const bool again = r0 + threadIdx.x < rows && __ldcg(a.redo + r0 + threadIdx.x) == 1;
        if (!__syncthreads_or(again)) continue;
        for (int w = 0; w < kWarps; ++w) {
            if (threadIdx.x / 32 == w) {
                const unsigned vote = __ballot_sync(kFull, again);
                if (threadIdx.x % 32 == 0) js.count[0] = static_cast<int>(vote);
            }
            __syncthreads();
            const unsigned vote = static_cast<unsigned>(js.count[0]);
            __syncthreads();
            for (int i = 0; i < 32; ++i)
                if (vote >> i & 1) {
                    const int64_t r = r0 + w * 32 + i;
                    one_row<E>(a, sh, static_cast<int>(r / a.q_heads), static_cast<int>(r % a.q_heads));
                }
        }
    }
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

template <typename F, typename... Args>
static cudaError_t launch_blocks(F fn, int64_t blocks, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

cudaError_t launch_span(const SpanArgs &a, bool vec, int elem, int sm_count, cudaStream_t s)
{
    const bool f16 = elem == GEMV_ELEM_F16;
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads, most = static_cast<int64_t>(sm_count) * 16;
    // a scale of 0 (or none) leaves the tiles no maximum to go by
    if (!(fabsf(a.scale_log2) > 0.f && fabsf(a.scale_log2) < INFINITY))
        return launch_blocks(f16 ? mbg_span_rows_kernel<GEMV_ELEM_F16> : mbg_span_rows_kernel<GEMV_ELEM_BF16>, rows < most ? rows : most, s, a);
    const int ctas = sm_count < kSpanMaxCtas ? sm_count : kSpanMaxCtas;
    const cudaError_t e = f16 ? launch_tile_f16(a, vec, ctas, s) : launch_tile_bf16(a, vec, ctas, s);
    if (e != cudaSuccess) return e;
    const int64_t tasks = static_cast<int64_t>(ctas) * span_streams(a.kv.dim) * (kSpanRows / kJoinRows);
    return launch_blocks(f16 ? mbg_span_finish_kernel<GEMV_ELEM_F16> : mbg_span_finish_kernel<GEMV_ELEM_BF16>, tasks, s, a, ctas);
}

}  // namespace mbg
