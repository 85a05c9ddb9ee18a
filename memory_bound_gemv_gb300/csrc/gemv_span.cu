// Attention of many tokens: what follows the tiles (gemv_tile.cuh).
//
// Blocks of rows that several CTAs shared are joined from their parts, in the
// order of their slots; rows behind a shared prefix with what their own slots
// give.  Bound by round trips: what parts there are, the rows' maxima and sums
// and their O, requested together for several parts; 11 us behind the tiles of a
// prompt of 9001 tokens, whose 150 cut blocks have 40 MB of parts.  And rows are computed one by one where a tile cannot:
// in the value product a weight of 0 meets the values that other rows of the tile
// see and this one does not, and 0 times an infinite value is NaN.  Rows with a
// NaN are therefore computed again, each for itself, slot by slot, in FP32.  So are
// rows that saw a page that does not exist.  That is slow: a prompt of 9001 tokens with a
// window of 2048 takes some 240 ms where all its rows are computed so, and a row that
// is joined from parts is computed once for each run of its elements that is written.
//
// A block takes such a row.  Its warps share the slots 32 at a time: a lane forms
// the score of one slot, the warp keeps a running maximum and sum, and adds the
// values weighted; the warps are joined at the end.  Nothing that a row does
// not see is read, so that infinities and NaN there leave no trace.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "gemv_decode.h"
#include "gemv_device.cuh"
#include "gemv_elem.cuh"
#include "gemv_span.cuh"

namespace mbg {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32, kMaxDim = 256, kOwn = kMaxDim / 32;
constexpr int kPiece = 1024;  // slots of a warp that are summed up before they join the others
constexpr unsigned kFull = 0xFFFFFFFFu;

struct Shared {
    float q[kMaxDim];
    float o[kWarps][kMaxDim];
    float m[kWarps], l[kWarps];
    int first[kWarps];
};

__device__ __forceinline__ float exp2_from(float x, float m)
{
    return exp2f(x - (m == -INFINITY ? 0.f : m));
}

__device__ __forceinline__ float lse_of(float m, float l)
{
    return l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// What a prefix and the slots behind it give together: factors of their O.
struct Both {
    float pre, own, m, l;
};
__device__ __forceinline__ Both both_of(const SpanArgs &a, int64_t index, float m, float l)
{
    const float *stat = a.own + (index + 1) * span_row(a.kv.dim) - 4;
    const float m2 = __ldcg(stat), l2 = __ldcg(stat + 1);
    Both r;
    r.m = fmaxf(m, m2);
    r.pre = exp2_from(m, r.m);
    r.own = l2 == 0.f ? 0.f : exp2_from(m2, r.m);  // (its O may not be there)
    r.l = l * r.pre + (l2 == 0.f ? 0.f : l2 * r.own);
    const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
    r.pre *= inv;
    r.own = l2 == 0.f ? 0.f : r.own * inv;
    return r;
}

// Whether the starts ascend (the whole block asks).
__device__ bool ascending(const SpanArgs &a)
{
    bool falls = false;
    for (int b = threadIdx.x; b < a.kv.batch; b += kThreads) falls = falls || __ldg(a.starts + b + 1) < __ldg(a.starts + b);
    return !__syncthreads_or(falls);
}

// The sequence that token t belongs to, if any does; -1: none does (the whole
// block asks).
__device__ int seq_of_token(const SpanArgs &a, Shared &sh, int t, bool ascend)
{
    if (a.prefix) return 0;
    const int batch = a.kv.batch, tid = threadIdx.x;
    if (ascend) {
        int lo = 0, hi = batch;  // the last b with starts[b] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (mid < batch && __ldg(a.starts + mid) <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    }
    // The first start or end above t is the sequence's end, and no start before the
    // sequence's lies above its own (span::seq_behind).
    int first = batch + 1;
    for (int i = tid; i <= batch && first > batch; i += kThreads)
        if (__ldg(a.starts + i) > t) first = i;
    first = __reduce_min_sync(kFull, first);
    __syncthreads();
    if (tid % 32 == 0) sh.first[tid / 32] = first;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) first = min(first, sh.first[w]);
    const int b = first > batch ? -1 : first - 1;
    bool above = false;
    for (int i = tid; i < b; i += kThreads) above = above || __ldg(a.starts + i) > __ldg(a.starts + b);
    return __syncthreads_or(above) ? -1 : b;
}

// (the whole block)
template <int E>
__device__ void one_row(const SpanArgs &a, Shared &sh, const span::Seq &s, int token, int head, int d0, int d1, bool joined)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dim = a.kv.dim;
    if (token < s.q0 || token >= s.q0 + s.m) return;
    const span::Seen seen = span::seen_by(a, s, token - s.q0);
    const KvView &kv = a.kv;
    const int h = head / a.group;
    for (int d = threadIdx.x; d < dim; d += kThreads)
        sh.q[d] = elem_load1<E>(a.q, token * a.q_st + head * a.q_sh + d);
    __syncthreads();
    // l and o: of the last kPiece slots that the warp has had at most; before: of those
    // ahead of them.  FP32 sums of 2^17 like values are off by far more than a step
    // of the output; of kPiece, and of so many pieces, they are not.
    float m = -INFINITY, l = 0.f, l_before = 0.f, o[kOwn], before[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) o[i] = before[i] = 0.f;
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
        l_before *= fix;
        l = l * fix + sum;
        m = mm;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) o[k] *= fix, before[k] *= fix;
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
        if ((i0 / kThreads + 1) % (kPiece / 32) == 0) {
            l_before += l;
            l = 0.f;
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                before[k] += o[k];
                o[k] = 0.f;
            }
        }
    }
    l += l_before;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) o[k] += before[k];
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
    // (the prefix of all rows: left for the joins; of a row that a join has sent here:
    // joined at once)
    Both f = {sum == 0.f ? 0.f : 1.f / sum, 0.f, top, sum};
    if (a.own && joined) f = both_of(a, row, top, sum);
    for (int d = d0 + threadIdx.x; d < d1; d += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sh.o[w][d];
        if (a.pre && !joined) {
            a.pre[row * span_row(dim) + d] = v;
            continue;
        }
        v *= f.pre;
        if (f.own != 0.f) v += __ldcg(a.own + row * span_row(dim) + d) * f.own;
        elem_store1<E>(a.out, token * a.o_st + head * a.o_sh + d, v);
    }
    if (threadIdx.x == 0 && joined) {  // the sums may differ from those of the tiles (a page that does not exist)
        if (d0 == 0 && a.lse) a.lse[row] = lse_of(f.m, f.l);
    } else if (threadIdx.x == 0) {
        if (a.pre) {
            a.pre[(row + 1) * span_row(dim) - 4] = top;
            a.pre[(row + 1) * span_row(dim) - 3] = sum;
        } else if (a.lse) {
            a.lse[row] = lse_of(top, sum);
        }
    }
    __syncthreads();
}

// A task joins a run of elements of all rows of a block, a thread per row: a warp
// reads 512 bytes of a part at a time, and has those of several parts under
// way.  Cut prompts: 16 elements of some two parts each; prefix: few blocks in many
// parts, four elements of eight parts at once.
constexpr int kPromptRun = 16, kPrefixRun = 4;
constexpr int kMaxParts = kSpanMaxCtas + 1;

struct JoinShared {
    int slot[kMaxParts];
    int count[kWarps];
    unsigned bad[kWarps];
};

// What the tiles have left of their parts, read once per block.
struct Parts {
    SpanInfo info[2 * kSpanMaxCtas];
    __device__ void read(const SpanArgs &a, int ctas)
    {
        constexpr int kMost = (2 * kSpanMaxCtas * sizeof(SpanInfo) / 16 + kThreads - 1) / kThreads;
        const int words = 2 * ctas * static_cast<int>(sizeof(SpanInfo)) / 16;
        uint4 w[kMost];
#pragma unroll
        for (int k = 0; k < kMost; ++k)
            if (threadIdx.x + k * kThreads < words) w[k] = __ldcg(reinterpret_cast<const uint4 *>(a.info) + threadIdx.x + k * kThreads);
#pragma unroll
        for (int k = 0; k < kMost; ++k)
            if (threadIdx.x + k * kThreads < words) reinterpret_cast<uint4 *>(info)[threadIdx.x + k * kThreads] = w[k];
        __syncthreads();
    }
};
static_assert(sizeof(SpanInfo) * 2 % 16 == 0, "");

// The numbers i < n for which f(i), in order, in list (no more than `most`).
template <typename F>
__device__ int collect(int n, int *list, int most, int *count, F f)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int have = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        const bool mine = i < n && f(i);
        const unsigned vote = __ballot_sync(kFull, mine);
        __syncthreads();
        if (lane == 0) count[warp] = __popc(vote);
        __syncthreads();
        int at = have;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += count[w];
            have += count[w];
        }
        at += __popc(vote & ((1u << lane) - 1));
        if (mine && at < most) list[at] = i;
    }
    __syncthreads();
    return min(have, most);
}

// A run of a row's output, from d on.
template <int E, int kRun>
__device__ __forceinline__ void store_run(const SpanArgs &a, int token, int head, int d, const float (&v)[kRun])
{
    uint16_t *to = static_cast<uint16_t *>(a.out) + token * a.o_st + head * a.o_sh + d;
    if (a.out_vec && d + kRun <= a.kv.dim) {
        uint32_t w[kRun / 2];
#pragma unroll
        for (int k = 0; k < kRun / 2; ++k) w[k] = elem_pack2<E>(v[2 * k], v[2 * k + 1]);
#pragma unroll
        for (int k = 0; k < kRun / 4; ++k) reinterpret_cast<uint2 *>(to)[k] = make_uint2(w[2 * k], w[2 * k + 1]);
    } else {
#pragma unroll
        for (int k = 0; k < kRun; ++k)
            if (d + k < a.kv.dim) elem_store1<E>(to, k, v[k]);
    }
}

// Run `run` of the rows of the block of cached head h that begins at row0 of
// sequence b's rows.
template <int E, int kRun, int kAtOnce>
__device__ void join_run(const SpanArgs &a, unsigned char *raw, const Parts &left, int ctas, int b, int h, int row0, int run)
{
    JoinShared &js = *reinterpret_cast<JoinShared *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, dim = a.kv.dim, d = run * kRun;
    const span::Seq s = span::seq_of(a, b, false);
    const int parts = collect(2 * ctas, js.slot, kMaxParts, js.count, [&](int i) {
        const SpanInfo &p = left.info[i];
        return p.tiles > 0 && p.b == b && p.h == h && p.row0 == row0;
    });
    const bool live = tid < span_streams(dim) * kSpanRows && row0 + tid < s.m * a.group;
    const int row = live ? row0 + tid : row0;
    const int token = s.q0 + row / a.group, head = h * a.group + row % a.group;
    const int64_t index = static_cast<int64_t>(token) * a.q_heads + head;
    bool bad = false;
    if (live) {
        // the row's place in a part
        const int stream = tid / kSpanRows, in = tid % kSpanRows;
        const float *part = a.part + stream * (a.part_stride / span_streams(dim));
        const float *stat = part + (dim + 15) / 16 * 16 * kSpanRows + in;
        const float *from = part + (static_cast<int64_t>(d / 4) * kSpanRows + in) * 4;
        float top = -INFINITY, sum = 0.f, v[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) v[k] = 0.f;
        for (int p0 = 0; p0 < parts; p0 += kAtOnce) {
            float m[kAtOnce], l[kAtOnce];
            float4 x[kAtOnce][kRun / 4];
#pragma unroll
            for (int p = 0; p < kAtOnce; ++p) {
                m[p] = -INFINITY, l[p] = 0.f;
#pragma unroll
                for (int k = 0; k < kRun / 4; ++k) x[p][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p0 + p >= parts) continue;
                const int64_t at = js.slot[p0 + p] * a.part_stride;
                m[p] = __ldcg(stat + at), l[p] = __ldcg(stat + at + kSpanRows);
#pragma unroll
                for (int k = 0; k < kRun / 4; ++k) x[p][k] = __ldcg(reinterpret_cast<const float4 *>(from + at + k * kSpanRows * 4));
            }
            float high = top;
#pragma unroll
            for (int p = 0; p < kAtOnce; ++p) high = fmaxf(high, m[p]);
            const float fix = exp2_from(top, high);
            sum *= fix;
#pragma unroll
            for (int k = 0; k < kRun; ++k) v[k] *= fix;
            top = high;
#pragma unroll
            for (int p = 0; p < kAtOnce; ++p) {
                const float w = exp2_from(m[p], top);
                sum += l[p] * w;
#pragma unroll
                for (int k = 0; k < kRun / 4; ++k) {
                    v[4 * k] += x[p][k].x * w, v[4 * k + 1] += x[p][k].y * w;
                    v[4 * k + 2] += x[p][k].z * w, v[4 * k + 3] += x[p][k].w * w;
                }
            }
        }
        if (parts == 0) {
            const float *pre = a.pre + index * span_row(dim);
            top = __ldcg(pre + span_row(dim) - 4);
            sum = __ldcg(pre + span_row(dim) - 3);
#pragma unroll
            for (int k = 0; k < kRun; ++k)
                if (d + k < dim) v[k] = __ldcg(pre + d + k);
            bad = ctas > 0 && __ldcg(a.redo + index) == 1;
        }
        Both f = {sum == 0.f ? 0.f : 1.f / sum, 0.f, top, sum};
        if (a.own) f = both_of(a, index, top, sum);
        const float *own = a.own + index * span_row(dim) + d;
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            bad = bad || (d + k < dim && v[k] != v[k] && sum == sum);
            v[k] *= f.pre;
            if (f.own != 0.f && d + k < dim) v[k] += __ldcg(own + k) * f.own;
        }
        store_run<E, kRun>(a, token, head, d, v);
        if (run == 0 && a.lse) a.lse[index] = lse_of(f.m, f.l);
    }
    // rows that need it, one by one: this run of them
    const unsigned vote = __ballot_sync(kFull, bad);
    if (lane == 0) js.bad[warp] = vote;
    if (!__syncthreads_or(bad)) return;
    unsigned again[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) again[w] = js.bad[w];
    __syncthreads();
    for (int i = 0; i < kThreads; ++i) {
        if (!(again[i / 32] >> i % 32 & 1)) continue;
        const int t = s.q0 + (row0 + i) / a.group, hd = h * a.group + (row0 + i) % a.group;
        one_row<E>(a, *reinterpret_cast<Shared *>(raw), s, t, hd, d, min(dim, d + kRun), true);
    }
}

// Prompts: the joins of all blocks that were cut, then the rows to be computed
// one by one.  Prefix: every row, joined with the slots behind it.
template <int E>
__global__ void __launch_bounds__(kThreads) mbg_span_finish_kernel(const __grid_constant__ SpanArgs a, int ctas)
{
    __shared__ __align__(16) unsigned char raw[sizeof(JoinShared) > sizeof(Shared) ? sizeof(JoinShared) : sizeof(Shared)];
    __shared__ int cuts[kSpanMaxCtas], count[kWarps];
    __shared__ __align__(16) Parts left;
    pdl_trigger();
    pdl_wait();
    const int block = span_streams(a.kv.dim) * kSpanRows, run = a.prefix ? kPrefixRun : kPromptRun, groups = (a.kv.dim + run - 1) / run;
    left.read(a, ctas);
    if (a.prefix) {
        const int blocks = static_cast<int>((static_cast<int64_t>(a.tokens) * a.group + block - 1) / block);
        const int64_t tasks = static_cast<int64_t>(blocks) * a.kv.kv_heads * groups;
        for (int64_t i = blockIdx.x; i < tasks; i += gridDim.x) {
            const int g = static_cast<int>(i % groups), h = static_cast<int>(i / groups % a.kv.kv_heads);
            join_run<E, kPrefixRun, 8>(a, raw, left, ctas, 0, h, static_cast<int>(i / groups / a.kv.kv_heads) * block, g);
            __syncthreads();
        }
        return;
    }
    // blocks whose beginning is a part
    const int n = collect(ctas, cuts, kSpanMaxCtas, count, [&](int c) { return left.info[2 * c + 1].tiles > 0; });
    for (int i = blockIdx.x; i < n * groups; i += gridDim.x) {
        const SpanInfo &p = left.info[2 * cuts[i / groups] + 1];
        join_run<E, kPromptRun, 4>(a, raw, left, ctas, p.b, p.h, p.row0, i % groups);
        __syncthreads();
    }
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kThreads; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * kThreads) {
        const bool again = r0 + threadIdx.x < rows && __ldcg(a.redo + r0 + threadIdx.x) == 1;
        if (!__syncthreads_or(again)) continue;
        const bool ascend = ascending(a);
        for (int w = 0; w < kWarps; ++w) {
            if (threadIdx.x / 32 == w) {
                const unsigned vote = __ballot_sync(kFull, again);
                if (threadIdx.x % 32 == 0) count[0] = static_cast<int>(vote);
            }
            __syncthreads();
            const unsigned vote = static_cast<unsigned>(count[0]);
            __syncthreads();
            for (int i = 0; i < 32; ++i)
                if (vote >> i & 1) {
                    const int64_t r = r0 + w * 32 + i;
                    const int t = static_cast<int>(r / a.q_heads);
                    Shared &sh = *reinterpret_cast<Shared *>(raw);
                    const int b = seq_of_token(a, sh, t, ascend);
                    if (b >= 0) one_row<E>(a, sh, span::seq_of(a, b, false), t, static_cast<int>(r % a.q_heads), 0, a.kv.dim, false);
                }
        }
    }
}

template <int E>
__global__ void __launch_bounds__(kThreads) mbg_span_rows_kernel(const __grid_constant__ SpanArgs a)
{
    __shared__ Shared sh;
    pdl_wait();
    pdl_trigger();  // as the tiles: what follows may go by this launch's wait
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < (a.prefix ? 1 : a.kv.batch); b += kThreads) span::seq_of(a, b, true);
    const bool ascend = a.prefix || ascending(a);
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int t = static_cast<int>(r / a.q_heads), b = seq_of_token(a, sh, t, ascend);
        if (b >= 0) one_row<E>(a, sh, span::seq_of(a, b, false), t, static_cast<int>(r % a.q_heads), 0, a.kv.dim, false);
    }
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

// A scale of 0 (or none) leaves the tiles no maximum to go by.
static bool tiled(const SpanArgs &a) { return fabsf(a.scale_log2) > 0.f && fabsf(a.scale_log2) < INFINITY; }
static int ctas_of(int sm_count) { return sm_count < kSpanMaxCtas ? sm_count : kSpanMaxCtas; }

// The driver's encoder of tensor maps; NULL where there is none.
static PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static std::atomic<void *> found{nullptr};
    void *f = found.load(std::memory_order_relaxed);
    if (!f) {
        cudaDriverEntryPointQueryResult result;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &result) != cudaSuccess ||
            result != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        found.store(f, std::memory_order_relaxed);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// A pool as a tensor of boxes of 64 elements x `box` tokens, rows of 128 bytes
// swizzled as the tensor core reads them.
static bool map_pool(CUtensorMap *map, const KvView &kv, void *pool, int64_t page, int64_t token, int64_t head, int elem, int box)
{
    const auto encode = encoder();
    // (a stride of 0, a pool broadcast along an axis, is not a map's)
    if (!encode || kv.num_pages < 1 || token < 1 || head < 1 || page < 1) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.dim), static_cast<cuuint64_t>(kv.page_size), static_cast<cuuint64_t>(kv.kv_heads),
                                static_cast<cuuint64_t>(kv.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(token) * 2, static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(page) * 2};
    const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), 1, 1}, steps[4] = {1, 1, 1, 1};
    return encode(map, elem == GEMV_ELEM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool, dims, strides, boxes,
                  steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Bulk copies go by boxes of 8 tokens or more that divide both a page and a
// tile; other pages, and pools that the maps cannot describe, are copied piece by piece.
static void map_pools(SpanArgs *a, bool vec, int elem)
{
    a->box = 0;
    int box = span_tile(a->kv.dim);
    while (box >= 8 && a->kv.page_size % box) box /= 2;
    if (!vec || box < 8 || a->kv.dim < 64) return;
    if (map_pool(&a->k_map, a->kv, a->kv.k, a->kv.ks_page, a->kv.ks_tok, a->kv.ks_head, elem, box) &&
        map_pool(&a->v_map, a->kv, a->kv.v, a->kv.vs_page, a->kv.vs_tok, a->kv.vs_head, elem, box))
        a->box = box;
}

cudaError_t launch_span(const SpanArgs &args, bool vec, int elem, int sm_count, cudaStream_t s)
{
    const bool f16 = elem == GEMV_ELEM_F16;
    SpanArgs a = args;
    if (tiled(a)) {
        map_pools(&a, vec, elem);
        return f16 ? launch_tile_f16(a, vec, ctas_of(sm_count), s) : launch_tile_bf16(a, vec, ctas_of(sm_count), s);
    }
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads, most = static_cast<int64_t>(sm_count) * 8;
    return launch_blocks(f16 ? mbg_span_rows_kernel<GEMV_ELEM_F16> : mbg_span_rows_kernel<GEMV_ELEM_BF16>, rows < most ? rows : most, s, a);
}

cudaError_t launch_span_finish(const SpanArgs &a, int elem, int sm_count, cudaStream_t s)
{
    if (!tiled(a) && !a.prefix) return cudaSuccess;
    const int64_t block = span_streams(a.kv.dim) * kSpanRows, rows = static_cast<int64_t>(a.tokens) * a.group;
    int64_t blocks = static_cast<int64_t>(sm_count) * 6;
    if (a.prefix) {
        const int64_t tasks = (rows + block - 1) / block * a.kv.kv_heads * ((a.kv.dim + kPrefixRun - 1) / kPrefixRun);
        if (tasks < blocks) blocks = tasks;
    }
    return launch_blocks(elem == GEMV_ELEM_F16 ? mbg_span_finish_kernel<GEMV_ELEM_F16> : mbg_span_finish_kernel<GEMV_ELEM_BF16>, blocks, s, a,
                         tiled(a) ? ctas_of(sm_count) : 0);
}

}  // namespace mbg
