// Eviction from a paged key-value cache by accumulated attention weight.
//
// Plan.  Of a row's n = length slots (one row per sequence and cached head)
// the first `keep` of this order stay: protected slots (stamp < sinks, or
// among the `recent` newest stamps), then the larger score, then the lower
// slot.  Slots that stay but lie at or behind `keep` move into the holes
// below `keep`, both lists in ascending order: the fewest rows move, no move
// reads what another writes, and the cache stays dense.  Attention over
// rotated keys does not depend on the slots' order; the stamps keep the
// tokens' own.
//
// The order's keep-th element is found by a radix select over the scores'
// bits mapped to unsigned integers (larger score, larger integer), on the one
// class (protected or not) that the budget cuts: four passes of 8 bits, then
// one pass in slot order that ranks ties and writes the moves.
#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"

namespace mbg {
namespace {

constexpr int kPlanThreads = 1024;

// Larger score, larger integer; NaN like -inf, -0 like 0.
__device__ __forceinline__ uint32_t score_key(float s)
{
    if (s != s) s = -INFINITY;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// Sum over the block, and the thread's exclusive prefix, of two counts packed
// into one 64-bit word.
__device__ uint64_t block_scan(uint64_t v, uint64_t *total, uint64_t *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t s = v;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
        const uint64_t n = __shfl_up_sync(0xFFFFFFFFu, s, x);
        if (lane >= x) s += n;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + s - v;
}

__global__ void __launch_bounds__(kPlanThreads) mbg_evict_plan_kernel(const __grid_constant__ EvictArgs a)
{
    __shared__ unsigned hist[256];
    __shared__ uint64_t warp_sums[kPlanThreads / 32];
    __shared__ int s_newest, s_protected;
    __shared__ unsigned s_prefix, s_left;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int b = static_cast<int>(row / a.kv.kv_heads);
    int n = __ldg(a.lengths + b);
    if (n < 0 || n > a.kv.capacity) {
        if (tid == 0) report_error(a.err, DEVERR_BAD_INDEX);
        n = n < 0 ? 0 : static_cast<int>(a.kv.capacity);
    }
    if (n <= a.keep) {
        if (tid == 0) a.counts[row] = 0;
        return;
    }
    const float *scores = a.scores + row * a.kv.capacity;
    const int32_t *stamps = a.stamps + row * a.kv.capacity;

    // newest stamp, and how many slots are protected
    if (tid == 0) {
        s_newest = INT32_MIN;
        s_protected = 0;
    }
    __syncthreads();
    int newest = INT32_MIN;
    for (int i = tid; i < n; i += kPlanThreads) newest = max(newest, __ldg(stamps + i));
    newest = __reduce_max_sync(0xFFFFFFFFu, newest);
    if ((tid & 31) == 0) atomicMax(&s_newest, newest);
    __syncthreads();
    const int64_t recent_from = static_cast<int64_t>(s_newest) - a.recent;
    auto is_protected = [&](int stamp) { return stamp < a.sinks || stamp > recent_from; };
    int mine = 0;
    for (int i = tid; i < n; i += kPlanThreads) mine += is_protected(__ldg(stamps + i));
    mine = __reduce_add_sync(0xFFFFFFFFu, mine);
    if ((tid & 31) == 0) atomicAdd(&s_protected, mine);
    __syncthreads();
    // the budget cuts one class; of it `left` slots stay
    const bool cut_protected = s_protected >= a.keep;
    unsigned left = cut_protected ? a.keep : a.keep - s_protected;

    // key of the left-th largest of that class
    unsigned prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kPlanThreads) {
            if (is_protected(__ldg(stamps + i)) != cut_protected) continue;
            const uint32_t key = score_key(__ldg(scores + i));
            if (shift < 24 && (key >> (shift + 8)) != prefix) continue;
            atomicAdd(&hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            unsigned rest = left;
            int d = 255;
            while (d > 0 && hist[d] < rest) rest -= hist[d--];
            s_prefix = (prefix << 8) | static_cast<unsigned>(d);
            s_left = rest;
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
    }
    // `left` of the slots with exactly this key stay, the lowest first
    const uint32_t limit = prefix;
    int32_t *moves = a.moves + 2 * row * a.max_moves;
    unsigned ties_before = 0, holes_before = 0, movers_before = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        bool in = i < n, cls = false, tie = false, above = false;
        if (in) {
            cls = is_protected(__ldg(stamps + i)) == cut_protected;
            const uint32_t key = score_key(__ldg(scores + i));
            tie = cls && key == limit;
            above = cls ? key > limit : !cut_protected;  // protected slots stay when the others are cut
        }
        uint64_t all;
        const uint64_t tie_rank = block_scan(tie, &all, warp_sums) + ties_before;
        ties_before += static_cast<unsigned>(all);
        const bool stays = in && (above || (tie && tie_rank < left));
        const bool hole = in && !stays && i < a.keep, mover = stays && i >= a.keep;
        const uint64_t pre = block_scan(static_cast<uint64_t>(hole) | (static_cast<uint64_t>(mover) << 32), &all,
                                        warp_sums);
        if (hole) {
            const unsigned at = holes_before + static_cast<unsigned>(pre);
            if (at < a.max_moves) moves[2 * static_cast<int64_t>(at) + 1] = i;
        }
        if (mover) {
            const unsigned at = movers_before + static_cast<unsigned>(pre >> 32);
            if (at < a.max_moves) moves[2 * static_cast<int64_t>(at)] = i;
        }
        holes_before += static_cast<unsigned>(all);
        movers_before += static_cast<unsigned>(all >> 32);
    }
    if (tid == 0) a.counts[row] = static_cast<int>(movers_before);
}

// Moves.  Sources lie at or behind `keep` and targets before it, so nothing
// is read that another thread writes and applying a plan twice changes
// nothing.  Bound by the bytes moved; one warp takes one move, half of it for
// K and half for V.
constexpr int kApplyThreads = 256;

__device__ __forceinline__ int64_t page_of(const KvView &kv, const int32_t *table, int slot, int *off)
{
    const int idx = kv.page_shift >= 0 ? slot >> kv.page_shift : slot / kv.page_size;
    *off = slot - idx * kv.page_size;
    const int page = __ldg(table + idx);
    return page >= 0 && page < kv.num_pages ? page : -1;
}

template <bool VEC>
__global__ void __launch_bounds__(kApplyThreads) mbg_evict_apply_kernel(const __grid_constant__ EvictApplyArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    const int h = blockIdx.y, b = blockIdx.z;
    const KvView &kv = a.kv;
    if (a.lengths && h == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        const int n = a.lengths[b];
        if (n > a.keep) a.lengths[b] = a.keep;
    }
    int count = __ldg(a.counts + row);
    if (count < 0 || count > a.max_moves) {
        if (threadIdx.x == 0) report_error(a.err, DEVERR_BAD_INDEX);
        count = count < 0 ? 0 : static_cast<int>(a.max_moves);
    }
    const int32_t *table = kv.table + b * kv.table_stride;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warps = kApplyThreads / 32;
    for (int i = blockIdx.x * warps + warp; i < count; i += gridDim.x * warps) {
        const int2 mv = __ldg(reinterpret_cast<const int2 *>(a.moves) + row * a.max_moves + i);
        if (mv.x < 0 || mv.x >= kv.capacity || mv.y < 0 || mv.y >= kv.capacity) {
            if (lane == 0) report_error(a.err, DEVERR_BAD_INDEX);
            continue;
        }
        int so, to;
        const int64_t sp = page_of(kv, table, mv.x, &so), tp = page_of(kv, table, mv.y, &to);
        if (sp < 0 || tp < 0) {
            if (lane == 0) report_error(a.err, DEVERR_BAD_INDEX);
            continue;
        }
        const bool is_v = lane >= 16;
        uint16_t *pool = static_cast<uint16_t *>(is_v ? kv.v : kv.k);
        const int64_t ps = is_v ? kv.vs_page : kv.ks_page, ts = is_v ? kv.vs_tok : kv.ks_tok,
                      hs = is_v ? kv.vs_head : kv.ks_head;
        const uint16_t *src = pool + sp * ps + so * ts + h * hs;
        uint16_t *dst = pool + tp * ps + to * ts + h * hs;
        if (VEC) {
            for (int d = (lane & 15) * 8; d < kv.dim; d += 128)
                *reinterpret_cast<uint4 *>(dst + d) = *reinterpret_cast<const uint4 *>(src + d);
        } else {
            for (int d = lane & 15; d < kv.dim; d += 16) dst[d] = src[d];
        }
        if (lane == 0 && a.scores) {
            float *sc = a.scores + row * kv.capacity;
            sc[mv.y] = sc[mv.x];
        }
        if (lane == 16 && a.stamps) {
            int32_t *st = a.stamps + row * kv.capacity;
            st[mv.y] = st[mv.x];
        }
    }
}

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*fn)(Params...), dim3 grid, int threads, cudaStream_t s, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace

cudaError_t launch_evict_plan(const EvictArgs &a, int sm_count, cudaStream_t s)
{
    (void)sm_count;
    return launch_pdl(mbg_evict_plan_kernel, dim3(static_cast<unsigned>(a.kv.batch) * a.kv.kv_heads), kPlanThreads, s,
                      a);
}

cudaError_t launch_evict_apply(const EvictApplyArgs &a, bool vec, int sm_count, cudaStream_t s)
{
    // enough blocks per row to fill the GPU a few times over, and no more
    // than the moves there can be
    const int64_t rows = static_cast<int64_t>(a.kv.batch) * a.kv.kv_heads;
    int64_t x = (16ll * sm_count + rows - 1) / rows;
    const int64_t most = (a.max_moves + kApplyThreads / 32 - 1) / (kApplyThreads / 32);
    if (x > most) x = most;
    if (x < 1) x = 1;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(a.kv.kv_heads), static_cast<unsigned>(a.kv.batch));
    return launch_pdl(vec ? mbg_evict_apply_kernel<true> : mbg_evict_apply_kernel<false>, grid, kApplyThreads, s, a);
}

}  // namespace mbg
