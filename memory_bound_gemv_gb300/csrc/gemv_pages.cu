// Page tables and slot maps from the lengths of requests.
//
// Request b has n slots in use and gets f new tokens: it holds ceil(n / P)
// pages and needs ceil((n + f) / P).  Prefix sums over the requests say which
// pages of the ring each of them takes, where its tokens stand in the slot
// map, and where the pages of those that are over go.
//
// Bound by latency: a few kilobytes behind a chain of reads (lengths, sums,
// ring) and one launch: 64 requests of a token each 6.3 us, 307 of which many
// bring prompts, 28272 tokens, 8.7 us.  Every block of one cluster makes the sums over all
// requests for itself, 1024 at a time, which costs less than handing them
// on, and then writes its share of the tokens and pages, for each of which a
// binary search among the chunk's sums finds the request.  What other blocks
// read (lengths, state, and with a full ring nothing else: pages are taken
// from the ring's front and put behind its end) is written behind a cluster
// barrier.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"

namespace mbg {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32, kMaxCluster = 8;
constexpr unsigned kFull = 0xFFFFFFFFu;

struct Sums {
    int64_t warp[2][kWarps];
};

// Sums over the block up to and with this thread's values.  A barrier has to
// lie between a call and the next one with the same buffer.
__device__ __forceinline__ void scan2(Sums &s, int64_t &a, int64_t &b, int64_t &all_a, int64_t &all_b)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
        const int64_t ua = __shfl_up_sync(kFull, a, x), ub = __shfl_up_sync(kFull, b, x);
        if (lane >= x) a += ua, b += ub;
    }
    if (lane == 31) s.warp[0][warp] = a, s.warp[1][warp] = b;
    __syncthreads();
    // every warp sums the warps' totals
    int64_t ta = s.warp[0][lane], tb = s.warp[1][lane];
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
        const int64_t ua = __shfl_up_sync(kFull, ta, x), ub = __shfl_up_sync(kFull, tb, x);
        if (lane >= x) ta += ua, tb += ub;
    }
    all_a = __shfl_sync(kFull, ta, 31);
    all_b = __shfl_sync(kFull, tb, 31);
    const int64_t pa = __shfl_sync(kFull, ta, warp ? warp - 1 : 0), pb = __shfl_sync(kFull, tb, warp ? warp - 1 : 0);
    if (warp) a += pa, b += pb;
}

// The request of a chunk whose range of a running sum holds i: the first
// whose end lies above it.
__device__ __forceinline__ int find(const int64_t *ends, int n, int64_t i)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > i)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Pages of n slots (below 2^31).
__device__ __forceinline__ int pages_of(int64_t n, int page_size)
{
    return n > 0 ? static_cast<int>((static_cast<uint32_t>(n) - 1) / static_cast<uint32_t>(page_size) + 1) : 0;
}

// Puts the pages that come back behind the ring's end, at `end`, once more and
// one request at a time, without those that do not exist; returns how many.  No more
// than `most` have a place.
__device__ __noinline__ int64_t put_back(const AssignArgs &a, Sums &s, int64_t end, int64_t most)
{
    int64_t put = 0;
    if (threadIdx.x == 0) report_error(a.err, DEVERR_BAD_INDEX);
    for (int b = 0; b < a.batch; ++b) {
        const int64_t n = a.lengths[b];
        if (a.fresh[b] >= 0 || n < 0 || n > a.capacity) continue;
        const int keep = a.shared ? max(0, a.shared[b]) / a.page_size : 0, have = pages_of(n, a.page_size);
        for (int i0 = keep; i0 < have; i0 += kThreads) {
            const int i = i0 + threadIdx.x;
            const int page = i < have ? a.table[b * a.table_stride + i] : -1;
            const bool there = page >= 0 && page < a.num_pages;
            int64_t sum = there, none = 0, all, none_all;
            scan2(s, sum, none, all, none_all);
            __syncthreads();
            if (there && put + sum <= most) {
                int64_t place = end + put + sum - 1;
                while (place >= a.ring_size) place -= a.ring_size;
                a.ring[place] = page;
            }
            put += all;
        }
    }
    return put < most ? put : most;
}

__global__ void __launch_bounds__(kThreads, 1) mbg_assign_kernel(const __grid_constant__ AssignArgs a)
{
    __shared__ Sums sums[2];
    __shared__ int64_t tok_end[kThreads], page_end[kThreads], gone_end[kThreads];
    __shared__ int from_slot[kThreads], from_page[kThreads];
    __shared__ int strays;  // (the first block's) of the pages that come back some do not exist
    const int tid = threadIdx.x, rank = blockIdx.x, blocks = gridDim.x;
    auto cluster = cooperative_groups::this_cluster();
    if (tid == 0) strays = 0;
    if (blocks > 1) cluster.barrier_arrive();  // waited for ahead of the first write to another block's memory
    pdl_trigger();
    pdl_wait();
    const int64_t at = a.state[0], count0 = a.state[1];
    // a state that cannot be: nothing is taken, nothing is put back
    const bool broken = at < 0 || count0 < 0 || count0 > a.ring_size || (at >= a.ring_size && a.ring_size > 0) ||
                        (a.ring_size == 0 && at != 0);
    const int64_t count = broken ? 0 : count0;
    if (broken && rank == 0 && tid == 0) report_error(a.err, DEVERR_BAD_INDEX);
    const int64_t behind = broken ? 0 : a.ring_size - count;  // places in the ring that hold no free page
    const int page_size = a.page_size, batch = a.batch;
    const int64_t capacity = a.capacity;
    // the page that this thread hands out first, whoever it goes to
    int ahead = -1;
    if (rank * kThreads + tid < count) {
        int64_t place = at + rank * kThreads + tid;
        if (place >= a.ring_size) place -= a.ring_size;
        ahead = a.ring[place];
    }
    int64_t needed = 0, wanted = 0, taken = 0, gone = 0, tokens = 0;  // sums of the chunks before
    bool stray = false;
    int after = 0;  // this thread's request of the last chunk: slots in use afterwards
    for (int b0 = 0; b0 < batch; b0 += kThreads) {
        const int b = b0 + tid, n_chunk = min(kThreads, batch - b0);
        int64_t n = 0, f = 0;
        int keep = 0;
        bool wrong = false;  // a length out of range: what its row holds is not known to be its own
        if (b < batch) {
            n = a.lengths[b];
            f = a.fresh[b];
            if (a.shared) keep = static_cast<int>(static_cast<uint32_t>(max(0, a.shared[b])) / static_cast<uint32_t>(page_size));
        }
        if (n < 0 || n > capacity || n + f > capacity) {
            if (rank == 0) report_error(a.err, DEVERR_BAD_INDEX);
            wrong = n < 0 || n > capacity;
            n = n < 0 ? 0 : n > capacity ? capacity : n;
            f = f < 0 ? f : 0;
        }
        const bool over = f < 0;
        if (over) f = 0;
        const int have = pages_of(n, page_size);
        int64_t need = pages_of(n + f, page_size) - have, back = over && !wrong && have > keep ? have - keep : 0;
        // first sums: pages needed, pages returned
        int64_t need_sum = need, back_sum = back, need_all, back_all;
        scan2(sums[0], need_sum, back_sum, need_all, back_all);
        if (need > 0 && needed + need_sum > count) f = need = 0;  // no page left: the request waits
        // second sums: tokens, and pages of those that have them
        int64_t tok_sum = f, take_sum = need, tok_all, take_all;
        scan2(sums[1], tok_sum, take_sum, tok_all, take_all);
        if (wanted + tok_sum > a.room) f = 0, need = 0;  // no room in the slot map: nor do those behind it fit
        // tokens and pages of those with room: the sums up to the last of them
        tok_end[tid] = f > 0 ? wanted + tok_sum : 0;
        page_end[tid] = f > 0 ? taken + take_sum : 0;
        gone_end[tid] = gone + back_sum;
        from_slot[tid] = static_cast<int>(n);
        from_page[tid] = over ? keep : have;
        const bool cut = wanted + tok_all > a.room;
        const int fit = cut ? __syncthreads_count(b < batch && wanted + tok_sum <= a.room) : n_chunk;
        __syncthreads();
        // requests behind `fit` got nothing, nor did waiting ones: their sums
        // repeat the one before
        if (f == 0) {
            const int64_t t = wanted + tok_sum, p = taken + take_sum;
            tok_end[tid] = tid < fit ? t : 0;
            page_end[tid] = tid < fit ? p : 0;
        }
        __syncthreads();
        const int64_t tok_last = fit ? tok_end[fit - 1] : tokens, page_last = fit ? page_end[fit - 1] : taken;
        if (tid >= fit) tok_end[tid] = tok_last, page_end[tid] = page_last;
        __syncthreads();
        const int step = kThreads * blocks, me = rank * kThreads + tid;
        // a token to a thread, or four side by side where there are more
        if (tok_last - tokens <= step) {
            const int64_t i = tokens + me;
            if (i < tok_last) {
                const int r = find(tok_end, n_chunk, i);
                a.slots[i] = from_slot[r] + static_cast<int>(i - (r ? tok_end[r - 1] : tokens));
                a.seq[i] = b0 + r;
            }
        } else {
            for (int64_t i0 = tokens / 4 * 4 + 4 * me; i0 < tok_last; i0 += 4 * step) {
                int r = find(tok_end, n_chunk, i0 < tokens ? tokens : i0), slot[4], seq[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t i = i0 + k;
                    if (i < tokens || i >= tok_last) continue;
                    while (tok_end[r] <= i) ++r;
                    slot[k] = from_slot[r] + static_cast<int>(i - (r ? tok_end[r - 1] : tokens));
                    seq[k] = b0 + r;
                }
                if (a.wide && i0 >= tokens && i0 + 4 <= tok_last) {
                    *reinterpret_cast<int4 *>(a.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
                    *reinterpret_cast<int4 *>(a.seq + i0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (i0 + k >= tokens && i0 + k < tok_last) a.slots[i0 + k] = slot[k], a.seq[i0 + k] = seq[k];
                }
            }
        }
        for (int64_t i = taken + me; i < page_last; i += step) {
            const int r = find(page_end, n_chunk, i);
            int page = ahead;
            if (i != me) {
                int64_t place = at + i;
                if (place >= a.ring_size) place -= a.ring_size;
                page = a.ring[place];
            }
            if (page < 0 || page >= a.num_pages) {
                report_error(a.err, DEVERR_BAD_INDEX);
                page = -1;
            }
            a.table[(b0 + r) * a.table_stride + from_page[r] + (i - (r ? page_end[r - 1] : taken))] = page;
        }
        for (int64_t i = gone + me; i < gone + back_all; i += step) {
            if (i >= behind) {  // more pages than the ring has lent
                report_error(a.err, DEVERR_BAD_INDEX);
                break;
            }
            const int r = find(gone_end, n_chunk, i);
            int64_t place = at + count + i;
            if (place >= a.ring_size) place -= a.ring_size;
            const int page = a.table[(b0 + r) * a.table_stride + from_page[r] + (i - (r ? gone_end[r - 1] : gone))];
            if (page < 0 || page >= a.num_pages) stray = true;
            a.ring[place] = page;
        }
        if (rank == 0 && b < batch) {
            a.starts[b + 1] = static_cast<int>(tok_end[tid]);
            if (b0 == 0 && tid == 0) a.starts[0] = 0;
        }
        after = over ? 0 : static_cast<int>(n + f);
        tokens = tok_last;
        taken = page_last;
        gone += back_all;
        needed += need_all;
        wanted += tok_all;
        __syncthreads();
    }
    if (batch == 0 && rank == 0 && tid == 0) a.starts[0] = 0;
    for (int64_t i = tokens + rank * kThreads + tid; i < a.room; i += kThreads * blocks) {
        a.slots[i] = -1;
        a.seq[i] = 0;
    }
    // lengths and state may be written where they were read
    if (blocks > 1) {
        cluster.barrier_wait();
        if (stray) *cluster.map_shared_rank(&strays, 0) = 1;
        cluster.sync();
    } else {
        if (stray) strays = 1;
        __syncthreads();
    }
    if (rank != 0) return;
    if (strays) gone = put_back(a, sums[0], at + count, behind);
    if (batch <= kThreads) {
        if (tid < batch) a.lengths_out[tid] = after;
    } else {
        for (int b = tid; b < batch; b += kThreads) {
            const int64_t n = a.lengths[b];
            const int f = a.fresh[b];
            a.lengths_out[b] = f < 0 ? 0 : static_cast<int>(n < 0 ? 0 : n > capacity ? capacity : n) + a.starts[b + 1] - a.starts[b];
        }
    }
    if (tid == 0) {
        if (broken) {
            a.state_out[0] = static_cast<int>(at);
            a.state_out[1] = static_cast<int>(count0);
        } else {
            int64_t front = at + taken;
            if (front >= a.ring_size) front -= a.ring_size;
            a.state_out[0] = static_cast<int>(front);
            a.state_out[1] = static_cast<int>(count - taken + (gone < behind ? gone : behind));
        }
    }
}

}  // namespace

cudaError_t launch_assign(const AssignArgs &a, cudaStream_t s)
{
    // one block where its threads write a few values each
    int blocks = 1;
    while (blocks < kMaxCluster && a.room > static_cast<int64_t>(4) * kThreads * blocks) blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mbg_assign_kernel, a);
}

}  // namespace mbg
