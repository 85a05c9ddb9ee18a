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
// class (protected or not) that the budget cuts: three histograms of 11, 11
// and 10 bits.  A row is read once, into registers; the passes, the ranking of
// ties and the numbering of holes and movers run on those.  The bytes (8 per
// slot) are few: what counts is the chain of dependent steps, so a long row
// is spread over a cluster of blocks, which add their histograms through
// distributed shared memory, and a row takes about a dozen barriers whatever
// its length.  Rows a few slots over the budget, as a decode step leaves them,
// have those picked one after another (128 rows of 2049 slots, plan and moves:
// 7.3 us, with the histograms 10.0 us).
#include <cooperative_groups.h>
#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"

namespace cg = cooperative_groups;

namespace mbg {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxCluster = 8;
constexpr int kBins = 2048;
// Up to this many slots over the budget are picked one by one: a decode step
// that appends a token and drops one does four barriers then, not ten.
constexpr int kFew = 4;

// Larger score, larger integer; NaN like -inf, -0 like 0.
__device__ __forceinline__ uint32_t score_key(float s)
{
    if (s != s) s = -INFINITY;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// Reductions over a warp and of two values.
struct OpMax {
    static constexpr unsigned none = 0u;
    __device__ unsigned operator()(unsigned v) const { return __reduce_max_sync(kAll, v); }
    __device__ unsigned two(unsigned a, unsigned b) const { return max(a, b); }
};
struct OpMin {
    static constexpr unsigned none = 0xFFFFFFFFu;
    __device__ unsigned operator()(unsigned v) const { return __reduce_min_sync(kAll, v); }
    __device__ unsigned two(unsigned a, unsigned b) const { return min(a, b); }
};
struct OpSum {
    static constexpr unsigned none = 0u;
    __device__ unsigned operator()(unsigned v) const { return __reduce_add_sync(kAll, v); }
    __device__ unsigned two(unsigned a, unsigned b) const { return a + b; }
};

// What the blocks of a cluster tell one another.  Every exchange has its own
// fields, so that one cluster barrier is enough for each.
struct PlanShared {
    uint4 hist[4][kBins / 4];
    unsigned scan[4][32];           // block scans of the histograms
    unsigned red[2 + 2 * kFew][32]; // reductions: each warp's value
    unsigned warp_ties[32], warp_holes[32], warp_movers[32];
    unsigned ties, holes, movers;   // this block's sums
    unsigned got[4][kPlanMaxCluster];  // the blocks' values as read here
    unsigned digit, left, count;    // a pass' result
    __device__ __forceinline__ unsigned *bins(int h) { return reinterpret_cast<unsigned *>(hist[h]); }
};

// KPT slots of a row per thread in registers; KPT 0: a row of any length, read
// again for each step.
template <int KPT>
__global__ void __launch_bounds__(kPlanThreads) mbg_evict_plan_kernel(const __grid_constant__ EvictArgs a)
{
    constexpr bool kReg = KPT > 0;
    constexpr int kWarps = kPlanThreads / 32;
    __shared__ PlanShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / blocks;
    pdl_trigger();
    for (int i = tid; i < kBins; i += kPlanThreads) (&sh.hist[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    pdl_wait();
    const int b = static_cast<int>(row / a.kv.kv_heads);
    int n = __ldg(a.lengths + b);
    if (n < 0 || n > a.kv.capacity) {
        if (tid == 0) report_error(a.err, DEVERR_BAD_INDEX);
        n = n < 0 ? 0 : static_cast<int>(a.kv.capacity);
    }
    if (n <= a.keep) {  // the whole cluster leaves here or none of it
        if (tid == 0 && rank == 0) a.counts[row] = 0;
        return;
    }
    const float *scores = a.scores + row * a.kv.capacity;
    const int32_t *stamps = a.stamps + row * a.kv.capacity;
    // each warp takes consecutive slots, 32 at a time
    const int warps = blocks * kWarps;
    const int steps = ((n + warps - 1) / warps + 31) / 32;
    const int64_t base = static_cast<int64_t>(rank * kWarps + warp) * steps * 32 + lane;
    constexpr int kHold = kReg ? KPT : 1;
    auto sync_all = [&]() {
        if (blocks > 1)
            cluster.sync();
        else
            __syncthreads();
    };

    uint32_t key[kHold];
    int newest = INT32_MIN;
    // short rows keep the stamps too; for long ones they are read a second
    // time, from L2
    constexpr bool kHoldStamps = kReg && KPT <= 8;
    int stamp[kHoldStamps ? KPT : 1];
    if (kReg) {
#pragma unroll
        for (int j = 0; j < kHold; ++j) {
            const int64_t i = base + 32 * j;
            if (j < steps && i < n) {
                const int st = __ldg(stamps + i);
                key[j] = score_key(__ldg(scores + i));
                newest = max(newest, st);
                if (kHoldStamps) stamp[kHoldStamps ? j : 0] = st;
            }
        }
    } else {
        for (int j = 0; j < steps; ++j)
            if (base + 32 * j < n) newest = max(newest, __ldg(stamps + base + 32 * j));
    }
    // joins a value of every thread of the cluster; one barrier
    auto reduce = [&](unsigned v, int slot, auto op) {
        v = op(v);
        if (lane == 0) sh.red[slot][warp] = v;
        sync_all();
        unsigned w = sh.red[slot][lane < kWarps ? lane : 0];
        if (lane >= kWarps) w = op.none;
        for (int k = 0; k < blocks; ++k) {
            if (k == rank) continue;
            const unsigned o = lane < kWarps ? *cluster.map_shared_rank(&sh.red[slot][lane], k) : op.none;
            w = op.two(w, o);
        }
        return op(w);
    };
    newest = static_cast<int>(reduce(static_cast<unsigned>(newest) ^ 0x80000000u, 0, OpMax()) ^ 0x80000000u);
    const int64_t recent_from = static_cast<int64_t>(newest) - a.recent;
    auto is_protected = [&](int st) { return st < a.sinks || st > recent_from; };
    uint32_t protected_bits = 0;
    if (kReg) {
#pragma unroll
        for (int j = 0; j < kHold; ++j) {
            const int64_t i = base + 32 * j;
            if (j < steps && i < n && is_protected(kHoldStamps ? stamp[kHoldStamps ? j : 0] : __ldg(stamps + i)))
                protected_bits |= 1u << j;
        }
    }
    // calls f(step, exists, key, protected) for each of the thread's slots,
    // in order and with the whole warp
    auto each = [&](auto f) {
        if (kReg) {
#pragma unroll
            for (int j = 0; j < kHold; ++j)
                if (j < steps) f(j, base + 32 * j < n, key[j], ((protected_bits >> j) & 1u) != 0);
        } else {
            for (int j = 0; j < steps; ++j) {
                const int64_t i = base + 32 * j;
                const bool in = i < n;
                f(j, in, in ? score_key(__ldg(scores + i)) : 0u, in && is_protected(__ldg(stamps + i)));
            }
        }
    };
    // adds a block value over the cluster (after sync_all)
    auto total_of = [&](const unsigned *mine, int slot, unsigned *before) {
        if (blocks == 1) {
            *before = 0;
            return *mine;
        }
        if (tid < blocks) sh.got[slot][tid] = *cluster.map_shared_rank(const_cast<unsigned *>(mine), tid);
        __syncthreads();
        unsigned sum = 0, pre = 0;
        for (int k = 0; k < blocks; ++k) {
            if (k < rank) pre += sh.got[slot][k];
            sum += sh.got[slot][k];
        }
        *before = pre;
        return sum;
    };
    // finds the digit that holds the left-th largest value of histogram h
    auto pick = [&](int h, unsigned left) {
        constexpr int kOwn = kBins / kPlanThreads;  // the thread's bins, from the top
        const int bin = kBins - kOwn - kOwn * tid;
        unsigned c[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) c[i] = 0;
        for (int k = 0; k < blocks; ++k) {
            const uint2 *p = reinterpret_cast<const uint2 *>(sh.bins(h) + bin);
            if (blocks > 1) p = cluster.map_shared_rank(const_cast<uint2 *>(p), k);
#pragma unroll
            for (int i = 0; i < kOwn / 2; ++i) {
                const uint2 v = p[i];
                c[2 * i] += v.x;
                c[2 * i + 1] += v.y;
            }
        }
        unsigned own = 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) own += c[i];
        unsigned s = own;
#pragma unroll
        for (int x = 1; x < 32; x *= 2) {
            const unsigned up = __shfl_up_sync(kAll, s, x);
            if (lane >= x) s += up;
        }
        if (lane == 31) sh.scan[h][warp] = s;
        __syncthreads();
        // sum over the warps before this one
        unsigned above = __reduce_add_sync(kAll, lane < warp ? sh.scan[h][lane] : 0u) + s - own;
#pragma unroll
        for (int i = kOwn - 1; i >= 0; --i) {
            if (above < left && left <= above + c[i]) {
                sh.digit = bin + i;
                sh.left = left - above;
                sh.count = c[i];
            }
            above += c[i];
        }
        __syncthreads();
    };

    if (kReg && n - a.keep <= kFew) {
        // how many protected slots there are: the others go first
        unsigned mine = 0;
        each([&](int, bool in, uint32_t, bool prot) { mine += in && prot; });
        const int open = n - static_cast<int>(reduce(mine, 1, OpSum()));
        uint32_t gone = 0;
        int victim[kFew];
#pragma unroll
        for (int r = 0; r < kFew; ++r) {
            victim[r] = INT32_MAX;
            if (r >= n - a.keep) continue;
            const bool cls = r >= open;
            unsigned low = 0xFFFFFFFFu, last = 0;
            each([&](int j, bool in, uint32_t k, bool prot) {
                if (in && prot == cls && !((gone >> j) & 1u)) low = min(low, k);
            });
            low = reduce(low, 2 + 2 * r, OpMin());
            each([&](int j, bool in, uint32_t k, bool prot) {
                if (in && prot == cls && !((gone >> j) & 1u) && k == low) last = static_cast<unsigned>(base + 32 * j);
            });
            victim[r] = static_cast<int>(reduce(last, 3 + 2 * r, OpMax()));
            each([&](int j, bool, uint32_t, bool) {
                if (base + 32 * j == victim[r]) gone |= 1u << j;
            });
        }
        if (tid == 0 && rank == 0) {
            // holes in ascending order, filled by what stays from `keep` on
#pragma unroll
            for (int i = 0; i < kFew; ++i)
#pragma unroll
                for (int k = 0; k + 1 < kFew; ++k)
                    if (victim[k] > victim[k + 1]) {
                        const int v = victim[k];
                        victim[k] = victim[k + 1];
                        victim[k + 1] = v;
                    }
            int2 *moves = reinterpret_cast<int2 *>(a.moves) + row * a.max_moves;
            int from = a.keep, count = 0;
#pragma unroll
            for (int i = 0; i < kFew; ++i) {
                if (victim[i] >= a.keep) continue;
                bool again = true;
                while (again) {
                    again = false;
#pragma unroll
                    for (int k = 0; k < kFew; ++k)
                        if (victim[k] == from) again = true;
                    if (again) ++from;
                }
                if (count < a.max_moves) moves[count] = make_int2(from, victim[i]);
                ++count;
                ++from;
            }
            a.counts[row] = count;
        }
        // no block leaves while another may still read its shared memory
        if (blocks > 1) cluster.sync();
        return;
    }

    // first digit, over the slots that are not protected; how many are
    unsigned mine = 0;
    each([&](int, bool in, uint32_t k, bool prot) {
        if (in && !prot) atomicAdd(sh.bins(0) + (k >> 21), 1u);
        mine += in && prot;
    });
    const unsigned protect = reduce(mine, 1, OpSum());
    const bool cut = protect >= static_cast<unsigned>(a.keep);  // does the budget cut the protected class
    unsigned left = cut ? a.keep : a.keep - protect;
    if (cut) {  // rare: more protected slots than the budget
        each([&](int, bool in, uint32_t k, bool prot) {
            if (in && prot) atomicAdd(sh.bins(1) + (k >> 21), 1u);
        });
        sync_all();
    }
    pick(cut ? 1 : 0, left);
    uint32_t limit = sh.digit;
    left = sh.left;
    each([&](int, bool in, uint32_t k, bool prot) {
        if (in && prot == cut && (k >> 21) == limit) atomicAdd(sh.bins(2) + ((k >> 10) & 2047u), 1u);
    });
    sync_all();
    pick(2, left);
    limit = (limit << 11) | sh.digit;
    left = sh.left;
    each([&](int, bool in, uint32_t k, bool prot) {
        if (in && prot == cut && (k >> 10) == limit) atomicAdd(sh.bins(3) + (k & 1023u), 1u);
    });
    sync_all();
    pick(3, left);
    limit = (limit << 10) | sh.digit;
    left = sh.left;
    // `left` of the slots with exactly this key stay, the lowest first
    const bool all_ties = left == sh.count;
    const unsigned below = (1u << lane) - 1;
    unsigned tie0 = 0;  // ties in front of this warp's slots
    if (!all_ties) {
        unsigned c = 0;
        each([&](int, bool in, uint32_t k, bool prot) { c += in && prot == cut && k == limit; });
        c = __reduce_add_sync(kAll, c);
        if (lane == 0) sh.warp_ties[warp] = c;
        __syncthreads();
        if (warp == 0) {
            const unsigned s = __reduce_add_sync(kAll, lane < kWarps ? sh.warp_ties[lane] : 0u);
            if (lane == 0) sh.ties = s;
        }
        sync_all();
        total_of(&sh.ties, 1, &tie0);
        tie0 += __reduce_add_sync(kAll, lane < warp ? sh.warp_ties[lane] : 0u);
    }
    // calls f(slot, hole, mover) in slot order
    auto decide = [&](auto f) {
        unsigned ties = tie0;
        each([&](int j, bool in, uint32_t k, bool prot) {
            const bool tie = in && prot == cut && k == limit;
            bool stays = in && (prot == cut ? k > limit : !cut);  // with the others cut, protected slots stay
            if (all_ties) {
                stays = stays || tie;
            } else {
                const unsigned m = __ballot_sync(kAll, tie);
                stays = stays || (tie && ties + __popc(m & below) < left);
                ties += __popc(m);
            }
            const int64_t i = base + 32 * j;
            f(static_cast<int>(i), in && !stays && i < a.keep, stays && i >= a.keep);
        });
    };
    unsigned nh = 0, nm = 0;
    decide([&](int, bool hole, bool mover) {
        nh += hole;
        nm += mover;
    });
    nh = __reduce_add_sync(kAll, nh);
    nm = __reduce_add_sync(kAll, nm);
    if (lane == 0) {
        sh.warp_holes[warp] = nh;
        sh.warp_movers[warp] = nm;
    }
    __syncthreads();
    if (warp == 0) {
        const unsigned h = __reduce_add_sync(kAll, lane < kWarps ? sh.warp_holes[lane] : 0u);
        const unsigned m = __reduce_add_sync(kAll, lane < kWarps ? sh.warp_movers[lane] : 0u);
        if (lane == 0) {
            sh.holes = h;
            sh.movers = m;
        }
    }
    sync_all();
    unsigned hole_at, mover_at;
    total_of(&sh.holes, 2, &hole_at);
    const unsigned movers = total_of(&sh.movers, 3, &mover_at);
    hole_at += __reduce_add_sync(kAll, lane < warp ? sh.warp_holes[lane] : 0u);
    mover_at += __reduce_add_sync(kAll, lane < warp ? sh.warp_movers[lane] : 0u);
    int32_t *moves = a.moves + 2 * row * a.max_moves;
    decide([&](int i, bool hole, bool mover) {
        const unsigned h = __ballot_sync(kAll, hole), m = __ballot_sync(kAll, mover);
        const int64_t at = hole ? hole_at + __popc(h & below) : mover_at + __popc(m & below);
        if ((hole || mover) && at < a.max_moves) moves[2 * at + (hole ? 1 : 0)] = i;
        hole_at += __popc(h);
        mover_at += __popc(m);
    });
    if (tid == 0 && rank == 0) a.counts[row] = static_cast<int>(movers);
    // no block leaves while another may still read its shared memory
    if (blocks > 1) cluster.sync();
}

// Moves.  Sources lie at or behind `keep` and targets before it, so nothing
// is read that another thread writes and applying a plan twice changes
// nothing.  Bound by the bytes moved, once enough of them are in flight: a
// warp's lanes look up the pages of kApplyLook moves side by side, then the
// rows of kApplyBatch moves are requested before the first is written.  Rows
// of 256 bytes from anywhere in the pool to anywhere: 74000 moves take some
// 20 us, half the rate of a plain copy.  Four rows in flight per warp and 32
// warps on an SM (plan and moves 36.6 us) beat eight and 24 (38.1 us), sixteen
// and 16 (45.3 us), and dealing all moves evenly to a fitting grid with the
// next group's pages looked up ahead (41.1 us).
constexpr int kApplyThreads = 256;
constexpr int kApplyBatch = 4, kApplyLook = 8;

// Page of a slot, and its place in the page; -1 where it has no valid one.
__device__ __forceinline__ int64_t page_of(const KvView &kv, const int32_t *table, int slot, int *off)
{
    const int idx = kv.page_shift >= 0 ? slot >> kv.page_shift : slot / kv.page_size;
    *off = slot - idx * kv.page_size;
    const int page = __ldg(table + idx);
    return page >= 0 && page < kv.num_pages ? page : -1;
}

template <bool VEC>
__global__ void __launch_bounds__(kApplyThreads, 4) mbg_evict_apply_kernel(const __grid_constant__ EvictApplyArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int h = blockIdx.y, b = blockIdx.z;
    const int64_t row = static_cast<int64_t>(b) * gridDim.y + h;
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
    const int2 *moves = reinterpret_cast<const int2 *>(a.moves) + row * a.max_moves;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stride = gridDim.x * (kApplyThreads / 32) * kApplyLook;
    // lanes 0..15 move K, the others V
    const bool is_v = lane >= 16;
    const int64_t ps = is_v ? kv.vs_page : kv.ks_page, ts = is_v ? kv.vs_tok : kv.ks_tok,
                  hs = is_v ? kv.vs_head : kv.ks_head;
    uint16_t *pool = static_cast<uint16_t *>(is_v ? kv.v : kv.k) + h * hs;
    for (int64_t i0 = (blockIdx.x * (kApplyThreads / 32) + warp) * kApplyLook; i0 < count; i0 += stride) {
        // lanes 0..7: a move each
        int sp = -1, tp = -1, so = 0, to = 0;
        if (lane < kApplyLook && i0 + lane < count) {
            const int2 mv = __ldg(moves + i0 + lane);
            const bool in = mv.x >= 0 && mv.x < kv.capacity && mv.y >= 0 && mv.y < kv.capacity;
            if (in) {
                sp = static_cast<int>(page_of(kv, table, mv.x, &so));
                tp = static_cast<int>(page_of(kv, table, mv.y, &to));
            }
            if (sp < 0 || tp < 0) {
                report_error(a.err, DEVERR_BAD_INDEX);
                sp = -1;
            } else {
                if (a.scores) {
                    float *sc = a.scores + row * kv.capacity;
                    sc[mv.y] = sc[mv.x];
                }
                if (a.stamps) {
                    int32_t *st = a.stamps + row * kv.capacity;
                    st[mv.y] = st[mv.x];
                }
            }
        }
        for (int k0 = 0; k0 < kApplyLook && i0 + k0 < count; k0 += kApplyBatch) {
            for (int d = (lane & 15) * (VEC ? 8 : 1); d - (lane & 15) * (VEC ? 8 : 1) < kv.dim; d += VEC ? 128 : 16) {
                uint4 v[kApplyBatch];
#pragma unroll
                for (int k = 0; k < kApplyBatch; ++k) {
                    const int page = __shfl_sync(kAll, sp, k0 + k), off = __shfl_sync(kAll, so, k0 + k);
                    const uint16_t *src = pool + page * ps + off * ts + d;
                    if (page >= 0 && d < kv.dim) {
                        if (VEC)
                            v[k] = *reinterpret_cast<const uint4 *>(src);
                        else
                            v[k].x = *src;
                    }
                }
#pragma unroll
                for (int k = 0; k < kApplyBatch; ++k) {
                    const int live = __shfl_sync(kAll, sp, k0 + k);
                    const int page = __shfl_sync(kAll, tp, k0 + k), off = __shfl_sync(kAll, to, k0 + k);
                    uint16_t *dst = pool + page * ps + off * ts + d;
                    if (live >= 0 && d < kv.dim) {
                        if (VEC)
                            *reinterpret_cast<uint4 *>(dst) = v[k];
                        else
                            *dst = static_cast<uint16_t>(v[k].x);
                    }
                }
            }
        }
    }
}

template <typename Args>
cudaError_t launch_pdl(void (*fn)(Args), dim3 grid, int threads, int cluster, cudaStream_t s, const Args &args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_evict_plan(const EvictArgs &a, cudaStream_t s)
{
    // the smallest cluster whose threads hold a row of the cache's capacity
    // eight slots each (32 rows of 30011 slots: 17 us; four slots and twice
    // the blocks take 19 us more, sixteen and half of them 6 us more), then more
    // slots per thread, then rows of any length
    const int64_t cap = a.kv.capacity;
    int cluster = 1;
    while (cluster < kPlanMaxCluster && cap > static_cast<int64_t>(cluster) * kPlanThreads * 8) cluster *= 2;
    const int64_t each = (cap + cluster * kPlanThreads - 1) / (cluster * kPlanThreads);
    auto fn = each <= 4    ? mbg_evict_plan_kernel<4>
              : each <= 8  ? mbg_evict_plan_kernel<8>
              : each <= 16 ? mbg_evict_plan_kernel<16>
              : each <= 24 ? mbg_evict_plan_kernel<24>
                           : mbg_evict_plan_kernel<0>;
    const dim3 grid(static_cast<unsigned>(a.kv.batch) * a.kv.kv_heads * cluster);
    return launch_pdl(fn, grid, kPlanThreads, cluster, s, a);
}

cudaError_t launch_evict_apply(const EvictApplyArgs &a, bool vec, int sm_count, cudaStream_t s)
{
    // enough blocks per row to fill the GPU a few times over, and no more
    // than the moves there can be
    const int64_t rows = static_cast<int64_t>(a.kv.batch) * a.kv.kv_heads;
    const int64_t per_block = kApplyThreads / 32 * kApplyLook;
    int64_t x = (16ll * sm_count + rows - 1) / rows;
    const int64_t most = (a.max_moves + per_block - 1) / per_block;
    if (x > most) x = most;
    if (x < 1) x = 1;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(a.kv.kv_heads), static_cast<unsigned>(a.kv.batch));
    return launch_pdl(vec ? mbg_evict_apply_kernel<true> : mbg_evict_apply_kernel<false>, grid, kApplyThreads, 1, s, a);
}

}  // namespace mbg
