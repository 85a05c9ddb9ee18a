// Attention of many tokens on the tensor cores: the new tokens of prompts, and a
// batch's tokens over the prefix that its sequences share.
//
//   S = Q K^T,  P = softmax(scale S),  O = P V
//
// for the rows of a cached head: the group's query heads of all tokens of a
// sequence (or of all sequences, over the prefix), 128 rows to a tile.  At a
// head size of 128 a row and 128 slots take 32768 flop for S and as many for O, and a
// slot 256 bytes of K and 256 of V, which all rows of a block share: from some 280
// rows on the products bound it, with fewer the cache's bytes.
//
// One pass over the slots: each row keeps a running maximum m and sum l, and O
// is multiplied by 2^(m - m') when m grows (Milakov & Gimelshein's online
// softmax) -- here only when it grows by more than kLazy powers of two, so
// that most tiles leave O alone; P then exceeds 1 by at most that.
//
// Work of a block's warps:
//   warps 0-3, 4-7  two streams of softmax, a thread per row: S from tensor
//                   memory, P back over it, at the end O;
//   warps 8-11      K and V from their pages into swizzled shared memory: by bulk
//                   tensor copies (TMA) of the tokens of a page, a warp each for
//                   K and V, or, where pages are not of a multiple of 8 tokens or
//                   heads are narrower than 64, 16 bytes at a time (cp.async), and
//                   unaligned pools element by element;
//   warp 12         issues the products;
//   warp 13         looks up what the block does next;
//   warps 14, 15    make what is copied piece by piece visible to the tensor core (a
//                   fence of some 0.2 us, during which the products would pause).
// While one stream's softmax runs, the other's products do.  The streams are two
// tiles of rows over the same slots, or with up to 128 rows one tile of
// rows over even and odd tiles of slots, joined at the end.  (Head sizes above
// 128: one stream with two buffers of S, O takes half of tensor memory.)
//
// What it measured: a tile of 128 slots for both streams takes 2.3 us (head size
// 128), of which the tensor core works 1.9 (48 instructions of 64 cycles; 0.93 us
// per stream are some 75 cycles each).  A stream's own chain is as long: S 0.31, the
// softmax 0.9, hand-overs 0.5, P V 0.62.  2000 new tokens behind up to 12000 cached ones, six
// sequences: 593 us, 869 TFLOP/s counted without P's second part; with copies
// piece by piece 835 us (a place of the ring is free for shorter than they
// need to be issued, 0.65 us, and to arrive).  Tiles of 64 slots with two
// buffers of S: 990 us -- the products' scores are read at half the width and their
// waits come twice as often.
//
// P enters the value product in two 16-bit parts, 16 bits (bf16) or 22 (f16) of
// FP32's 24: one part would add an error as large as the output's own rounding.
// The second one is a third of the products.  In f16 P is multiplied by
// 2^11, so that what is small beside the largest weight is kept down to 2^-35 of it.
//
// A weight of 0 times an infinite value is NaN, and a tile's values meet the rows
// that do not see them too: rows with a NaN are computed once more, alone
// (gemv_span.cu).  So are the rows of a segment in which a page does not exist: its
// slots are copied as zeros, and the rows become NaN on purpose.  (Scores of such slots
// set to -inf tile by tile, by bits beside K, keep the tiles' speed there and cost
// it everywhere else: a prompt of 9001 tokens 439 -> 485 us, so 461.)
//
// Blocks of rows are cut between the CTAs: all tiles of a call are numbered and
// each CTA takes an equal share of consecutive ones, whatever the lengths (read
// on the device).  A block inside one share is written at once, others
// leave (O, m, l) in the workspace for a second launch, in a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "gemv_decode.h"
#include "gemv_device.cuh"
#include "gemv_span.cuh"
#include "gemv_tcgen05.cuh"

namespace mbg {
namespace tile {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 512, kRows = 128;
constexpr uint32_t kSegs = 4;  // segments looked up ahead
constexpr uint32_t kSkipped = 2;  // the tile of K that the test hook withholds

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// DC: head sizes up to 64 DC.
template <int DC>
struct Shape {
    static constexpr int kStreams = DC <= 2 ? 2 : 1;
    static constexpr int kTok = DC <= 2 ? 128 : 64;  // slots of a tile
    static constexpr int kBufs = DC <= 2 ? 1 : 2;    // tiles of S or P that a stream has in tensor memory
    static constexpr int kQBytes = kRows * DC * 128; // a tile of rows
    static constexpr int kKvBytes = kTok * DC * 128;
    static constexpr int kStages = DC == 1 ? 4 : DC == 3 ? 3 : 2;  // tiles of K, and of V, in shared memory
    static constexpr int kBlock = kStreams * kRows;  // rows of a block
    static constexpr int kMost = 32768 / kTok;       // tiles of a segment
    static constexpr int kOColumn = 256;
};

// A block of rows and its tiles of slots: tile j is tile j of the sequence for
// j < sink_tiles, and tile j + skip behind them.
struct Block {
    int tiles, sink_tiles, skip;
    int lo, hi, sinks;  // some row sees [lo, hi) and, before hi, [0, sinks)
    int rows;
};

// What a CTA does next: tiles [t0, t1) of a block.  Not more than 32768 slots at
// a time: the tensor core adds products to O with the bits that O leaves
// them, cut off, so that a long sum comes out too small (equal weights, positive
// values, binary16: by 0.1 of 2^-12 after 32768 slots, by 2.3 after 131072, by 27
// after 2^20).  What has been summed up is put aside and joined in FP32.  (And
// no wait of another warp lasts longer than a few segments.)
struct Segment {
    span::Seq seq;
    Block block;
    int h, row0;      // cached head, first row among its sequence's
    int t0, t1;
    int slot;         // of the part; -1: the whole block
    int aside;        // where sums are put aside
    int more, merge;  // some tiles follow; others came before
    int stop;         // nothing is left
    int missing;      // rows see a slot whose page does not exist
};

// The block, and the cached head, that is looked at next.
struct Cursor {
    int64_t before;   // cost of what lies before the block, per cached head
    int b, row0, h;
    int done;         // tiles of this CTA's share of it that are behind
    int top;          // the largest start of a sequence so far
    span::Seq seq;
    Block block;
};

struct Limits {
    int shortest, longest;  // prefix: lengths of the batch
};

template <int DC>
__device__ __forceinline__ Block block_of(const SpanArgs &a, const span::Seq &s, int row0, const Limits &lim)
{
    constexpr int T = Shape<DC>::kTok;
    Block k;
    k.rows = min(Shape<DC>::kBlock, s.m * a.group - row0);
    if (a.prefix) {
        k.lo = a.window > 0 && lim.shortest > a.window ? lim.shortest - a.window : 0;
        k.hi = min(s.n, lim.longest);
    } else {
        k.lo = span::seen_by(a, s, row0 / a.group).lo;
        k.hi = span::seen_by(a, s, (row0 + k.rows - 1) / a.group).hi;
    }
    k.sinks = min(a.sinks, k.hi);
    if (k.lo <= k.sinks) k.lo = k.sinks = 0;
    k.sink_tiles = (k.sinks + T - 1) / T;
    const int first = k.lo / T, last = (k.hi + T - 1) / T;
    if (k.lo >= k.hi) {
        k.tiles = k.sink_tiles;
        k.skip = 0;
    } else if (first < k.sink_tiles) {  // they meet in a tile
        k.tiles = last;
        k.sink_tiles = k.skip = 0;
    } else {
        k.tiles = k.sink_tiles + last - first;
        k.skip = first - k.sink_tiles;
    }
    return k;
}

// Costs, in units of some 0.5 us: a tile of slots for two tiles of rows, for
// one, and a block's beginning and end.
constexpr int kLead = 12;
template <int DC>
__device__ __forceinline__ int per_tile(const Block &k) { return k.rows > kRows ? 5 : 4; }
template <int DC>
__device__ __forceinline__ int cost_of(const Block &k) { return kLead + k.tiles * per_tile<DC>(k); }

template <int DC>
struct Shared {
    // of each place in the rings of K and V: copied; visible to the tensor core; free
    alignas(8) uint64_t kthere[Shape<DC>::kStages], kfull[Shape<DC>::kStages], kempty[Shape<DC>::kStages];
    alignas(8) uint64_t vthere[Shape<DC>::kStages], vfull[Shape<DC>::kStages], vempty[Shape<DC>::kStages];
    alignas(8) uint64_t sready[2][2], pready[2][2], vdone[2], qready, meet, last, segfull[kSegs], segempty[kSegs];
    uint32_t tmem;
    int abort;
    Segment seg[kSegs];
    Limits lim;
    Cursor first;     // where the CTA's share begins
    int64_t warp_sum[2][kThreads / 32];
    int ends[kThreads];
    float join_m[kRows], join_l[kRows];
};

// One share: [x0, x1) of the call's total.
struct Share {
    int64_t x0, x1;
    int near;  // cuts that leave so few tiles of a block move to its end
};

template <typename T, int DC, bool VEC>
struct Kernel {
    using S = Shape<DC>;
    static constexpr bool kBf16 = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value;
    static constexpr int kTok = S::kTok;
    // P is at most 2^kLazy times kUp: in f16 below 2^16
    static constexpr float kLazy = kBf16 ? 8.f : 4.f, kUp = kBf16 ? 0.f : 11.f;

    static __device__ __forceinline__ bool wait(Shared<DC> &sh, uint64_t &bar, uint32_t parity, const SpanArgs &a)
    {
        if (mbar_wait_bounded(smem_addr(&bar), parity, a.wait_limit_ns)) return true;
        report_error(a.err, DEVERR_TIMEOUT);
        sh.abort = 1;
        return false;
    }

    // Sum over the block up to and with this thread's value; one barrier.
    static __device__ int64_t scan(Shared<DC> &sh, int &turn, int64_t v, int64_t *all)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int64_t *sums = sh.warp_sum[turn];
        turn ^= 1;
#pragma unroll
        for (int x = 1; x < 32; x *= 2) {
            const int64_t u = __shfl_up_sync(kFull, v, x);
            if (lane >= x) v += u;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        int64_t t = lane < kThreads / 32 ? sums[lane] : 0;
#pragma unroll
        for (int x = 1; x < kThreads / 32; x *= 2) {
            const int64_t u = __shfl_up_sync(kFull, t, x);
            if (lane >= x) t += u;
        }
        *all = __shfl_sync(kFull, t, kThreads / 32 - 1);
        const int64_t before = __shfl_sync(kFull, t, warp ? warp - 1 : 0);
        return warp ? before + v : v;
    }

    // All blocks of rows in order, kThreads at a time: f(sequence, first row,
    // block, cost of the blocks before) is called by one thread for each.
    // Returns their cost together; *once: no thread had more than one.
    template <typename F>
    static __device__ int64_t for_blocks(const SpanArgs &a, Shared<DC> &sh, F f, bool *once)
    {
        const int batch = a.prefix ? 1 : a.kv.batch, tid = threadIdx.x;
        int64_t before = 0;
        int turn = 0, top = 0;
        bool ascend = true;
        *once = batch <= kThreads;
        for (int b0 = 0; b0 < batch; b0 += kThreads) {
            int64_t blocks = 0, all = 0;
            span::Seq own = {0, 0, 0, 0};
            int from = 0;
            bool falls = false;
            if (b0 + tid < batch) {
                own = span::seq_of(a, b0 + tid, blockIdx.x == 0);
                blocks = (static_cast<int64_t>(own.m) * a.group + S::kBlock - 1) / S::kBlock;
                from = __ldg(a.starts + b0 + tid);
                falls = __ldg(a.starts + b0 + tid + 1) < from;
            }
            ascend = !__syncthreads_or(falls) && ascend;
            if (!ascend) {  // sequences that begin below an earlier one's start have no tokens
                sh.ends[tid] = from;
                __syncthreads();
                int high = top;
                for (int i = 0; i < min(kThreads, batch - b0); ++i) {
                    if (i == tid && from < high) blocks = 0;
                    high = max(high, sh.ends[i]);
                }
                top = high;
                __syncthreads();
            } else {
                top = max(top, __ldg(a.starts + min(b0 + kThreads, batch)));
            }
            const int64_t end = scan(sh, turn, blocks, &all);
            sh.ends[tid] = static_cast<int>(end);
            __syncthreads();
            if (all > kThreads) *once = false;
            for (int64_t i0 = 0; i0 < all; i0 += kThreads) {
                const int64_t i = i0 + tid;
                int cost = 0;
                span::Seq s;
                Block k;
                int row0 = 0;
                if (i < all) {
                    int lo = 0, hi = min(kThreads, batch - b0) - 1;  // the first whose end lies above i
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (sh.ends[mid] > i)
                            hi = mid;
                        else
                            lo = mid + 1;
                    }
                    row0 = static_cast<int>(i - (lo ? sh.ends[lo - 1] : 0)) * S::kBlock;
                    s = span::seq_of(a, b0 + lo, false);
                    k = block_of<DC>(a, s, row0, sh.lim);
                    cost = cost_of<DC>(k);
                }
                int64_t sum;
                const int64_t to = scan(sh, turn, cost, &sum);
                if (i < all) f(s, row0, k, before + to - cost);
                before += sum;
            }
            __syncthreads();
        }
        return before;
    }

    // The tile before which a block that begins at r0 is cut at x.
    static __device__ __forceinline__ int cut(const Block &k, int64_t r0, int64_t x, int near)
    {
        if (x <= r0) return 0;
        if (x >= r0 + cost_of<DC>(k)) return k.tiles;
        const int t = max(0, static_cast<int>(x - r0) - kLead) / per_tile<DC>(k);
        return t <= near ? 0 : k.tiles - t <= near ? k.tiles : t;
    }

    // Looks up the CTA's next segment (one thread).
    static __device__ void advance(const SpanArgs &a, const Shared<DC> &sh, const Share &w, Cursor &at, Segment &out)
    {
        const int batch = a.prefix ? 1 : a.kv.batch;
        while (at.b < batch) {
            if (at.h == a.kv.kv_heads) {  // the next block
                at.before += cost_of<DC>(at.block);
                at.row0 += S::kBlock;
                at.h = 0;
                while (at.row0 >= at.seq.m * a.group) {
                    at.row0 = 0;
                    if (++at.b >= batch) break;
                    at.seq = span::seq_behind(a, at.b, at.top);
                }
                if (at.b >= batch) break;
                at.block = block_of<DC>(a, at.seq, at.row0, sh.lim);
            }
            const Block &k = at.block;
            const int64_t r0 = at.before * a.kv.kv_heads + static_cast<int64_t>(at.h) * cost_of<DC>(k);
            if (r0 >= w.x1) break;
            const int t0 = cut(k, r0, w.x0, w.near), t1 = cut(k, r0, w.x1, w.near);
            // (a block without slots is its beginning's)
            if (t0 < t1 || (k.tiles == 0 && r0 >= w.x0)) {
                const int mine = 2 * static_cast<int>(blockIdx.x);
                out.seq = at.seq;
                out.block = k;
                out.h = at.h;
                out.row0 = at.row0;
                out.t0 = t0 + at.done;
                out.t1 = min(t1, out.t0 + S::kMost);
                out.slot = t0 == 0 && t1 == k.tiles ? -1 : mine + (t0 == 0 ? 1 : 0);
                out.aside = out.slot >= 0 ? out.slot : mine + 1;  // (a part there would be the CTA's last)
                out.merge = at.done > 0;
                out.more = out.t1 < t1;
                out.stop = out.missing = 0;
                at.done = out.more ? out.t1 - t0 : 0;
                if (!out.more) ++at.h;
                return;
            }
            ++at.h;
        }
        at.b = batch;
        out.stop = 1;
    }

    // ---------------------------------------------------------------- loading

    static __device__ __forceinline__ uint32_t swizzled(int rows, int row, int chunk)
    {
        return static_cast<uint32_t>((chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    }

    static __device__ __forceinline__ uint4 load8(const uint16_t *p, int left)
    {
        if (VEC) return left > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < left ? p[2 * i] : 0, hi = 2 * i + 1 < left ? p[2 * i + 1] : 0;
            w[i] = lo | hi << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }

    static __device__ __forceinline__ void st_shared(uint32_t addr, uint4 v)
    {
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    }

    // OWN of ROWS rows in shared memory, from row0 on: those that begin at `at`
    // (a lane each; -1: zeros).
    template <int OWN, int ROWS>
    static __device__ __forceinline__ void load_rows(uint32_t dst, const uint16_t *base, int64_t at, int dim, int row0, int lane)
    {
        constexpr int kLanes = DC == 1 ? 8 : DC == 2 ? 16 : 32;   // of a row
        constexpr int kAtOnce = 32 / kLanes;
        const int chunk = lane % kLanes, sub = lane / kLanes;
#pragma unroll 4
        for (int i = 0; i < OWN; i += kAtOnce) {
            const int own = i + sub;
            const int64_t from = __shfl_sync(kFull, at, own);
            if (chunk >= DC * 8) continue;
            const int left = from >= 0 ? dim - chunk * 8 : 0;
            const uint32_t to = dst + swizzled(ROWS, row0 + own, chunk);
            const uint16_t *p = base + (left > 0 ? from + chunk * 8 : 0);
            if (VEC) {
                asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(left > 0 ? 16 : 0)
                             : "memory");
            } else {
                st_shared(to, left > 0 ? load8(p, left) : make_uint4(0, 0, 0, 0));
            }
        }
    }

    static __device__ void loader(const SpanArgs &a, Shared<DC> &sh, uint32_t ks, uint32_t vs)
    {
        const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 8;
        const KvView &kv = a.kv;
        constexpr int kOwn = kTok / 4;
        // arrives when this thread's copies so far have landed
        auto issued = [&](uint64_t &bar) {
            if (VEC) {
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&bar)) : "memory");
            } else {
                mbar_arrive(smem_addr(&bar));
            }
        };
        auto free_place = [&](uint64_t &bar, uint32_t parity) { return static_cast<bool>(__all_sync(kFull, wait(sh, bar, parity, a))); };
        uint32_t nk = 0, nv = 0;
        for (uint32_t n = 0;; ++n) {
            if (!__all_sync(kFull, wait(sh, sh.segfull[n % kSegs], n / kSegs & 1, a))) break;
            const Segment &g = sh.seg[n % kSegs];
            if (g.stop) break;
            const int32_t *table = kv.table + g.seq.b * kv.table_stride;
            const int t0 = g.t0, t1 = g.t1, sink_tiles = g.block.sink_tiles, skip = g.block.skip;
            const int lo = g.block.lo, hi = g.block.hi, sinks = g.block.sinks;
            const uint16_t *kb = static_cast<const uint16_t *>(kv.k) + g.h * kv.ks_head;
            const uint16_t *vb = static_cast<const uint16_t *>(kv.v) + g.h * kv.vs_head;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.segempty[n % kSegs]));
            bool ok = true;
            // this lane's slot of a tile: its page (-1: none) and place there
            auto look_up = [&](int j, int &off) {
                const int slot = (j < sink_tiles ? j : j + skip) * kTok + warp * kOwn + lane;
                int page = -1;
                off = 0;
                if (j < t1 && lane < kOwn && slot < hi && (slot >= lo || slot < sinks)) {
                    const int idx = kv.page_shift >= 0 ? slot >> kv.page_shift : slot / kv.page_size;
                    off = slot - idx * kv.page_size;
                    page = __ldg(table + idx);
                }
                return page;
            };
            auto checked = [&](int page) {
                if (page < -1 || page >= kv.num_pages) page = -1;
                return page;
            };
            auto report = [&](int j, int page, int off) {
                const int slot = (j < sink_tiles ? j : j + skip) * kTok + warp * kOwn + lane;
                if (j < t1 && lane < kOwn && slot < hi && (slot >= lo || slot < sinks) && (page < 0 || page >= kv.num_pages)) {
                    report_error(a.err, DEVERR_BAD_INDEX);
                    sh.seg[n % kSegs].missing = 1;  // (the softmax keeps the segment until its rows are written)
                }
            };
            int off_k = 0, off_v = 0, page_v = -1;
            int page_k = look_up(t0, off_k);
            report(t0, page_k, off_k);
            page_k = checked(page_k);
            for (int j = t0; j <= t1 && ok; ++j) {  // K of tile j, then V of tile j - 1
                int off_next = 0, page_next = -1;
                if (j < t1) {
                    page_next = look_up(j + 1, off_next);
                    const int st = nk % S::kStages;
                    if (a.skip_tile && nk == kSkipped) {
                        ok = false;
                        break;
                    }
                    ok = free_place(sh.kempty[st], (nk / S::kStages & 1) ^ 1);
                    if (!ok) break;
                    load_rows<kOwn, kTok>(ks + st * S::kKvBytes, kb, page_k < 0 ? -1 : page_k * kv.ks_page + off_k * kv.ks_tok, kv.dim,
                                          warp * kOwn, lane);
                    issued(sh.kthere[st]);
                    ++nk;
                }
                if (j > t0) {
                    const int st = nv % S::kStages;
                    ok = free_place(sh.vempty[st], (nv / S::kStages & 1) ^ 1);
                    if (!ok) break;
                    load_rows<kOwn, kTok>(vs + st * S::kKvBytes, vb, page_v < 0 ? -1 : page_v * kv.vs_page + off_v * kv.vs_tok, kv.dim,
                                          warp * kOwn, lane);
                    issued(sh.vthere[st]);
                    ++nv;
                }
                page_v = page_k;
                off_v = off_k;
                report(j + 1, page_next, off_next);
                page_k = checked(page_next);
                off_k = off_next;
            }
            if (!ok) break;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }

    // Bulk copies, K's and V's by a warp each.  A lane takes one box: `box` tokens
    // of a page x 64 elements.  Boxes that no row sees, and pages that do not
    // exist, are asked for outside the pool, which gives zeros.  They arrive by
    // themselves at `full`; a tile of V in which a sequence ends inside a box goes
    // by `there` and zero_v.
    static __device__ void bulk_loader(const SpanArgs &a, Shared<DC> &sh, uint32_t dst, bool is_v)
    {
        const int lane = threadIdx.x & 31, box = a.box, boxes = kTok / box;  // of 64 elements of a tile
        const KvView &kv = a.kv;
        uint64_t *full = is_v ? sh.vfull : sh.kfull, *empty = is_v ? sh.vempty : sh.kempty;
        const CUtensorMap *map = is_v ? &a.v_map : &a.k_map;
        const int group = lane % boxes, chunk = lane / boxes;
        uint32_t count = 0, edges = 0;  // edges: the places whose last tile went by `there`, and the phases of those
        uint32_t phases = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            ok = __all_sync(kFull, wait(sh, sh.segfull[n % kSegs], n / kSegs & 1, a));
            if (!ok) break;
            const Segment &g = sh.seg[n % kSegs];
            if (g.stop) break;
            const int32_t *table = kv.table + g.seq.b * kv.table_stride;
            const int t0 = g.t0, t1 = g.t1, h = g.h;
            const int length = g.seq.n;
            const Block k = g.block;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.segempty[n % kSegs]));
            // this lane's box of a tile: its page (num_pages: none) and place there
            auto look_up = [&](int j, int &off) {
                const int slot = slot_of(k, j) + group * box;
                int page = -1;
                off = 0;
                if (j < t1 && (max(slot, k.lo) < min(slot + box, k.hi) || slot < min(k.sinks, k.hi))) {
                    const int idx = kv.page_shift >= 0 ? slot >> kv.page_shift : slot / kv.page_size;
                    off = slot - idx * kv.page_size;
                    page = __ldg(table + idx);
                    if (page < 0 || page >= kv.num_pages) {
                        if (!is_v && chunk == 0) {
                            report_error(a.err, DEVERR_BAD_INDEX);
                            sh.seg[n % kSegs].missing = 1;  // (the softmax keeps the segment until its rows are written)
                        }
                        page = -1;
                    }
                }
                return page < 0 ? static_cast<int>(kv.num_pages) : page;
            };
            int off = 0, page = look_up(t0, off);
            for (int j = t0; j < t1; ++j, ++count) {
                const int st = count % S::kStages;
                if (a.skip_tile && !is_v && count == kSkipped) {
                    ok = false;
                    break;
                }
                ok = __all_sync(kFull, wait(sh, empty[st], (count / S::kStages & 1) ^ 1, a));
                if (!ok) break;
                const bool edge = is_v && ends_in(slot_of(k, j), length, box);
                uint64_t *bar = edge ? &sh.vthere[st] : &full[st];
                edges = (edges & ~(1u << st)) | static_cast<uint32_t>(edge) << st;
                if (edge) phases ^= 1u << st;
                if (lane == 0) mbar_arrive_expect_tx(smem_addr(bar), S::kKvBytes);
                __syncwarp();
                if (lane < boxes * DC)
                    tc::load_box(dst + st * S::kKvBytes + chunk * (kTok * 128) + group * box * 128, map, chunk * 64, off, h, page,
                                 smem_addr(bar));
                page = look_up(j + 1, off);
            }
        }
        // no copy is left under way, had others given up too
        for (uint32_t i = count > S::kStages ? count - S::kStages : 0; i < count; ++i) {
            const int st = i % S::kStages;
            const bool edge = edges >> st & 1;
            const bool done = wait(sh, edge ? sh.vthere[st] : full[st], edge ? (phases >> st & 1) ^ 1 : i / S::kStages & 1, a);
            if (!__all_sync(kFull, done) && lane == 0) report_error(a.err, DEVERR_UNDRAINED);
        }
    }

    static __device__ __forceinline__ int slot_of(const Block &k, int j) { return (j < k.sink_tiles ? j : j + k.skip) * kTok; }

    // Does a sequence of so many slots end inside a box of this tile?
    static __device__ __forceinline__ bool ends_in(int slot, int length, int box)
    {
        return length > slot && length < slot + kTok && length % box != 0;
    }

    // What lies in the box behind a sequence's last slot was perhaps never written:
    // it becomes zeros.  (Other slots that a row does not see hold values, whose
    // weights are 0.)
    static __device__ void zero_v(const SpanArgs &a, Shared<DC> &sh, uint32_t vs)
    {
        const int lane = threadIdx.x & 31, box = a.box;
        uint32_t count = 0, phases = 0;
        for (uint32_t n = 0;; ++n) {
            if (!__all_sync(kFull, wait(sh, sh.segfull[n % kSegs], n / kSegs & 1, a))) return;
            const Segment &g = sh.seg[n % kSegs];
            if (g.stop) return;
            const int t0 = g.t0, t1 = g.t1, length = g.seq.n;
            const Block k = g.block;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.segempty[n % kSegs]));
            for (int j = t0; j < t1; ++j, ++count) {
                const int st = count % S::kStages, first = slot_of(k, j);
                if (!ends_in(first, length, box)) continue;
                if (!__all_sync(kFull, wait(sh, sh.vthere[st], phases >> st & 1, a))) return;
                phases ^= 1u << st;
                for (int r = length - first; r % box != 0; ++r)
                    if (lane < DC * 8) st_shared(vs + st * S::kKvBytes + swizzled(kTok, r, lane), make_uint4(0, 0, 0, 0));
                tc::fence_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.vfull[st]));
            }
        }
    }

    // --------------------------------------------------------------- products

    // Tiles that have been copied (to `there`) are made visible to the tensor core.
    static __device__ void pass_on(const SpanArgs &a, Shared<DC> &sh, uint64_t *there, uint64_t *full)
    {
        uint32_t n = 0;
        for (uint32_t k = 0;; ++k) {
            if (!wait(sh, sh.segfull[k % kSegs], k / kSegs & 1, a)) return;
            if (sh.seg[k % kSegs].stop) return;
            const int tiles = sh.seg[k % kSegs].t1 - sh.seg[k % kSegs].t0;
            mbar_arrive(smem_addr(&sh.segempty[k % kSegs]));
            for (int j = 0; j < tiles; ++j, ++n) {
                if (!wait(sh, there[n % S::kStages], n / S::kStages & 1, a)) return;
                tc::fence_smem();
                mbar_arrive(smem_addr(&full[n % S::kStages]));
            }
        }
    }

    // One warp issues all products; none is under way when it leaves.
    static __device__ void products(const SpanArgs &a, Shared<DC> &sh, uint32_t qs, uint32_t ks, uint32_t vs)
    {
        issue(a, sh, qs, ks, vs);
        __syncwarp();
        if (tc::elect()) tc::commit(smem_addr(&sh.last));
        wait(sh, sh.last, 0, a);
    }

    static __device__ __forceinline__ bool warp_wait(Shared<DC> &sh, uint64_t &bar, uint32_t parity, const SpanArgs &a)
    {
        return __all_sync(kFull, wait(sh, bar, parity, a));
    }

    // The whole warp goes through this with the same values, so that operands and
    // descriptors are kept once per warp, as the instruction takes them; they
    // differ by constants within a tile, and the loops are unrolled.  An
    // instruction of 64 cycles has to be issued in less: by one thread of
    // a diverged warp it takes 90.
    static __device__ void issue(const SpanArgs &a, Shared<DC> &sh, uint32_t qs, uint32_t ks, uint32_t vs)
    {
        const int lane = threadIdx.x & 31;
        const uint32_t tmem = tc::uniform(sh.tmem);
        qs = tc::uniform(qs), ks = tc::uniform(ks), vs = tc::uniform(vs);
        const int k16 = (a.kv.dim + 15) / 16;
        // (a negative scale: the scores' signs change, the softmax goes by its size)
        const uint32_t s_instr = tc::instruction<kBf16>(kTok, false, a.scale_log2 < 0.f);
        const uint32_t o_instr = tc::instruction<kBf16>(k16 * 16, true, false);
        uint32_t nk = 0, nv = 0, nq = 0, np = 0;  // np: a bit per buffer of P, the phase of the next wait
        for (uint32_t n = 0;; ++n) {
            if (!warp_wait(sh, sh.segfull[n % kSegs], n / kSegs & 1, a)) return;
            const Segment &g = sh.seg[n % kSegs];
            if (tc::uniform(g.stop)) return;
            const int tiles = tc::uniform(g.t1 - g.t0);
            const bool both = tc::uniform(g.block.rows > kRows);
            if (tc::elect()) mbar_arrive(smem_addr(&sh.segempty[n % kSegs]));
            if (tiles == 0) continue;
            if (!warp_wait(sh, sh.qready, nq++ & 1, a)) return;
            tc::fence_after();
            // step s: stream s % kStreams, whose tiles go through its buffers in turn
            const int steps = both ? 2 * tiles : tiles;
            auto scores = [&](int s) {
                const int w = s % S::kStreams, buf = s / S::kStreams % S::kBufs, st = nk % S::kStages;
                const uint64_t q = tc::descriptor(qs + (both ? w * S::kQBytes : 0), 16), k = tc::descriptor(ks + st * S::kKvBytes, 16);
                const uint32_t d = tmem + (w * S::kBufs + buf) * kTok;
                const bool last = !both || w == 1;  // of those that read this tile
                if (tc::elect()) {
#pragma unroll
                    for (int i = 0; i < DC * 4; ++i)
                        if (i < k16)
                            tc::mma_ss(d, tc::further(q, (i >> 2) * (kRows * 128) + (i & 3) * 32),
                                       tc::further(k, (i >> 2) * (kTok * 128) + (i & 3) * 32), s_instr, i > 0);
                    tc::commit(smem_addr(&sh.sready[w][buf]));
                    if (last) tc::commit(smem_addr(&sh.kempty[st]));
                }
                if (last) ++nk;
            };
            constexpr int kAhead = S::kBufs * S::kStreams;
            bool ok = true;
            for (int s = 0; s < kAhead && s < steps && ok; ++s) {
                if (!both || s % S::kStreams == 0) ok = warp_wait(sh, sh.kfull[nk % S::kStages], nk / S::kStages & 1, a);
                if (ok) scores(s);
            }
            for (int s = 0; s < steps && ok; ++s) {
                const int w = s % S::kStreams, buf = s / S::kStreams % S::kBufs, st = nv % S::kStages, b = w * S::kBufs + buf;
                // P, V and K of the buffer's next tile are waited for at once, a lane each
                const bool begins = !both || w == 0;  // of the steps that read these tiles
                uint64_t *bar = &sh.pready[w][buf];
                uint32_t parity = np >> b & 1;
                if (lane == 1 && begins) bar = &sh.vfull[st], parity = nv / S::kStages & 1;
                if (lane == 2 && begins && s + kAhead < steps) bar = &sh.kfull[nk % S::kStages], parity = nk / S::kStages & 1;
                ok = warp_wait(sh, *bar, parity, a);
                np ^= 1u << b;
                if (!ok) break;
                tc::fence_after();
                const uint64_t v = tc::descriptor(vs + st * S::kKvBytes, kTok * 128);
                const uint32_t p = tmem + b * kTok, o = tmem + S::kOColumn + w * (DC * 64);
                const bool add = s >= S::kStreams, last = !both || w == 1;
                if (tc::elect()) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int i = 0; i < kTok / 16; ++i)
                            tc::mma_ts(o, p + i / 2 * 32 + part * 16 + i % 2 * 8, tc::further(v, i * 2048), o_instr,
                                       add || part > 0 || i > 0);
                    tc::commit(smem_addr(&sh.vdone[w]));
                    if (last) tc::commit(smem_addr(&sh.vempty[st]));
                }
                if (last) ++nv;
                if (s + kAhead < steps) scores(s + kAhead);
            }
            if (!ok) return;
        }
    }

    // ---------------------------------------------------------------- softmax

    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        uint32_t r;
        if (kBf16)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        else
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }

    // Two weights as 16-bit parts whose sum they are, but for the last part's rounding.
    static __device__ __forceinline__ void split(float p0, float p1, uint32_t &hi, uint32_t &lo)
    {
        if (kBf16) {
            hi = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
            const float2 rest = apart(add2(two(p0, p1), two(__uint_as_float((__float_as_uint(p0) & 0xFFFF0000u) ^ 0x80000000u),
                                                            __uint_as_float((__float_as_uint(p1) & 0xFFFF0000u) ^ 0x80000000u))));
            lo = pack(rest.x, rest.y);
        } else {
            hi = pack(p0, p1);
            const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            lo = pack(p0 - back.x, p1 - back.y);
        }
    }

    // The lowest n bits of 32.
    static __device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

    // Two FP32 operations in one instruction.
    static __device__ __forceinline__ uint64_t two(float a, float b)
    {
        uint64_t r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
        return r;
    }
    static __device__ __forceinline__ float2 apart(uint64_t v)
    {
        float2 r;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
        return r;
    }
    static __device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
    {
        uint64_t r;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
        return r;
    }
    static __device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
    {
        uint64_t r;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
        return r;
    }

    // This thread's row of a segment: a query head of a token.
    struct Row {
        bool live;
        int token, head;
    };
    static __device__ __forceinline__ Row row_of(const SpanArgs &a, const Segment &g, int stream, int row)
    {
        Row r;
        const int i = g.row0 + (g.block.rows > kRows ? stream * kRows : 0) + row;
        r.live = i < g.row0 + g.block.rows;
        r.token = r.live ? i / a.group : 0;
        r.head = g.h * a.group + (r.live ? i - r.token * a.group : 0);
        return r;
    }

    // Requests a warp's 32 rows of Q (those of stream 1 only where it has rows of its own).
    static __device__ __forceinline__ void load_q(const SpanArgs &a, const Segment &g, const Row &r, uint32_t qs, int stream, int row, int lane)
    {
        const bool both = g.block.rows > kRows;
        if (g.t0 == g.t1 || (!both && stream == 1)) return;
        const int64_t at = r.live ? (g.seq.q0 + r.token) * a.q_st + r.head * a.q_sh : -1;
        load_rows<32, kRows>(qs + (both ? stream * S::kQBytes : 0), static_cast<const uint16_t *>(a.q), at, a.kv.dim, row & 96, lane);
    }

    // Multiplies this warp's rows of O by f.
    static __device__ __forceinline__ void scale_o(uint32_t o, float f, int dim)
    {
        for (int c = 0; c < dim; c += 16) {
            float x[16];
            tc::load16(o + c, x);
            tc::wait_ld();
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(x[i] * f);
            tc::store16(o + c, y);
        }
        tc::wait_st();
    }

    // The streams' threads meet.
    static __device__ __forceinline__ bool all_softmax(const SpanArgs &a, Shared<DC> &sh, uint32_t &count)
    {
        mbar_arrive(smem_addr(&sh.meet));
        return __all_sync(kFull, wait(sh, sh.meet, count++ & 1, a));
    }

    static __device__ void softmax(const SpanArgs &a, Shared<DC> &sh, uint32_t qs, unsigned char *q_generic)
    {
        const int stream = threadIdx.x >> 7, row = threadIdx.x & 127, lane = threadIdx.x & 31;
        const uint32_t tmem = sh.tmem + (static_cast<uint32_t>(row & 96) << 16);
        const uint32_t o_at = tmem + S::kOColumn + stream * (DC * 64);
        const KvView &kv = a.kv;
        // phases: of the buffers of S (a bit each), of the products with V, of the
        // streams' meetings
        uint32_t ns = 0, nv = 0, nm = 0;
        if (stream >= S::kStreams) return;
        if (!next_segment(a, sh, 0, stream, row, lane, qs)) return;
        for (uint32_t n = 0; !sh.seg[n % kSegs].stop; ++n) {
            // (what a loop over the tiles does not need is looked up again behind it:
            // 128 scores leave few registers)
            const Segment &g = sh.seg[n % kSegs];
            const int tiles = g.t1 - g.t0, from = g.t0, sink_tiles = g.block.sink_tiles, skip = g.block.skip;
            const bool both = g.block.rows > kRows;
            asm volatile("cp.async.wait_all;" ::: "memory");
            tc::fence_smem();
            // neither stream runs ahead: Q is one barrier's business
            if (S::kStreams == 2 && !all_softmax(a, sh, nm)) return;
            if (tiles > 0) mbar_arrive(smem_addr(&sh.qready));
            // rows that do not exist see everything, of which nothing is kept
            span::Seen seen = {0, INT32_MAX};
            {
                const Row r = row_of(a, g, stream, row);
                if (r.live) seen = span::seen_by(a, g.seq, r.token);
            }
            const float scale = fabsf(a.scale_log2);
            float m = -INFINITY, l = 0.f;  // m: what P is relative to, less kUp
            const int first = both || S::kStreams == 1 ? 0 : stream, step = both || S::kStreams == 1 ? 1 : 2;
            int buf = 0;
            for (int j = first; j < tiles; j += step, buf = S::kBufs - 1 - buf) {
                if (!__all_sync(kFull, wait(sh, sh.sready[stream][buf], ns >> buf & 1, a))) return;
                ns ^= 1u << buf;
                tc::fence_after();
                const uint32_t s_at = tmem + (S::kBufs * stream + buf) * kTok;
                float s[kTok];
#pragma unroll
                for (int c = 0; c < kTok; c += 32) tc::load32(s_at + c, s + c);
                tc::wait_ld();
                const int jj = from + j, t0 = (jj < sink_tiles ? jj : jj + skip) * kTok;
                const bool clear = t0 + kTok <= seen.hi && (t0 >= seen.lo || t0 + kTok <= a.sinks);
                if (!__all_sync(kFull, clear)) {
#pragma unroll
                    for (int c = 0; c < kTok; c += 32) {
                        const int at = t0 + c;
                        const uint32_t see = below(seen.hi - at) & (~below(seen.lo - at) | below(a.sinks - at));
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[c + i] = see & 1u << i ? s[c + i] : -INFINITY;
                    }
                }
                float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < kTok; ++i) top[i & 3] = fmaxf(top[i & 3], s[i]);
                const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale - kUp;
                const bool grow = high > m + kLazy || (m == -INFINITY && high != m);
                // The product before the last is done (these scores were issued behind
                // it), with two buffers the last one may be under way: it is waited for where O is
                // changed, and ahead of the last P, so that no phase is missed.
                const bool changes = __any_sync(kFull, grow);
                if (j != first && (changes || j + step >= tiles) &&
                    !__all_sync(kFull, wait(sh, sh.vdone[stream], (nv & 1) ^ 1, a)))
                    return;
                if (changes) {
                    tc::fence_after();
                    const float to = grow ? high : m;
                    const float f = grow ? exp2_approx(m - (to == -INFINITY ? 0.f : to)) : 1.f;
                    if (j != first) scale_o(o_at, f, kv.dim);
                    l *= f;
                    m = to;
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const uint64_t scale2 = two(scale, scale), ref2 = two(-ref, -ref);
                uint64_t sum[2] = {0, 0};
                // the P of 32 scores takes their place: 16 columns of first parts, 16 of
                // second ones
#pragma unroll
                for (int c = 0; c < kTok; c += 32) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 x = apart(fma2(two(s[c + 2 * i], s[c + 2 * i + 1]), scale2, ref2));
                        const float p0 = exp2_approx(x.x), p1 = exp2_approx(x.y);
                        sum[i & 1] = add2(sum[i & 1], two(p0, p1));
                        split(p0, p1, hi[i], lo[i]);
                    }
                    tc::store16(s_at + c, hi);
                    tc::store16(s_at + c + 16, lo);
                }
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(smem_addr(&sh.pready[stream][buf]));
                ++nv;
                const float2 sums = apart(add2(sum[0], sum[1]));
                l += sums.x + sums.y;
            }
            const bool any = first < tiles;
            if (any && !__all_sync(kFull, wait(sh, sh.vdone[stream], (nv & 1) ^ 1, a))) return;
            tc::fence_after();
            float own = 1.f, other = 0.f;  // factors of this stream's O and the other's
            const bool join = !both && S::kStreams == 2 && tiles > 1;
            float *shared_o = reinterpret_cast<float *>(q_generic);  // [dim][rows]
            if (join) {
                if (!all_softmax(a, sh, nm)) return;  // both streams are done with Q
                if (stream == 1) {
                    sh.join_m[row] = m;
                    sh.join_l[row] = l;
                    for (int c = 0; c < kv.dim; c += 16) {
                        float x[16];
                        tc::load16(o_at + c, x);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < kv.dim) shared_o[(c + i) * kRows + row] = x[i];
                    }
                }
                if (!all_softmax(a, sh, nm)) return;
                if (stream == 0) {
                    const float m2 = sh.join_m[row], mm = fmaxf(m, m2), base = mm == -INFINITY ? 0.f : mm;
                    own = exp2_approx(m - base);
                    other = exp2_approx(m2 - base);
                    l = l * own + sh.join_l[row] * other;
                    m = mm;
                }
            }
            // The next segment's Q is requested before the present rows are
            // written; the streams' joint buffer lies where it goes.
            if (!join && !next_segment(a, sh, n + 1, stream, row, lane, qs)) return;
            if (both || stream == 0) {
                const Row r = row_of(a, g, stream, row);
                if (g.merge)
                    finish<true>(a, g, o_at, any, stream, row, r.live, r.token, r.head, m, l, own, other, join ? shared_o : nullptr);
                else
                    finish<false>(a, g, o_at, any, stream, row, r.live, r.token, r.head, m, l, own, other, join ? shared_o : nullptr);
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.segempty[n % kSegs]));
            if (join) {
                if (!all_softmax(a, sh, nm)) return;
                if (!next_segment(a, sh, n + 1, stream, row, lane, qs)) return;
            }
        }
    }

    // Waits for a segment and requests its Q.
    static __device__ __forceinline__ bool next_segment(const SpanArgs &a, Shared<DC> &sh, uint32_t n, int stream, int row, int lane, uint32_t qs)
    {
        if (!__all_sync(kFull, wait(sh, sh.segfull[n % kSegs], n / kSegs & 1, a))) return false;
        const Segment &g = sh.seg[n % kSegs];
        if (!g.stop) load_q(a, g, row_of(a, g, stream, row), qs, stream, row, lane);
        return true;
    }

    // Writes a row: its output, its part of the prefix, or a part of a cut block.
    template <bool MERGE>
    static __device__ __forceinline__ void finish(const SpanArgs &a, const Segment &g, uint32_t o_at, bool any, int stream, int row, bool live,
                                                  int token, int head, float m, float l, float own, float other, const float *buf)
    {
        const int dim = a.kv.dim;
        const int64_t t = g.seq.q0 + token, index = t * a.q_heads + head;
        float *part = a.part + g.aside * a.part_stride + stream * (a.part_stride / S::kStreams);
        float *part_stat = part + (dim + 15) / 16 * 16 * kRows;
        const bool aside = g.more || g.slot >= 0;
        float now = 1.f, then = 0.f;  // factors of this segment's O and of what this thread put aside
        if (MERGE && live) {
            const float m1 = part_stat[row], l1 = part_stat[kRows + row], mm = fmaxf(m, m1), base = mm == -INFINITY ? 0.f : mm;
            now = exp2_approx(m - base);
            then = exp2_approx(m1 - base);
            l = l * now + l1 * then;
            m = mm;
        }
        // (a thread of the copies has written it ahead of the tile's K)
        const bool missing = *const_cast<const volatile int *>(&g.missing) != 0;
        if (missing) l = 1.f;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        bool nan = false;
        for (int c = 0; c < dim; c += 16) {
            float x[16];
            __syncwarp();
            if (any) {
                tc::load16(o_at + c, x);
                tc::wait_ld();
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = 0.f;
            }
            if (buf) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < dim) x[i] = x[i] * own + buf[(c + i) * kRows + row] * other;
            }
            if (missing) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __int_as_float(0x7FFFFFFF);
            }
            if (live) {
                if (MERGE) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 y = *reinterpret_cast<const float4 *>(part + ((c + i) / 4 * kRows + row) * 4);
                        x[i] = x[i] * now + y.x * then, x[i + 1] = x[i + 1] * now + y.y * then;
                        x[i + 2] = x[i + 2] * now + y.z * then, x[i + 3] = x[i + 3] * now + y.w * then;
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) nan = nan || (c + i < dim && x[i] != x[i]);
                if (aside) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4 *>(part + ((c + i) / 4 * kRows + row) * 4) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                } else if (a.pre) {
                    float *p = a.pre + index * span_row(dim) + c;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < dim) p[i] = x[i];
                } else {
                    uint16_t *p = static_cast<uint16_t *>(a.out) + t * a.o_st + head * a.o_sh + c;
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = pack(x[2 * i] * inv, x[2 * i + 1] * inv);
                    if (a.out_vec == 2 && c + 16 <= dim) {  // a whole sector
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                     : "memory");
                    } else if (a.out_vec && c + 16 <= dim) {
                        reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < dim) p[i] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
                    }
                }
            }
        }
        __syncwarp();
        if (!live) return;
        if (aside) {
            part_stat[row] = m;
            part_stat[kRows + row] = l;
            a.redo[index] = 0;  // the join's business
            return;
        }
        // a value that another row of the block sees may be infinite where this row's
        // weight is 0: such rows are computed again, one by one
        a.redo[index] = nan && l == l;
        if (a.pre) {
            float *stat = a.pre + (index + 1) * span_row(dim) - 4;
            stat[0] = m;
            stat[1] = l;
        } else if (a.lse) {
            a.lse[index] = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
    }

    static __device__ void run(const SpanArgs &a, unsigned char *raw)
    {
        unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
        unsigned char *kgen = base + S::kStreams * S::kQBytes;
        Shared<DC> &sh = *reinterpret_cast<Shared<DC> *>(kgen + 2 * S::kStages * S::kKvBytes);
        const uint32_t qs = smem_addr(base), ks = smem_addr(kgen), vs = ks + S::kStages * S::kKvBytes;
        const int tid = threadIdx.x, warp = tc::uniform(tid >> 5), lane = tid & 31;
        const bool bulk = VEC && a.box > 0;
        if (tid == 0) {
            for (int i = 0; i < S::kStages; ++i) {
                mbar_init(smem_addr(&sh.kthere[i]), 128);
                mbar_init(smem_addr(&sh.vthere[i]), bulk ? 1 : 128);
                mbar_init(smem_addr(&sh.kfull[i]), 1);
                mbar_init(smem_addr(&sh.vfull[i]), 1);
                mbar_init(smem_addr(&sh.kempty[i]), 1);
                mbar_init(smem_addr(&sh.vempty[i]), 1);
            }
            for (int i = 0; i < 2; ++i) {
                for (int k = 0; k < 2; ++k) {
                    mbar_init(smem_addr(&sh.sready[i][k]), 1);
                    mbar_init(smem_addr(&sh.pready[i][k]), kRows);
                }
                mbar_init(smem_addr(&sh.vdone[i]), 1);
            }
            for (int i = 0; i < kSegs; ++i) {
                mbar_init(smem_addr(&sh.segfull[i]), 1);
                mbar_init(smem_addr(&sh.segempty[i]), (bulk ? 3 : 6) + 1 + 4 * S::kStreams);
            }
            mbar_init(smem_addr(&sh.qready), kRows * S::kStreams);
            mbar_init(smem_addr(&sh.meet), kRows * S::kStreams);
            mbar_init(smem_addr(&sh.last), 1);
            sh.abort = 0;
            sh.lim.shortest = INT32_MAX;
            sh.lim.longest = 0;
            sh.seg[0].stop = 1;
        }
        if (warp == 0) tc::alloc(smem_addr(&sh.tmem), 512);
        // the next launch may start once this one's wait is over: then nothing
        // before this launch is under way any more
        pdl_wait();
        pdl_trigger();
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
        if (a.prefix) {
            int lo = INT32_MAX, hi = 0;
            for (int b = tid; b < a.tokens; b += kThreads) {
                const int n = min(max(__ldg(a.lengths + b), 0), static_cast<int>(a.kv.capacity));
                if (n > 0) lo = min(lo, n);  // (an empty sequence sees nothing)
                hi = max(hi, n);
            }
            atomicMin(&sh.lim.shortest, __reduce_min_sync(kFull, lo));
            atomicMax(&sh.lim.longest, __reduce_max_sync(kFull, hi));
            __syncthreads();
        }
        // the call's work, and where this CTA's share of it begins
        Cursor mine;
        mine.before = -1;
        auto take = [&](const span::Seq &q, int row0, const Block &k, int64_t before) {
            mine.done = 0;
            mine.before = before;
            mine.b = q.b;
            mine.row0 = row0;
            mine.top = q.q0;  // (one that has tokens starts at or above all before it)
            mine.seq = q;
            mine.block = k;
        };
        bool once = true, again;
        int64_t total;
        span::Seq all;
        int blocks = 0;
        if (a.prefix) {  // one sequence, whose blocks but for the last are alike
            all = span::seq_of(a, 0, blockIdx.x == 0 && tid == 0);
            blocks = (all.m * a.group + S::kBlock - 1) / S::kBlock;
            const int first = blocks > 1 ? cost_of<DC>(block_of<DC>(a, all, 0, sh.lim)) : 0;
            total = (static_cast<int64_t>(first) * (blocks - 1) + cost_of<DC>(block_of<DC>(a, all, (blocks - 1) * S::kBlock, sh.lim))) * a.kv.kv_heads;
            if (tid == 0) mine.before = first;
        } else {
            total = for_blocks(a, sh, take, &once) * a.kv.kv_heads;
        }
        const int ctas = gridDim.x, cta = blockIdx.x;
        Share w;
        w.x0 = total * cta / ctas;
        w.x1 = total * (cta + 1) / ctas;
        const int64_t near = total / ctas / 40;
        w.near = near > 2 ? 2 : static_cast<int>(near);
        auto find = [&]() {
            if (mine.before < 0) return;
            const int64_t r0 = mine.before * a.kv.kv_heads;
            const int cost = cost_of<DC>(mine.block);
            if (w.x0 < w.x1 && r0 <= w.x0 && w.x0 < r0 + static_cast<int64_t>(cost) * a.kv.kv_heads) {
                mine.h = static_cast<int>((w.x0 - r0) / cost);
                advance(a, sh, w, mine, sh.seg[0]);
                sh.first = mine;
            }
        };
        if (a.prefix) {
            if (tid == 0) {
                const int64_t each = mine.before, per = each * a.kv.kv_heads;
                const int i = per > 0 ? static_cast<int>(min(w.x0 / per, static_cast<int64_t>(blocks - 1))) : 0;
                take(all, i * S::kBlock, block_of<DC>(a, all, i * S::kBlock, sh.lim), i * each);
                find();
            }
        } else if (once) {
            find();
        } else {
            for_blocks(a, sh, [&](const span::Seq &q, int row0, const Block &k, int64_t before) {
                take(q, row0, k, before);
                find();
            }, &again);
        }
        if (tid < 2) a.info[2 * cta + tid].tiles = 0;  // no parts yet
        __syncthreads();
        if (tid == 0) mbar_arrive(smem_addr(&sh.segfull[0]));  // the first segment is there
        if (warp < 8) {
            tc::set_registers_up<208>();
            softmax(a, sh, qs, base);
            asm volatile("cp.async.wait_all;" ::: "memory");  // (given up: Q may be under way)
        } else if (warp < 12) {
            tc::set_registers_down<56>();
            if (!bulk)
                loader(a, sh, ks, vs);
            else if (warp < 10)
                bulk_loader(a, sh, warp == 9 ? vs : ks, warp == 9);
        } else {
            tc::set_registers_down<40>();
            if (warp == 12) products(a, sh, qs, ks, vs);
            if (warp == 13 && lane == 0) schedule(a, sh, w);
            if (warp == 14 && lane == 0 && !bulk) pass_on(a, sh, sh.kthere, sh.kfull);
            if (warp == 15 && lane == 0 && !bulk) pass_on(a, sh, sh.vthere, sh.vfull);
            if (warp == 15 && bulk) zero_v(a, sh, vs);
        }
        __syncwarp();
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
        if (warp == 0) tc::dealloc(sh.tmem, 512);
    }

    static __device__ void schedule(const SpanArgs &a, Shared<DC> &sh, const Share &w)
    {
        Cursor at = sh.first;
        for (uint32_t n = 0;; ++n) {
            if (n >= kSegs && !wait(sh, sh.segempty[n % kSegs], (n / kSegs & 1) ^ 1, a)) {
                sh.seg[n % kSegs].stop = 1;
                mbar_arrive(smem_addr(&sh.segfull[n % kSegs]));
                return;
            }
            Segment &g = sh.seg[n % kSegs];
            if (n > 0) advance(a, sh, w, at, g);  // (the first is there)
            if (sh.abort && n > 0) g.stop = 1;
            if (!g.stop && g.slot >= 0) {
                SpanInfo &i = a.info[g.slot];
                i.b = g.seq.b;
                i.h = g.h;
                i.row0 = g.row0;
                i.t0 = g.t0;
                i.t1 = g.t1;
                i.tiles = g.block.tiles;
            }
            if (n > 0) mbar_arrive(smem_addr(&sh.segfull[n % kSegs]));
            if (g.stop) return;
        }
    }
};

template <typename T, int DC, bool VEC>
__global__ void __launch_bounds__(kThreads, 1) mbg_tile_kernel(const __grid_constant__ SpanArgs a)
{
    extern __shared__ __align__(1024) unsigned char raw[];
    Kernel<T, DC, VEC>::run(a, raw);
}

template <typename T, int DC, bool VEC>
cudaError_t launch_one(const SpanArgs &a, int ctas, cudaStream_t s)
{
    using S = Shape<DC>;
    constexpr int smem = 1024 + S::kStreams * S::kQBytes + 2 * S::kStages * S::kKvBytes + sizeof(Shared<DC>);
    static_assert(smem <= 227 * 1024, "");
    auto fn = mbg_tile_kernel<T, DC, VEC>;
    static std::atomic<uint64_t> ready{0};  // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(ready.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) ready.fetch_or(uint64_t{1} << (dev & 63), std::memory_order_relaxed);
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <typename T>
cudaError_t launch(const SpanArgs &a, bool vec, int ctas, cudaStream_t s)
{
    switch ((a.kv.dim + 63) / 64) {
    case 1: return vec ? launch_one<T, 1, true>(a, ctas, s) : launch_one<T, 1, false>(a, ctas, s);
    case 2: return vec ? launch_one<T, 2, true>(a, ctas, s) : launch_one<T, 2, false>(a, ctas, s);
    case 3: return vec ? launch_one<T, 3, true>(a, ctas, s) : launch_one<T, 3, false>(a, ctas, s);
    default: return vec ? launch_one<T, 4, true>(a, ctas, s) : launch_one<T, 4, false>(a, ctas, s);
    }
}

}  // namespace tile
}  // namespace mbg
