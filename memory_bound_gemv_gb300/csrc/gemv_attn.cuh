// Attention of one new token over a paged key-value cache.
//
//   s_t = scale * q . k_t,  p = softmax(s),  o = sum_t p_t v_t
//
// over the tokens t in [max(0, len - window), len) of a sequence, and with
// sinks those in [0, sinks), G query heads sharing one cached head.  Behind a
// prefix that is attended to elsewhere only the tokens from its end on are
// read, and O, m and l are left in FP32 for the join (gemv_span.cu).  One pass over the cache: each warp keeps a
// running maximum m, denominator l and output O of its own tokens and rescales
// by 2^(m - m') when m grows (Milakov & Gimelshein's online softmax); the
// warps, then the blocks, that share a row are joined by the same rule.
//
// What bounds it: K and V are read once and nothing else is large; a cached
// element takes 2 G flop.  With G up to 16 that needs at most ~100 TFLOP/s at
// HBM speed, which the warp-level MMA instruction (m16n8k16) has to spare,
// while FP32 FMAs would not keep up from G = 8 on.
//
// K and V go from global memory straight into the registers that the MMA
// reads, with no shared memory and no barriers in the loop:
//   S^T = K Q^T: 16 tokens x 8 heads per MMA.  Thread (g, t) = (lane / 4,
//     lane % 4) holds rows g and g + 8 of K.  The contraction over d may run in
//     any order, so each thread takes 8 consecutive d per row with one
//     16-byte load and feeds them to two MMAs; Q is laid out the same way.
//   O^T = V^T P^T: 16 d x 8 heads per MMA over 16 tokens.  Thread (g, t) loads 8
//     consecutive d of tokens 2t, 2t + 1, 2t + 8, 2t + 9; byte permutes pair
//     the tokens.  P comes out of S^T's registers by a transposing move
//     (movmatrix).
// P is split into 16-bit parts, an MMA per V tile each: a rounding of P to 8
// (bf16) or 11 (f16) bits would be as large as that of the output itself.  In
// bf16 three parts hold the 24 bits of FP32.  In f16 two parts are off by 2^-21
// relative; P is multiplied by 2^15 first, so that the smallest f16 steps lie at
// 2^-39 of the warp's largest weight (unscaled at 2^-24, where weights behind
// a token that leads by 17 nats, a sink say, would vanish from O).
//
// The next tile's K is requested while the present tile's softmax and V
// product run, and the next V after that: about 8 KB in flight per warp at a
// head size of 128.
//
// Split over the length: the rows (sequence x cached head) are cut into tiles
// of 16 or 32 tokens; all tiles of the call are numbered and each CTA takes an equal
// share of consecutive ones, whatever the lengths (they are read on the
// device, so a captured graph serves any lengths).  A share's border that
// falls close to a row's end moves there, so that short rows are not cut, nor
// are others that spread evenly over the CTAs whole.  A row inside one CTA's
// share is written at once; otherwise each CTA leaves (O, m, l) in the workspace
// and the last to arrive joins them, always in the same order, so results do
// not depend on the order of arrival.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "gemv_decode.h"
#include "gemv_device.cuh"

namespace mbg {
namespace attn {

constexpr unsigned kFull = 0xFFFFFFFFu;

// 8x8 matrix of 16-bit elements, one row per four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t w)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
    return r;
}

template <typename T>
struct Mma;

template <>
struct Mma<__half> {
    static __device__ __forceinline__ void run(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
    // Two weights in parts, transposed for the value product; kUnscale times the
    // parts' sum are the weights.  Parts of a weight above 0 are above 0 (the high
    // part is rounded down, the steps at the lower end are the least they can
    // be): times an infinite value, a part of 0 would be NaN.
    static constexpr int kParts = 2;
    static constexpr float kUnscale = 1.f / 32768.f;
    static __device__ __forceinline__ void split(float p0, float p1, uint32_t (&w)[kParts])
    {
        constexpr float kStep = 1.f / 16777216.f;
        const float s0 = p0 > 0.f ? kStep : 0.f, s1 = p1 > 0.f ? kStep : 0.f;
        p0 = fmaxf(p0 * 32768.f, s0);
        p1 = fmaxf(p1 * 32768.f, s1);
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w[0]) : "f"(p1), "f"(p0));
        const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&w[0]));
        const __half2 rest = __floats2half2_rn(fmaxf(p0 - back.x, s0), fmaxf(p1 - back.y, s1));
        w[0] = transpose8x8(w[0]);
        w[1] = transpose8x8(*reinterpret_cast<const uint32_t *>(&rest));
    }
    static __device__ __forceinline__ uint16_t bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
};

template <>
struct Mma<__nv_bfloat16> {
    static __device__ __forceinline__ void run(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
    // Eight bits of the significand each: the upper halves of p, of what is left
    // of it, and of what is left of that, which has no more than eight.  What
    // is left of a weight above 0 (they are 2^-126 or more) counts as that much.
    static constexpr int kParts = 3;
    static constexpr float kUnscale = 1.f;
    static __device__ __forceinline__ void split(float p0, float p1, uint32_t (&w)[kParts])
    {
        // the transposing moves take the halves of p, of which the upper ones are
        // the first parts; the others are made afterwards (parts made first are
        // three moves and 80 bytes of spilled registers: 384 rows of 1000 tokens of
        // 128 41.2 us, so 39.8)
        w[0] = transpose8x8(__byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632));
        const uint32_t low = transpose8x8(__byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x5410));
        const uint32_t b0 = w[0] << 16, b1 = w[0] & 0xFFFF0000u;
        p0 = __uint_as_float(__byte_perm(low, w[0], 0x5410));
        p1 = __uint_as_float(__byte_perm(low, w[0], 0x7632));
        const float s0 = fminf(p0, 1.17549435e-38f), s1 = fminf(p1, 1.17549435e-38f);
        p0 = fmaxf(p0 - __uint_as_float(b0), s0);
        p1 = fmaxf(p1 - __uint_as_float(b1), s1);
        const uint32_t c0 = __float_as_uint(p0), c1 = __float_as_uint(p1);
        w[1] = __byte_perm(c0, c1, 0x7632);
        p0 = fmaxf(p0 - __uint_as_float(c0 & 0xFFFF0000u), s0);
        p1 = fmaxf(p1 - __uint_as_float(c1 & 0xFFFF0000u), s1);
        w[2] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
    }
    static __device__ __forceinline__ uint16_t bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 2^(x - m) where m = -inf stands for "nothing seen yet" (then x = -inf too,
// and the answer is 0).
__device__ __forceinline__ float exp2_from(float x, float m)
{
    return exp2_approx(x - (m == -INFINITY ? 0.f : m));
}

// log2 of the sum of 2^s, -inf for a row without weights.
__device__ __forceinline__ float lse2_of(float m, float l) { return l > 0.f || l != l ? m + log2f(l) : -INFINITY; }

// 16 bytes of a cached row, read once.  (Asking L2 for the whole 256 bytes
// around them brings other heads' rows along when a row is shorter: 16 x 32768
// tokens of four heads of 64 take 115 us then, 92 us without, and rows of 256
// bytes gain nothing from it.)
__device__ __forceinline__ uint4 ld_row16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight consecutive 16-bit elements at p, of which the first `left` exist.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int left)
{
    if (VEC) return ld_row16(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < left ? __ldg(p + 2 * i) : 0;
        const uint32_t hi = 2 * i + 1 < left ? __ldg(p + 2 * i + 1) : 0;
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The tokens of a sequence that are attended to, and their tiles of TOKENS
// tokens.  Tile t of the sequence's tiles is tile begin / TOKENS + t of the
// cache for t < sink_tiles, of which the tokens before `sinks` count, and tile0
// + t behind them.  (Sinks and window may meet in one tile of the cache,
// which is then gone through twice.)
struct RowSpan {
    int first, len;         // tokens [first, len)
    int begin, sinks;       // and [begin, sinks), sinks < first; none if sink_tiles is 0
    int sink_tiles;
    int tile0, tiles;       // first / TOKENS - sink_tiles; the tiles' number
};

template <int TOKENS, bool SINKS = true, bool OWN = false>
__device__ __forceinline__ RowSpan row_span(const AttnArgs &a, int b)
{
    RowSpan r;
    int len = __ldg(a.lengths + b);
    if (len < 0) len = 0;
    if (len > a.kv.capacity) len = static_cast<int>(a.kv.capacity);
    r.len = len;
    r.first = (a.window > 0 && len > a.window) ? len - a.window : 0;
    r.begin = 0;
    if (OWN) r.begin = min(max(__ldg(a.prefix), 0), len);
    if (SINKS && r.first <= max(a.sinks, r.begin)) r.first = r.begin;
    r.sinks = SINKS && r.first > r.begin && a.sinks > r.begin ? a.sinks : r.begin;
    r.sink_tiles = r.sinks > r.begin ? (r.sinks + TOKENS - 1) / TOKENS - r.begin / TOKENS : 0;
    r.tile0 = r.first / TOKENS - r.sink_tiles;
    r.tiles = len > r.first ? (len + TOKENS - 1) / TOKENS - r.tile0 : 0;
    return r;
}

// Where a tile's tokens are; page -1: nowhere.  WHOLE (pages of a multiple of
// 16 tokens, so that a tile lies in one): the page, the place of its first
// token there, and which of its 16 tokens count: lo <= r < hi.  Otherwise
// lanes 0..15, and again 16..31, hold the page and place of one token each.
struct TilePlace {
    int page, off, lo, hi;
};

template <bool WHOLE>
__device__ __forceinline__ TilePlace place_of(const KvView &kv, const int32_t *table, int tile, bool wanted, int first,
                                              int len, unsigned int *err)
{
    TilePlace p = {-1, 0, 0, 0};
    const int slot = tile * 16 + (WHOLE ? 0 : threadIdx.x & 15);
    if (wanted && slot < len && slot + (WHOLE ? 15 : 0) >= first) {
        const int idx = kv.page_shift >= 0 ? slot >> kv.page_shift : slot / kv.page_size;
        p.off = slot - idx * kv.page_size;
        p.page = __ldg(table + idx);
        if (p.page < 0 || p.page >= kv.num_pages) {
            p.page = -1;
            report_error(err, DEVERR_BAD_INDEX);
        } else if (WHOLE) {
            p.lo = first - slot;
            p.hi = len - slot;
        }
    }
    return p;
}

template <int DC, int NT>
constexpr int kTilesAtOnce = DC * NT == 1 ? 2 : 1;

template <typename T, int DC, int NT, int NW, bool VEC, bool WHOLE, bool SINKS, bool OWN>
struct Kernel {
    static constexpr int kWarps = NW, kThreads = NW * 32;
    // tiles of 16 tokens that a warp takes at once: two of narrow heads, so that
    // as many bytes are under way as with wide ones
    static constexpr int MT = kTilesAtOnce<DC, NT>, kTokens = 16 * MT;
    // CTAs whose parts of a row are joined first, before the groups are
    static constexpr int kGroupCtas = 4 * NW;
    static constexpr int kHeads = 8 * NT;           // query heads of one tile
    static constexpr int kRegs = NT * DC * 16;      // O values per thread
    static constexpr int kQWords = NT * DC * 8;     // Q words per thread
    // Q of wide heads or of two head tiles comes from shared memory: as
    // registers it would not fit beside K, V and O
    static constexpr bool kQInSmem = NT * DC > 2;

    // parts joined at once: a group, or the groups of a row
    static constexpr int kMaxParts = kAttnMaxCtas / kGroupCtas > kGroupCtas ? kAttnMaxCtas / kGroupCtas : kGroupCtas;

    // This CTA's part of the call's work.  A row of n tiles counts `lead` + n:
    // starting a row costs about that many tiles.  CTA c's share ends where CTA
    // c + 1's begins, at total * c / ctas -- or at an end of the row there, if
    // that is at most kNear tiles away (one round of the warps: 160 rows of 2000
    // tokens of 128 35.8 us, two rounds 36.7; 128 of 500 17.2 and 18.4).  A cut
    // costs as much as some kUncut tiles: rows of no more have none (384 rows of
    // 256 tokens: 16.0 us, cut 23.9), nor has any row where the CTA with most to
    // do would then have no more than that above the mean (384 rows of 400 tokens
    // 20.7 us, cut 27.7; of 1000 39.8 and 43.4; but 512 of 1000 66.7 and 53.8,
    // 800 ragged ones of up to 800 46.3 and 40.1).
    static constexpr int kNear = kWarps, kUncut = 16;
    struct Share {
        int64_t total, x0, x1;
        int ctas, cta, lead;
        int uncut;  // rows of up to so many tiles are not cut
    };
    // The row that is looked at next; `before` counts what lies before its
    // sequence, per cached head.
    struct Cursor {
        int64_t before;
        int b, hk;
    };
    // Tiles [t0, t1) of a row; none are left when t0 = t1.
    struct Segment {
        int64_t r0;             // where the row begins
        int b, hk, t0, t1;
        int first, len, begin, sinks, sink_tiles, tile0, tiles;
    };

    struct Shared {
        float o[kWarps][kRegs][32];
        float m[kWarps][kHeads];
        float l[kWarps][kHeads];
        uint32_t q[kQInSmem ? kQWords : 1][32];
        float part_m[kMaxParts][kHeads];
        float part_l[kMaxParts][kHeads];
        int scan[kWarps];
        int last;
        uint64_t call;    // the call's number, as counters carry it
        Share share;
        Cursor cursor;
        Segment seg[3];   // the present one, the next, and the one being looked up
    };

    struct Row {
        int b, hk;        // sequence; cached head * head_tiles + tile
        int head0, heads; // first query head and how many of the tile exist
    };

    static __device__ __forceinline__ Row row_of(const AttnArgs &a, int b, int hk)
    {
        Row r;
        r.b = b;
        r.hk = hk;
        const int h = hk / a.head_tiles, ht = hk - h * a.head_tiles;
        r.head0 = h * a.group + ht * kHeads;
        r.heads = min(kHeads, a.group - ht * kHeads);
        return r;
    }

    // Where a row's O, maximum and denominator go that are to be joined with its prefix's.
    static __device__ __forceinline__ float *own_of(const AttnArgs &a, const Row &r, int head)
    {
        return a.own + (static_cast<int64_t>(r.b) * a.q_heads + r.head0 + head) * span_row(a.kv.dim);
    }

    // Output value pair: fragment register idx of a lane is O[head][d].
    //   idx = ((nt * DC + c) * 4 + i) * 4 + e;  head = nt * 8 + 2t + (e & 1),
    //   d = c * 64 + 8g + 2i + (e >> 1)
    static __device__ void store_out(const AttnArgs &a, const Row &r, int idx0, const float (&o)[4], int lane,
                                     const float (&inv)[2])
    {
        const int g = lane >> 2, t = lane & 3;
        const int i = (idx0 >> 2) & 3, c = (idx0 >> 4) % DC, nt = (idx0 >> 4) / DC;
        const int d = c * 64 + 8 * g + 2 * i;
        uint16_t *out = static_cast<uint16_t *>(a.out) + r.b * a.o_sb;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int head = nt * 8 + 2 * t + e;
            if (head >= r.heads) continue;
            if (OWN) {  // (d is even, and a row there a multiple of four)
                if (d < a.kv.dim)
                    *reinterpret_cast<float2 *>(own_of(a, r, head) + d) = make_float2(o[e] * inv[e], o[e + 2] * inv[e]);
                continue;
            }
            uint16_t *p = out + (r.head0 + head) * a.o_sh + d;
            if (d < a.kv.dim) p[0] = Mma<T>::bits(o[e] * inv[e]);
            if (d + 1 < a.kv.dim) p[1] = Mma<T>::bits(o[e + 2] * inv[e]);
        }
    }

    // Statistics of a finished row: log2 of the denominator for the weights,
    // the natural logarithm for the caller.  An empty row has -inf there, and
    // +inf for the weights (every weight is then 2^-inf = 0).
    static __device__ void store_stats(const AttnArgs &a, const Row &r, int head, float m, float l)
    {
        const float lse2 = lse2_of(m, l);
        if (a.scores_out) {
            const int64_t row = static_cast<int64_t>(r.b) * a.kv.kv_heads * a.head_tiles + r.hk;
            a.row_lse[row * kHeads + head] = lse2 == -INFINITY ? INFINITY : lse2;
        }
        if (a.lse && head < r.heads)
            a.lse[static_cast<int64_t>(r.b) * a.q_heads + r.head0 + head] = lse2 * 0.69314718055994531f;
    }

    static __device__ void empty_rows(const AttnArgs &a)
    {
        for (int b = blockIdx.x; b < a.kv.batch; b += gridDim.x) {
            const int len = __ldg(a.lengths + b);
            if ((len < 0 || len > a.kv.capacity) && threadIdx.x == 0) report_error(a.err, DEVERR_BAD_INDEX);
            if (OWN) {
                if (row_span<kTokens, SINKS, OWN>(a, b).tiles > 0) continue;
                for (int h = threadIdx.x; h < a.q_heads; h += kThreads) {
                    float *stat = a.own + (static_cast<int64_t>(b) * a.q_heads + h) * span_row(a.kv.dim) + span_row(a.kv.dim) - 4;
                    stat[0] = -INFINITY;
                    stat[1] = 0.f;
                }
                continue;
            }
            if (len > 0 && a.kv.capacity > 0) continue;
            uint16_t *out = static_cast<uint16_t *>(a.out) + b * a.o_sb;
            for (int i = threadIdx.x; i < a.q_heads * a.kv.dim; i += kThreads) {
                const int h = i / a.kv.dim;
                out[h * a.o_sh + (i - h * a.kv.dim)] = 0;
            }
            if (a.lse)
                for (int h = threadIdx.x; h < a.q_heads; h += kThreads)
                    a.lse[static_cast<int64_t>(b) * a.q_heads + h] = -INFINITY;
        }
    }

    static __device__ __forceinline__ int64_t border(const Share &w, int64_t x, int64_t r0, int64_t r1)
    {
        const int64_t d0 = x - r0 - w.lead, d1 = r1 - x;
        const int64_t tiles = r1 - r0 - w.lead, near = tiles <= w.uncut ? tiles : kNear;
        if (d0 <= d1) return d0 <= near ? r0 : x;
        return d1 <= near ? r1 : x;
    }

    // Looks up the CTA's next segment (one thread).
    static __device__ void advance(const AttnArgs &a, const Share &w, Cursor &at, Segment &out)
    {
        const int hks = a.kv.kv_heads * a.head_tiles;
        while (at.b < a.kv.batch) {  // (the last share ends with the last row)
            const RowSpan span = row_span<kTokens, SINKS, OWN>(a, at.b);
            const int n = span.tiles, cost = n + w.lead;
            if (n == 0) {
                ++at.b;
                continue;
            }
            const int hk = at.hk, b = at.b;
            const int64_t r0 = at.before * hks + static_cast<int64_t>(hk) * cost, r1 = r0 + cost;
            const int64_t from = w.x0 > r0 ? border(w, w.x0, r0, r1) : r0;
            const int64_t to = w.x1 >= r1 ? r1 : border(w, w.x1, r0, r1);
            if (++at.hk == hks) {
                at.hk = 0;
                ++at.b;
                at.before += cost;
            }
            if (w.x1 <= r1) at.b = a.kv.batch;
            if (from < to) {
                out.r0 = r0;
                out.b = b;
                out.hk = hk;
                out.t0 = from == r0 ? 0 : static_cast<int>(from - r0 - w.lead);
                out.t1 = static_cast<int>(to - r0 - w.lead);
                out.first = span.first;
                out.len = span.len;
                out.begin = span.begin;
                out.sinks = span.sinks;
                out.sink_tiles = span.sink_tiles;
                out.tile0 = span.tile0;
                out.tiles = n;
                if (out.t0 < out.t1) return;
            }
        }
        out.b = out.hk = out.t0 = out.t1 = 0;
    }

    // The CTA's segments, one after another.  A warp requests the first tiles
    // of its next segment before it joins the present one, so that the loads
    // never pause between rows.
    static __device__ void stream(const AttnArgs &a, Shared &sh, uint64_t ticket)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int g = lane >> 2, t = lane & 3;
        const KvView &kv = a.kv;

        uint4 q[kQInSmem ? 1 : NT][kQInSmem ? 1 : 2 * DC];
        auto load_q = [&](const Row &r) {
            const uint16_t *qb = static_cast<const uint16_t *>(a.q) + r.b * a.q_sb;
            if (kQInSmem) {
                for (int w = warp; w < NT * 2 * DC; w += kWarps) {
                    const int nt = w / (2 * DC), j = w - nt * 2 * DC;
                    const int head = nt * 8 + g, d = j * 32 + t * 8;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (head < r.heads && d < kv.dim) v = load8<VEC>(qb + (r.head0 + head) * a.q_sh + d, kv.dim - d);
                    sh.q[4 * w + 0][lane] = v.x;
                    sh.q[4 * w + 1][lane] = v.y;
                    sh.q[4 * w + 2][lane] = v.z;
                    sh.q[4 * w + 3][lane] = v.w;
                }
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2 * DC; ++j) {
                        const int head = nt * 8 + g, d = j * 32 + t * 8;
                        q[kQInSmem ? 0 : nt][kQInSmem ? 0 : j] =
                            (head < r.heads && d < kv.dim)
                                ? load8<VEC>(qb + (r.head0 + head) * a.q_sh + d, kv.dim - d)
                                : make_uint4(0, 0, 0, 0);
                    }
            }
        };
        uint4 kx[MT][2][2 * DC], vx[MT][DC][4];
        struct Places {
            TilePlace t[MT];
        };
        auto place = [&](const Segment &s, int tile) {
            Places p;
            const bool sink = SINKS && tile < s.sink_tiles;
            const int begin = OWN ? s.begin : 0;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                p.t[i] = place_of<WHOLE>(kv, kv.table + s.b * kv.table_stride,
                                         ((sink ? begin / kTokens : s.tile0) + tile) * MT + i, tile < s.t1,
                                         sink ? begin : s.first, sink ? s.sinks : s.len, a.err);
            return p;
        };
        // does token r of a tile count, and its place relative to p's
        auto token = [&](const TilePlace &p, int r, int *page, int *off) {
            if (WHOLE) {
                *page = p.page;
                *off = p.off + r;
                return r >= p.lo && r < p.hi;
            }
            *page = __shfl_sync(kFull, p.page, r);
            *off = __shfl_sync(kFull, p.off, r);
            return *page >= 0;
        };
        auto load_k16 = [&](const TilePlace &p, int h, uint4(&x)[2][2 * DC]) {
            const uint16_t *base = static_cast<const uint16_t *>(kv.k) + h * kv.ks_head;
            if (WHOLE) base += p.page * kv.ks_page + p.off * kv.ks_tok;
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                int page, off;
                const bool live = token(p, g + 8 * rr, &page, &off);
                const uint16_t *row = WHOLE ? base + (g + 8 * rr) * kv.ks_tok : base + page * kv.ks_page + off * kv.ks_tok;
#pragma unroll
                for (int j = 0; j < 2 * DC; ++j) {
                    const int d = j * 32 + t * 8;
                    x[rr][j] = (live && d < kv.dim) ? load8<VEC>(row + d, kv.dim - d) : make_uint4(0, 0, 0, 0);
                }
            }
        };
        auto load_v16 = [&](const TilePlace &p, int h, uint4(&x)[DC][4]) {
            const uint16_t *base = static_cast<const uint16_t *>(kv.v) + h * kv.vs_head;
            if (WHOLE) base += p.page * kv.vs_page + p.off * kv.vs_tok;
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) {
                const int tok = 2 * t + (rr & 1) + 8 * (rr >> 1);
                int page, off;
                const bool live = token(p, tok, &page, &off);
                const uint16_t *row = WHOLE ? base + tok * kv.vs_tok : base + page * kv.vs_page + off * kv.vs_tok;
#pragma unroll
                for (int c = 0; c < DC; ++c) {
                    const int d = c * 64 + g * 8;
                    x[c][rr] = (live && d < kv.dim) ? load8<VEC>(row + d, kv.dim - d) : make_uint4(0, 0, 0, 0);
                }
            }
        };

        auto load_k = [&](const Places &p, int h) {
#pragma unroll
            for (int i = 0; i < MT; ++i) load_k16(p.t[i], h, kx[i]);
        };
        auto load_v = [&](const Places &p, int h) {
#pragma unroll
            for (int i = 0; i < MT; ++i) load_v16(p.t[i], h, vx[i]);
        };

        Places here, next;
#pragma unroll
        for (int i = 0; i < MT; ++i) here.t[i] = next.t[i] = {-1, 0, 0, 0};
        bool first_segment = true;
        bool primed = false;  // the present segment's first tiles are already requested
        if (sh.seg[0].t0 < sh.seg[0].t1) load_q(row_of(a, sh.seg[0].b, sh.seg[0].hk));
        for (int i = 0;; i = i == 2 ? 0 : i + 1) {
            const Segment seg = sh.seg[i];
            const Segment &after = sh.seg[i == 2 ? 0 : i + 1];
            if (seg.t0 >= seg.t1) break;
            const int h = seg.hk / a.head_tiles;
            int tile = seg.t0 + warp;
            if (!primed) {
                here = place(seg, tile);
                load_k(here, h);
                load_v(here, h);
            }
            if (first_segment) {  // the second segment is looked up while the first loads are under way
                if (threadIdx.x == 0) advance(a, sh.share, sh.cursor, sh.seg[1]);
                if (threadIdx.x == kTicketThread) sh.call = (ticket / kTickets + 1) << 2 * kCountBits;
                __syncthreads();
                first_segment = false;
            }
            if (threadIdx.x == 0) advance(a, sh.share, sh.cursor, sh.seg[i == 0 ? 2 : i - 1]);
            // this warp's tiles of the segment
            int left = (seg.t1 - tile + kWarps - 1) / kWarps;
            if (!primed || left == 1) next = left > 1 ? place(seg, tile + kWarps) : place(after, after.t0 + warp);
            primed = left > 0;
            const int h_after = after.hk / a.head_tiles;

            float o[NT * DC * 4][4];
            float m[NT][2], l[NT][2];
#pragma unroll
            for (int k = 0; k < NT * DC * 4; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt][0] = m[nt][1] = -INFINITY;
                l[nt][0] = l[nt][1] = 0.f;
            }
            for (; left > 0; --left, tile += kWarps) {
                // S^T = K Q^T
                float s[MT][NT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float odd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
                        for (int j = 0; j < 2 * DC; ++j) {
                            uint4 b;
                            if (kQInSmem) {
                                const int w = 4 * (nt * 2 * DC + j);
                                b = make_uint4(sh.q[kQInSmem ? w : 0][lane], sh.q[kQInSmem ? w + 1 : 0][lane],
                                               sh.q[kQInSmem ? w + 2 : 0][lane], sh.q[kQInSmem ? w + 3 : 0][lane]);
                            } else {
                                b = q[kQInSmem ? 0 : nt][kQInSmem ? 0 : j];
                            }
                            const uint4 k0 = kx[mt][0][j], k1 = kx[mt][1][j];
                            Mma<T>::run(s[mt][nt], k0.x, k1.x, k0.y, k1.y, b.x, b.y);
                            Mma<T>::run(odd, k0.z, k1.z, k0.w, k1.w, b.z, b.w);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][nt][e] += odd[e];
                    }
                const Places old = here;
                here = next;
                load_k(here, left > 1 ? h : h_after);
                next = left > 2 ? place(seg, tile + 2 * kWarps) : place(after, after.t0 + warp + (2 - left) * kWarps);

                // scale, mask, running maximum
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    int page, off;
                    const bool live0 = token(old.t[mt], g, &page, &off), live1 = token(old.t[mt], g + 8, &page, &off);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[mt][nt][e] = (e < 2 ? live0 : live1) ? s[mt][nt][e] * a.scale_log2 : -INFINITY;
                }
                if (a.scores_out) {
                    const int64_t row = static_cast<int64_t>(seg.b) * kv.kv_heads * a.head_tiles + seg.hk;
                    const bool sink = SINKS && tile < seg.sink_tiles;
                    const int begin = OWN ? seg.begin : 0;
                    const int at0 = ((sink ? begin / kTokens : seg.tile0) + tile) * MT * 16 + g;
                    const int first = sink ? begin : seg.first, len = sink ? seg.sinks : seg.len;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int rr = 0; rr < 2; ++rr) {
                                const int head = nt * 8 + 2 * t, at = at0 + mt * 16 + 8 * rr;
                                if (head < a.logit_heads && at < len && at >= first)
                                    *reinterpret_cast<float2 *>(a.logits + (row * kv.capacity + at) * a.logit_heads + head) =
                                        make_float2(s[mt][nt][2 * rr], s[mt][nt][2 * rr + 1]);
                            }
                }
                uint32_t part[MT][NT][2][Mma<T>::kParts];
                bool grew = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top[e & 1] = fmaxf(top[e & 1], s[mt][nt][e]);
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) {
                        top[0] = fmaxf(top[0], __shfl_xor_sync(kFull, top[0], x));
                        top[1] = fmaxf(top[1], __shfl_xor_sync(kFull, top[1], x));
                    }
                    float fix[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m2 = fmaxf(m[nt][e], top[e]);
                        grew = grew || m2 != m[nt][e];
                        fix[e] = exp2_from(m[nt][e], m2);
                        m[nt][e] = m2;
                        l[nt][e] *= fix[e];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const float p0 = exp2_from(s[mt][nt][e], m2), p1 = exp2_from(s[mt][nt][e + 2], m2);
                            l[nt][e] += p0 + p1;
                            s[mt][nt][e] = p0;
                            s[mt][nt][e + 2] = p1;
                        }
                    }
                    if (__any_sync(kFull, grew)) {
#pragma unroll
                        for (int k = 0; k < DC * 4; ++k)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt * DC * 4 + k][e] *= fix[e & 1];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            Mma<T>::split(s[mt][nt][2 * rr], s[mt][nt][2 * rr + 1], part[mt][nt][rr]);
                        }
                }
                // O^T += V^T P^T
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int c = 0; c < DC; ++c) {
                        const uint32_t *w[4] = {reinterpret_cast<const uint32_t *>(&vx[mt][c][0]),
                                                reinterpret_cast<const uint32_t *>(&vx[mt][c][1]),
                                                reinterpret_cast<const uint32_t *>(&vx[mt][c][2]),
                                                reinterpret_cast<const uint32_t *>(&vx[mt][c][3])};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t a0 = __byte_perm(w[0][k], w[1][k], 0x5410);
                            const uint32_t a1 = __byte_perm(w[0][k], w[1][k], 0x7632);
                            const uint32_t a2 = __byte_perm(w[2][k], w[3][k], 0x5410);
                            const uint32_t a3 = __byte_perm(w[2][k], w[3][k], 0x7632);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float(&acc)[4] = o[(nt * DC + c) * 4 + k];
#pragma unroll
                                for (int i = 0; i < Mma<T>::kParts; ++i)
                                    Mma<T>::run(acc, a0, a1, a2, a3, part[mt][nt][0][i], part[mt][nt][1][i]);
                            }
                        }
                    }
                load_v(here, left > 1 ? h : h_after);
            }

            if (!kQInSmem && after.t0 < after.t1) load_q(row_of(a, after.b, after.hk));

            // join the warps
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], x);
                    if (g == 0) {
                        sh.m[warp][nt * 8 + 2 * t + e] = m[nt][e];
                        sh.l[warp][nt * 8 + 2 * t + e] = l[nt][e];
                    }
                }
            __syncthreads();
            float top[NT][2], sum[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int head = nt * 8 + 2 * t + e;
                    float mm = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sh.m[w][head]);
                    float ll = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) ll += sh.l[w][head] * exp2_from(sh.m[w][head], mm);
                    const float fix = exp2_from(m[nt][e], mm);
#pragma unroll
                    for (int i = 0; i < DC * 4; ++i) {
                        sh.o[warp][(nt * DC * 4 + i) * 4 + e][lane] = o[nt * DC * 4 + i][e] * fix;
                        sh.o[warp][(nt * DC * 4 + i) * 4 + e + 2][lane] = o[nt * DC * 4 + i][e + 2] * fix;
                    }
                    top[nt][e] = mm;
                    sum[nt][e] = ll;
                }
            if (kQInSmem && after.t0 < after.t1) load_q(row_of(a, after.b, after.hk));
            __syncthreads();

            const bool whole = seg.t0 == 0 && seg.t1 == seg.tiles;
            const Row r = row_of(a, seg.b, seg.hk);
            finish(a, sh, r, whole ? -1 : 2 * sh.share.cta + (seg.t0 == 0 ? 1 : 0), top, sum);
            if (!whole) join(a, sh, seg, r);
            __syncthreads();  // shared memory is free again
        }
    }

    // Sums the warps' O in shared memory (relative to `top`) and writes the
    // row's output (slot < 0) or a part.
    static __device__ __forceinline__ void finish(const AttnArgs &a, const Shared &sh, const Row &r, int slot,
                                                  const float (&top)[NT][2], const float (&sum)[NT][2])
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float *mine = a.part + slot * a.part_stride;
        for (int i4 = warp; i4 < kRegs / 4; i4 += kWarps) {
            const int nt = i4 / (DC * 4);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v[e] += sh.o[w][i4 * 4 + e][lane];
            }
            if (slot < 0) {
                float inv[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ll = NT == 1 || nt == 0 ? sum[0][e] : sum[NT - 1][e];
                    inv[e] = OWN ? Mma<T>::kUnscale : ll == 0.f ? 0.f : Mma<T>::kUnscale / ll;
                }
                store_out(a, r, i4 * 4, v, lane, inv);
            } else {
                *reinterpret_cast<float4 *>(mine + (i4 * 32 + lane) * 4) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        if (warp == 0 && lane < 4) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int head = nt * 8 + 2 * lane + e;
                    if (slot < 0) {
                        if (!OWN) {
                            store_stats(a, r, head, top[nt][e], sum[nt][e]);
                        } else if (head < r.heads) {
                            float *stat = own_of(a, r, head) + span_row(a.kv.dim) - 4;
                            stat[0] = top[nt][e];
                            stat[1] = sum[nt][e];
                        }
                    } else {
                        mine[kRegs * 32 + head] = top[nt][e];
                        mine[kRegs * 32 + kHeads + head] = sum[nt][e];
                    }
                }
        }
    }

    // A counter holds the number of the call that last used it and, in
    // kCountBits each, two counts of that call.  What an earlier call has left there
    // (one whose lengths changed meanwhile leaves arrivals that no one waited for)
    // is below the present call's number and gives way to it.  The number comes from
    // the tickets that every CTA of a call draws, kTickets in all; CTA 0 draws
    // what the others leave.
    static constexpr int kCountBits = 11;
    static constexpr unsigned kTickets = 2 * kAttnMaxCtas, kTicketThread = 32;
    static_assert(kAttnMaxCtas < 1 << kCountBits && kTicketThread < kThreads, "");

    static __device__ __forceinline__ uint64_t draw_ticket(const AttnArgs &a)
    {
        // a part's slot 0 begins no group (join): its counter is free for the tickets
        const unsigned long long n = blockIdx.x == 0 ? kTickets - (gridDim.x - 1) : 1;
        return atomicAdd(reinterpret_cast<unsigned long long *>(a.arrived), n);
    }

    // Has every one of `expected` CTAs arrived at this counter's first or second
    // count?  True for the last, for which the others' parts are visible then.
    static __device__ __forceinline__ bool last_of(Shared &sh, uint64_t *counter, int which, int expected)
    {
        // the barrier orders the block's writes before thread 0's release, which
        // is cumulative; its acquire orders the others' parts before what the
        // block reads after the second barrier
        __syncthreads();
        if (threadIdx.x == 0) {
            const int shift = which * kCountBits;
            uint64_t seen;
            asm volatile("red.relaxed.gpu.global.max.u64 [%0], %1;" ::"l"(counter), "l"(sh.call) : "memory");
            asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;"
                         : "=l"(seen)
                         : "l"(counter), "l"(uint64_t{1} << shift)
                         : "memory");
            sh.last = static_cast<int>(seen >> shift & ((1 << kCountBits) - 1)) == expected - 1;
        }
        __syncthreads();
        return sh.last != 0;
    }

    // Joins n parts, the i-th at slot_of(i), into the row's output (into < 0) or
    // into a part's slot.  The warps take the parts in turn, several of each
    // in flight; the order of the sums is fixed by n.
    template <typename F>
    static __device__ void combine(const AttnArgs &a, Shared &sh, const Row &r, int n, F slot_of, int into)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3;
        for (int i = threadIdx.x; i < n * 2 * kHeads; i += kThreads) {
            const int p = i / (2 * kHeads), k = i - p * 2 * kHeads;
            const float v = __ldcg(a.part + slot_of(p) * a.part_stride + kRegs * 32 + k);
            if (k < kHeads)
                sh.part_m[p][k] = v;
            else
                sh.part_l[p][k - kHeads] = v;
        }
        __syncthreads();
        float top[NT][2], sum[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int head = nt * 8 + 2 * t + e;
                float mm = -INFINITY, ll = 0.f;
                for (int p = 0; p < n; ++p) mm = fmaxf(mm, sh.part_m[p][head]);
                for (int p = 0; p < n; ++p) ll += sh.part_l[p][head] * exp2_from(sh.part_m[p][head], mm);
                top[nt][e] = mm;
                sum[nt][e] = ll;
            }
        float v[kRegs];
#pragma unroll
        for (int i = 0; i < kRegs; ++i) v[i] = 0.f;
        for (int p = warp; p < n; p += kWarps) {
            const float *part = a.part + slot_of(p) * a.part_stride;
            float4 x[kRegs / 4];
#pragma unroll
            for (int i = 0; i < kRegs / 4; ++i) x[i] = __ldcg(reinterpret_cast<const float4 *>(part + (i * 32 + lane) * 4));
#pragma unroll
            for (int i = 0; i < kRegs / 4; ++i) {
                const int nt = i / (DC * 4);
                const float f0 = exp2_from(sh.part_m[p][nt * 8 + 2 * t], top[nt][0]);
                const float f1 = exp2_from(sh.part_m[p][nt * 8 + 2 * t + 1], top[nt][1]);
                v[4 * i] += x[i].x * f0;
                v[4 * i + 1] += x[i].y * f1;
                v[4 * i + 2] += x[i].z * f0;
                v[4 * i + 3] += x[i].w * f1;
            }
        }
#pragma unroll
        for (int i = 0; i < kRegs; ++i) sh.o[warp][i][lane] = v[i];
        __syncthreads();
        finish(a, sh, r, into, top, sum);
    }

    // A row that several CTAs share.  The last CTA of each group of kGroupCtas
    // to arrive joins the group's parts, the last group to arrive joins the
    // groups: one CTA joining all parts of a long row one after another took
    // 20 us and more of latency.
    static __device__ void join(const AttnArgs &a, Shared &sh, const Segment &seg, const Row &r)
    {
        // borders inside the row: the first and the last CTA that begins in it
        const Share &w = sh.share;
        const int64_t tile0 = seg.r0 + w.lead, r1 = tile0 + seg.tiles;
        const int first_in = static_cast<int>(((tile0 + kNear + 1) * w.ctas + w.total - 1) / w.total);
        const int last_in = static_cast<int>(((r1 - kNear) * w.ctas - 1) / w.total);
        const int c0 = first_in - 1, n = last_in - c0 + 1;
        if (c0 < 0 || c0 > w.cta || last_in < w.cta || last_in >= w.ctas) {
            // lengths that changed during the call: no part is where it should be
            if (threadIdx.x == 0) report_error(a.err, DEVERR_BAD_INDEX);
            return;
        }
        // a CTA's part that begins a row is its second slot, any other its first
        auto slot = [&](int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); };
        const int first = (w.cta - c0) / kGroupCtas * kGroupCtas, members = min(kGroupCtas, n - first);
        const int groups = (n + kGroupCtas - 1) / kGroupCtas;
        // level 0: the members of the group; level 1: the groups, counted beside the first one's members
        for (int level = 0; level < 2; ++level) {
            const bool members_only = level == 0;
            if (!last_of(sh, a.arrived + slot(members_only ? first : 0), level, members_only ? members : groups)) return;
            const bool done = !members_only || groups == 1;
            if (done || members > 1) {
                combine(a, sh, r, members_only ? members : groups,
                        [&](int i) { return slot(members_only ? first + i : i * kGroupCtas); }, done ? -1 : slot(first));
                __syncthreads();
            }
            if (done) return;
        }
    }

    // Sum over the block of one int per thread, and the thread's prefix.
    static __device__ int scan(Shared &sh, int v, int *total)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int s = v;
#pragma unroll
        for (int x = 1; x < 32; x *= 2) {
            const int n = __shfl_up_sync(kFull, s, x);
            if (lane >= x) s += n;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = s;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sh.scan[w];
            all += sh.scan[w];
        }
        *total = all;
        return before + s - v;
    }

    static __device__ void run(const AttnArgs &a, Shared &sh)
    {
        pdl_trigger();
        if (!OWN) pdl_wait();
        uint64_t ticket = 0;
        if (threadIdx.x == kTicketThread) ticket = draw_ticket(a);  // needed late
        empty_rows(a);
        const int hks = a.kv.kv_heads * a.head_tiles;
        // up to 32 sequences: one per lane, every warp for itself
        const bool few = a.kv.batch <= 32;
        const int step = few ? 32 : kThreads, own = few ? threadIdx.x & 31 : threadIdx.x;
        // tiles and rows per cached head over all sequences
        int64_t tiles = 0, rows = 0;
        int longest = 0;
        for (int b0 = 0; b0 < a.kv.batch; b0 += step) {
            const int n = b0 + own < a.kv.batch ? row_span<kTokens, SINKS, OWN>(a, b0 + own).tiles : 0;
            longest = max(longest, n);
            if (few) {
                tiles = __reduce_add_sync(kFull, n);
                rows = __popc(__ballot_sync(kFull, n > 0));
            } else {
                int all;
                scan(sh, n, &all);
                tiles += all;
                rows += __syncthreads_count(n > 0);
            }
        }
        longest = __reduce_max_sync(kFull, longest);
        if (!few) {
            __syncthreads();
            if ((threadIdx.x & 31) == 0) sh.scan[threadIdx.x >> 5] = longest;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) longest = max(longest, sh.scan[w]);
        }
        // shares of a round of the block's warps at least, but for short rows
        const int64_t most = max(tiles * hks / kWarps, rows * hks);
        const int ctas = static_cast<int>(min(most, static_cast<int64_t>(gridDim.x))), cta = blockIdx.x;
        if (tiles == 0 || cta >= ctas) return;
        const int64_t total = (tiles + rows * a.lead) * hks;
        const int64_t x0 = total * cta / ctas;
        if (threadIdx.x == 0) {
            sh.share.total = total;
            sh.share.x0 = x0;
            sh.share.x1 = total * (cta + 1) / ctas;
            sh.share.ctas = ctas;
            sh.share.cta = cta;
            sh.share.lead = a.lead;
            // uncut rows go to CTAs as evenly as their number allows
            const int64_t each = (rows * hks + ctas - 1) / ctas;
            sh.share.uncut = (each * longest - kUncut) * ctas <= tiles * hks ? INT32_MAX : kUncut;
            sh.cursor.b = a.kv.batch;
            sh.seg[0].t0 = sh.seg[0].t1 = 0;
        }
        __syncthreads();
        // the sequence that holds x0
        int64_t before = 0;
        for (int b0 = 0; b0 < a.kv.batch && x0 >= before * hks; b0 += step) {
            const int b = b0 + own, n = b < a.kv.batch ? row_span<kTokens, SINKS, OWN>(a, b).tiles : 0, cost = n > 0 ? n + a.lead : 0;
            int all, pre;
            if (few) {
                pre = cost;
#pragma unroll
                for (int x = 1; x < 32; x *= 2) {
                    const int up = __shfl_up_sync(kFull, pre, x);
                    if (own >= x) pre += up;
                }
                pre -= cost;
                all = 0;
            } else {
                pre = scan(sh, cost, &all);
            }
            const int64_t from = (before + pre) * hks;
            if (n > 0 && from <= x0 && x0 < from + static_cast<int64_t>(cost) * hks && (!few || threadIdx.x < 32)) {
                sh.cursor.before = before + pre;
                sh.cursor.b = b;
                sh.cursor.hk = static_cast<int>((x0 - from) / cost);
                advance(a, sh.share, sh.cursor, sh.seg[0]);
            }
            before += all;
        }
        __syncthreads();
        stream(a, sh, ticket);
    }
};

// Warps that fit on an SM by their registers (168 at a head size of 128), as
// one block or as blocks of four.
template <int DC, int NT>
constexpr int warps_per_sm()
{
    return DC * NT <= 2 ? 12 : 8;
}

template <typename T, int DC, int NT, int NW, bool VEC, bool WHOLE, bool SINKS, bool OWN>
__global__ void __launch_bounds__(NW * 32, warps_per_sm<DC, NT>() / NW)
    mbg_attn_kernel(const __grid_constant__ AttnArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    using K = Kernel<T, DC, NT, NW, VEC, WHOLE, SINKS, OWN>;
    K::run(a, *reinterpret_cast<typename K::Shared *>(raw));
    // The launch before it attends to the prefix, which nothing here depends on.  Each
    // of its blocks lets others start only behind its own wait, when what was launched
    // before it is done and its writes (lengths, table, K, V, the last call's use of the
    // workspace) are visible on the device; no block of this launch runs
    // earlier.  Who waits for this launch waits for both.
    if (OWN) pdl_wait();
}

template <typename T, int DC, int NT, int NW, bool VEC, bool WHOLE, bool SINKS, bool OWN>
cudaError_t launch_one(const AttnArgs &a, int sm_count, cudaStream_t s)
{
    constexpr int smem = sizeof(typename Kernel<T, DC, NT, NW, VEC, WHOLE, SINKS, OWN>::Shared);
    auto fn = mbg_attn_kernel<T, DC, NT, NW, VEC, WHOLE, SINKS, OWN>;
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> ready{0};  // a bit per device
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && !(ready.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e == cudaSuccess) ready.fetch_or(uint64_t{1} << (dev & 63), std::memory_order_relaxed);
        }
        if (e != cudaSuccess) return e;
    }
    int ctas = sm_count * (warps_per_sm<DC, NT>() / NW);
    if (ctas > kAttnMaxCtas) ctas = kAttnMaxCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

// big: one block of all an SM's warps instead of blocks of four.
template <typename T, int DC, int NT, bool SINKS, bool OWN>
cudaError_t launch_shape(const AttnArgs &a, bool big, int sm_count, cudaStream_t s)
{
    constexpr int kBig = warps_per_sm<DC, NT>();
    if (a.kv.page_size % 16 == 0)
        return big ? launch_one<T, DC, NT, kBig, true, true, SINKS, OWN>(a, sm_count, s)
                   : launch_one<T, DC, NT, 4, true, true, SINKS, OWN>(a, sm_count, s);
    return big ? launch_one<T, DC, NT, kBig, true, false, SINKS, OWN>(a, sm_count, s)
               : launch_one<T, DC, NT, 4, true, false, SINKS, OWN>(a, sm_count, s);
}

// SINKS: with first slots that stay visible; OWN: the slots behind a prefix.
template <typename T, bool SINKS, bool OWN>
cudaError_t launch(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s)
{
    const int dc = (a.kv.dim + 63) / 64;
    if (vec && nt == 2) return dc == 1 ? launch_shape<T, 1, 2, SINKS, OWN>(a, big, sm_count, s) : launch_shape<T, 2, 2, SINKS, OWN>(a, big, sm_count, s);
    if (vec) {
        switch (dc) {
        case 1: return launch_shape<T, 1, 1, SINKS, OWN>(a, big, sm_count, s);
        case 2: return launch_shape<T, 2, 1, SINKS, OWN>(a, big, sm_count, s);
        case 3: return launch_shape<T, 3, 1, SINKS, OWN>(a, big, sm_count, s);
        default: return launch_shape<T, 4, 1, SINKS, OWN>(a, big, sm_count, s);
        }
    }
    switch (dc) {
    case 1: return launch_one<T, 1, 1, 4, false, false, SINKS, OWN>(a, sm_count, s);
    case 2: return launch_one<T, 2, 1, 4, false, false, SINKS, OWN>(a, sm_count, s);
    case 3: return launch_one<T, 3, 1, 4, false, false, SINKS, OWN>(a, sm_count, s);
    default: return launch_one<T, 4, 1, 4, false, false, SINKS, OWN>(a, sm_count, s);
    }
}

}  // namespace attn
}  // namespace mbg
