// Attention of one new token over a paged key-value cache.
//
//   s_t = scale * q . k_t,  p = softmax(s),  o = sum_t p_t v_t
//
// over the tokens t in [max(0, len - window), len) of a sequence, G query
// heads sharing one cached head.  One pass over the cache: each warp keeps a
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
// P is split into two 16-bit parts (high and the rest), two MMAs per V tile:
// a rounding of P to 8 (bf16) or 11 (f16) bits would be as large as that of
// the output itself; with the rest added the error is 2^-16 or less.
//
// The next tile's K is requested while the present tile's softmax and V
// product run, and the next V after that: about 8 KB in flight per warp at a
// head size of 128.
//
// Split over the length: the rows (sequence x cached head) are cut into blocks
// of NW * 16 tokens; all blocks of the call are numbered and each CTA takes an
// equal share of consecutive ones, whatever the lengths (they are read on the
// device, so a captured graph serves any lengths).  A row inside one CTA's
// share is written at once; otherwise each CTA leaves (O, m, l) in the
// workspace and the last to arrive joins them, always in the same order, so
// results do not depend on the order of arrival.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"

namespace mbg {
namespace attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xFFFFFFFFu;
// CTAs whose parts of a row are joined first, before the groups are.
constexpr int kGroupCtas = 16;

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
    // Two values rounded to 16 bits, first one in the low half.
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
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
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
    }
    static __device__ __forceinline__ uint16_t bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};

// 8x8 matrix of 16-bit elements, one row per four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t w)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
    return r;
}

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

// Eight consecutive 16-bit elements at p, of which the first `left` exist.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int left)
{
    if (VEC) return ld_stream16(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < left ? __ldg(p + 2 * i) : 0;
        const uint32_t hi = 2 * i + 1 < left ? __ldg(p + 2 * i + 1) : 0;
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// First tile of 16 tokens, number of tiles and of blocks of a sequence.
struct RowSpan {
    int first, len;         // tokens [first, len)
    int tile0, tiles;       // 16-token tiles, tile0 = first / 16
    __device__ __forceinline__ int blocks() const { return (tiles + kWarps - 1) / kWarps; }
};

__device__ __forceinline__ RowSpan row_span(const AttnArgs &a, int b)
{
    RowSpan r;
    int len = __ldg(a.lengths + b);
    if (len < 0) len = 0;
    if (len > a.kv.capacity) len = static_cast<int>(a.kv.capacity);
    r.len = len;
    r.first = (a.window > 0 && len > a.window) ? len - a.window : 0;
    r.tile0 = r.first >> 4;
    r.tiles = len > r.first ? ((len + 15) >> 4) - r.tile0 : 0;
    return r;
}

// Page of one token, and its place in the page; page -1 where there is none.
struct TokenPlace {
    int page, off;
};

__device__ __forceinline__ TokenPlace place_of(const KvView &kv, const int32_t *table, int slot, bool wanted,
                                               unsigned int *err)
{
    TokenPlace p;
    p.page = -1;
    p.off = 0;
    if (wanted) {
        const int idx = kv.page_shift >= 0 ? slot >> kv.page_shift : slot / kv.page_size;
        p.off = slot - idx * kv.page_size;
        const int page = __ldg(table + idx);
        if (page >= 0 && page < kv.num_pages)
            p.page = page;
        else
            report_error(err, DEVERR_BAD_INDEX);
    }
    return p;
}

template <typename T, int DC, int NT, bool VEC>
struct Kernel {
    static constexpr int kHeads = 8 * NT;           // query heads of one tile
    static constexpr int kRegs = NT * DC * 16;      // O values per thread
    static constexpr int kQWords = NT * DC * 8;     // Q words per thread
    // Q of wide heads or of two head tiles comes from shared memory: as
    // registers it would not fit beside K, V and O
    static constexpr bool kQInSmem = NT * DC > 2;

    // parts joined at once: a group, or the groups of a row
    static constexpr int kMaxParts = kAttnMaxCtas / kGroupCtas;

    struct Shared {
        float o[kWarps][kRegs][32];
        float m[kWarps][kHeads];
        float l[kWarps][kHeads];
        uint32_t q[kQInSmem ? kQWords : 1][32];
        float part_m[kMaxParts][kHeads];
        float part_l[kMaxParts][kHeads];
        int scan[kWarps];
        int pick[2];
        int last;
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
        const float lse2 = l > 0.f || l != l ? m + log2f(l) : -INFINITY;
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
            if (len > 0) continue;
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

    // Blocks [k0, k1) of a row.
    static __device__ void segment(const AttnArgs &a, Shared &sh, const RowSpan &span, const Row &r, int k0, int k1,
                                   int64_t unit0, int64_t units, int ctas, int cta)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int g = lane >> 2, t = lane & 3;
        const KvView &kv = a.kv;
        const int h = r.hk / a.head_tiles;
        const uint16_t *kbase = static_cast<const uint16_t *>(kv.k) + h * kv.ks_head;
        const uint16_t *vbase = static_cast<const uint16_t *>(kv.v) + h * kv.vs_head;
        const int32_t *table = kv.table + r.b * kv.table_stride;

        uint4 q[kQInSmem ? 1 : NT][kQInSmem ? 1 : 2 * DC];
        {
            const uint16_t *qb = static_cast<const uint16_t *>(a.q) + r.b * a.q_sb;
            if (kQInSmem) {
                __syncthreads();
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
                __syncthreads();
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
        }

        float o[NT * DC * 4][4];
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int i = 0; i < NT * DC * 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }

        uint4 kx[2][2 * DC], vx[DC][4];
        const int tile_end = min(span.tiles, k1 * kWarps);
        // lanes 0..15 (and again 16..31) hold the places of the tile's tokens
        auto place = [&](int tile) {
            const int slot = (span.tile0 + tile) * 16 + (lane & 15);
            return place_of(kv, table, slot, tile < tile_end && slot >= span.first && slot < span.len, a.err);
        };
        auto load_k = [&](const TokenPlace &p) {
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int page = __shfl_sync(kFull, p.page, g + 8 * rr);
                const int off = __shfl_sync(kFull, p.off, g + 8 * rr);
                const uint16_t *row = kbase + page * kv.ks_page + off * kv.ks_tok;
#pragma unroll
                for (int j = 0; j < 2 * DC; ++j) {
                    const int d = j * 32 + t * 8;
                    kx[rr][j] = (page >= 0 && d < kv.dim) ? load8<VEC>(row + d, kv.dim - d) : make_uint4(0, 0, 0, 0);
                }
            }
        };
        auto load_v = [&](const TokenPlace &p) {
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) {
                const int tok = 2 * t + (rr & 1) + 8 * (rr >> 1);
                const int page = __shfl_sync(kFull, p.page, tok);
                const int off = __shfl_sync(kFull, p.off, tok);
                const uint16_t *row = vbase + page * kv.vs_page + off * kv.vs_tok;
#pragma unroll
                for (int c = 0; c < DC; ++c) {
                    const int d = c * 64 + g * 8;
                    vx[c][rr] = (page >= 0 && d < kv.dim) ? load8<VEC>(row + d, kv.dim - d) : make_uint4(0, 0, 0, 0);
                }
            }
        };

        int tile = k0 * kWarps + warp;
        TokenPlace here = place(tile), next = place(tile + kWarps);
        load_k(here);
        load_v(here);
        for (; tile < tile_end; tile += kWarps) {
            // S^T = K Q^T
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float odd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
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
                    Mma<T>::run(s[nt], kx[0][j].x, kx[1][j].x, kx[0][j].y, kx[1][j].y, b.x, b.y);
                    Mma<T>::run(odd, kx[0][j].z, kx[1][j].z, kx[0][j].w, kx[1][j].w, b.z, b.w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] += odd[e];
            }
            const TokenPlace old = here;
            here = next;
            load_k(here);
            next = place(tile + 2 * kWarps);

            // scale, mask, running maximum
            const bool live0 = __shfl_sync(kFull, old.page, g) >= 0;
            const bool live1 = __shfl_sync(kFull, old.page, g + 8) >= 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool live = e < 2 ? live0 : live1;
                    s[nt][e] = live ? s[nt][e] * a.scale_log2 : -INFINITY;
                }
            }
            if (a.scores_out) {
                const int64_t row = static_cast<int64_t>(r.b) * kv.kv_heads * a.head_tiles + r.hk;
                const int slot = (span.tile0 + tile) * 16 + g;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr) {
                        const int head = nt * 8 + 2 * t, at = slot + 8 * rr;
                        if (head < a.logit_heads && at < span.len && at >= span.first)
                            *reinterpret_cast<float2 *>(a.logits + (row * kv.capacity + at) * a.logit_heads + head) =
                                make_float2(s[nt][2 * rr], s[nt][2 * rr + 1]);
                    }
            }
            uint32_t phi[NT][2], plo[NT][2];
            bool grew = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float top[2] = {fmaxf(s[nt][0], s[nt][2]), fmaxf(s[nt][1], s[nt][3])};
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
                    const float p0 = exp2_from(s[nt][e], m2), p1 = exp2_from(s[nt][e + 2], m2);
                    l[nt][e] = l[nt][e] * fix[e] + (p0 + p1);
                    s[nt][e] = p0;
                    s[nt][e + 2] = p1;
                }
                if (__any_sync(kFull, grew)) {
#pragma unroll
                    for (int i = 0; i < DC * 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nt * DC * 4 + i][e] *= fix[e & 1];
                }
#pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
                    const uint32_t hi = Mma<T>::pack(s[nt][2 * rr], s[nt][2 * rr + 1]);
                    const float2 back = Mma<T>::unpack(hi);
                    const uint32_t lo = Mma<T>::pack(s[nt][2 * rr] - back.x, s[nt][2 * rr + 1] - back.y);
                    phi[nt][rr] = transpose8x8(hi);
                    plo[nt][rr] = transpose8x8(lo);
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int c = 0; c < DC; ++c) {
                const uint32_t *w[4] = {reinterpret_cast<const uint32_t *>(&vx[c][0]),
                                        reinterpret_cast<const uint32_t *>(&vx[c][1]),
                                        reinterpret_cast<const uint32_t *>(&vx[c][2]),
                                        reinterpret_cast<const uint32_t *>(&vx[c][3])};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = __byte_perm(w[0][i], w[1][i], 0x5410);
                    const uint32_t a1 = __byte_perm(w[0][i], w[1][i], 0x7632);
                    const uint32_t a2 = __byte_perm(w[2][i], w[3][i], 0x5410);
                    const uint32_t a3 = __byte_perm(w[2][i], w[3][i], 0x7632);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        Mma<T>::run(o[(nt * DC + c) * 4 + i], a0, a1, a2, a3, phi[nt][0], phi[nt][1]);
                        Mma<T>::run(o[(nt * DC + c) * 4 + i], a0, a1, a2, a3, plo[nt][0], plo[nt][1]);
                    }
                }
            }
            load_v(here);
        }

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
        __syncthreads();

        const bool whole = k0 == 0 && k1 == span.blocks();
        const int slot = 2 * cta + (k0 == 0 ? 1 : 0);
        finish(a, sh, r, whole ? -1 : slot, top, sum);
        if (!whole) join(a, sh, span, r, unit0, units, ctas, cta);
        __syncthreads();  // shared memory is free again
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
                    inv[e] = ll == 0.f ? 0.f : 1.f / ll;
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
                        store_stats(a, r, head, top[nt][e], sum[nt][e]);
                    } else {
                        mine[kRegs * 32 + head] = top[nt][e];
                        mine[kRegs * 32 + kHeads + head] = sum[nt][e];
                    }
                }
        }
    }

    // CTA whose share holds a block: the largest c with units * c / ctas <= u.
    static __device__ __forceinline__ int cta_of(int64_t u, int64_t units, int ctas)
    {
        return static_cast<int>(((u + 1) * ctas - 1) / units);
    }

    // Has every one of `expected` CTAs arrived at this counter?  True for the
    // last, for which the others' parts are visible then.
    static __device__ __forceinline__ bool last_of(Shared &sh, unsigned int *counter, int expected)
    {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            sh.last = atomicAdd(counter, 1u) == static_cast<unsigned>(expected - 1);
            if (sh.last) *counter = 0;  // ready for the next call
        }
        __syncthreads();
        if (!sh.last) return false;
        __threadfence();
        return true;
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
#pragma unroll 2
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
    // 20 us and more of latency, two levels take about 3.  unit0: number of the
    // row's first block.
    static __device__ void join(const AttnArgs &a, Shared &sh, const RowSpan &span, const Row &r, int64_t unit0,
                                int64_t units, int ctas, int cta)
    {
        const int c0 = cta_of(unit0, units, ctas), n = cta_of(unit0 + span.blocks() - 1, units, ctas) - c0 + 1;
        // a CTA's part that begins a row is its second slot, any other its first
        auto slot = [&](int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); };
        const int first = (cta - c0) / kGroupCtas * kGroupCtas, members = min(kGroupCtas, n - first);
        const int groups = (n + kGroupCtas - 1) / kGroupCtas;
        if (!last_of(sh, a.arrived_group + slot(first), members)) return;
        if (groups == 1) {
            combine(a, sh, r, n, slot, -1);
            return;
        }
        if (members > 1) {
            combine(a, sh, r, members, [&](int i) { return slot(first + i); }, slot(first));
            __syncthreads();
        }
        const int64_t row = static_cast<int64_t>(r.b) * a.kv.kv_heads * a.head_tiles + r.hk;
        if (!last_of(sh, a.arrived + row, groups)) return;
        combine(a, sh, r, groups, [&](int i) { return slot(i * kGroupCtas); }, -1);
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
        pdl_wait();
        empty_rows(a);
        const int hks = a.kv.kv_heads * a.head_tiles;
        // blocks per cached head over all sequences
        int64_t blocks = 0;
        for (int b0 = 0; b0 < a.kv.batch; b0 += kThreads) {
            const int b = b0 + threadIdx.x;
            int all;
            scan(sh, b < a.kv.batch ? row_span(a, b).blocks() : 0, &all);
            blocks += all;
        }
        const int64_t units = blocks * hks;
        if (units == 0) return;
        // no CTA without a block, so that a row's CTAs are all that lie between
        // its first and its last
        const int ctas = static_cast<int>(min(units, static_cast<int64_t>(gridDim.x)));
        const int cta = blockIdx.x;
        if (cta >= ctas) return;
        int64_t u = units * cta / ctas;
        const int64_t u_end = units * (cta + 1) / ctas;
        // the sequence that holds block u
        int64_t before = 0;
        int b = 0;
        for (int b0 = 0; b0 < a.kv.batch; b0 += kThreads) {
            const int mine = b0 + threadIdx.x;
            const int n = mine < a.kv.batch ? row_span(a, mine).blocks() : 0;
            int all;
            const int pre = scan(sh, n, &all);
            if (u < (before + all) * hks) {
                if (n > 0 && (before + pre) * hks <= u && u < (before + pre + n) * hks) {
                    sh.pick[0] = mine;
                    sh.pick[1] = pre;
                }
                __syncthreads();
                b = sh.pick[0];
                before += sh.pick[1];
                break;
            }
            before += all;
        }
        while (u < u_end) {
            const RowSpan span = row_span(a, b);
            const int n = span.blocks();
            if (n == 0) {
                ++b;
                continue;
            }
            const int64_t base = before * hks;
            int64_t rem = u - base;
            while (rem < static_cast<int64_t>(n) * hks && u < u_end) {
                const int hk = static_cast<int>(rem / n), k0 = static_cast<int>(rem - static_cast<int64_t>(hk) * n);
                const int k1 = static_cast<int>(min(static_cast<int64_t>(n), k0 + (u_end - u)));
                segment(a, sh, span, row_of(a, b, hk), k0, k1, base + static_cast<int64_t>(hk) * n, units, ctas, cta);
                u += k1 - k0;
                rem += k1 - k0;
            }
            before += n;
            ++b;
        }
    }
};

template <int DC, int NT>
constexpr int ctas_per_sm()
{
    return DC * NT <= 1 ? 4 : DC * NT <= 2 ? 3 : 2;
}

template <typename T, int DC, int NT, bool VEC>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<DC, NT>()) mbg_attn_kernel(const __grid_constant__ AttnArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Kernel<T, DC, NT, VEC>::run(a, *reinterpret_cast<typename Kernel<T, DC, NT, VEC>::Shared *>(raw));
}

template <typename T, int DC, int NT, bool VEC>
cudaError_t launch_one(const AttnArgs &a, cudaStream_t s)
{
    constexpr int smem = sizeof(typename Kernel<T, DC, NT, VEC>::Shared);
    auto fn = mbg_attn_kernel<T, DC, NT, VEC>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
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
cudaError_t launch(const AttnArgs &a, bool vec, int nt, cudaStream_t s)
{
    const int dc = (a.kv.dim + 63) / 64;
    if (vec && nt == 2) return dc == 1 ? launch_one<T, 1, 2, true>(a, s) : launch_one<T, 2, 2, true>(a, s);
    if (vec) {
        switch (dc) {
        case 1: return launch_one<T, 1, 1, true>(a, s);
        case 2: return launch_one<T, 2, 1, true>(a, s);
        case 3: return launch_one<T, 3, 1, true>(a, s);
        default: return launch_one<T, 4, 1, true>(a, s);
        }
    }
    switch (dc) {
    case 1: return launch_one<T, 1, 1, false>(a, s);
    case 2: return launch_one<T, 2, 1, false>(a, s);
    case 3: return launch_one<T, 3, 1, false>(a, s);
    default: return launch_one<T, 4, 1, false>(a, s);
    }
}

}  // namespace attn
}  // namespace mbg
