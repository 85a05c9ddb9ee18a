// Internal declarations of the decode-step operators (paged attention, cache
// eviction, rotary append, residual norms).  Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gemv.h"

namespace mbg {

// What the decode-step entry points need of the current device; nullptr on
// failure (the CUDA error is recorded for gemv_last_cuda_error).
struct DecodeDevice {
    unsigned int *status;  // device status word
    int sm_count;
    uint64_t wait_limit_ns;    // bound of every device-side wait
    unsigned int skip_copies;  // test hook (SKIP_*)
};
bool decode_device(DecodeDevice *d);
gemv_status_t decode_cuda_fail(cudaError_t e, gemv_status_t code);

// The cache as the kernels see it.  All strides in elements.
struct KvView {
    void *k, *v;
    int64_t ks_page, ks_tok, ks_head;
    int64_t vs_page, vs_tok, vs_head;
    const int32_t *table;
    int64_t table_stride;
    int64_t num_pages;
    int page_size, page_shift;  // page_shift < 0: not a power of two
    int max_pages;
    int batch, kv_heads, dim;
    int64_t capacity;           // max_pages * page_size
};

struct AttnArgs {
    KvView kv;
    const void *q;
    int64_t q_sb, q_sh;
    void *out;
    int64_t o_sb, o_sh;
    const int32_t *lengths;
    float *lse;                 // [batch][q_heads] natural log, or NULL
    const float *scores_in;     // accumulated weights
    float *scores_out;          // NULL: not accumulated
    int q_heads, group;         // query heads per cached head
    int head_tiles;             // tiles of 8 * NT query heads per cached head
    int window;                 // 0: none
    int sinks;                  // first slots that stay visible behind a window
    float scale_log2;           // scale * log2(e)
    unsigned int *err;
    // workspace
    float *part;                // [2 * ctas][part_stride]: O in fragment order, then m and l per head
    int64_t part_stride;
    uint64_t *arrived;          // [2 * kAttnMaxCtas], by a part's slot; zero before the first call
    float *row_lse;             // same rows x 8 * NT heads: log2 of the softmax denominator
    float *logits;              // [rows][capacity][logit_heads], log2 units; weights only
    int logit_heads;
    int lead;                   // tiles that a row's beginning counts like
    // a prefix that is attended to elsewhere: only slots from *prefix on are read
    const int32_t *prefix;      // NULL: none
    float *own;                 // instead of out, [batch * q_heads][span_row(dim)]
};
// A row of FP32 results: O, and from the last four on the maximum (log2 units)
// and the denominator that it is relative to.
__host__ __device__ constexpr int span_row(int dim) { return (dim + 3) / 4 * 4 + 4; }

// Launches for one cache type; vec: 16-byte loads are possible; big: one block
// per SM instead of several small ones.
cudaError_t launch_attn_f16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s);
cudaError_t launch_attn_bf16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s);
// The same with a.sinks, and for the slots behind a.prefix, into a.own.  Kernels of
// their own: with all forms in one, chosen at run time, the plain one spilled registers
// (bf16, 128: 88 bytes) and 24 sequences of heads of 256 took 121.5 us, not 114.7; with
// sinks in it 119.7.
cudaError_t launch_attn_sinks_f16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s);
cudaError_t launch_attn_sinks_bf16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s);
cudaError_t launch_attn_own_f16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s);
cudaError_t launch_attn_own_bf16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s);
cudaError_t launch_attn_weights(const AttnArgs &a, int nt, cudaStream_t s);
constexpr int kAttnMaxCtas = 512;

// A part of a block of rows that several CTAs share (tiles 0: none).
struct SpanInfo {
    int b, h, row0, t0, t1, tiles;
};
constexpr int kSpanMaxCtas = 160;

// Attention of many tokens over one table row's slots: of the new tokens of
// each sequence (starts), or of a batch's tokens over the prefix that its
// sequences share (prefix).
struct SpanArgs {
    KvView kv;
    const void *q;
    int64_t q_st, q_sh;
    void *out;
    int64_t o_st, o_sh;
    float *lse;                 // [tokens][q_heads] natural log, or NULL
    float *pre;                 // prefix: blocks that are not cut, [tokens * q_heads][span_row(dim)]
    const float *own;           // prefix: what the slots behind it give, alike
    const int32_t *starts;      // [batch + 1]; NULL: prefix
    const int32_t *lengths;     // [batch]
    const int32_t *prefix;
    int tokens;
    int q_heads, group;
    int window, sinks;
    float scale_log2;
    int out_vec;                // out takes stores of 16 bytes (1), of 32 (2)
    unsigned int *err;
    // workspace
    float *part;                // [2 * ctas][part_stride]: per tile of rows O [dim / 4][row][4], m and l [row]
    int64_t part_stride;
    SpanInfo *info;             // [2 * ctas]
    uint8_t *redo;              // [tokens * q_heads]: rows to be computed one by one
    // K and V as tensors (element, token of a page, head, page) for bulk copies of
    // `box` tokens of a page at a time; box 0: copied piece by piece
    int box;
    uint64_t wait_limit_ns;     // bound of every wait
    int skip_tile;              // test hook (SKIP_TILE)
    CUtensorMap k_map, v_map;
};
// Rows of a tile of query rows, and how many tiles a block of them has.
constexpr int kSpanRows = 128;
__host__ __device__ constexpr int span_streams(int dim) { return dim <= 128 ? 2 : 1; }
// Slots of a tile.
__host__ __device__ constexpr int span_tile(int dim) { return dim <= 128 ? 128 : 64; }
// Floats of a part.
__host__ __device__ constexpr int64_t span_part(int dim) { return static_cast<int64_t>(span_streams(dim)) * kSpanRows * ((dim + 15) / 16 * 16 + 2); }
cudaError_t launch_tile_f16(const SpanArgs &a, bool vec, int ctas, cudaStream_t s);
cudaError_t launch_tile_bf16(const SpanArgs &a, bool vec, int ctas, cudaStream_t s);
// The tiles, and what follows them (and for a prefix the attention behind it):
// joins, and rows computed one by one.
cudaError_t launch_span(const SpanArgs &a, bool vec, int elem, int sm_count, cudaStream_t s);
cudaError_t launch_span_finish(const SpanArgs &a, int elem, int sm_count, cudaStream_t s);

struct EvictArgs {
    KvView kv;
    const float *scores;
    const int32_t *stamps;
    const int32_t *lengths;
    int keep, sinks, recent;
    int32_t *moves;             // [batch][kv_heads][max_moves][2]
    int32_t *counts;            // [batch][kv_heads]
    int64_t max_moves;
    unsigned int *err;
};
cudaError_t launch_evict_plan(const EvictArgs &a, cudaStream_t s);

struct EvictApplyArgs {
    KvView kv;
    float *scores;              // NULL: not moved
    int32_t *stamps;
    int32_t *lengths;           // NULL: not written
    int keep;
    const int32_t *moves;
    const int32_t *counts;
    int64_t max_moves;
    unsigned int *err;
};
cudaError_t launch_evict_apply(const EvictApplyArgs &a, bool vec, int sm_count, cudaStream_t s);

struct RopeArgs {
    KvView kv;
    const void *q, *k, *v;
    int src_elem, dst_elem;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;
    void *q_out;
    int64_t qo_st, qo_sh;
    const int32_t *positions;   // [axes][tokens], rows pos_stride apart
    int64_t pos_stride;
    const int32_t *slots;       // [tokens]
    const int32_t *seq;         // [tokens] or NULL (token t belongs to sequence t)
    const int32_t *stamps;      // [tokens] or NULL
    float *scores_cache;        // NULL: not initialised
    int32_t *stamps_cache;
    const uint64_t *turns;      // [rot / 2]: 2^64 * frequency / (2 pi)
    const uint8_t *axis;        // [rot / 2]
    int tokens, q_heads, rot, axes, pairs;
    // norms of q's and k's heads before they are turned
    int norm, unit_offset;
    const void *q_weight, *k_weight;  // [dim] or NULL (1)
    int q_weight_e, k_weight_e;
    float eps;
    unsigned int *err;
};
cudaError_t launch_rope(const RopeArgs &a, bool vec, int sm_count, cudaStream_t s);

struct AssignArgs {
    int32_t *table;             // [batch][max_pages]
    int64_t table_stride, capacity;
    int64_t num_pages;
    int batch, page_size;
    const int32_t *lengths, *fresh;
    const int32_t *shared;      // NULL: none
    int32_t *lengths_out;       // may be lengths
    int32_t *ring;              // free pages, from state[0] on, state[1] of them
    int64_t ring_size;
    const int32_t *state;
    int32_t *state_out;         // may be state
    int32_t *starts;            // [batch + 1]
    int32_t *slots, *seq;       // [room]
    int64_t room;
    int wide;                   // both take 16-byte stores
    unsigned int *err;
};
cudaError_t launch_assign(const AssignArgs &a, cudaStream_t s);

struct NormArgs {
    const void *y, *r, *gate, *post_w, *pre_w, *pre_b;
    void *out, *h;
    int y_e, r_e, gate_e, post_e, pre_w_e, pre_b_e, h_e;
    int64_t y_s, r_s, gate_s, post_s, pre_w_s, pre_b_s, out_s, h_s;  // row strides (0: one row for all)
    int64_t rows;
    int width;
    int post, layer, unit_offset;
    int staged;  // bits 0..3: post_w, gate, pre_w, pre_b stand in shared memory
    float alpha, eps;
};
cudaError_t launch_norm(const NormArgs &a, bool vec, int sm_count, cudaStream_t s);

}  // namespace mbg
