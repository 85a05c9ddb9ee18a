// Internal declarations of the decode-step operators (paged attention, cache
// eviction, rotary append, residual norms).  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gemv.h"

namespace mbg {

// What the decode-step entry points need of the current device; nullptr on
// failure (the CUDA error is recorded for gemv_last_cuda_error).
struct DecodeDevice {
    unsigned int *status;  // device status word
    int sm_count;
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
};

// Launches for one cache type; vec: 16-byte loads are possible; big: one block
// per SM instead of several small ones.
cudaError_t launch_attn_f16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s);
cudaError_t launch_attn_bf16(const AttnArgs &a, bool vec, int nt, bool big, int sm_count, cudaStream_t s);
cudaError_t launch_attn_weights(const AttnArgs &a, int nt, cudaStream_t s);
constexpr int kAttnMaxCtas = 512;

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
    unsigned int *err;
};
cudaError_t launch_rope(const RopeArgs &a, bool vec, int sm_count, cudaStream_t s);

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
