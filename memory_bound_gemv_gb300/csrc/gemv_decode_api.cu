// C-ABI entry points of the decode-step operators (include/gemv.h): argument
// checks, the choice between vector and element-wise loads, launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>

#include "../../include/gemv.h"
#include "gemv_decode.h"
#include "gemv_internal.h"

namespace mbg {
namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is_elem(int e) { return e == GEMV_ELEM_F32 || e == GEMV_ELEM_F16 || e == GEMV_ELEM_BF16; }
int elem_bytes(int e) { return e == GEMV_ELEM_F32 ? 4 : 2; }
// Alignment of eight elements that are moved at once.
int vec_bytes(int e) { return 8 * elem_bytes(e); }

bool mult8(const int64_t *stride, int n)
{
    for (int i = 0; i < n; ++i)
        if (stride[i] % 8) return false;
    return true;
}

bool negative(const gemv_heads_t &h) { return h.stride[0] < 0 || h.stride[1] < 0; }

// Checks a cache and fills the kernels' view of it.
gemv_status_t view_of(const gemv_kv_t *kv, KvView *v, bool need_data = true)
{
    if (!kv) return GEMV_ERR_INVALID_VALUE;
    if (kv->elem != GEMV_ELEM_F16 && kv->elem != GEMV_ELEM_BF16) return GEMV_ERR_INVALID_VALUE;
    if (kv->batch < 0 || kv->kv_heads < 1 || kv->head_dim < 1 || kv->page_size < 1 || kv->max_pages < 0 ||
        kv->num_pages < 0 || kv->table_stride < 0)
        return GEMV_ERR_INVALID_VALUE;
    for (int i = 0; i < 3; ++i)
        if (kv->k_stride[i] < 0 || kv->v_stride[i] < 0) return GEMV_ERR_INVALID_VALUE;
    if (kv->head_dim > 256) return GEMV_ERR_UNSUPPORTED;
    const int64_t capacity = static_cast<int64_t>(kv->page_size) * kv->max_pages;
    // slots, rows and page numbers are 32-bit on the device
    if (capacity > INT_MAX - 4096 || kv->num_pages > INT_MAX ||
        static_cast<int64_t>(kv->batch) * kv->kv_heads > INT_MAX / 64 || kv->batch > 65535 || kv->kv_heads > 65535)
        return GEMV_ERR_UNSUPPORTED;
    if (need_data && kv->batch > 0) {
        if (!kv->k || !kv->v || (kv->max_pages > 0 && !kv->page_table)) return GEMV_ERR_INVALID_VALUE;
        if (!aligned(kv->k, 2) || !aligned(kv->v, 2) || !aligned(kv->page_table, 4) || !aligned(kv->scores, 4) ||
            !aligned(kv->stamps, 4))
            return GEMV_ERR_MISALIGNED;
    }
    v->k = kv->k;
    v->v = kv->v;
    v->ks_page = kv->k_stride[0];
    v->ks_tok = kv->k_stride[1];
    v->ks_head = kv->k_stride[2];
    v->vs_page = kv->v_stride[0];
    v->vs_tok = kv->v_stride[1];
    v->vs_head = kv->v_stride[2];
    v->table = kv->page_table;
    v->table_stride = kv->table_stride;
    v->num_pages = kv->num_pages;
    v->page_size = kv->page_size;
    v->page_shift = -1;
    for (int s = 0; s < 31; ++s)
        if (kv->page_size == 1 << s) v->page_shift = s;
    v->max_pages = kv->max_pages;
    v->batch = kv->batch;
    v->kv_heads = kv->kv_heads;
    v->dim = kv->head_dim;
    v->capacity = capacity;
    return GEMV_OK;
}

bool cache_vec(const gemv_kv_t *kv)
{
    return kv->head_dim % 8 == 0 && aligned(kv->k, 16) && aligned(kv->v, 16) && mult8(kv->k_stride, 3) &&
           mult8(kv->v_stride, 3);
}

// Heads that the kernels' 32-bit counts of heads and of their elements can hold.
bool too_many_heads(int heads, int dim)
{
    return heads > 1 << 24 || static_cast<int64_t>(heads) * dim > INT_MAX;
}

// Query heads per tile: two MMA tiles of eight where a cached head has more
// than eight and the accumulators of both fit in registers.
int head_tile(int dim, int group, bool vec) { return vec && group > 8 && dim <= 128 ? 2 : 1; }

struct AttnPlan {
    int nt, head_tiles, logit_heads;
    int64_t part_stride, rows;
    size_t part, row_lse, logits, total;  // offsets and size in bytes
};

// The element-wise kernel takes single tiles: sized for the larger need.
AttnPlan attn_plan(const KvView &v, int group, int nt, bool weights)
{
    AttnPlan p;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const int dc = (v.dim + 63) / 64, heads = 8 * nt;
    p.nt = nt;
    p.head_tiles = (group + heads - 1) / heads;
    p.logit_heads = group >= heads ? heads : (group + 1) / 2 * 2;
    p.part_stride = static_cast<int64_t>(nt) * dc * 16 * 32 + 2 * heads;
    p.rows = static_cast<int64_t>(v.batch) * v.kv_heads * p.head_tiles;
    // The counters stand ahead of all else, whatever the tiles: calls whose q
    // allows wide loads and calls whose q does not share a workspace.
    static_assert(2 * kAttnMaxCtas * sizeof(uint64_t) == GEMV_ATTN_COUNTER_BYTES, "");
    p.part = GEMV_ATTN_COUNTER_BYTES;
    p.row_lse = p.part + up(static_cast<size_t>(2) * kAttnMaxCtas * p.part_stride * 4);
    p.logits = p.row_lse + (weights ? up(static_cast<size_t>(p.rows) * heads * 4) : 0);
    p.total = p.logits + (weights ? up(static_cast<size_t>(p.rows) * v.capacity * p.logit_heads * 4) : 0);
    return p;
}

// Workspace of the attention of many tokens: offsets and size in bytes.
struct SpanPlan {
    size_t info, redo, pre, own, total;
};

SpanPlan span_plan(const KvView &v, int64_t tokens, int q_heads, bool prefix)
{
    SpanPlan p;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = static_cast<size_t>(tokens) * q_heads;
    p.info = up(static_cast<size_t>(2) * kSpanMaxCtas * span_part(v.dim) * 4);
    p.redo = p.info + up(2 * kSpanMaxCtas * sizeof(SpanInfo));
    p.pre = p.redo + up(rows);
    p.own = p.pre + (prefix ? up(rows * span_row(v.dim) * 4) : 0);
    p.total = p.own + (p.own - p.pre);
    return p;
}

void place_span(SpanArgs *a, const SpanPlan &p, void *workspace)
{
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a->part = reinterpret_cast<float *>(ws);
    a->part_stride = span_part(a->kv.dim);
    a->info = reinterpret_cast<SpanInfo *>(ws + p.info);
    a->redo = ws + p.redo;
}

// Stores of how many 16 bytes at once an output's rows take.
int out_vec(const gemv_heads_t &h)
{
    if (!aligned(h.data, 16) || !mult8(h.stride, 2)) return 0;
    return aligned(h.data, 32) && h.stride[0] % 16 == 0 && h.stride[1] % 16 == 0 ? 2 : 1;
}

// Rows that the kernels' 32-bit counts can hold: they are rounded up to blocks of
// at most 256, and the row behind the last block is formed too.
bool too_many_rows(int64_t tokens, int q_heads) { return tokens > INT_MAX / 64 || tokens * q_heads > INT_MAX - 1024; }

// prefix: the slots before *prefix are attended to by a launch of their own, whose
// results stand behind the workspace of the others.
gemv_status_t attn_paged(const gemv_kv_t *kv, const gemv_attn_t *args, const int32_t *prefix, int sinks, void *stream)
{
    AttnArgs a{};
    gemv_status_t st = view_of(kv, &a.kv);
    if (st != GEMV_OK) return st;
    if (!args) return GEMV_ERR_INVALID_VALUE;
    const gemv_heads_t &q = args->q, &out = args->out;
    const int q_heads = args->q_heads;
    if (q_heads < 1 || q_heads % a.kv.kv_heads || args->window < 0 || sinks < 0 || negative(q) || negative(out))
        return GEMV_ERR_INVALID_VALUE;
    if (too_many_heads(q_heads, a.kv.dim)) return GEMV_ERR_UNSUPPORTED;
    if (a.kv.batch == 0) return GEMV_OK;
    if (!q.data || !args->lengths || !out.data || !args->workspace || (args->scores_out && !kv->scores))
        return GEMV_ERR_INVALID_VALUE;
    if (!aligned(q.data, 2) || !aligned(out.data, 2) || !aligned(args->lengths, 4) || !aligned(args->lse, 4) ||
        !aligned(args->scores_out, 4) || !aligned(args->workspace, 256))
        return GEMV_ERR_MISALIGNED;
    const int group = q_heads / a.kv.kv_heads;
    const bool vec = cache_vec(kv) && aligned(q.data, 16) && mult8(q.stride, 2);
    const int nt = head_tile(a.kv.dim, group, vec);
    const AttnPlan p = attn_plan(a.kv, group, nt, args->scores_out != nullptr);
    if (p.rows > INT_MAX || (prefix && too_many_rows(a.kv.batch, q_heads))) return GEMV_ERR_UNSUPPORTED;
    const size_t total = prefix ? gemv_attn_shared_workspace(kv, q_heads) : p.total;
    if (args->workspace_bytes < total || total == 0) return GEMV_ERR_INVALID_VALUE;
    DecodeDevice dev;
    if (!decode_device(&dev)) return GEMV_ERR_CUDA;
    a.q = q.data;
    a.q_sb = q.stride[0];
    a.q_sh = q.stride[1];
    a.out = out.data;
    a.o_sb = out.stride[0];
    a.o_sh = out.stride[1];
    a.lengths = args->lengths;
    a.lse = args->lse;
    a.scores_in = kv->scores;
    a.scores_out = args->scores_out;
    a.q_heads = q_heads;
    a.group = group;
    a.head_tiles = p.head_tiles;
    a.window = args->window;
    a.sinks = sinks;
    a.scale_log2 = args->scale * 1.4426950408889634f;
    a.err = dev.status;
    unsigned char *ws = static_cast<unsigned char *>(args->workspace);
    a.arrived = reinterpret_cast<uint64_t *>(ws);
    a.part = reinterpret_cast<float *>(ws + p.part);
    a.part_stride = p.part_stride;
    a.row_lse = reinterpret_cast<float *>(ws + p.row_lse);
    a.logits = reinterpret_cast<float *>(ws + p.logits);
    a.logit_heads = p.logit_heads;
    // Few rows: one block of all an SM's warps, a third of the parts to join
    // (8 rows of 131001 tokens of 128: 88.4 us, with blocks of four warps 94.1).
    // Many rows: blocks of four warps, one joins while the others load (384
    // rows of 1000 tokens: 39.8 us against 48.2).
    const bool big = vec && p.rows <= dev.sm_count / 2;
    // A row's beginning counts like `lead` tiles (48 ragged sequences of up to 6000
    // tokens with their weights: 111.5 us, 120.4 us with none).
    a.lead = big ? 16 : 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    SpanArgs g{};
    if (prefix) {
        const SpanPlan sp = span_plan(a.kv, a.kv.batch, q_heads, true);
        unsigned char *mine = ws + (total - sp.total);
        g.kv = a.kv;
        place_span(&g, sp, mine);
        g.q = a.q, g.q_st = a.q_sb, g.q_sh = a.q_sh;
        g.out = a.out, g.o_st = a.o_sb, g.o_sh = a.o_sh;
        g.out_vec = out_vec(out);
        g.lse = a.lse;
        g.pre = reinterpret_cast<float *>(mine + sp.pre);
        g.own = a.own = reinterpret_cast<float *>(mine + sp.own);
        g.lengths = a.lengths;
        g.prefix = a.prefix = prefix;
        g.tokens = a.kv.batch;
        g.q_heads = q_heads;
        g.group = group;
        g.window = args->window;
        g.sinks = sinks;
        g.scale_log2 = a.scale_log2;
        g.err = a.err;
        g.wait_limit_ns = dev.wait_limit_ns;
        g.skip_tile = (dev.skip_copies & SKIP_TILE) != 0;
        const cudaError_t e = launch_span(g, vec, kv->elem, dev.sm_count, s);
        if (e != cudaSuccess) return decode_cuda_fail(e, GEMV_ERR_LAUNCH);
    }
    const bool f16 = kv->elem == GEMV_ELEM_F16;
    const auto attend = prefix                         ? f16 ? launch_attn_own_f16 : launch_attn_own_bf16
                        : a.sinks > 0 && a.window > 0 ? f16 ? launch_attn_sinks_f16 : launch_attn_sinks_bf16
                        : f16                          ? launch_attn_f16
                                                       : launch_attn_bf16;
    cudaError_t e = attend(a, vec, nt, big, dev.sm_count, s);
    if (e == cudaSuccess && a.scores_out && a.kv.capacity > 0) e = launch_attn_weights(a, nt, s);
    if (e == cudaSuccess && prefix) e = launch_span_finish(g, kv->elem, dev.sm_count, s);
    return e == cudaSuccess ? GEMV_OK : decode_cuda_fail(e, GEMV_ERR_LAUNCH);
}

gemv_status_t rope_append(const gemv_kv_t *kv, const gemv_rope_t *r, const gemv_head_norm_t *norm, void *stream)
{
    RopeArgs a{};
    const gemv_status_t st = view_of(kv, &a.kv);
    if (st != GEMV_OK) return st;
    if (!r || !is_elem(r->src_elem) || r->tokens < 0 || r->q_heads < 0 || r->axes < 1 || r->rot < 0 || r->rot % 2 ||
        r->rot > a.kv.dim || r->pos_stride < 0)
        return GEMV_ERR_INVALID_VALUE;
    if (negative(r->q) || negative(r->k) || negative(r->v) || negative(r->q_out)) return GEMV_ERR_INVALID_VALUE;
    if (!r->seq && r->tokens > a.kv.batch) return GEMV_ERR_INVALID_VALUE;
    if (norm && ((norm->q_weight && !is_elem(norm->q_elem)) || (norm->k_weight && !is_elem(norm->k_elem))))
        return GEMV_ERR_INVALID_VALUE;
    // a block looks up to 64 steps of the grid ahead, in 32 bits
    if (r->tokens > INT_MAX - (1 << 20) || too_many_heads(r->q_heads, a.kv.dim)) return GEMV_ERR_UNSUPPORTED;
    if (r->tokens == 0) return GEMV_OK;
    if ((r->q_heads > 0 && (!r->q.data || !r->q_out.data)) || !r->k.data || !r->v.data || !r->positions || !r->slots ||
        (r->rot > 0 && (!r->turns || !r->axis)) || !kv->k || !kv->v)
        return GEMV_ERR_INVALID_VALUE;
    const int eb = elem_bytes(r->src_elem);
    if (!aligned(r->q.data, eb) || !aligned(r->k.data, eb) || !aligned(r->v.data, eb) || !aligned(r->q_out.data, 2) ||
        !aligned(r->positions, 4) || !aligned(r->slots, 4) || !aligned(r->seq, 4) || !aligned(r->stamps, 4) ||
        !aligned(r->turns, 8))
        return GEMV_ERR_MISALIGNED;
    if (norm && ((norm->q_weight && !aligned(norm->q_weight, elem_bytes(norm->q_elem))) ||
                 (norm->k_weight && !aligned(norm->k_weight, elem_bytes(norm->k_elem)))))
        return GEMV_ERR_MISALIGNED;
    DecodeDevice dev;
    if (!decode_device(&dev)) return GEMV_ERR_CUDA;
    if (norm) {
        a.norm = 1;
        a.unit_offset = norm->unit_offset != 0;
        a.q_weight = norm->q_weight, a.q_weight_e = norm->q_elem;
        a.k_weight = norm->k_weight, a.k_weight_e = norm->k_elem;
        a.eps = norm->eps;
    }
    a.q = r->q.data, a.q_st = r->q.stride[0], a.q_sh = r->q.stride[1];
    a.k = r->k.data, a.k_st = r->k.stride[0], a.k_sh = r->k.stride[1];
    a.v = r->v.data, a.v_st = r->v.stride[0], a.v_sh = r->v.stride[1];
    a.q_out = r->q_out.data, a.qo_st = r->q_out.stride[0], a.qo_sh = r->q_out.stride[1];
    a.src_elem = r->src_elem;
    a.dst_elem = kv->elem;
    a.positions = r->positions;
    a.pos_stride = r->pos_stride;
    a.slots = r->slots;
    a.seq = r->seq;
    a.stamps = r->stamps;
    a.scores_cache = kv->scores;
    a.stamps_cache = kv->stamps;
    a.turns = r->turns;
    a.axis = r->axis;
    a.tokens = r->tokens;
    a.q_heads = r->q_heads;
    a.rot = r->rot;
    a.axes = r->axes;
    a.pairs = r->pairs != 0;
    a.err = dev.status;
    bool vec = cache_vec(kv) && r->rot % 16 == 0;
    for (const gemv_heads_t *h : {&r->q, &r->k, &r->v, &r->q_out})
        vec = vec && aligned(h->data, h == &r->q_out ? 16 : vec_bytes(r->src_elem)) && mult8(h->stride, 2);
    const cudaError_t e = launch_rope(a, vec, dev.sm_count, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMV_OK : decode_cuda_fail(e, GEMV_ERR_LAUNCH);
}

}  // namespace
}  // namespace mbg

using namespace mbg;

extern "C" {

size_t gemv_attn_paged_workspace(const gemv_kv_t *kv, int q_heads, int weights)
{
    KvView v;
    if (view_of(kv, &v, false) != GEMV_OK || q_heads < 1 || q_heads % v.kv_heads || too_many_heads(q_heads, v.dim))
        return 0;
    const int group = q_heads / v.kv_heads;
    const AttnPlan a = attn_plan(v, group, 1, weights != 0);
    if (v.dim > 128 || group <= 8) return a.total;
    const AttnPlan b = attn_plan(v, group, 2, weights != 0);
    return a.total > b.total ? a.total : b.total;
}

uint64_t gemv_capture_id(void *stream)
{
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, &id) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return status == cudaStreamCaptureStatusActive ? id : 0;
}

gemv_status_t gemv_attn_paged(const gemv_kv_t *kv, const gemv_attn_t *args, void *stream)
{
    return gemv_attn_paged_sinks(kv, args, 0, stream);
}

gemv_status_t gemv_attn_paged_sinks(const gemv_kv_t *kv, const gemv_attn_t *args, int sinks, void *stream)
{
    return attn_paged(kv, args, nullptr, sinks, stream);
}

size_t gemv_attn_shared_workspace(const gemv_kv_t *kv, int q_heads)
{
    const size_t own = gemv_attn_paged_workspace(kv, q_heads, 0);
    KvView v;
    if (own == 0 || view_of(kv, &v, false) != GEMV_OK || too_many_rows(v.batch, q_heads)) return 0;
    return own + span_plan(v, v.batch, q_heads, true).total;
}

gemv_status_t gemv_attn_shared(const gemv_kv_t *kv, const gemv_attn_t *args, const int32_t *prefix, int sinks, void *stream)
{
    if (!args || !prefix || args->scores_out) return GEMV_ERR_INVALID_VALUE;
    if (!aligned(prefix, 4)) return GEMV_ERR_MISALIGNED;
    return attn_paged(kv, args, prefix, sinks, stream);
}

size_t gemv_attn_prompt_workspace(const gemv_kv_t *kv, int64_t tokens, int q_heads)
{
    KvView v;
    if (view_of(kv, &v, false) != GEMV_OK || q_heads < 1 || q_heads % v.kv_heads || too_many_heads(q_heads, v.dim) ||
        tokens < 0 || too_many_rows(tokens, q_heads))
        return 0;
    return span_plan(v, tokens, q_heads, false).total;
}

gemv_status_t gemv_attn_prompt(const gemv_kv_t *kv, const gemv_prompt_t *g, void *stream)
{
    SpanArgs a{};
    const gemv_status_t st = view_of(kv, &a.kv);
    if (st != GEMV_OK) return st;
    if (!g || g->q_heads < 1 || g->q_heads % a.kv.kv_heads || g->tokens < 0 || g->window < 0 || g->sinks < 0 ||
        negative(g->q) || negative(g->out))
        return GEMV_ERR_INVALID_VALUE;
    if (too_many_heads(g->q_heads, a.kv.dim) || too_many_rows(g->tokens, g->q_heads)) return GEMV_ERR_UNSUPPORTED;
    if (a.kv.batch == 0 || g->tokens == 0) return GEMV_OK;
    if (!g->q.data || !g->out.data || !g->starts || !g->lengths || !g->workspace) return GEMV_ERR_INVALID_VALUE;
    if (!aligned(g->q.data, 2) || !aligned(g->out.data, 2) || !aligned(g->starts, 4) || !aligned(g->lengths, 4) ||
        !aligned(g->lse, 4) || !aligned(g->workspace, 256))
        return GEMV_ERR_MISALIGNED;
    const SpanPlan p = span_plan(a.kv, g->tokens, g->q_heads, false);
    if (g->workspace_bytes < p.total) return GEMV_ERR_INVALID_VALUE;
    DecodeDevice dev;
    if (!decode_device(&dev)) return GEMV_ERR_CUDA;
    a.q = g->q.data, a.q_st = g->q.stride[0], a.q_sh = g->q.stride[1];
    a.out = g->out.data, a.o_st = g->out.stride[0], a.o_sh = g->out.stride[1];
    a.lse = g->lse;
    a.starts = g->starts;
    a.lengths = g->lengths;
    a.tokens = static_cast<int>(g->tokens);
    a.q_heads = g->q_heads;
    a.group = g->q_heads / a.kv.kv_heads;
    a.window = g->window;
    a.sinks = g->sinks;
    a.scale_log2 = g->scale * 1.4426950408889634f;
    a.err = dev.status;
    a.out_vec = out_vec(g->out);
    a.wait_limit_ns = dev.wait_limit_ns;
    a.skip_tile = (dev.skip_copies & SKIP_TILE) != 0;
    place_span(&a, p, g->workspace);
    const bool vec = cache_vec(kv) && aligned(g->q.data, 16) && mult8(g->q.stride, 2);
    cudaError_t e = launch_span(a, vec, kv->elem, dev.sm_count, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = launch_span_finish(a, kv->elem, dev.sm_count, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMV_OK : decode_cuda_fail(e, GEMV_ERR_LAUNCH);
}

gemv_status_t gemv_kv_evict_plan(const gemv_kv_t *kv, const int32_t *lengths, int keep, int sinks, int recent,
                                 int32_t *moves, int64_t max_moves, int32_t *counts, void *stream)
{
    EvictArgs a{};
    const gemv_status_t st = view_of(kv, &a.kv);
    if (st != GEMV_OK) return st;
    if (keep < 1 || sinks < 0 || recent < 0 || max_moves < 0) return GEMV_ERR_INVALID_VALUE;
    const int64_t behind = a.kv.capacity - keep;
    if (behind > 0 && max_moves < (keep < behind ? keep : behind)) return GEMV_ERR_INVALID_VALUE;
    if (a.kv.batch == 0) return GEMV_OK;
    if (!lengths || !counts || !kv->scores || !kv->stamps || (max_moves > 0 && !moves)) return GEMV_ERR_INVALID_VALUE;
    if (!aligned(lengths, 4) || !aligned(counts, 4) || !aligned(moves, 8)) return GEMV_ERR_MISALIGNED;
    DecodeDevice dev;
    if (!decode_device(&dev)) return GEMV_ERR_CUDA;
    a.scores = kv->scores;
    a.stamps = kv->stamps;
    a.lengths = lengths;
    a.keep = keep;
    a.sinks = sinks;
    a.recent = recent;
    a.moves = moves;
    a.max_moves = max_moves;
    a.counts = counts;
    a.err = dev.status;
    const cudaError_t e = launch_evict_plan(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMV_OK : decode_cuda_fail(e, GEMV_ERR_LAUNCH);
}

gemv_status_t gemv_kv_evict_apply(const gemv_kv_t *kv, const int32_t *moves, int64_t max_moves, const int32_t *counts,
                                  int32_t *lengths, int keep, void *stream)
{
    EvictApplyArgs a{};
    const gemv_status_t st = view_of(kv, &a.kv);
    if (st != GEMV_OK) return st;
    if (keep < 1 || max_moves < 0) return GEMV_ERR_INVALID_VALUE;
    if (a.kv.batch == 0) return GEMV_OK;
    if (!counts || (max_moves > 0 && !moves)) return GEMV_ERR_INVALID_VALUE;
    if (!aligned(lengths, 4) || !aligned(counts, 4) || !aligned(moves, 8)) return GEMV_ERR_MISALIGNED;
    DecodeDevice dev;
    if (!decode_device(&dev)) return GEMV_ERR_CUDA;
    a.scores = kv->scores;
    a.stamps = kv->stamps;
    a.lengths = lengths;
    a.keep = keep;
    a.moves = moves;
    a.max_moves = max_moves;
    a.counts = counts;
    a.err = dev.status;
    const cudaError_t e = launch_evict_apply(a, cache_vec(kv), dev.sm_count, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMV_OK : decode_cuda_fail(e, GEMV_ERR_LAUNCH);
}

gemv_status_t gemv_rope_append(const gemv_kv_t *kv, const gemv_rope_t *r, void *stream)
{
    return rope_append(kv, r, nullptr, stream);
}

gemv_status_t gemv_rope_append_norm(const gemv_kv_t *kv, const gemv_rope_t *r, const gemv_head_norm_t *norm, void *stream)
{
    if (!norm) return GEMV_ERR_INVALID_VALUE;
    return rope_append(kv, r, norm, stream);
}

gemv_status_t gemv_kv_assign(const gemv_kv_t *kv, const gemv_assign_t *g, void *stream)
{
    KvView v;
    // the pools are not touched: they may be missing, not so the table
    const gemv_status_t st = view_of(kv, &v, false);
    if (st != GEMV_OK) return st;
    if (!g || g->room < 0 || g->ring_size < 0) return GEMV_ERR_INVALID_VALUE;
    if (g->room > INT_MAX - (1 << 20) || g->ring_size > INT_MAX) return GEMV_ERR_UNSUPPORTED;
    if (!g->state || !g->state_out || !g->starts || (g->ring_size > 0 && !g->ring) || (g->room > 0 && (!g->slots || !g->seq)) ||
        (v.batch > 0 && (!g->lengths || !g->lengths_out || !g->fresh || (v.max_pages > 0 && !v.table))))
        return GEMV_ERR_INVALID_VALUE;
    if (v.batch > 1 && v.table_stride < v.max_pages) return GEMV_ERR_INVALID_VALUE;  // rows that are written must not lie on one another
    for (const void *p : {static_cast<const void *>(v.table), static_cast<const void *>(g->ring), static_cast<const void *>(g->state),
                          static_cast<const void *>(g->state_out), static_cast<const void *>(g->starts),
                          static_cast<const void *>(g->slots), static_cast<const void *>(g->seq),
                          static_cast<const void *>(g->lengths), static_cast<const void *>(g->lengths_out),
                          static_cast<const void *>(g->fresh), static_cast<const void *>(g->shared)})
        if (!aligned(p, 4)) return GEMV_ERR_MISALIGNED;
    DecodeDevice dev;
    if (!decode_device(&dev)) return GEMV_ERR_CUDA;
    AssignArgs a{};
    a.table = const_cast<int32_t *>(v.table);
    a.table_stride = v.table_stride;
    a.capacity = v.capacity;
    a.num_pages = v.num_pages;
    a.batch = v.batch;
    a.page_size = v.page_size;
    a.lengths = g->lengths;
    a.fresh = g->fresh;
    a.shared = g->shared;
    a.lengths_out = g->lengths_out;
    a.ring = g->ring;
    a.ring_size = g->ring_size;
    a.state = g->state;
    a.state_out = g->state_out;
    a.starts = g->starts;
    a.slots = g->slots;
    a.seq = g->seq;
    a.room = g->room;
    a.wide = aligned(g->slots, 16) && aligned(g->seq, 16);
    a.err = dev.status;
    const cudaError_t e = launch_assign(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMV_OK : decode_cuda_fail(e, GEMV_ERR_LAUNCH);
}

gemv_status_t gemv_norm_residual(const gemv_norm_t *n, void *stream)
{
    if (!n || n->rows < 0 || n->width < 0 || (n->flags & ~7u)) return GEMV_ERR_INVALID_VALUE;
    const gemv_rows_t *all[8] = {&n->y, &n->x, &n->gate, &n->post_weight, &n->pre_weight, &n->pre_bias, &n->out, &n->h};
    for (const gemv_rows_t *r : all)
        if (r->data && (!is_elem(r->elem) || r->row_stride < 0)) return GEMV_ERR_INVALID_VALUE;
    if (n->rows == 0 || n->width == 0) return GEMV_OK;
    if (!n->y.data || !n->x.data || !n->out.data || n->out.elem != n->x.elem) return GEMV_ERR_INVALID_VALUE;
    if (n->width > (1 << 24) || n->rows >= (1 << 28)) return GEMV_ERR_UNSUPPORTED;
    // rows that are written must not lie on one another
    if (n->rows > 1 && (n->out.row_stride < n->width || (n->h.data && n->h.row_stride < n->width)))
        return GEMV_ERR_INVALID_VALUE;
    bool vec = n->width % 8 == 0;
    for (const gemv_rows_t *r : all) {
        if (!r->data) continue;
        if (!aligned(r->data, elem_bytes(r->elem))) return GEMV_ERR_MISALIGNED;
        if (!aligned(r->data, vec_bytes(r->elem)) || r->row_stride % 8) vec = false;
    }
    NormArgs a{};
    a.y = n->y.data, a.y_e = n->y.elem, a.y_s = n->y.row_stride;
    a.r = n->x.data, a.r_e = n->x.elem, a.r_s = n->x.row_stride;
    a.gate = n->gate.data, a.gate_e = n->gate.elem, a.gate_s = n->gate.row_stride;
    a.post_w = n->post_weight.data, a.post_e = n->post_weight.elem, a.post_s = n->post_weight.row_stride;
    a.pre_w = n->pre_weight.data, a.pre_w_e = n->pre_weight.elem, a.pre_w_s = n->pre_weight.row_stride;
    a.pre_b = n->pre_bias.data, a.pre_b_e = n->pre_bias.elem, a.pre_b_s = n->pre_bias.row_stride;
    a.out = n->out.data, a.out_s = n->out.row_stride;
    a.h = n->h.data, a.h_e = n->h.elem, a.h_s = n->h.row_stride;
    a.rows = n->rows;
    a.width = static_cast<int>(n->width);
    a.layer = (n->flags & GEMV_NORM_LAYER) != 0;
    a.post = (n->flags & GEMV_NORM_POST) != 0;
    a.unit_offset = (n->flags & GEMV_NORM_UNIT_OFFSET) != 0;
    a.alpha = n->alpha;
    a.eps = n->eps;
    DecodeDevice dev;
    if (!decode_device(&dev)) return GEMV_ERR_CUDA;
    const cudaError_t e = launch_norm(a, vec, dev.sm_count, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMV_OK : decode_cuda_fail(e, GEMV_ERR_LAUNCH);
}

}  // extern "C"
