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
    AttnArgs a{};
    gemv_status_t st = view_of(kv, &a.kv);
    if (st != GEMV_OK) return st;
    if (!args) return GEMV_ERR_INVALID_VALUE;
    const gemv_heads_t &q = args->q, &out = args->out;
    const int q_heads = args->q_heads;
    if (q_heads < 1 || q_heads % a.kv.kv_heads || args->window < 0 || negative(q) || negative(out))
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
    if (p.rows > INT_MAX) return GEMV_ERR_UNSUPPORTED;
    if (args->workspace_bytes < p.total) return GEMV_ERR_INVALID_VALUE;
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
    cudaError_t e = kv->elem == GEMV_ELEM_F16 ? launch_attn_f16(a, vec, nt, big, dev.sm_count, s)
                                              : launch_attn_bf16(a, vec, nt, big, dev.sm_count, s);
    if (e == cudaSuccess && a.scores_out && a.kv.capacity > 0) e = launch_attn_weights(a, nt, s);
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
    RopeArgs a{};
    const gemv_status_t st = view_of(kv, &a.kv);
    if (st != GEMV_OK) return st;
    if (!r || !is_elem(r->src_elem) || r->tokens < 0 || r->q_heads < 0 || r->axes < 1 || r->rot < 0 || r->rot % 2 ||
        r->rot > a.kv.dim || r->pos_stride < 0)
        return GEMV_ERR_INVALID_VALUE;
    if (negative(r->q) || negative(r->k) || negative(r->v) || negative(r->q_out)) return GEMV_ERR_INVALID_VALUE;
    if (!r->seq && r->tokens > a.kv.batch) return GEMV_ERR_INVALID_VALUE;
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
    DecodeDevice dev;
    if (!decode_device(&dev)) return GEMV_ERR_CUDA;
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
