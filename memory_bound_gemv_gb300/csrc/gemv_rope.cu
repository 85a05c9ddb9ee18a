// Rotary positions with several axes, and the append to the paged cache.
//
// Pair i of a head is turned by the angle pos[axis(i)] * f_i.  A position can
// be millions of turns' worth of radians, where FP32 (and the argument of
// FP32 sine) has lost the angle.  The table therefore holds f_i / (2 pi) as a
// 64-bit fixed-point fraction of a turn: pos * turns mod 2^64 is the exact
// fraction of a turn left over (integer products wrap as angles do), off by
// at most |pos| * 2^-65 turns from the table's rounding.  Its upper 32 bits
// go to sincospif.
//
// Bound by the bytes of q, k and v read and written once.  A block takes one
// token and some of its heads.  Each thread requests its first heads' part,
// the block computes the token's sines and cosines into shared memory while
// those are under way, then they are turned and written.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"
#include "gemv_elem.cuh"

namespace mbg {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxPairs = 128;

// A head is cut into units of 16 elements: two runs of eight, at d0 and d1, of
// which n0 and n1 exist.  Turned units are eight pairs (style "halves":
// elements i..i+7 and those rot / 2 behind them; "pairs": 16 consecutive
// ones); the others are copied.
struct Unit {
    int d0, d1, n0, n1;
    bool turned;
    __device__ __forceinline__ Unit(const RopeArgs &a, int u, bool is_v)
    {
        const int half = a.rot >> 1, dim = a.kv.dim, turn_units = (half + 7) >> 3;
        turned = !is_v && u < turn_units;
        if (!turned) {
            d0 = is_v ? u * 16 : a.rot + (u - turn_units) * 16;
            d1 = d0 + 8;
            n0 = min(8, dim - d0);
            n1 = min(8, dim - d1);
        } else if (a.pairs) {
            d0 = u * 16;
            d1 = d0 + 8;
            n0 = min(8, a.rot - d0);
            n1 = min(8, a.rot - d1);
        } else {
            d0 = u * 8;
            d1 = half + d0;
            n0 = n1 = min(8, half - d0);
        }
    }
};

// blockDim.x = units per head x heads that are worked on side by side.  A
// thread keeps to one unit, so its sines and cosines stay in registers while
// it goes through the heads, HEADS of them requested at once.
template <bool VEC, int SRC, int DST, int HEADS>
__global__ void __launch_bounds__(kMaxThreads)
    mbg_rope_kernel(const __grid_constant__ RopeArgs a, int heads_per_block, int per_head)
{
    __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
    pdl_trigger();
    pdl_wait();
    const KvView &kv = a.kv;
    const int t = blockIdx.x, threads = blockDim.x;
    const int half = a.rot >> 1;
    const int side = threads / per_head, lane_head = threadIdx.x / per_head, u = threadIdx.x - lane_head * per_head;
    const int head0 = blockIdx.y * heads_per_block;
    const int head1 = min(head0 + heads_per_block, a.q_heads + 2 * kv.kv_heads);
    const int first_v = a.q_heads + kv.kv_heads;
    const Unit uqk(a, u, false), uv(a, u, true);
    float x[HEADS][8], y[HEADS][8];
    auto request = [&](int h0) {
#pragma unroll
        for (int k = 0; k < HEADS; ++k) {
            const int head = h0 + k * side;
            if (head >= head1) continue;
            const bool is_v = head >= first_v;
            const void *src = head < a.q_heads ? a.q : is_v ? a.v : a.k;
            const int h = head < a.q_heads ? head : is_v ? head - first_v : head - a.q_heads;
            const int64_t st = head < a.q_heads ? a.q_st : is_v ? a.v_st : a.k_st;
            const int64_t sh = head < a.q_heads ? a.q_sh : is_v ? a.v_sh : a.k_sh;
            const int64_t at = t * st + h * sh;
            elem_load8<VEC, SRC>(src, at + (is_v ? uv.d0 : uqk.d0), is_v ? uv.n0 : uqk.n0, x[k]);
            elem_load8<VEC, SRC>(src, at + (is_v ? uv.d1 : uqk.d1), is_v ? uv.n1 : uqk.n1, y[k]);
        }
    };
    int head = head0 + lane_head;
    if (lane_head >= side) head = head1;  // threads beyond the last whole head
    request(head);
    // where the token goes
    const int seq = a.seq ? __ldg(a.seq + t) : t;
    const int slot = __ldg(a.slots + t);
    int64_t page = -1;
    int off = 0;
    if (slot >= 0) {  // a negative slot is padding: nothing is written
        bool ok = seq >= 0 && seq < kv.batch && slot < kv.capacity;
        if (ok) {
            const int idx = kv.page_shift >= 0 ? slot >> kv.page_shift : slot / kv.page_size;
            off = slot - idx * kv.page_size;
            page = __ldg(kv.table + seq * kv.table_stride + idx);
            ok = page >= 0 && page < kv.num_pages;
        }
        if (!ok) {
            page = -1;
            if (threadIdx.x == 0) report_error(a.err, DEVERR_BAD_INDEX);
        }
    }
    for (int i = threadIdx.x; i < half; i += threads) {
        int ax = __ldg(a.axis + i);
        if (ax >= a.axes) {
            if (t == 0) report_error(a.err, DEVERR_BAD_INDEX);
            ax = 0;
        }
        const int pos = __ldg(a.positions + ax * a.pos_stride + t);
        const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * __ldg(a.turns + i);
        // the nearest 2^-32 turns, as half turns in [-1, 1)
        const int32_t part = static_cast<int32_t>((turn + 0x80000000ull) >> 32);
        float sn, cs;
        sincospif(static_cast<float>(part) * 4.656612873077393e-10f, &sn, &cs);
        s_cos[i] = cs;
        s_sin[i] = sn;
    }
    if (blockIdx.y == 0 && page >= 0) {
        for (int h = threadIdx.x; h < kv.kv_heads; h += threads) {
            const int64_t at = (static_cast<int64_t>(seq) * kv.kv_heads + h) * kv.capacity + slot;
            if (a.scores_cache) a.scores_cache[at] = 0.f;
            if (a.stamps_cache) a.stamps_cache[at] = a.stamps ? __ldg(a.stamps + t) : slot;
        }
    }
    __syncthreads();
    float c[8], s[8];
    if (uqk.turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // pairs past the last turn elements that do not exist
            const int i = min(u * 8 + e, half - 1);
            c[e] = s_cos[VEC ? u * 8 + e : i];
            s[e] = s_sin[VEC ? u * 8 + e : i];
        }
    }
    for (; head < head1;) {
#pragma unroll
        for (int k = 0; k < HEADS; ++k) {
            const int hd = head + k * side;
            const bool is_v = hd >= first_v;
            if (hd >= head1 || (hd >= a.q_heads && page < 0)) continue;
            if (uqk.turned && !is_v) {
                if (a.pairs) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = x[k][2 * e], q = x[k][2 * e + 1], v = y[k][2 * e], w = y[k][2 * e + 1];
                        x[k][2 * e] = p * c[e] - q * s[e];
                        x[k][2 * e + 1] = p * s[e] + q * c[e];
                        y[k][2 * e] = v * c[e + 4] - w * s[e + 4];
                        y[k][2 * e + 1] = v * s[e + 4] + w * c[e + 4];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float p = x[k][e], q = y[k][e];
                        x[k][e] = p * c[e] - q * s[e];
                        y[k][e] = p * s[e] + q * c[e];
                    }
                }
            }
            uint16_t *dst;
            if (hd < a.q_heads)
                dst = static_cast<uint16_t *>(a.q_out) + t * a.qo_st + hd * a.qo_sh;
            else if (!is_v)
                dst = static_cast<uint16_t *>(kv.k) + page * kv.ks_page + off * kv.ks_tok + (hd - a.q_heads) * kv.ks_head;
            else
                dst = static_cast<uint16_t *>(kv.v) + page * kv.vs_page + off * kv.vs_tok + (hd - first_v) * kv.vs_head;
            elem_store8<VEC, DST>(dst, is_v ? uv.d0 : uqk.d0, is_v ? uv.n0 : uqk.n0, x[k]);
            elem_store8<VEC, DST>(dst, is_v ? uv.d1 : uqk.d1, is_v ? uv.n1 : uqk.n1, y[k]);
        }
        head += HEADS * side;
        request(head);
    }
}

template <bool VEC, int SRC, int DST, int HEADS>
cudaError_t launch_heads(const RopeArgs &a, dim3 grid, int threads, int per, int per_head, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mbg_rope_kernel<VEC, SRC, DST, HEADS>, a, per, per_head);
}

template <bool VEC, int SRC, int DST>
cudaError_t launch(const RopeArgs &a, int sm_count, cudaStream_t s)
{
    // few tokens: spread the heads of one over several blocks, so that the
    // call is as long as one block's few loads
    const int heads = a.q_heads + 2 * a.kv.kv_heads;
    int per = heads;
    while (per > 4 && static_cast<int64_t>(a.tokens) * ((heads + per - 1) / per) < sm_count) per = (per + 1) / 2;
    const int half = a.rot / 2;
    const int units = (half + 7) / 8 + (a.kv.dim - a.rot + 15) / 16, v_units = (a.kv.dim + 15) / 16;
    const int per_head = units > v_units ? units : v_units;
    const dim3 grid(static_cast<unsigned>(a.tokens), static_cast<unsigned>((heads + per - 1) / per));
    // many heads per block: each thread takes three or more, three requested
    // at once
    const bool deep = VEC && per >= 12;
    int side = deep ? (per + 2) / 3 : per;
    while (side > 1 && side * per_head > (deep ? 192 : kMaxThreads)) side = (side + 1) / 2;
    const int threads = (side * per_head + 31) / 32 * 32;
    if (deep) return launch_heads<VEC, SRC, DST, VEC ? 3 : 1>(a, grid, threads, per, per_head, s);
    return launch_heads<VEC, SRC, DST, 1>(a, grid, threads, per, per_head, s);
}

template <int SRC, int DST>
cudaError_t pick(const RopeArgs &a, bool vec, int sm_count, cudaStream_t s)
{
    return vec ? launch<true, SRC, DST>(a, sm_count, s) : launch<false, SRC, DST>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool vec, int sm_count, cudaStream_t s)
{
    if (a.dst_elem == GEMV_ELEM_F16) {
        if (a.src_elem == GEMV_ELEM_F32) return pick<GEMV_ELEM_F32, GEMV_ELEM_F16>(a, vec, sm_count, s);
        if (a.src_elem == GEMV_ELEM_F16) return pick<GEMV_ELEM_F16, GEMV_ELEM_F16>(a, vec, sm_count, s);
        return pick<GEMV_ELEM_BF16, GEMV_ELEM_F16>(a, vec, sm_count, s);
    }
    if (a.src_elem == GEMV_ELEM_F32) return pick<GEMV_ELEM_F32, GEMV_ELEM_BF16>(a, vec, sm_count, s);
    if (a.src_elem == GEMV_ELEM_F16) return pick<GEMV_ELEM_F16, GEMV_ELEM_BF16>(a, vec, sm_count, s);
    return pick<GEMV_ELEM_BF16, GEMV_ELEM_BF16>(a, vec, sm_count, s);
}

}  // namespace mbg
