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
// token and some of its heads: it computes the token's sines and cosines once
// into shared memory, then every thread turns eight pairs of a head at a
// time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"
#include "gemv_elem.cuh"

namespace mbg {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

template <bool VEC, int SRC, int DST>
__global__ void __launch_bounds__(kThreads) mbg_rope_kernel(const __grid_constant__ RopeArgs a, int heads_per_block)
{
    __shared__ float s_cos[kMaxPairs], s_sin[kMaxPairs];
    pdl_trigger();
    pdl_wait();
    const KvView &kv = a.kv;
    const int t = blockIdx.x;
    const int half = a.rot >> 1, dim = kv.dim;
    for (int i = threadIdx.x; i < half; i += kThreads) {
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
    // where the token goes
    int seq = a.seq ? __ldg(a.seq + t) : t;
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
    if (blockIdx.y == 0 && page >= 0) {
        for (int h = threadIdx.x; h < kv.kv_heads; h += kThreads) {
            const int64_t at = (static_cast<int64_t>(seq) * kv.kv_heads + h) * kv.capacity + slot;
            if (a.scores_cache) a.scores_cache[at] = 0.f;
            if (a.stamps_cache) a.stamps_cache[at] = a.stamps ? __ldg(a.stamps + t) : slot;
        }
    }
    __syncthreads();
    // a head is cut into units of 16 elements: eight pairs, or 16 elements
    // that are not turned.  (Style "halves": elements i..i+7 and those rot / 2
    // behind them; style "pairs": 16 consecutive ones.)
    const int turn_units = (half + 7) >> 3, rest_units = (dim - a.rot + 15) >> 4;
    const int units = turn_units + rest_units, v_units = (dim + 15) >> 4;
    const int head0 = blockIdx.y * heads_per_block;
    const int head1 = min(head0 + heads_per_block, a.q_heads + 2 * kv.kv_heads);
    const int per_head = max(units, v_units);
    for (int w = threadIdx.x; w < (head1 - head0) * per_head; w += kThreads) {
        const int hi = w / per_head, u = w - hi * per_head, head = head0 + hi;
        const void *src;
        uint16_t *dst;
        int64_t so;
        bool turned = true;
        if (head < a.q_heads) {
            src = a.q;
            so = t * a.q_st + head * a.q_sh;
            dst = static_cast<uint16_t *>(a.q_out) + t * a.qo_st + head * a.qo_sh;
        } else if (head < a.q_heads + kv.kv_heads) {
            const int h = head - a.q_heads;
            if (page < 0) continue;
            src = a.k;
            so = t * a.k_st + h * a.k_sh;
            dst = static_cast<uint16_t *>(kv.k) + page * kv.ks_page + off * kv.ks_tok + h * kv.ks_head;
        } else {
            const int h = head - a.q_heads - kv.kv_heads;
            if (page < 0) continue;
            src = a.v;
            so = t * a.v_st + h * a.v_sh;
            dst = static_cast<uint16_t *>(kv.v) + page * kv.vs_page + off * kv.vs_tok + h * kv.vs_head;
            turned = false;
        }
        // two runs of eight elements, at d0 and d1, with n0 and n1 of them
        int d0, d1, n0, n1;
        if (!turned || u >= turn_units) {
            if (u >= (turned ? units : v_units)) continue;
            d0 = turned ? a.rot + (u - turn_units) * 16 : u * 16;
            d1 = d0 + 8;
            n0 = min(8, dim - d0);
            n1 = min(8, dim - d1);
            turned = false;
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
        float x[8], y[8];
        elem_load8<VEC, SRC>(src, so + d0, n0, x);
        elem_load8<VEC, SRC>(src, so + d1, n1, y);
        if (turned && a.pairs) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = u * 8 + e;
                if (i < half) {
                    const float c = s_cos[i], s = s_sin[i], p = x[2 * e], q = x[2 * e + 1];
                    x[2 * e] = p * c - q * s;
                    x[2 * e + 1] = p * s + q * c;
                }
                if (i + 4 < half) {
                    const float c = s_cos[i + 4], s = s_sin[i + 4], p = y[2 * e], q = y[2 * e + 1];
                    y[2 * e] = p * c - q * s;
                    y[2 * e + 1] = p * s + q * c;
                }
            }
        } else if (turned) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = u * 8 + e;
                if (i < half) {
                    const float c = s_cos[i], s = s_sin[i], p = x[e], q = y[e];
                    x[e] = p * c - q * s;
                    y[e] = p * s + q * c;
                }
            }
        }
        elem_store8<VEC, DST>(dst, d0, n0, x);
        elem_store8<VEC, DST>(dst, d1, n1, y);
    }
}

template <bool VEC, int SRC, int DST>
cudaError_t launch(const RopeArgs &a, int sm_count, cudaStream_t s)
{
    // few tokens: spread the heads of one over several blocks, so that the
    // call is as long as one block's few loads
    const int heads = a.q_heads + 2 * a.kv.kv_heads;
    int per = heads;
    while (per > 4 && static_cast<int64_t>(a.tokens) * ((heads + per - 1) / per) < sm_count) per = (per + 1) / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.tokens), static_cast<unsigned>((heads + per - 1) / per));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mbg_rope_kernel<VEC, SRC, DST>, a, per);
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
