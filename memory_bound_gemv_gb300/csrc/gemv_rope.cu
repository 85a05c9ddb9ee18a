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
// Bound by the bytes of q, k and v read and written once.  A thread keeps one
// head and one unit of 16 of its elements, so that its addresses and its part
// of the work are settled once, and goes through tokens: a block's loads of
// the next tokens are under way while it turns the present one, whose sines
// and cosines were computed into shared memory during the one before.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "gemv_decode.h"
#include "gemv_device.cuh"
#include "gemv_elem.cuh"

namespace mbg {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kMaxPairs = 128;

// A head is cut into runs of eight elements, and a unit is two of them, at d0
// and d1, of which n0 and n1 elements exist: runs u and u + (half of them), so
// that neighbouring threads load neighbouring runs (two neighbouring runs in
// one thread would fetch and write every 32-byte sector in two halves).  Turned
// units are eight pairs: style "halves" elements i..i+7 and those rot / 2
// behind them, "pairs" four pairs in each run.  The others are copied.
struct Unit {
    int d0, d1, n0, n1;
    int pair0, pair1;  // first pairs of the runs
    bool turned;
    __device__ __forceinline__ Unit(const RopeArgs &a, int u, bool is_v)
    {
        const int half = a.rot >> 1, dim = a.kv.dim, turn_units = (half + 7) >> 3;
        turned = !is_v && u < turn_units;
        pair0 = pair1 = 8 * u;
        if (turned && !a.pairs) {
            d0 = u * 8;
            d1 = half + d0;
            n0 = n1 = min(8, half - d0);
        } else {
            const int from = is_v || turned ? 0 : a.rot, to = turned ? a.rot : dim, first = is_v || turned ? u : u - turn_units;
            const int units = (to - from + 15) >> 4;
            d0 = from + first * 8;
            d1 = d0 + units * 8;
            n0 = min(8, to - d0);
            n1 = min(8, to - d1);
            pair0 = 4 * u;
            pair1 = 4 * (u + units);
        }
        if (u >= (is_v ? (dim + 15) >> 4 : turn_units + ((dim - a.rot + 15) >> 4))) n0 = n1 = 0;
    }
};

// Eight elements as loaded.
template <int E>
struct Raw8 {
    uint4 a, b;  // b: FP32 only
    template <bool VEC>
    __device__ __forceinline__ void load(const void *base, int64_t at, int n)
    {
        const int size = E == GEMV_ELEM_F32 ? 4 : 2;
        if (VEC) {
            if (n < 8) return;
            const unsigned char *p = static_cast<const unsigned char *>(base) + at * size;
            if (E == GEMV_ELEM_F32) {
                uint32_t w[8];
                ld_global32(p, w);
                a = make_uint4(w[0], w[1], w[2], w[3]);
                b = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
                a = ld_stream16(p);
            }
        } else {
            float x[8];
            elem_load8<false, E>(base, at, n, x);
            a = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            b = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
        }
    }
    template <bool VEC>
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (!VEC || E == GEMV_ELEM_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = elem_unpack2<E>(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
};

// What a block knows of a token before it turns it.
struct Place {
    int seq, slot, page, off;  // page -1: not written
};

// All warps but the last turn; the last one looks ahead: it computes the next
// token's sines and cosines and its place in the cache, whose indices it has
// read for 32 tokens at a time.  7001 tokens of 48 heads of 128 in bf16: 29.8 us,
// 5.8 TB/s; with these reads token by token 33.6 us, with the sines in every
// thread (100 registers, 12 warps on an SM) 62.8 us.
template <bool VEC, int SRC, int DST>
__global__ void __launch_bounds__(kMaxThreads + 32, 3)
    mbg_rope_kernel(const __grid_constant__ RopeArgs a, int heads_per_block, int per_head)
{
    __shared__ __align__(16) float s_cos[2][kMaxPairs], s_sin[2][kMaxPairs];
    __shared__ Place s_place[2];
    pdl_trigger();
    pdl_wait();
    const KvView &kv = a.kv;
    const int tid = threadIdx.x, half = a.rot >> 1, step = gridDim.x;

    if (tid >= static_cast<int>(blockDim.x) - 32) {
        const int lane = tid & 31;
        constexpr int kPairs = kMaxPairs / 32, kAxes = 4;
        uint64_t turns[kPairs];
        int ax[kPairs];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int pair = lane + 32 * i;
            turns[i] = pair < half ? __ldg(a.turns + pair) : 0;
            ax[i] = pair < half ? __ldg(a.axis + pair) : 0;
            if (ax[i] >= a.axes) {
                report_error(a.err, DEVERR_BAD_INDEX);
                ax[i] = 0;
            }
        }
        // what is to be known of 32 tokens, one per lane: places, and positions
        // on the first axes (those on further axes are read when needed)
        struct Ahead {
            Place p;
            int pos[kAxes];
        };
        auto ahead = [&](int t) {
            Ahead w = {{0, -1, -1, 0}, {0, 0, 0, 0}};
            if (t >= a.tokens) return w;
#pragma unroll
            for (int x = 0; x < kAxes; ++x)
                if (x < a.axes) w.pos[x] = __ldg(a.positions + x * a.pos_stride + t);
            w.p.seq = a.seq ? __ldg(a.seq + t) : t;
            w.p.slot = __ldg(a.slots + t);
            if (w.p.slot < 0) return w;  // a negative slot is padding: nothing is written
            if (w.p.seq >= 0 && w.p.seq < kv.batch && w.p.slot < kv.capacity) {
                const int idx = kv.page_shift >= 0 ? w.p.slot >> kv.page_shift : w.p.slot / kv.page_size;
                w.p.off = w.p.slot - idx * kv.page_size;
                w.p.page = __ldg(kv.table + w.p.seq * kv.table_stride + idx);  // checked when the token's turn comes
            }
            return w;
        };
        int t = blockIdx.x;
        Ahead now = ahead(t + lane * step), then = ahead(t + (32 + lane) * step);
        for (int n = 0; t < a.tokens; t += step, ++n) {
            const int l = n & 31, buf = n & 1;
            if (n > 0 && l == 0) {
                now = then;
                then = ahead(t + (32 + lane) * step);
            }
            int at[kAxes];
#pragma unroll
            for (int x = 0; x < kAxes; ++x) at[x] = __shfl_sync(0xFFFFFFFFu, now.pos[x], l);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                if (lane + 32 * i >= half) continue;
                int pos = at[0];
#pragma unroll
                for (int x = 1; x < kAxes; ++x)
                    if (ax[i] == x) pos = at[x];
                if (ax[i] >= kAxes) pos = __ldg(a.positions + ax[i] * a.pos_stride + t);
                const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns[i];
                // the nearest 2^-32 turns, as half turns in [-1, 1)
                const int32_t part = static_cast<int32_t>((turn + 0x80000000ull) >> 32);
                sincospif(static_cast<float>(part) * 4.656612873077393e-10f, &s_sin[buf][lane + 32 * i],
                          &s_cos[buf][lane + 32 * i]);
            }
            Place here;
            here.seq = __shfl_sync(0xFFFFFFFFu, now.p.seq, l);
            here.slot = __shfl_sync(0xFFFFFFFFu, now.p.slot, l);
            here.page = __shfl_sync(0xFFFFFFFFu, now.p.page, l);
            here.off = __shfl_sync(0xFFFFFFFFu, now.p.off, l);
            if (here.page < 0 || here.page >= kv.num_pages) {
                if (here.slot >= 0 && lane == 0) report_error(a.err, DEVERR_BAD_INDEX);
                here.page = -1;
            }
            if (lane == 0) s_place[buf] = here;
            __syncthreads();
            if (blockIdx.y == 0 && here.page >= 0) {
                for (int i = lane; i < kv.kv_heads; i += 32) {
                    const int64_t slot = (static_cast<int64_t>(here.seq) * kv.kv_heads + i) * kv.capacity + here.slot;
                    if (a.scores_cache) a.scores_cache[slot] = 0.f;
                    if (a.stamps_cache) a.stamps_cache[slot] = a.stamps ? __ldg(a.stamps + t) : here.slot;
                }
            }
        }
        return;
    }

    // this thread's head and unit
    const int lane_head = tid / per_head, u = tid - lane_head * per_head;
    const int head = blockIdx.y * heads_per_block + lane_head, first_v = a.q_heads + kv.kv_heads;
    const bool is_q = head < a.q_heads, is_v = head >= first_v;
    const bool mine = lane_head < heads_per_block && head < first_v + kv.kv_heads;
    const int h = is_q ? head : is_v ? head - first_v : head - a.q_heads;
    const Unit un(a, u, is_v);
    const int n0 = mine ? un.n0 : 0, n1 = mine ? un.n1 : 0;
    constexpr int kSize = SRC == GEMV_ELEM_F32 ? 4 : 2;
    const int64_t src_token = is_q ? a.q_st : is_v ? a.v_st : a.k_st;
    const unsigned char *src = static_cast<const unsigned char *>(is_q ? a.q : is_v ? a.v : a.k) +
                               (h * (is_q ? a.q_sh : is_v ? a.v_sh : a.k_sh) + blockIdx.x * src_token) * kSize;
    const int64_t src_step = step * src_token * kSize;
    uint16_t *dst = is_q ? static_cast<uint16_t *>(a.q_out) + h * a.qo_sh + blockIdx.x * a.qo_st
                    : is_v ? static_cast<uint16_t *>(kv.v) + h * kv.vs_head
                           : static_cast<uint16_t *>(kv.k) + h * kv.ks_head;
    const int64_t d_page = is_v ? kv.vs_page : kv.ks_page, d_tok = is_v ? kv.vs_tok : kv.ks_tok;
    constexpr int kAhead = SRC == GEMV_ELEM_F32 ? 1 : 2;  // tokens requested ahead
    Raw8<SRC> x[kAhead], y[kAhead];
    auto request = [&](int k, int t) {
        if (t < a.tokens) {
            x[k].template load<VEC>(src, un.d0, n0);
            y[k].template load<VEC>(src, un.d1, n1);
            src += src_step;
        }
    };
    int t = blockIdx.x;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) request(k, t + k * step);
    for (int buf = 0; t < a.tokens;) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (t >= a.tokens) break;
            __syncthreads();
            float v[8], w[8];
            x[k].template floats<VEC>(v);
            y[k].template floats<VEC>(w);
            request(k, t + kAhead * step);
            if (un.turned) {
                // pairs past the last turn elements that do not exist
                const int last = half - 1;
                if (a.pairs) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int p0 = min(un.pair0 + e, last), p1 = min(un.pair1 + e, last);
                        const float c0 = s_cos[buf][p0], s0 = s_sin[buf][p0], c1 = s_cos[buf][p1], s1 = s_sin[buf][p1];
                        const float f = v[2 * e], g = v[2 * e + 1], i = w[2 * e], j = w[2 * e + 1];
                        v[2 * e] = f * c0 - g * s0;
                        v[2 * e + 1] = f * s0 + g * c0;
                        w[2 * e] = i * c1 - j * s1;
                        w[2 * e + 1] = i * s1 + j * c1;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = min(un.pair0 + e, last);
                        const float c = s_cos[buf][i], s = s_sin[buf][i], f = v[e], g = w[e];
                        v[e] = f * c - g * s;
                        w[e] = f * s + g * c;
                    }
                }
            }
            const int page = s_place[buf].page, off = s_place[buf].off;
            if (mine && (is_q || page >= 0)) {
                uint16_t *to = is_q ? dst : dst + page * d_page + off * d_tok;
                elem_store8<VEC, DST>(to, un.d0, n0, v);
                elem_store8<VEC, DST>(to, un.d1, n1, w);
            }
            if (is_q) dst += step * a.qo_st;
            t += step;
            buf ^= 1;
        }
    }
}

template <bool VEC, int SRC, int DST>
cudaError_t launch(const RopeArgs &a, int sm_count, cudaStream_t s)
{
    const int heads = a.q_heads + 2 * a.kv.kv_heads, half = a.rot / 2;
    const int units = (half + 7) / 8 + (a.kv.dim - a.rot + 15) / 16, v_units = (a.kv.dim + 15) / 16;
    const int per_head = units > v_units ? units : v_units;
    // few tokens: spread the heads of one over several blocks, so that the
    // call is as long as one block's few loads
    int per = heads;
    while (per * per_head > kMaxThreads || (per > 4 && static_cast<int64_t>(a.tokens) * ((heads + per - 1) / per) < sm_count))
        per = (per + 1) / 2;
    const int threads = (per * per_head + 31) / 32 * 32 + 32, groups = (heads + per - 1) / per;
    // blocks that fit on the GPU at once go through the tokens
    auto fn = mbg_rope_kernel<VEC, SRC, DST>;
    static std::atomic<int> fit[kMaxThreads / 32 + 2];  // blocks per SM, by warps (0: not asked yet)
    int per_sm = fit[threads / 32].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, threads, 0);
        if (e != cudaSuccess) return e;
        if (per_sm < 1) per_sm = 1;
        fit[threads / 32].store(per_sm, std::memory_order_relaxed);
    }
    int64_t blocks = static_cast<int64_t>(per_sm) * sm_count / groups;
    if (blocks < 1) blocks = 1;
    if (blocks > a.tokens) blocks = a.tokens;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(groups));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a, per, per_head);
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
