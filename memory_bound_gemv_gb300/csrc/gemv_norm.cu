// Norms around a block, fused with its gate, the residual's scale and the
// residual:
//
//   u = y;  u = norm(u) * w_post  (when asked);  u = u * gate
//   x' = x + alpha * u            -> out
//   h  = norm(x') * w_pre + b_pre -> h (the next block's input)
//
// norm is x / rms(x), or (x - mean) / std (LayerNorm).  Statistics and all
// arithmetic are FP32; h is computed from the unrounded x', so out and h are
// each rounded once.  The variance is taken around the mean that was computed
// first: sums of squares minus squared sums lose the small variance of a row
// with a large mean.
//
// Bound by the bytes: y, x and the row-wise gate, scale and shift are read
// once, out and h written once.  One block takes one row and keeps it in
// registers, eight neighbouring elements per thread and step; y and x are
// requested before the first reduction, and what the row alone has of the
// other operands is prefetched into L2.
#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"
#include "gemv_elem.cuh"

namespace mbg {
namespace {

// Eight elements as loaded; converted after the loads of the whole row are
// under way.
struct Raw {
    uint4 a, b;
};

template <bool VEC>
__device__ __forceinline__ Raw raw_load(const void *base, int elem, int64_t at, int n)
{
    Raw r;
    r.a = r.b = make_uint4(0u, 0u, 0u, 0u);
    if (n <= 0) return r;
    if (VEC) {
        if (elem == GEMV_ELEM_F32) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
            r.a = p[0];
            r.b = p[1];
        } else {
            r.a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
        }
        return r;
    }
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (elem == GEMV_ELEM_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i] = static_cast<const uint32_t *>(base)[at + i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                w[i >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t *>(base)[at + i]) << (16 * (i & 1));
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    r.b = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}

__device__ __forceinline__ void raw_floats(const Raw &r, int elem, float (&x)[8])
{
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (elem == GEMV_ELEM_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = elem == GEMV_ELEM_F16 ? elem_unpack2<GEMV_ELEM_F16>(w[i]) : elem_unpack2<GEMV_ELEM_BF16>(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store_as(void *base, int elem, int64_t at, int n, const float (&x)[8])
{
    if (elem == GEMV_ELEM_F32)
        elem_store8<VEC, GEMV_ELEM_F32>(base, at, n, x);
    else if (elem == GEMV_ELEM_F16)
        elem_store8<VEC, GEMV_ELEM_F16>(base, at, n, x);
    else
        elem_store8<VEC, GEMV_ELEM_BF16>(base, at, n, x);
}

// Sum over the block; `turn` numbers the reductions of a kernel so that one
// barrier is enough for each.
struct Sums {
    float w[4][32];
};

__device__ __forceinline__ float block_sum(float v, Sums &s, int turn)
{
#pragma unroll
    for (int x = 16; x > 0; x /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, x);
    if ((threadIdx.x & 31) == 0) s.w[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5;
    float t = 0.f;
    for (int i = 0; i < warps; ++i) t += s.w[turn][i];
    return t;
}

// x -> (x - mean) / sqrt(var + eps), or x / sqrt(mean of squares + eps), for
// values held in registers; cnt[k] of the eight values of step k exist.
template <int K>
__device__ __forceinline__ void normalise(float (&x)[K][8], const int (&cnt)[K], const NormArgs &a, Sums &s, int turn)
{
    const float inv_n = 1.f / static_cast<float>(a.width);
    if (a.layer) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) t += x[k][e];  // elements that do not exist are 0
        const float mean = block_sum(t, s, turn) * inv_n;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = e < cnt[k] ? x[k][e] - mean : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(x[k][e], x[k][e], q);
    const float r = 1.f / sqrtf(block_sum(q, s, turn + 1) * inv_n + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] *= r;
}

// 16 bytes that are read once.  Not the read-only path: out may be x, h may
// be y.
__device__ __forceinline__ uint4 ld_once16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Types of y and x known at compile time (16 bits or FP32) halve the
// registers that their loads wait in.
template <bool VEC, bool WIDE>
struct Stream {
    Raw r;
    __device__ __forceinline__ void load(const void *base, int elem, int64_t at, int n)
    {
        if (!VEC) {
            r = raw_load<false>(base, elem, at, n);
        } else if (n > 0) {
            if (WIDE) {
                const unsigned char *p = reinterpret_cast<const unsigned char *>(static_cast<const float *>(base) + at);
                r.a = ld_once16(p);
                r.b = ld_once16(p + 16);
            } else {
                r.a = ld_once16(static_cast<const uint16_t *>(base) + at);
            }
        } else {
            r.a = r.b = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __device__ __forceinline__ void floats(int elem, float (&x)[8]) const
    {
        if (VEC && !WIDE) {
            const Raw t = {r.a, make_uint4(0u, 0u, 0u, 0u)};
            raw_floats(t, elem == GEMV_ELEM_F16 ? GEMV_ELEM_F16 : GEMV_ELEM_BF16, x);
        } else {
            raw_floats(r, VEC ? GEMV_ELEM_F32 : elem, x);
        }
    }
};

template <int K, int MAXT, bool VEC, bool Y32, bool X32>
__global__ void __launch_bounds__(MAXT) mbg_norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ Sums sums;
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    int at[K], cnt[K];
    Stream<VEC, Y32> y[K];
    Stream<VEC, X32> r[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        at[k] = (threadIdx.x + k * blockDim.x) * 8;
        cnt[k] = min(8, a.width - at[k]);
        y[k].load(a.y, a.y_e, row * a.y_s + at[k], cnt[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) r[k].load(a.r, a.r_e, row * a.r_s + at[k], cnt[k]);
    if (VEC && threadIdx.x == 0) {
        // operands of this row alone that are needed late: into L2 meanwhile
        auto early = [&](const void *p, int e, int64_t stride) {
            const int size = e == GEMV_ELEM_F32 ? 4 : 2;
            if (p && stride) prefetch_l2(static_cast<const unsigned char *>(p) + row * stride * size, a.width * size);
        };
        early(a.gate, a.gate_e, a.gate_s);
        early(a.pre_w, a.pre_w_e, a.pre_w_s);
        early(a.pre_b, a.pre_b_e, a.pre_b_s);
    }
    float x[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) y[k].floats(a.y_e, x[k]);
    if (a.post) {
        normalise<K>(x, cnt, a, sums, 0);
        if (a.post_w) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float w[8];
                raw_floats(raw_load<VEC>(a.post_w, a.post_e, row * a.post_s + at[k], cnt[k]), a.post_e, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[k][e] *= w[e];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float t[8];
        if (a.gate) {
            raw_floats(raw_load<VEC>(a.gate, a.gate_e, row * a.gate_s + at[k], cnt[k]), a.gate_e, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] *= t[e];
        }
        r[k].floats(a.r_e, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = e < cnt[k] ? fmaf(a.alpha, x[k][e], t[e]) : 0.f;
        store_as<VEC>(a.out, a.r_e, row * a.out_s + at[k], cnt[k], x[k]);
    }
    if (!a.h) return;
    normalise<K>(x, cnt, a, sums, 2);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float t[8];
        if (a.pre_w) {
            raw_floats(raw_load<VEC>(a.pre_w, a.pre_w_e, row * a.pre_w_s + at[k], cnt[k]), a.pre_w_e, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] *= a.unit_offset ? 1.f + t[e] : t[e];
        }
        if (a.pre_b) {
            raw_floats(raw_load<VEC>(a.pre_b, a.pre_b_e, row * a.pre_b_s + at[k], cnt[k]), a.pre_b_e, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] += t[e];
        }
        store_as<VEC>(a.h, a.h_e, row * a.h_s + at[k], cnt[k], x[k]);
    }
}

// Rows that registers cannot hold: every pass computes x' again from the
// inputs (through L2), and out and h are written in the last one, so that out
// may be the residual itself.
constexpr int kLongThreads = 1024;

template <bool VEC>
__global__ void __launch_bounds__(kLongThreads) mbg_norm_long_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ Sums sums;
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const float inv_n = 1.f / static_cast<float>(a.width);
    float mean_y = 0.f, r_y = 1.f, mean_x = 0.f;
    auto load = [&](const void *p, int e, int64_t stride, int at, int n, float(&t)[8]) {
        raw_floats(raw_load<VEC>(p, e, row * stride + at, n), e, t);
    };
    auto sum_y = [&](int at, int n, bool square) {
        float t[8], s = 0.f;
        load(a.y, a.y_e, a.y_s, at, n, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = e < n ? t[e] - mean_y : 0.f;
            s += square ? d * d : d;
        }
        return s;
    };
    auto stream = [&](int at, int n, float(&x)[8]) {
        float t[8];
        load(a.y, a.y_e, a.y_s, at, n, x);
        if (a.post) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (x[e] - mean_y) * r_y;
            if (a.post_w) {
                load(a.post_w, a.post_e, a.post_s, at, n, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= t[e];
            }
        }
        if (a.gate) {
            load(a.gate, a.gate_e, a.gate_s, at, n, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= t[e];
        }
        load(a.r, a.r_e, a.r_s, at, n, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e < n ? fmaf(a.alpha, x[e], t[e]) : 0.f;
    };
    const int step = kLongThreads * 8, first = threadIdx.x * 8;
    if (a.post) {
        float s = 0.f;
        if (a.layer) {
            for (int at = first; at < a.width; at += step) s += sum_y(at, min(8, a.width - at), false);
            mean_y = block_sum(s, sums, 0) * inv_n;
            s = 0.f;
        }
        for (int at = first; at < a.width; at += step) s += sum_y(at, min(8, a.width - at), true);
        r_y = 1.f / sqrtf(block_sum(s, sums, 1) * inv_n + a.eps);
    }
    float x[8], r_x = 1.f;
    if (a.h) {
        float s = 0.f;
        if (a.layer) {
            for (int at = first; at < a.width; at += step) {
                stream(at, min(8, a.width - at), x);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += x[e];
            }
            mean_x = block_sum(s, sums, 2) * inv_n;
            s = 0.f;
        }
        for (int at = first; at < a.width; at += step) {
            const int n = min(8, a.width - at);
            stream(at, n, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < n ? x[e] - mean_x : 0.f;
                s = fmaf(d, d, s);
            }
        }
        r_x = 1.f / sqrtf(block_sum(s, sums, 3) * inv_n + a.eps);
    }
    for (int at = first; at < a.width; at += step) {
        const int n = min(8, a.width - at);
        float t[8];
        stream(at, n, x);
        store_as<VEC>(a.out, a.r_e, row * a.out_s + at, n, x);
        if (!a.h) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (x[e] - mean_x) * r_x;
        if (a.pre_w) {
            load(a.pre_w, a.pre_w_e, a.pre_w_s, at, n, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= a.unit_offset ? 1.f + t[e] : t[e];
        }
        if (a.pre_b) {
            load(a.pre_b, a.pre_b_e, a.pre_b_s, at, n, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += t[e];
        }
        store_as<VEC>(a.h, a.h_e, row * a.h_s + at, n, x);
    }
}

cudaError_t launch_rows(void (*fn)(NormArgs), const NormArgs &a, int threads, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <bool VEC, bool Y32, bool X32>
cudaError_t launch(const NormArgs &a, int sm_count, cudaStream_t s)
{
    const int chunks = (a.width + 7) / 8;
    auto threads = [&](int k) { return ((chunks + k - 1) / k + 31) / 32 * 32; };
    // Few rows: a row's latency counts, and more threads shorten it.  Many
    // rows: small blocks with four steps per thread, so that several rows are
    // in different phases on one SM and loads are always under way.
    const bool many = a.rows > 2 * sm_count;
    if (chunks <= (many ? 128 : 512)) return launch_rows(mbg_norm_kernel<1, 512, VEC, Y32, X32>, a, threads(1), s);
    if (chunks <= (many ? 256 : 1024)) return launch_rows(mbg_norm_kernel<2, 512, VEC, Y32, X32>, a, threads(2), s);
    if (chunks <= 2048) return launch_rows(mbg_norm_kernel<4, 512, VEC, Y32, X32>, a, threads(4), s);
    return launch_rows(mbg_norm_long_kernel<VEC>, a, kLongThreads, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, bool vec, int sm_count, cudaStream_t s)
{
    if (!vec) return launch<false, true, true>(a, sm_count, s);
    const bool y32 = a.y_e == GEMV_ELEM_F32, x32 = a.r_e == GEMV_ELEM_F32;
    if (y32) return x32 ? launch<true, true, true>(a, sm_count, s) : launch<true, true, false>(a, sm_count, s);
    return x32 ? launch<true, false, true>(a, sm_count, s) : launch<true, false, false>(a, sm_count, s);
}

}  // namespace mbg
