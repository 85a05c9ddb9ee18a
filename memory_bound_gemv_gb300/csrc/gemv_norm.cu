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
// registers, eight neighbouring elements per thread and step.  Next to the
// bytes it is the instructions that count, some twenty per element: types are
// chosen outside the loops, addresses once per row and operand (8192 x 4096 in
// bf16: 46.6 us; with both inside the loops 83 us).
#include <stdint.h>

#include <atomic>

#include "gemv_decode.h"
#include "gemv_device.cuh"
#include "gemv_elem.cuh"

namespace mbg {
namespace {

// f(type's constant) for a type known at run time: one branch around all of a
// thread's steps.  (With the choice inside, the compiler converts every
// element both ways and selects.)
template <int E>
struct ElemTag {
    static constexpr int value = E;
};
template <typename F>
__device__ __forceinline__ void by_elem(int elem, F f)
{
    if (elem == GEMV_ELEM_F32)
        f(ElemTag<GEMV_ELEM_F32>());
    else if (elem == GEMV_ELEM_F16)
        f(ElemTag<GEMV_ELEM_F16>());
    else
        f(ElemTag<GEMV_ELEM_BF16>());
}

__device__ __forceinline__ const unsigned char *row_of(const void *base, int elem, int64_t row, int64_t stride)
{
    return static_cast<const unsigned char *>(base) + (row * stride << (elem == GEMV_ELEM_F32 ? 2 : 1));
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

// Rows that do not all begin at a 16-byte border (an odd width, say).  Their
// steps of eight elements are counted from the border before the row's
// beginning in out, which is where its beginning in the other tensors of the
// same layout has one too: those are moved whole, and only the row's first and
// last elements one by one.  Operands shared by all rows lie otherwise: a block
// lays them out once in shared memory (Staged).  What does not fit there is
// loaded in the aligned windows that hold it, and the first `skip` elements are
// shifted out.  8192 x 4001 in bf16: 73.9 us; with windows for the shared
// operands too 93.0 us, with loads and stores of single elements 250.8 us.
template <int E>
struct Window {
    static constexpr int kSize = E == GEMV_ELEM_F32 ? 4 : 2;
    static constexpr int kWords = E == GEMV_ELEM_F32 ? 12 : 8, kWhole = E == GEMV_ELEM_F32 ? 8 : 4;
    uint32_t w[kWords];
    int skip;
    // elements [at, at + 8) of a row of `width`; those outside it read 0
    __device__ __forceinline__ void load(const unsigned char *row, int at, int width)
    {
        const unsigned char *p = row + static_cast<int64_t>(at) * kSize;
        skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / kSize;
        const uint4 *q = reinterpret_cast<const uint4 *>(p - skip * kSize);
        if (skip == 0 && at >= 0 && at + 8 <= width) {
#pragma unroll
            for (int i = 0; i < kWhole / 4; ++i) set(i, q[i]);
#pragma unroll
            for (int i = kWhole; i < kWords; ++i) w[i] = 0u;
        } else if (at >= skip && at - skip + kWords * 4 / kSize <= width) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) set(i, q[i]);
        } else {
            skip = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (at + i < 0 || at + i >= width) continue;
                if (E == GEMV_ELEM_F32)
                    w[i] = reinterpret_cast<const uint32_t *>(p)[i];
                else
                    w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << (16 * (i & 1));
            }
        }
    }
    __device__ __forceinline__ void set(int i, const uint4 &v)
    {
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const { shifted(__any_sync(0xFFFFFFFFu, skip != 0), x); }
    // the same where the warp's lanes are not all here
    __device__ __forceinline__ void floats_one(float (&x)[8]) const { shifted(skip != 0, x); }
    __device__ __forceinline__ void shifted(bool any, float (&x)[8]) const
    {
        uint32_t t[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) t[i] = w[i];
        if (any) {
            const int words = E == GEMV_ELEM_F32 ? skip : skip >> 1;
#pragma unroll
            for (int d = 2; d > 0; d /= 2)
#pragma unroll
                for (int i = 0; i + d < kWords; ++i) t[i] = (words & d) ? t[i + d] : t[i];
            if (E != GEMV_ELEM_F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = (skip & 1) ? __funnelshift_r(t[i], t[i + 1], 16) : t[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if (E == GEMV_ELEM_F32) {
                x[i] = __uint_as_float(t[i]), x[i + 1] = __uint_as_float(t[i + 1]);
            } else {
                const float2 f = elem_unpack2<E == GEMV_ELEM_F32 ? GEMV_ELEM_F16 : E>(t[i / 2]);
                x[i] = f.x, x[i + 1] = f.y;
            }
        }
    }
};

// Elements between the border before a row's beginning and that beginning.
__device__ __forceinline__ int border_shift(const unsigned char *row, int elem)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(row);
    return static_cast<int>(elem == GEMV_ELEM_F32 ? (p & 31) >> 2 : (p & 15) >> 1);
}

// A thread's eight elements [at, at + 8) of a row.  VEC: all there (n = 8) or
// none, and aligned.
template <bool VEC, int E>
__device__ __forceinline__ void load_step(const unsigned char *row, int at, int n, int width, float (&x)[8])
{
    if (VEC) {
        elem_load8<true, E>(row, at, n, x);
    } else {
        Window<E> v;
        v.load(row, at, width);
        v.floats(x);
    }
}

template <bool VEC, int E>
__device__ __forceinline__ void store_step(unsigned char *row, int at, int n, int width, const float (&x)[8])
{
    unsigned char *p = row + static_cast<int64_t>(at) * (E == GEMV_ELEM_F32 ? 4 : 2);
    if (VEC) {
        elem_store8<true, E>(row, at, n, x);
    } else if (at >= 0 && at + 8 <= width && (reinterpret_cast<uintptr_t>(p) & (E == GEMV_ELEM_F32 ? 31 : 15)) == 0) {
        elem_store8<true, E>(p, 0, 8, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i >= 0 && at + i < width) elem_store1<E>(p, i, x[i]);
    }
}

// Eight elements as loaded, converted after the row's loads are under way.
// WIDE: FP32, else one of the 16-bit types.
template <bool VEC, bool WIDE>
struct Stream {
    uint4 a, b;  // b: FP32
    __device__ __forceinline__ void load(const unsigned char *row, int at, int n, int)
    {
        a = b = make_uint4(0u, 0u, 0u, 0u);
        if (n <= 0) return;
        if (WIDE) {
            uint32_t w[8];
            ld_global32(row + static_cast<int64_t>(at) * 4, w);
            a = make_uint4(w[0], w[1], w[2], w[3]);
            b = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            a = ld_once16(row + static_cast<int64_t>(at) * 2);
        }
    }
    template <int E>
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (WIDE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = elem_unpack2<E == GEMV_ELEM_F32 ? GEMV_ELEM_F16 : E>(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
};

// The same for rows that begin anywhere: whole pieces where they lie at a
// border, single elements where not; those outside the row read 0.
template <bool WIDE>
struct Stream<false, WIDE> {
    static constexpr int kSize = WIDE ? 4 : 2, kWords = WIDE ? 8 : 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const unsigned char *row, int at, int, int width)
    {
        const unsigned char *p = row + static_cast<int64_t>(at) * kSize;
        if (at >= 0 && at + 8 <= width && (reinterpret_cast<uintptr_t>(p) & (8 * kSize - 1)) == 0) {
            if constexpr (WIDE) {
                ld_global32(p, w);
            } else {
                const uint4 v = ld_once16(p);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (at + i < 0 || at + i >= width) continue;
            if constexpr (WIDE)
                w[i] = reinterpret_cast<const uint32_t *>(p)[i];
            else
                w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << (16 * (i & 1));
        }
    }
    template <int E>
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if constexpr (WIDE) {
                x[i] = __uint_as_float(w[i]), x[i + 1] = __uint_as_float(w[i + 1]);
            } else {
                const float2 f = elem_unpack2<E == GEMV_ELEM_F32 ? GEMV_ELEM_F16 : E>(w[i / 2]);
                x[i] = f.x, x[i + 1] = f.y;
            }
        }
    }
};

// An operand shared by all rows, in shared memory as FP32: element j stands in
// line (j + 8) % 8, column (j + 8) / 8, zeros around the row.  Whatever the row's
// shift, neighbouring threads then read neighbouring words, one element of each
// thread's eight at a time, and no instruction goes into shifting.
__device__ __forceinline__ void stage_operand(float *to, int columns, const void *from, int elem, int width)
{
    by_elem(elem, [&](auto e) {
        for (int c = threadIdx.x; c < columns; c += blockDim.x) {
            Window<decltype(e)::value> v;
            float t[8];
            v.load(static_cast<const unsigned char *>(from), 8 * c - 8, width);
            v.floats_one(t);
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i * columns + c] = t[i];
        }
    });
}

// The type of y or x where WIDE leaves only two.
template <bool WIDE, typename F>
__device__ __forceinline__ void by_stream(int elem, F f)
{
    if (WIDE)
        f(ElemTag<GEMV_ELEM_F32>());
    else if (elem == GEMV_ELEM_F16)
        f(ElemTag<GEMV_ELEM_F16>());
    else
        f(ElemTag<GEMV_ELEM_BF16>());
}

// Sum over the block.  `turn` numbers the reductions, so that one barrier is
// enough for each; a block that goes through several rows alternates between
// two sets of four.  (A row spread over a cluster of blocks, joined through
// distributed shared memory, takes longer: 331 rows of 14336 in clusters of
// two 21.5 us, in blocks 18.1 us.)
struct Sums {
    float w[8][32];
};

__device__ __forceinline__ float row_sum(float v, Sums &s, int turn)
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
// values held in registers.  Elements that do not exist are 0 before and after
// (every operand reads 0 there; where a factor is infinite or NaN, so is the row).
template <int K, bool VEC, bool FULL>
__device__ __forceinline__ void normalise(float (&x)[K][8], const int (&at)[K], int shift_by, const NormArgs &a, Sums &s,
                                          int turn)
{
    const float inv_n = 1.f / static_cast<float>(a.width);
    if (a.layer) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) t += x[k][e];
        const float mean = row_sum(t, s, turn) * inv_n;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[k][e] = FULL || static_cast<unsigned>(at[k] - shift_by + (VEC ? 0 : e)) < static_cast<unsigned>(a.width)
                              ? x[k][e] - mean
                              : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(x[k][e], x[k][e], q);
    const float r = 1.f / sqrtf(row_sum(q, s, turn + 1) * inv_n + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] *= r;
}

// A block goes through rows and requests the next row's y and x while it
// works on the present one (MINB 1); or MINB blocks are on an SM, each with one
// row, or with rows that begin anywhere several, one after another;
// what else differs from row to row is prefetched into L2, what does not comes
// from L1.  FULL: every thread has all of its K steps.
template <int K, int MAXT, int MINB, bool VEC, bool FULL, bool Y32, bool X32>
__global__ void __launch_bounds__(MAXT, MINB) mbg_norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ Sums sums;
    pdl_trigger();
    pdl_wait();
    constexpr bool kLoop = MINB == 1 || !VEC;  // otherwise a block for each row
    constexpr bool kNext = MINB == 1;          // rows ahead
    int64_t row = blockIdx.x;
    int at[K], cnt[K];
    Stream<VEC, Y32> y[K];
    Stream<VEC, X32> r[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        at[k] = (k * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8;
        cnt[k] = FULL ? 8 : min(8, a.width - at[k]);  // VEC: 8 or none
    }
    // operands of a row alone that are needed late
    auto prefetch = [&](int64_t rw) {
        if (!VEC || threadIdx.x != 0 || rw >= a.rows) return;
        auto one = [&](const void *p, int e, int64_t stride) {
            if (p && stride) prefetch_l2(row_of(p, e, rw, stride), a.width << (e == GEMV_ELEM_F32 ? 2 : 1));
        };
        one(a.post_w, a.post_e, a.post_s);
        one(a.gate, a.gate_e, a.gate_s);
        one(a.pre_w, a.pre_w_e, a.pre_w_s);
        one(a.pre_b, a.pre_b_e, a.pre_b_s);
    };
    // where the steps are counted from
    auto shift_of = [&](int64_t rw) { return VEC ? 0 : border_shift(row_of(a.out, a.r_e, rw, a.out_s), a.r_e); };
    auto request_y = [&](int64_t rw) {
        const unsigned char *p = row_of(a.y, a.y_e, rw, a.y_s);
        const int from = shift_of(rw);
#pragma unroll
        for (int k = 0; k < K; ++k) y[k].load(p, at[k] - from, cnt[k], a.width);
    };
    auto request_r = [&](int64_t rw) {
        const unsigned char *p = row_of(a.r, a.r_e, rw, a.r_s);
        const int from = shift_of(rw);
#pragma unroll
        for (int k = 0; k < K; ++k) r[k].load(p, at[k] - from, cnt[k], a.width);
    };
    // operands shared by all rows, where those begin anywhere
    extern __shared__ float staged[];
    const int columns = K * static_cast<int>(blockDim.x) + 1;
    // x[k][i] = f(x[k][i], operand)
    float x[K][8];
    int shift = 0;
    auto with = [&](int which, const void *base, int elem, int64_t stride, auto f) {
        if (!VEC && ((a.staged >> which) & 1)) {
            const float *lines = staged + __popc(a.staged & ((1 << which) - 1)) * 8 * columns;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int line = (i - shift) & 7, col = line > i ? 0 : 1;
                const float *from = lines + line * columns + col + threadIdx.x;
#pragma unroll
                for (int k = 0; k < K; ++k) x[k][i] = f(x[k][i], from[k * blockDim.x]);
            }
            return;
        }
        const unsigned char *p = row_of(base, elem, row, stride);
        by_elem(elem, [&](auto e) {
            float t[K][8];
#pragma unroll
            for (int k = 0; k < K; ++k) load_step<VEC, decltype(e)::value>(p, at[k] - shift, cnt[k], a.width, t[k]);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[k][i] = f(x[k][i], t[k][i]);
        });
    };
    auto product = [](float v, float w) { return v * w; };
    prefetch(row);
    request_y(row);
    request_r(row);
    if (!VEC) {
        int n = 0;
        auto stage = [&](int which, const void *from, int elem) {
            if ((a.staged >> which) & 1) stage_operand(staged + n++ * 8 * columns, columns, from, elem, a.width);
        };
        stage(0, a.post_w, a.post_e);
        stage(1, a.gate, a.gate_e);
        stage(2, a.pre_w, a.pre_w_e);
        stage(3, a.pre_b, a.pre_b_e);
        if (n > 0) __syncthreads();
    }
    for (int turn = 0;; turn ^= 4) {
        shift = shift_of(row);
        const int64_t next = kLoop ? row + gridDim.x : a.rows;
        if (kNext) prefetch(next);
        by_stream<Y32>(a.y_e, [&](auto e) {
#pragma unroll
            for (int k = 0; k < K; ++k) y[k].template floats<decltype(e)::value>(x[k]);
        });
        if (kNext && next < a.rows) request_y(next);
        if (a.post) {
            normalise<K, VEC, FULL>(x, at, shift, a, sums, turn);
            if (a.post_w) with(0, a.post_w, a.post_e, a.post_s, product);
        }
        if (a.gate) with(1, a.gate, a.gate_e, a.gate_s, product);
        by_stream<X32>(a.r_e, [&](auto e) {
            constexpr int E = decltype(e)::value;
            unsigned char *p = const_cast<unsigned char *>(row_of(a.out, E, row, a.out_s));
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float t[8];
                r[k].template floats<E>(t);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[k][i] = fmaf(a.alpha, x[k][i], t[i]);
                store_step<VEC, E>(p, at[k] - shift, cnt[k], a.width, x[k]);
            }
        });
        if (kNext && next < a.rows) request_r(next);
        if (a.h) {
            normalise<K, VEC, FULL>(x, at, shift, a, sums, turn + 2);
            if (a.pre_w) {
                const float unit = a.unit_offset ? 1.f : 0.f;
                with(2, a.pre_w, a.pre_w_e, a.pre_w_s, [&](float v, float w) { return v * (w + unit); });
            }
            if (a.pre_b) with(3, a.pre_b, a.pre_b_e, a.pre_b_s, [](float v, float w) { return v + w; });
            by_elem(a.h_e, [&](auto e) {
                constexpr int E = decltype(e)::value;
                unsigned char *p = const_cast<unsigned char *>(row_of(a.h, E, row, a.h_s));
#pragma unroll
                for (int k = 0; k < K; ++k) store_step<VEC, E>(p, at[k] - shift, cnt[k], a.width, x[k]);
            });
        }
        if (!kLoop || next >= a.rows) break;
        row = next;
        if (!kNext) {
            request_y(row);
            request_r(row);
        }
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
    const int shift = VEC ? 0 : border_shift(row_of(a.out, a.r_e, row, a.out_s), a.r_e);
    const int steps = (a.width + shift + kLongThreads * 8 - 1) / (kLongThreads * 8);
    auto step_at = [&](int step) { return (step * kLongThreads + static_cast<int>(threadIdx.x)) * 8 - shift; };
    auto exists = [&](int at, int e) { return static_cast<unsigned>(at + e) < static_cast<unsigned>(a.width); };
    auto load = [&](const void *p, int elem, int64_t stride, int at, int n, float(&t)[8]) {
        by_elem(elem, [&](auto e) {
            load_step<VEC, decltype(e)::value>(row_of(p, elem, row, stride), at, n, a.width, t);
        });
    };
    auto store = [&](void *p, int elem, int64_t stride, int at, int n, const float(&t)[8]) {
        by_elem(elem, [&](auto e) {
            store_step<VEC, decltype(e)::value>(const_cast<unsigned char *>(row_of(p, elem, row, stride)), at, n, a.width, t);
        });
    };
    auto sum_y = [&](int at, int n, bool square) {
        float t[8], s = 0.f;
        load(a.y, a.y_e, a.y_s, at, n, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = exists(at, e) ? t[e] - mean_y : 0.f;
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
        for (int e = 0; e < 8; ++e) x[e] = exists(at, e) ? fmaf(a.alpha, x[e], t[e]) : 0.f;
    };
    if (a.post) {
        float s = 0.f;
        if (a.layer) {
            for (int c = 0; c < steps; ++c) s += sum_y(step_at(c), min(8, a.width - step_at(c)), false);
            mean_y = row_sum(s, sums, 0) * inv_n;
            s = 0.f;
        }
        for (int c = 0; c < steps; ++c) s += sum_y(step_at(c), min(8, a.width - step_at(c)), true);
        r_y = 1.f / sqrtf(row_sum(s, sums, 1) * inv_n + a.eps);
    }
    float x[8], r_x = 1.f;
    if (a.h) {
        float s = 0.f;
        if (a.layer) {
            for (int c = 0; c < steps; ++c) {
                const int at = step_at(c);
                stream(at, min(8, a.width - at), x);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += x[e];
            }
            mean_x = row_sum(s, sums, 2) * inv_n;
            s = 0.f;
        }
        for (int c = 0; c < steps; ++c) {
            const int at = step_at(c), n = min(8, a.width - at);
            stream(at, n, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = exists(at, e) ? x[e] - mean_x : 0.f;
                s = fmaf(d, d, s);
            }
        }
        r_x = 1.f / sqrtf(row_sum(s, sums, 3) * inv_n + a.eps);
    }
    for (int c = 0; c < steps; ++c) {
        const int at = step_at(c), n = min(8, a.width - at);
        float t[8];
        stream(at, n, x);
        store(a.out, a.r_e, a.out_s, at, n, x);
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
        store(a.h, a.h_e, a.h_s, at, n, x);
    }
}

cudaError_t launch_rows(void (*fn)(NormArgs), const NormArgs &a, int64_t blocks, int threads, cudaStream_t s,
                        size_t smem = 0)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

// Shared memory that an SM's staged operands may take.
constexpr int kStageBytes = 224 * 1024;

// Blocks that fit on the GPU at once, each going through rows.
template <int K, int MAXT, int MINB, bool VEC, bool FULL, bool Y32, bool X32>
cudaError_t launch_fitting(NormArgs a, int threads, int sm_count, cudaStream_t s)
{
    auto fn = mbg_norm_kernel<K, MAXT, MINB, VEC, FULL, Y32, X32>;
    static std::atomic<int> fit[MAXT / 32 + 1][5];  // blocks per SM, by warps and staged operands (0: not asked yet)
    const int each = 32 * (K * threads + 1);       // bytes of a staged operand
    int count = 0, smem = 0;
    auto blocks = [&](int64_t *n) {
        int per_sm = fit[threads / 32][count].load(std::memory_order_relaxed);
        if (per_sm == 0) {
            const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, threads, smem);
            if (e != cudaSuccess) return e;
            if (per_sm < 1) per_sm = 1;
            fit[threads / 32][count].store(per_sm, std::memory_order_relaxed);
        }
        *n = static_cast<int64_t>(per_sm) * sm_count;
        return cudaSuccess;
    };
    int64_t most = 0;
    cudaError_t e = blocks(&most);
    a.staged = 0;
    // Staging pays from the third row of a block on (1500 x 4001 in binary16,
    // 2.5 rows a block: 19.0 us against 20.9; 600 rows, one a block: 8.8
    // against 7.5; in FP32, two a block, 10.5 against 10.2).
    if (!VEC && e == cudaSuccess && a.rows > 2 * most) {
        const bool shared[4] = {a.post_w && !a.post_s, a.gate && !a.gate_s, a.pre_w && !a.pre_w_s, a.pre_b && !a.pre_b_s};
        for (int i = 0; i < 4; ++i)
            if (shared[i] && (count + 1) * each <= kStageBytes / MINB) {
                a.staged |= 1 << i;
                ++count;
            }
        smem = count * each;
        static std::atomic<uint64_t> ready{0};  // a bit per device
        int dev = 0;
        if (count > 0) e = cudaGetDevice(&dev);
        if (count > 0 && e == cudaSuccess && !(ready.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageBytes);
            if (e == cudaSuccess) ready.fetch_or(uint64_t{1} << (dev & 63), std::memory_order_relaxed);
        }
        if (count > 0 && e == cudaSuccess) e = blocks(&most);
    }
    if (e != cudaSuccess) return e;
    return launch_rows(fn, a, a.rows < most ? a.rows : most, threads, s, smem);
}

template <int K, bool VEC, bool Y32, bool X32>
cudaError_t launch_steps(const NormArgs &a, int sm_count, cudaStream_t s)
{
    const int chunks = (a.width + (VEC ? 7 : 14)) / 8, threads = ((chunks + K - 1) / K + 31) / 32 * 32;
    // Rows of more than 256 threads: one such block at a time on an SM leaves it
    // idle at every sum, so two of fewer registers each take turns.  A block
    // per row, without rows ahead (2000 x 9216 in bf16 29.8 us against 37.3, 200
    // rows 6.2 against 6.5; 100 rows 4.9 against 4.2: not with shared operands
    // on fewer rows than SMs); where rows begin anywhere, blocks that keep their
    // staged operands (2000 x 9001 50.6 us against 66.7), up to 320 threads.  Up
    // to 384 registers spill and an SM has no room to stage three operands twice:
    // two blocks where nothing is staged (11908 wide in bf16: 200 rows 8.2 us
    // against 10.1, 608 19.6 against 21.9, though 400 17.2 against 16.3) or both
    // streams are FP32 (2000 x 10501 71.8 against 90.6, 12281 90.3 against 97.7),
    // one for more rows of other types (in bf16 1000 x 11908 35.2 against 37.5,
    // 2000 65.3 against 63.1; FP32 and binary16 2000 x 12281 60.9 against 75.9).  Operands of each row are loaded late in
    // it, which blocks hide better than rows ahead do (2000 x 8192 with gate,
    // weight and bias of each row 38.3 us against 42.7; with shared ones 28.1
    // against 26.7).  400 x 4096, all rows at once on the GPU, is faster without
    // (5.4 us against 6.4).
    const bool each = a.gate_s || a.pre_w_s || a.pre_b_s;
    if constexpr (!VEC && K == 4) {
        if (threads > 256 && threads <= 320 && a.rows > sm_count)
            return launch_fitting<4, 320, 2, false, false, Y32, X32>(a, threads, sm_count, s);
        if (threads > 320 && threads <= 384 && a.rows > sm_count && (a.rows <= 4 * sm_count || (Y32 && X32)))
            return launch_fitting<4, 384, 2, false, false, Y32, X32>(a, threads, sm_count, s);
    }
    if constexpr (VEC && K == 4) {
        if (threads <= 448 && (threads > 256 ? each || a.rows > sm_count : each && a.rows > 8 * sm_count))
            return launch_rows(chunks == threads * K ? mbg_norm_kernel<4, 448, 2, true, true, Y32, X32>
                                                     : mbg_norm_kernel<4, 448, 2, true, false, Y32, X32>,
                               a, a.rows, threads, s);
    }
    if (VEC && chunks == threads * K) return launch_fitting<K, 512, 1, VEC, VEC, Y32, X32>(a, threads, sm_count, s);
    return launch_fitting<K, 512, 1, VEC, false, Y32, X32>(a, threads, sm_count, s);
}

template <bool VEC, bool Y32, bool X32>
cudaError_t launch(const NormArgs &a, int sm_count, cudaStream_t s)
{
    const int chunks = (a.width + (VEC ? 7 : 14)) / 8;  // a row may begin up to seven elements into its first step
    if (chunks > 2048) return launch_rows(mbg_norm_long_kernel<VEC>, a, a.rows, kLongThreads, s);
    // Few rows: a row's latency counts, and more threads shorten it.  Many
    // rows: small blocks with several steps per thread, so that several rows
    // are in different phases on one SM.
    const bool many = a.rows > 2 * sm_count;
    if (chunks > 1024 || (many && !Y32 && !X32 && chunks > 256)) return launch_steps<4, VEC, Y32, X32>(a, sm_count, s);
    if (chunks > (many ? 128 : 512)) return launch_steps<2, VEC, Y32, X32>(a, sm_count, s);
    return launch_steps<1, VEC, Y32, X32>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, bool vec, int sm_count, cudaStream_t s)
{
    const bool y32 = a.y_e == GEMV_ELEM_F32, x32 = a.r_e == GEMV_ELEM_F32;
    auto pick = [&](auto v) {
        constexpr bool V = decltype(v)::value != 0;
        if (y32) return x32 ? launch<V, true, true>(a, sm_count, s) : launch<V, true, false>(a, sm_count, s);
        return x32 ? launch<V, false, true>(a, sm_count, s) : launch<V, false, false>(a, sm_count, s);
    };
    return vec ? pick(ElemTag<1>()) : pick(ElemTag<0>());
}

}  // namespace mbg
