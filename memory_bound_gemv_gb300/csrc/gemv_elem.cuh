// Loads and stores of eight elements of a type chosen at compile time
// (GEMV_ELEM_*), as FP32 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gemv_decode.h"

namespace mbg {

// 32 bytes at once (32-byte aligned): eight FP32 values of a thread as one
// whole sector; two 16-byte accesses would move every sector in two halves.
__device__ __forceinline__ void ld_global32(const void *p, uint32_t (&w)[8])
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}

__device__ __forceinline__ void st_global32(void *p, const float (&x)[8])
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

// 32 bits holding two 16-bit elements -> two floats (bf16 is the upper half
// of an FP32 value).
template <int E>
__device__ __forceinline__ float2 elem_unpack2(uint32_t w)
{
    if (E == GEMV_ELEM_F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <int E>
__device__ __forceinline__ uint32_t elem_pack2(float lo, float hi)
{
    if (E == GEMV_ELEM_F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int E>
__device__ __forceinline__ float elem_load1(const void *base, int64_t at)
{
    if (E == GEMV_ELEM_F32) return static_cast<const float *>(base)[at];
    const uint32_t b = static_cast<const uint16_t *>(base)[at];
    return elem_unpack2<E>(b).x;
}

template <int E>
__device__ __forceinline__ void elem_store1(void *base, int64_t at, float v)
{
    if (E == GEMV_ELEM_F32)
        static_cast<float *>(base)[at] = v;
    else
        static_cast<uint16_t *>(base)[at] = static_cast<uint16_t>(elem_pack2<E>(v, 0.f));
}

// Elements [at, at + 8) of which the first n exist (the others read 0).  VEC:
// `at` is a multiple of 8 from a 16-byte aligned base (FP32: 32) and n is 8 or
// less than 1.
template <bool VEC, int E>
__device__ __forceinline__ void elem_load8(const void *base, int64_t at, int n, float (&x)[8])
{
    if (VEC) {
        if (n < 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
        } else if (E == GEMV_ELEM_F32) {
            uint32_t w[8];
            ld_global32(static_cast<const float *>(base) + at, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
            const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = elem_unpack2<E>(ws[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < n ? elem_load1<E>(base, at + i) : 0.f;
    }
}

template <bool VEC, int E>
__device__ __forceinline__ void elem_store8(void *base, int64_t at, int n, const float (&x)[8])
{
    if (VEC) {
        if (n < 8) return;
        if (E == GEMV_ELEM_F32) {
            st_global32(static_cast<float *>(base) + at, x);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) =
                make_uint4(elem_pack2<E>(x[0], x[1]), elem_pack2<E>(x[2], x[3]), elem_pack2<E>(x[4], x[5]),
                           elem_pack2<E>(x[6], x[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) elem_store1<E>(base, at + i, x[i]);
    }
}

}  // namespace mbg
