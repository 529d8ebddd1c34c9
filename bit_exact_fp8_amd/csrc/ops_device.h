// ops_device.h -- loads, stores and reductions shared by the operators' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/emu_operators.h"

namespace emu {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// An element type and its vector of 8.  Rows start where the caller's
// leading dimension puts them, so vectors are accessed with the element's
// alignment only: the GPU runs in unaligned-access mode, where the same
// 16-byte instructions serve both.
template <typename E>
struct Vec8 {
    typedef E type __attribute__((ext_vector_type(8)));
    typedef type mem __attribute__((aligned(sizeof(E))));
};

template <typename E>
__device__ __forceinline__ f32x8 load8(const E *p)
{
    const typename Vec8<E>::type v = *reinterpret_cast<const typename Vec8<E>::mem *>(p);
    return __builtin_convertvector(v, f32x8);
}

// The first `valid` (0..8) of 8 elements; the rest are `fill`.
template <typename E>
__device__ __forceinline__ f32x8 load8_part(const E *p, int valid, float fill = 0.0f)
{
    f32x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = i < valid ? (float)p[i] : fill;
    return r;
}

// As stored, for values that wait in registers before they are used.
template <typename E>
__device__ __forceinline__ typename Vec8<E>::type load8_raw(const E *row, int64_t c, int64_t n)
{
    if (c + 8 <= n) return *reinterpret_cast<const typename Vec8<E>::mem *>(row + c);
    typename Vec8<E>::type r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = c + i < n ? row[c + i] : (E)0.0f;
    return r;
}

template <typename E>
__device__ __forceinline__ f32x8 load8_row(const E *row, int64_t c, int64_t n, float fill = 0.0f)
{
    if (c + 8 <= n) return load8(row + c);
    return load8_part(row + c, c < n ? (int)(n - c) : 0, fill);
}

// The same with the type known at run time only (uniform over the launch).
__device__ __forceinline__ f32x8 load8_any(const void *row, int dtype, int64_t c, int64_t n)
{
    if (dtype == EMU_DT_BF16) return load8_row(static_cast<const __bf16 *>(row), c, n);
    if (dtype == EMU_DT_FP16) return load8_row(static_cast<const _Float16 *>(row), c, n);
    return load8_row(static_cast<const float *>(row), c, n);
}

template <typename E>
__device__ __forceinline__ void store8_row(E *row, int64_t c, int64_t n, const f32x8 &v)
{
    const typename Vec8<E>::type r = __builtin_convertvector(v, typename Vec8<E>::type);
    if (c + 8 <= n) {
        *reinterpret_cast<typename Vec8<E>::mem *>(row + c) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n) row[c + i] = r[i];
    }
}

// Reductions over a wave's 64 lanes; every lane gets the result, the same
// bits in each (the butterfly's sums are symmetric).
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
// A NaN in any lane wins.
__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v = __builtin_elementwise_maximum(v, __shfl_xor(v, o));
    return v;
}

// Over the W waves of a row, through W words of LDS; W = 1 needs neither LDS
// nor a barrier.  Two reductions in a row need two arrays.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *lds, int wave, int lane)
{
    v = wave_sum(v);
    if (W == 1) return v;
    if (lane == 0) lds[wave] = v;
    __syncthreads();
    float s = lds[0];
#pragma unroll
    for (int i = 1; i < W; ++i) s += lds[i];
    return s;
}
template <int W>
__device__ __forceinline__ float row_max(float v, float *lds, int wave, int lane)
{
    v = wave_max(v);
    if (W == 1) return v;
    if (lane == 0) lds[wave] = v;
    __syncthreads();
    float s = lds[0];
#pragma unroll
    for (int i = 1; i < W; ++i) s = __builtin_elementwise_maximum(s, lds[i]);
    return s;
}

}  // namespace emu
