// ops_device.h -- loads, stores and reductions shared by the operators' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/emu_operators.h"

namespace emu {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// The index of this thread's wave in its workgroup, known to be the same for all its lanes.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// An element type and its vector of 8.  Rows start where the caller's
// leading dimension puts them, so vectors are accessed with the element's
// alignment only: the GPU runs in unaligned-access mode, where the same
// 16-byte instructions serve both (512 MiB: loads 6.5 TB/s aligned to 4
// bytes, 4.6 to 2; stores 4.3 and 3.4).
template <typename E>
struct Vec8 {
    typedef E type __attribute__((ext_vector_type(8)));
    typedef type mem __attribute__((aligned(sizeof(E))));
};
template <typename E>
using Raw8 = typename Vec8<E>::type;

template <typename E>
__device__ __forceinline__ Raw8<E> load8(const E *p)
{
    return *reinterpret_cast<const typename Vec8<E>::mem *>(p);
}
// ONCE: what is read or written once, and would not fit the last-level cache,
// passes by it (the launches say from where on, and what it measured).
template <bool ONCE, typename E>
__device__ __forceinline__ Raw8<E> load8(const E *p)
{
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const typename Vec8<E>::mem *>(p));
    return load8(p);
}
// (the vector's lower alignment belongs to its typedef and is lost where that
// is a template's argument, so the pointer is made here)
template <bool ONCE, typename E>
__device__ __forceinline__ void store8(E *p, const Raw8<E> &v)
{
    typedef typename Vec8<E>::mem mem;
    if constexpr (ONCE)
        __builtin_nontemporal_store(v, reinterpret_cast<mem *>(p));
    else
        *reinterpret_cast<mem *>(p) = v;
}
// f(std::true_type) or f(std::false_type)
template <typename F>
__device__ __forceinline__ void with_bool(bool b, F f)
{
    if (b)
        f(std::true_type{});
    else
        f(std::false_type{});
}
template <typename E>
__device__ __forceinline__ f32x8 widen(const Raw8<E> &v)
{
    return __builtin_convertvector(v, f32x8);
}

// Moves v down by k (0..8) elements, `fill` after.
__device__ __forceinline__ f32x8 moved(f32x8 v, int k, float fill = 0.0f)
{
    if (k & 1) v = f32x8{v[1], v[2], v[3], v[4], v[5], v[6], v[7], fill};
    if (k & 2) v = f32x8{v[2], v[3], v[4], v[5], v[6], v[7], fill, fill};
    if (k & 4) v = f32x8{v[4], v[5], v[6], v[7], fill, fill, fill, fill};
    if (k & 8) v = fill;
    return v;
}

// Elements c .. c + 7 of a row of n in two steps, so that all of a lane's
// loads are under way before the first is used: fetch8 reads them, or, where
// the row ends before, its last eight, with the same instruction; settle8
// then moves those into place, zeros past the end.
template <bool ONCE = false, typename E>
__device__ __forceinline__ Raw8<E> fetch8(const E *row, int c, int n)
{
    if (n >= 8) return load8<ONCE>(row + (c + 8 <= n ? c : n - 8));
    Raw8<E> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = c + i < n ? row[c + i] : (E)0.0f;
    return r;
}
__device__ __forceinline__ f32x8 settled(const f32x8 &v, int c, int n)
{
    if (n < 8 || c + 8 <= n) return v;
    return moved(v, c + 8 - n < 8 ? c + 8 - n : 8);
}
template <typename E>
__device__ __forceinline__ f32x8 settle8(const Raw8<E> &raw, int c, int n)
{
    return settled(widen<E>(raw), c, n);
}

// The same where the type is known at run time only (uniform over the launch).
struct AnyRaw8 {
    Raw8<float> v;  // binary32, or 8 elements of 16 bits in the first half
};
__device__ __forceinline__ AnyRaw8 fetch8_any(const void *row, int dtype, int c, int n)
{
    if (dtype == EMU_DT_FP32) return AnyRaw8{fetch8(static_cast<const float *>(row), c, n)};
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
    u16x8 h;
    const uint16_t *r = static_cast<const uint16_t *>(row);
    if (n >= 8) {
        typedef u16x8 mem __attribute__((aligned(2)));
        h = *reinterpret_cast<const mem *>(r + (c + 8 <= n ? c : n - 8));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = c + i < n ? r[c + i] : (uint16_t)0;
    }
    const f32x4 q = __builtin_bit_cast(f32x4, h);
    return AnyRaw8{f32x8{q[0], q[1], q[2], q[3], 0.0f, 0.0f, 0.0f, 0.0f}};
}
__device__ __forceinline__ f32x8 settle8_any(const AnyRaw8 &raw, int dtype, int c, int n)
{
    f32x8 v = raw.v;
    if (dtype != EMU_DT_FP32) {
        typedef float f32x4 __attribute__((ext_vector_type(4)));
        const f32x4 q = {v[0], v[1], v[2], v[3]};
        v = dtype == EMU_DT_BF16 ? widen<__bf16>(__builtin_bit_cast(Raw8<__bf16>, q))
                                 : widen<_Float16>(__builtin_bit_cast(Raw8<_Float16>, q));
    }
    return settled(v, c, n);
}

// Elements c .. c + 7, those past n (or all of them) not stored; past the end in pieces of 4, 2 and 1.
template <bool ONCE = false, typename E>
__device__ __forceinline__ void store8_row(E *row, int c, int n, f32x8 v)
{
    E *p = row + c;
    if (c + 8 <= n) {
        store8<ONCE>(p, __builtin_convertvector(v, Raw8<E>));
        return;
    }
    const int left = c < n ? n - c : 0;
    if (left & 4) {
        typedef E e4 __attribute__((ext_vector_type(4)));
        typedef e4 mem __attribute__((aligned(sizeof(E))));
        *reinterpret_cast<mem *>(p) = e4{(E)v[0], (E)v[1], (E)v[2], (E)v[3]};
        p += 4;
        v = moved(v, 4);
    }
    if (left & 2) {
        typedef E e2 __attribute__((ext_vector_type(2)));
        typedef e2 mem __attribute__((aligned(sizeof(E))));
        *reinterpret_cast<mem *>(p) = e2{(E)v[0], (E)v[1]};
        p += 2;
        v = moved(v, 2);
    }
    if (left & 1) *p = (E)v[0];
}

// Reductions over a wave's 64 lanes, all of them active; every lane gets the
// result, the same bits in each (f(a, b) and f(b, a) are the same).  Lanes
// 1, 2, 4 and 8 apart meet by DPP (the mirrors do for 4 and 8 once the lanes
// between agree), rows of 16 and halves by swaps: no step goes through LDS.
template <typename T, typename F>
__device__ __forceinline__ T by_words(const T &v, F f)
{
    constexpr int N = sizeof(T) / 4;
    struct Words {
        uint32_t w[N];
    };
    Words x = __builtin_bit_cast(Words, v);
#pragma unroll
    for (int i = 0; i < N; ++i) x.w[i] = f(x.w[i]);
    return __builtin_bit_cast(T, x);
}
template <int CTRL, typename T>
__device__ __forceinline__ T by_dpp(const T &v)
{
    return by_words(v, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, CTRL, 0xF, 0xF, true); });
}
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, F f)
{
    v = f(v, by_dpp<0xB1>(v));   // quad_perm 1 0 3 2
    v = f(v, by_dpp<0x4E>(v));   // quad_perm 2 3 0 1
    v = f(v, by_dpp<0x141>(v));  // row_half_mirror
    v = f(v, by_dpp<0x140>(v));  // row_mirror
    v = f(by_words(v, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_permlane16_swap(w, w, false, false)[0]; }),
          by_words(v, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_permlane16_swap(w, w, false, false)[1]; }));
    return f(by_words(v, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_permlane32_swap(w, w, false, false)[0]; }),
             by_words(v, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_permlane32_swap(w, w, false, false)[1]; }));
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v)
{
    return wave_reduce(v, [](T a, T b) { return a + b; });
}
// A NaN in any lane wins.
__device__ __forceinline__ float wave_max(float v)
{
    return wave_reduce(v, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
}

// Over the W waves of a row, through W words of LDS; W = 1 needs neither LDS
// nor a barrier.  Two reductions in a row need two arrays.
template <int W, typename T>
__device__ __forceinline__ T row_sum(T v, T *lds, int wave, int lane)
{
    v = wave_sum(v);
    if (W == 1) return v;
    if (lane == 0) lds[wave] = v;
    __syncthreads();
    T s = lds[0];
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
