// emu_norm.hip -- emu_add_rms_norm_quant and its gradient.
//
// Forward: v = x + residual, y = v r w with r = 1 / sqrt(mean(v^2) + eps),
// codes of y / scale.  Each value is needed three times (for the mean, for
// the row's largest |y|, for its code), so a row is held in registers and
// read once; the weight is read again for the codes, since to hold the products'
// rests instead takes a workgroup off each CU (16384 x 8192: 176 us, 163 now, 5.8 TB/s).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops_device.h"
#include "ops_internal.h"

namespace emu {

namespace {

// A row's way from v to codes: u = v 2^e w with 2^e near r (the power of two
// changes no digit and keeps v w from overflowing), held with what its
// rounding cut off, then u f with f = r 2^-e / scale, made in 64 bits and kept
// as the sum of two binary32 values.  Where the product lies on a border it is
// rounded to odd, so that the code's rounding after it is that of the whole
// value and no code falls to the other side (rounded to nearest, some one in
// 2 million does; this costs 2%), and no division is left.  A scale under 2^-100, whose f may
// overflow, divides.
// Where r is 0 (the squares of the row overflowed) the power is 0 and the rest
// 1: finite values become 0 whatever their weights, an infinity NaN.
struct Factor {
    double whole;         // r 2^-e
    float power, hi, lo;  // 2^e; f
    float rest, scale;    // r 2^-e
};
__device__ __forceinline__ Factor factor_of(double r)
{
    Factor f;
    const int e = r > 0.0 && r < 1e300 ? __builtin_amdgcn_frexp_exp(r) : 0;
    f.power = r == 0.0 ? 0.0f : __builtin_amdgcn_ldexpf(1.0f, e);
    f.whole = r == 0.0 ? 1.0 : __builtin_amdgcn_ldexp(r, -e);
    f.rest = (float)f.whole;
    f.hi = f.lo = f.scale = 0.0f;
    return f;
}
__device__ __forceinline__ void set_scale(Factor &f, float scale)
{
    const double q = f.whole / (double)scale;
    f.hi = (float)q;
    f.lo = (float)(q - (double)f.hi);
    f.scale = scale;
}

// Cut to +-Q; the comparisons keep a NaN (fmin / fmax drop it).
template <int Q>
__device__ __forceinline__ float cut(float v)
{
    constexpr float most = Q == EMU_DT_INT8 ? 127.0f : Q == EMU_DT_E4M3FN ? 448.0f : 57344.0f;
    return v > most ? most : v < -most ? -most : v;
}

// u f rounded to odd: to the neighbour with an odd last digit where it is not exact.
__device__ __forceinline__ float product_to_odd(float u, float rest, const Factor &f)
{
    // (an infinite u has no rest)
    const float t = __builtin_fabsf(u) < INFINITY ? __builtin_fmaf(u, f.lo, rest * f.hi) : 0.0f;
    const float y = __builtin_fmaf(u, f.hi, t);
    const float off = __builtin_fmaf(u, f.hi, -y) + t;  // the value less y
    const uint32_t bits = __float_as_uint(y);
    const uint32_t toward = bits - ((__float_as_uint(off) ^ bits) >> 31);  // the value lies beyond it, away from 0
    const bool plain = __builtin_fabsf(y) > 1e-30f && __builtin_fabsf(y) < INFINITY;  // (below, the code is 0 anyway)
    return off != 0.0f && plain ? __uint_as_float(toward | 1) : y;
}

// 8 codes of u + rest, rounded to nearest even.
template <int Q>
__device__ __forceinline__ uint2 codes8(const f32x8 &u, const f32x8 &rest, const Factor &f)
{
    f32x8 y;
    if (f.scale >= 7.888609052e-31f) {
        // A product to nearest has its code on the wrong side only if it lies
        // on a border, whose last 19 (int8: 16) bits are 0: where any does
        // (an infinity and a NaN of it too), all are made again.  To round
        // every one to odd costs 16384 x 8192 10%.
        uint32_t least = ~0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = __builtin_fmaf(u[i], f.hi, __builtin_fmaf(u[i], f.lo, rest[i] * f.hi));
            const uint32_t last = __float_as_uint(y[i]) & (Q == EMU_DT_INT8 ? 0xFFFFu : 0x7FFFFu);
            least = last < least ? last : least;
        }
        if (__any(least == 0)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = product_to_odd(u[i], rest[i], f);
        }
    } else {
        y = u * f.rest / f.scale;
    }
    uint32_t r[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = cut<Q>(y[4 * j + i]);
        if (Q == EMU_DT_INT8) {
            uint32_t b = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float k = c[i] == c[i] ? c[i] : 0.0f;
                b |= ((uint32_t)(int)rintf(k) & 0xFFu) << (8 * i);
            }
            r[j] = b;
        } else if (Q == EMU_DT_E4M3FN) {
            int b = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
            r[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], b, true);
        } else {
            int b = __builtin_amdgcn_cvt_pk_bf8_f32(c[0], c[1], 0, false);
            r[j] = (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c[2], c[3], b, true);
        }
    }
    return make_uint2(r[0], r[1]);
}

template <typename T>
struct Bytes {
    T v;
} __attribute__((packed, aligned(1)));

template <bool ONCE = false>
__device__ __forceinline__ void store_codes(uint8_t *row, int c, int n, const uint2 &r)
{
    uint64_t v = (uint64_t)r.y << 32 | r.x;
    uint8_t *p = row + c;
    if (c + 8 <= n) {
        if (ONCE)
            __builtin_nontemporal_store(v, &reinterpret_cast<Bytes<uint64_t> *>(p)->v);
        else
            reinterpret_cast<Bytes<uint64_t> *>(p)->v = v;
        return;
    }
    const int left = c < n ? n - c : 0;
    if (left & 4) {
        reinterpret_cast<Bytes<uint32_t> *>(p)->v = (uint32_t)v;
        p += 4;
        v >>= 32;
    }
    if (left & 2) {
        reinterpret_cast<Bytes<uint16_t> *>(p)->v = (uint16_t)v;
        p += 2;
        v >>= 16;
    }
    if (left & 1) *p = (uint8_t)v;
}

__device__ __forceinline__ uint2 codes8_any(int q_dtype, const f32x8 &u, const f32x8 &rest, const Factor &f)
{
    if (q_dtype == EMU_DT_INT8) return codes8<EMU_DT_INT8>(u, rest, f);
    if (q_dtype == EMU_DT_E4M3FN) return codes8<EMU_DT_E4M3FN>(u, rest, f);
    return codes8<EMU_DT_E5M2>(u, rest, f);
}
// u and rest of 8 values
__device__ __forceinline__ f32x8 scaled(const f32x8 &v, const f32x8 &w, const Factor &f, f32x8 &rest)
{
    const f32x8 x = v * f.power, u = x * w;
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = __builtin_fmaf(x[i], w[i], -u[i]);
    return u;
}

__device__ __forceinline__ float most_of(int q_dtype)
{
    return q_dtype == EMU_DT_INT8 ? 127.0f : q_dtype == EMU_DT_E4M3FN ? 448.0f : 57344.0f;
}

// Smallest own scale: a row of zeros divides by it and gives zeros.
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126
__device__ __forceinline__ float own_scale(float most, const Factor &f, int q_dtype)
{
    return __builtin_elementwise_maximum(most * f.rest / most_of(q_dtype), kLeastScale);
}

// W waves hold one row, VPT vectors of 8 values in each lane: n <= W * VPT * 512.
// R: no residual, or its element type.
struct NoRes {};
template <typename X, typename R, int W, int VPT>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_rows(NormParams p)
{
    constexpr bool kRes = !__is_same(R, NoRes);
    __shared__ double sums[W];
    __shared__ float maxima[W];
    const int lane = threadIdx.x & 63;
    const int wave = W == 1 ? 0 : wave_index();
    const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + wave_index() : blockIdx.x;
    if (W == 1 && row >= p.T) return;
    const int n = (int)p.n;
    __builtin_assume(n >= 8);
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    const int c0 = (wave * 64 + lane) * 8;

    f32x8 v[VPT];
    {
        Raw8<X> xr[VPT];
        Raw8<std::conditional_t<kRes, R, X>> rr[VPT];
        with_bool(p.once, [&](auto once) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = c0 + i * (W * 512);
                xr[i] = fetch8<once()>(x, c, n);
                if constexpr (kRes) rr[i] = fetch8<once()>(static_cast<const R *>(p.res) + row * p.ldres, c, n);
            }
        });
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = c0 + i * (W * 512);
            v[i] = settle8<X>(xr[i], c, n);
            if constexpr (kRes) v[i] += settle8<R>(rr[i], c, n);
        }
    }

    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[i][j] * v[i][j];
    const double r = 1.0 / sqrt(row_sum<W>((double)s, sums, wave, lane) / (double)n + (double)p.eps);

    if constexpr (kRes) {
        if (p.h) {
            R *h = static_cast<R *>(p.h) + row * p.ldh;
            with_bool(p.once, [&](auto once) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) store8_row<once()>(h, c0 + i * (W * 512), n, v[i]);
            });
        }
    }
    Factor f = factor_of(r);
    const auto weight = [&](int c) { return settle8_any(fetch8_any(p.weight, p.w_dtype, c, n), p.w_dtype, c, n); };
    float scale;
    if (p.scale) {
        scale = *p.scale;
    } else {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const f32x8 u = v[i] * f.power * weight(c0 + i * (W * 512));
#pragma unroll
            for (int j = 0; j < 8; ++j) a = __builtin_elementwise_maximum(a, __builtin_fabsf(u[j]));
        }
        scale = own_scale(row_max<W>(a, maxima, wave, lane), f, p.q_dtype);
        if (wave == 0 && lane == 0) p.row_scales[row] = scale;
    }
    set_scale(f, scale);
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.ldq;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = c0 + i * (W * 512);
        if (c >= n) continue;
        f32x8 rest;
        const f32x8 u = scaled(v[i], weight(c), f, rest);
        const uint2 codes = codes8_any(p.q_dtype, u, rest, f);
        with_bool(p.once, [&](auto once) { store_codes<once()>(q, c, n, codes); });
    }
}

// Rows too long for registers (or of fewer than 8 values): three passes over
// the row, by one workgroup.
// h is stored in the last one, after its element's last load, since it may be
// the residual.
template <typename X, typename R>
__global__ __launch_bounds__(1024) void norm_long_rows(NormParams p)
{
    constexpr bool kRes = !__is_same(R, NoRes);
    __shared__ double sums[16];
    __shared__ float maxima[16];
    const int lane = threadIdx.x & 63, wave = wave_index();
    const int64_t row = blockIdx.x;
    const int n = (int)p.n;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    const auto weight = [&](int c) { return settle8_any(fetch8_any(p.weight, p.w_dtype, c, n), p.w_dtype, c, n); };
    const auto value = [&](int c) {
        const Raw8<X> xr = fetch8(x, c, n);
        if constexpr (kRes) {
            const Raw8<R> rr = fetch8(static_cast<const R *>(p.res) + row * p.ldres, c, n);
            return settle8<X>(xr, c, n) + settle8<R>(rr, c, n);
        } else {
            return settle8<X>(xr, c, n);
        }
    };
    double s = 0.0;
    for (int c = threadIdx.x * 8; c < n; c += 8192) {
        const f32x8 v = value(c);
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t += v[j] * v[j];
        s += (double)t;
    }
    const double r = 1.0 / sqrt(row_sum<16>(s, sums, wave, lane) / (double)n + (double)p.eps);
    Factor f = factor_of(r);
    float scale;
    if (p.scale) {
        scale = *p.scale;
    } else {
        float a = 0.0f;
        for (int c = threadIdx.x * 8; c < n; c += 8192) {
            const f32x8 u = value(c) * f.power * weight(c);
#pragma unroll
            for (int j = 0; j < 8; ++j) a = __builtin_elementwise_maximum(a, __builtin_fabsf(u[j]));
        }
        scale = own_scale(row_max<16>(a, maxima, wave, lane), f, p.q_dtype);
        if (threadIdx.x == 0) p.row_scales[row] = scale;
    }
    set_scale(f, scale);
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.ldq;
    for (int c = threadIdx.x * 8; c < n; c += 8192) {
        const f32x8 v = value(c);
        if constexpr (kRes) {
            if (p.h) store8_row(static_cast<R *>(p.h) + row * p.ldh, c, n, v);
        }
        f32x8 rest;
        const f32x8 u = scaled(v, weight(c), f, rest);
        store_codes(q, c, n, codes8_any(p.q_dtype, u, rest, f));
    }
}

// Few waves with more values each need fewer barriers, many with few have
// more rows in flight: 16384 x 2048 takes 44 us on 2 waves of 16 values a
// lane, 62 on 4 of 8; 4096 x 16384 98 us on 8 of 32, 117 on 16 of 16; 16384 x
// 4096 84 us on 4 of 16, 92 on 2 of 32.
template <typename X, typename R>
hipError_t launch_norm_of(const NormParams &p, hipStream_t stream)
{
    const int64_t n = p.n, T = p.T;
    const dim3 rows((unsigned)T), rows4((unsigned)((T + 3) / 4));
    if (n < 8 || n > 16384)
        hipLaunchKernelGGL((norm_long_rows<X, R>), rows, dim3(1024), 0, stream, p);
    else if (n <= 512)
        hipLaunchKernelGGL((norm_rows<X, R, 1, 1>), rows4, dim3(256), 0, stream, p);
    else if (n <= 1024)
        hipLaunchKernelGGL((norm_rows<X, R, 1, 2>), rows4, dim3(256), 0, stream, p);
    else if (n <= 2048)
        hipLaunchKernelGGL((norm_rows<X, R, 2, 2>), rows, dim3(128), 0, stream, p);
    else if (n <= 4096)
        hipLaunchKernelGGL((norm_rows<X, R, 4, 2>), rows, dim3(256), 0, stream, p);
    else if (n <= 8192)
        hipLaunchKernelGGL((norm_rows<X, R, 8, 2>), rows, dim3(512), 0, stream, p);
    else
        hipLaunchKernelGGL((norm_rows<X, R, 8, 4>), rows, dim3(512), 0, stream, p);
    return hipGetLastError();
}

template <typename X>
hipError_t launch_norm_x(int res_dtype, const NormParams &p, hipStream_t stream)
{
    if (!p.res) return launch_norm_of<X, NoRes>(p, stream);
    if (res_dtype == EMU_DT_FP32) return launch_norm_of<X, float>(p, stream);
    return launch_norm_of<X, X>(p, stream);
}

// ---- the gradient ------------------------------------------------------
//
// grad_in = r (u - n mean(u n)) + grad_h needs two sums of its row first, and
// grad_weight adds g n over all rows.  A workgroup takes rows blockIdx,
// blockIdx + parts, ... of the grid, holds a row in registers while its two
// sums are made (together, one barrier), and adds its rows' g n in binary32
// registers; it stores them once, and grad_weight_kernel adds the parts.
// Enough workgroups share a CU for one's loads to cover the other's sums: to
// read the next row ahead as well gains nothing.  8192 x 8192 bf16 with
// grad_h: 101 + 5 us, 5.1 TB/s, the rate of a large copy.

// A part's place in the workspace, whole cache lines (1023 x 1925: 8.0 us, 9.0 without).
__host__ __device__ constexpr int64_t part_ld(int64_t n) { return (n + 31) / 32 * 32; }

// D: grad_h's type.  W waves hold a row, as in norm_rows; a workgroup has ROWS
// rows at a time, and the sums of all of them go into its one part.
template <typename G, typename H, typename D, int W, int VPT, int ROWS>
__global__ __launch_bounds__(W * ROWS * 64, 4) void norm_grad_rows(NormGradParams p, int64_t parts)
{
    __shared__ float2 lds[2][ROWS][W];
    __shared__ float share[ROWS > 1 ? (ROWS - 1) * W * VPT * 512 : 1];
    const int lane = threadIdx.x & 63, wave = wave_index() % W, group = wave_index() / W;
    const int n = (int)p.n;
    __builtin_assume(n >= 8);
    const int c0 = (wave * 64 + lane) * 8;

    f32x8 gw[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) gw[i] = 0.0f;
    const auto weight = [&](int c) { return settle8_any(fetch8_any(p.weight, p.w_dtype, c, n), p.w_dtype, c, n); };
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * ROWS; first < p.T; first += parts * ROWS, turn ^= 1) {
        // (a group past the last row goes along to the barriers)
        const bool mine = first + group < p.T;
        const int64_t row = mine ? first + group : p.T - 1;
        f32x8 gv[VPT], hv[VPT];
        Raw8<G> gr[VPT];
        Raw8<H> hr[VPT];
        Raw8<D> dr[VPT];
        with_bool(p.once, [&](auto once) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = c0 + i * (W * 512);
                gr[i] = fetch8<once()>(static_cast<const G *>(p.g) + row * p.ldg, c, n);
                hr[i] = fetch8<once()>(static_cast<const H *>(p.h) + row * p.ldh, c, n);
                // (before the first store, since it may be grad_in)
                if (p.gh) dr[i] = fetch8<once()>(static_cast<const D *>(p.gh) + row * p.ldgh, c, n);
            }
        });
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = c0 + i * (W * 512);
            gv[i] = settle8<G>(gr[i], c, n);
            hv[i] = settle8<H>(hr[i], c, n);
            const f32x8 u = gv[i] * weight(c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sq += hv[i][j] * hv[i][j];
                dot += u[j] * hv[i][j];
            }
        }
        sq = wave_sum(sq);
        dot = wave_sum(dot);
        if (W > 1) {
            if (lane == 0) lds[turn][group][wave] = make_float2(sq, dot);
            __syncthreads();  // two arrays in turn: a wave is at most one barrier ahead
            sq = dot = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                sq += lds[turn][group][i].x;
                dot += lds[turn][group][i].y;
            }
        }
        if (ROWS > 1 && !mine) continue;
        const float r = 1.0f / sqrtf(sq / (float)n + p.eps);
        const float mean = dot * r / (float)n;
        G *gi = static_cast<G *>(p.gi) + row * p.ldgi;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = c0 + i * (W * 512);
            const f32x8 nv = hv[i] * r;
            gw[i] += gv[i] * nv;
            f32x8 d = (gv[i] * weight(c) - nv * mean) * r;
            if (p.gh) d += settle8<D>(dr[i], c, n);
            store8_row(gi, c, n, d);
        }
    }
    if (ROWS > 1) {  // the groups' sums, in their order
        float *at = share + wave * VPT * 512 + lane;
        if (group) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) at[(group - 1) * W * VPT * 512 + (i * 8 + j) * 64] = gw[i][j];
        }
        __syncthreads();
        if (group) return;
        for (int o = 0; o < ROWS - 1; ++o)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) gw[i][j] += at[o * W * VPT * 512 + (i * 8 + j) * 64];
    }
    float *part = p.part + blockIdx.x * part_ld(n);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        store8_row(part, c0 + i * (W * 512), n, gw[i]);
}

// Rows too long for registers (or of fewer than 8 values): the row is read
// twice, and the workgroup's own
// part in the workspace takes the place of the sums in registers.
template <typename G, typename H>
__global__ __launch_bounds__(1024) void norm_grad_long_rows(NormGradParams p, int64_t parts)
{
    __shared__ float lds[2][2][16];
    const int lane = threadIdx.x & 63, wave = wave_index();
    const int n = (int)p.n;
    float *part = p.part + blockIdx.x * part_ld(n);
    const auto weight = [&](int c) { return settle8_any(fetch8_any(p.weight, p.w_dtype, c, n), p.w_dtype, c, n); };
    int turn = 0;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.T; row += parts, turn ^= 1, first = false) {
        const G *g = static_cast<const G *>(p.g) + row * p.ldg;
        const H *h = static_cast<const H *>(p.h) + row * p.ldh;
        float sq = 0.0f, dot = 0.0f;
        for (int c = threadIdx.x * 8; c < n; c += 8192) {
            const f32x8 gv = settle8<G>(fetch8(g, c, n), c, n), hv = settle8<H>(fetch8(h, c, n), c, n), w = weight(c);
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a += hv[j] * hv[j];
                b += gv[j] * w[j] * hv[j];
            }
            sq += a;
            dot += b;
        }
        sq = row_sum<16>(sq, lds[turn][0], wave, lane);
        dot = row_sum<16>(dot, lds[turn][1], wave, lane);
        const float r = 1.0f / sqrtf(sq / (float)n + p.eps);
        const float mean = dot * r / (float)n;
        for (int c = threadIdx.x * 8; c < n; c += 8192) {
            const f32x8 gv = settle8<G>(fetch8(g, c, n), c, n), nv = settle8<H>(fetch8(h, c, n), c, n) * r;
            f32x8 d = (gv * weight(c) - nv * mean) * r;
            if (p.gh) {
                const char *gh = static_cast<const char *>(p.gh) + row * p.ldgh * (p.gh_dtype == EMU_DT_FP32 ? 4 : 2);
                d += settle8_any(fetch8_any(gh, p.gh_dtype, c, n), p.gh_dtype, c, n);
            }
            f32x8 t = gv * nv;
            if (!first) t += settle8<float>(fetch8(part, c, n), c, n);
            store8_row(part, c, n, t);
            store8_row(static_cast<G *>(p.gi) + row * p.ldgi, c, n, d);
        }
    }
}

// grad_weight: 32 columns a workgroup, whose 32 rows of threads each add every
// 32nd part, joined in their order.  (16 or 64 columns: the same up to 4,096,
// 7.6 and 4.8 us against 4.9 at 8192.)
__global__ __launch_bounds__(1024) void grad_weight_kernel(NormGradParams p, int64_t parts)
{
    constexpr int COLS = 32, ROWS = 1024 / COLS;
    __shared__ float lds[ROWS][COLS + 1];
    const int col = threadIdx.x % COLS, row = threadIdx.x / COLS;
    const int64_t c = (int64_t)blockIdx.x * COLS + col, ld = part_ld(p.n);
    float s = 0.0f;
    if (c < p.n) {
#pragma unroll 8
        for (int64_t i = row; i < parts; i += ROWS) s += p.part[i * ld + c];
    }
    lds[row][col] = s;
    __syncthreads();
    if (row || c >= p.n) return;
#pragma unroll 16
    for (int i = 1; i < ROWS; ++i) s += lds[i][col];
    if (p.w_dtype == EMU_DT_BF16)
        static_cast<__bf16 *>(p.gw)[c] = (__bf16)s;
    else if (p.w_dtype == EMU_DT_FP16)
        static_cast<_Float16 *>(p.gw)[c] = (_Float16)s;
    else
        static_cast<float *>(p.gw)[c] = s;
}

// Rows at a time in a workgroup.
int64_t grad_rows_at_once(int64_t n) { return n < 8 ? 1 : n <= 1024 ? 4 : n <= 4096 ? 2 : 1; }

template <typename G, typename H, typename D, int W, int VPT, int ROWS>
void launch_grad_rows(const NormGradParams &p, int64_t parts, hipStream_t stream)
{
    hipLaunchKernelGGL((norm_grad_rows<G, H, D, W, VPT, ROWS>), dim3((unsigned)parts), dim3(W * ROWS * 64), 0, stream, p, parts);
}

template <typename G, typename H, typename D>
void launch_norm_grad_of(const NormGradParams &p, int64_t parts, hipStream_t stream)
{
    const int64_t n = p.n;
    if (n < 8 || n > 16384)
        hipLaunchKernelGGL((norm_grad_long_rows<G, H>), dim3((unsigned)parts), dim3(1024), 0, stream, p, parts);
    else if (n <= 512)
        launch_grad_rows<G, H, D, 1, 1, 4>(p, parts, stream);
    else if (n <= 1024)
        launch_grad_rows<G, H, D, 1, 2, 4>(p, parts, stream);
    else if (n <= 2048)
        launch_grad_rows<G, H, D, 4, 1, 2>(p, parts, stream);
    else if (n <= 4096)
        launch_grad_rows<G, H, D, 8, 1, 2>(p, parts, stream);
    else if (n <= 8192)
        launch_grad_rows<G, H, D, 8, 2, 1>(p, parts, stream);
    else
        launch_grad_rows<G, H, D, 16, 2, 1>(p, parts, stream);
}

template <typename G, typename H>
void launch_norm_grad_gh(const NormGradParams &p, int64_t parts, hipStream_t stream)
{
    if (p.gh && p.gh_dtype == EMU_DT_FP32)
        launch_norm_grad_of<G, H, float>(p, parts, stream);
    else
        launch_norm_grad_of<G, H, G>(p, parts, stream);
}

}  // namespace

// Workgroups of the gradient, each with a part of grad_weight in the
// workspace: 16 waves for each CU (rows of up to 1,024 values take four for
// that, which is done only where each workgroup gets 8 turns), and no more than have rows.
int64_t norm_grad_part_ld(int64_t n) { return part_ld(n); }

int64_t norm_grad_parts(int64_t T, int64_t n)
{
    const int64_t at_once = grad_rows_at_once(n), most = (T + at_once - 1) / at_once;
    int64_t parts = n <= 1024 ? 1024 : n <= 2048 ? 512 : n <= 4096 ? 256 : n <= 8192 ? 512 : 256;
    if (parts > 512 && parts > T / 8) parts = T / 8 > 512 ? T / 8 : 512;
    return most < parts ? most : parts;
}

hipError_t launch_norm_grad(int g_dtype, int h_dtype, const NormGradParams &params, hipStream_t stream)
{
    NormGradParams p = params;
    const int64_t size = (g_dtype == EMU_DT_FP32 ? 4 : 2) * (p.gh ? 3 : 2) + (h_dtype == EMU_DT_FP32 ? 4 : 2);
    // (8192 x 8192 bf16: 100 us past the cache, 110 through it)
    p.once = p.T * p.n * size > kOnceBytes;
    const int64_t parts = norm_grad_parts(p.T, p.n);
    if (parts > 0) {
        if (g_dtype == EMU_DT_FP32)
            launch_norm_grad_gh<float, float>(p, parts, stream);
        else if (g_dtype == EMU_DT_BF16 && h_dtype == EMU_DT_FP32)
            launch_norm_grad_gh<__bf16, float>(p, parts, stream);
        else if (g_dtype == EMU_DT_BF16)
            launch_norm_grad_gh<__bf16, __bf16>(p, parts, stream);
        else if (h_dtype == EMU_DT_FP32)
            launch_norm_grad_gh<_Float16, float>(p, parts, stream);
        else
            launch_norm_grad_gh<_Float16, _Float16>(p, parts, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(grad_weight_kernel, dim3((unsigned)((p.n + 31) / 32)), dim3(1024), 0, stream, p, parts);
    return hipGetLastError();
}

hipError_t launch_norm(int x_dtype, int res_dtype, const NormParams &params, hipStream_t stream)
{
    NormParams p = params;
    const int64_t res = !p.res ? 0 : res_dtype == EMU_DT_FP32 ? 4 : 2;
    // (after x's producer, 8192 x 8192 bf16: 79 us past the cache, 84 through
    // it; 4096 x 8192: 38 and 44)
    p.once = p.T * p.n * ((x_dtype == EMU_DT_FP32 ? 4 : 2) + res + (p.h ? res : 0) + 1) > kOnceBytes;
    if (x_dtype == EMU_DT_BF16) return launch_norm_x<__bf16>(res_dtype, p, stream);
    if (x_dtype == EMU_DT_FP16) return launch_norm_x<_Float16>(res_dtype, p, stream);
    return launch_norm_x<float>(res_dtype, p, stream);
}

}  // namespace emu
