// emu_norm.hip -- emu_add_rms_norm_quant and its gradient.
//
// Forward: v = x + residual, y = v r w with r = 1 / sqrt(mean(v^2) + eps),
// codes of y / scale.  Each value is needed three times (for the mean, for
// the row's largest |y|, for its code), so a row is held in registers and
// read once.
#include <hip/hip_runtime.h>

#include "ops_device.h"
#include "ops_internal.h"

namespace emu {

namespace {

// 8 codes of y / scale, cut to +-Q and rounded to nearest even.  The division
// is IEEE's, not a product with the reciprocal: codes are those of the
// definition also next to a tie, and at some 10 instructions a value it hides
// behind the row's loads.  The comparisons keep a NaN (fmin / fmax drop it).
template <int Q>
__device__ __forceinline__ float cut(float v, float scale)
{
    constexpr float most = Q == EMU_DT_INT8 ? 127.0f : Q == EMU_DT_E4M3FN ? 448.0f : 57344.0f;
    v = v / scale;
    return v > most ? most : v < -most ? -most : v;
}

template <int Q>
__device__ __forceinline__ uint2 codes8(const f32x8 &y, float scale)
{
    uint32_t r[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = cut<Q>(y[4 * j + i], scale);
        if (Q == EMU_DT_INT8) {
            uint32_t b = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = c[i] == c[i] ? c[i] : 0.0f;
                b |= ((uint32_t)(int)rintf(f) & 0xFFu) << (8 * i);
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

struct uint2_u {
    uint32_t x, y;
} __attribute__((packed, aligned(1)));

__device__ __forceinline__ void store_codes(uint8_t *row, int64_t c, int64_t n, const uint2 &r)
{
    if (c + 8 <= n) {
        *reinterpret_cast<uint2_u *>(row + c) = uint2_u{r.x, r.y};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n) row[c + i] = (uint8_t)((i < 4 ? r.x : r.y) >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ uint2 codes8_any(int q_dtype, const f32x8 &y, float scale)
{
    if (q_dtype == EMU_DT_INT8) return codes8<EMU_DT_INT8>(y, scale);
    if (q_dtype == EMU_DT_E4M3FN) return codes8<EMU_DT_E4M3FN>(y, scale);
    return codes8<EMU_DT_E5M2>(y, scale);
}

__device__ __forceinline__ float most_of(int q_dtype)
{
    return q_dtype == EMU_DT_INT8 ? 127.0f : q_dtype == EMU_DT_E4M3FN ? 448.0f : 57344.0f;
}

// Smallest own scale: a row of zeros divides by it and gives zeros.
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126

// W waves hold one row, VPT vectors of 8 values in each lane: n <= W * VPT * 512.
// R: no residual, or its element type.
struct NoRes {};
template <typename X, typename R, int W, int VPT>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_rows(NormParams p)
{
    constexpr bool kRes = !__is_same(R, NoRes);
    __shared__ float lds[2][W];
    const int lane = threadIdx.x & 63;
    const int wave = W == 1 ? 0 : threadIdx.x >> 6;
    const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (W == 1 && row >= p.T) return;
    const int64_t n = p.n;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    const int64_t c0 = (int64_t)(wave * 64 + lane) * 8;

    f32x8 v[VPT], w[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = load8_row(x, c0 + i * (W * 512), n);
    if constexpr (kRes) {
        const R *res = static_cast<const R *>(p.res) + row * p.ldres;
#pragma unroll
        for (int i = 0; i < VPT; ++i) v[i] += load8_row(res, c0 + i * (W * 512), n);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) w[i] = load8_any(p.weight, p.w_dtype, c0 + i * (W * 512), n);

    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[i][j] * v[i][j];
    s = row_sum<W>(s, lds[0], wave, lane);
    const float r = 1.0f / sqrtf(s / (float)n + p.eps);

    if constexpr (kRes) {
        if (p.h) {
            R *h = static_cast<R *>(p.h) + row * p.ldh;
#pragma unroll
            for (int i = 0; i < VPT; ++i) store8_row(h, c0 + i * (W * 512), n, v[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = v[i] * r * w[i];

    float scale;
    if (p.scale) {
        scale = *p.scale;
    } else {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) a = __builtin_elementwise_maximum(a, __builtin_fabsf(v[i][j]));
        a = row_max<W>(a, lds[1], wave, lane);
        scale = __builtin_elementwise_maximum(a / most_of(p.q_dtype), kLeastScale);
        if (wave == 0 && lane == 0) p.row_scales[row] = scale;
    }
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.ldq;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t c = c0 + i * (W * 512);
        if (c < n) store_codes(q, c, n, codes8_any(p.q_dtype, v[i], scale));
    }
}

// Rows too long for registers: three passes over the row, by one workgroup.
// h is stored in the last one, after its element's last load, since it may be
// the residual.
template <typename X, typename R>
__global__ __launch_bounds__(1024) void norm_long_rows(NormParams p)
{
    constexpr bool kRes = !__is_same(R, NoRes);
    __shared__ float lds[2][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x, n = p.n;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    const auto value = [&](int64_t c) {
        f32x8 v = load8_row(x, c, n);
        if constexpr (kRes) v += load8_row(static_cast<const R *>(p.res) + row * p.ldres, c, n);
        return v;
    };
    float s = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
        const f32x8 v = value(c);
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t += v[j] * v[j];
        s += t;
    }
    s = row_sum<16>(s, lds[0], wave, lane);
    const float r = 1.0f / sqrtf(s / (float)n + p.eps);
    float scale;
    if (p.scale) {
        scale = *p.scale;
    } else {
        float a = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
            const f32x8 y = value(c) * r * load8_any(p.weight, p.w_dtype, c, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) a = __builtin_elementwise_maximum(a, __builtin_fabsf(y[j]));
        }
        a = row_max<16>(a, lds[1], wave, lane);
        scale = __builtin_elementwise_maximum(a / most_of(p.q_dtype), kLeastScale);
        if (threadIdx.x == 0) p.row_scales[row] = scale;
    }
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.ldq;
    for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
        const f32x8 v = value(c);
        if constexpr (kRes) {
            if (p.h) store8_row(static_cast<R *>(p.h) + row * p.ldh, c, n, v);
        }
        store_codes(q, c, n, codes8_any(p.q_dtype, v * r * load8_any(p.weight, p.w_dtype, c, n), scale));
    }
}

template <typename X, typename R>
hipError_t launch_norm_of(const NormParams &p, hipStream_t stream)
{
    const int64_t n = p.n, T = p.T;
    const dim3 rows((unsigned)T), rows4((unsigned)((T + 3) / 4));
    if (n <= 512)
        hipLaunchKernelGGL((norm_rows<X, R, 1, 1>), rows4, dim3(256), 0, stream, p);
    else if (n <= 1024)
        hipLaunchKernelGGL((norm_rows<X, R, 1, 2>), rows4, dim3(256), 0, stream, p);
    else if (n <= 2048)
        hipLaunchKernelGGL((norm_rows<X, R, 4, 1>), rows, dim3(256), 0, stream, p);
    else if (n <= 4096)
        hipLaunchKernelGGL((norm_rows<X, R, 4, 2>), rows, dim3(256), 0, stream, p);
    else if (n <= 8192)
        hipLaunchKernelGGL((norm_rows<X, R, 8, 2>), rows, dim3(512), 0, stream, p);
    else if (n <= 16384)
        hipLaunchKernelGGL((norm_rows<X, R, 16, 2>), rows, dim3(1024), 0, stream, p);
    else
        hipLaunchKernelGGL((norm_long_rows<X, R>), rows, dim3(1024), 0, stream, p);
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
// registers; it stores them once, and grad_weight_kernel adds the parts.  The
// next row's loads are issued before this row's sums are waited for.

template <typename E>
__device__ __forceinline__ f32x8 widen(const E &v)
{
    return __builtin_convertvector(v, f32x8);
}

template <typename G, typename H, int W, int VPT>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_grad_rows(NormGradParams p, int64_t parts)
{
    constexpr int kRows = W == 1 ? 4 : 1;  // rows at a time in a workgroup
    __shared__ float2 lds[2][W];
    __shared__ float share[W == 1 ? 3 * VPT * 512 : 1];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int wave = W == 1 ? 0 : wv;
    const int64_t n = p.n, step = parts * kRows;
    const int64_t c0 = (int64_t)(wave * 64 + lane) * 8;
    const G *g = static_cast<const G *>(p.g);
    const H *h = static_cast<const H *>(p.h);

    f32x8 gw[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) gw[i] = 0.0f;
    typename Vec8<G>::type gn[VPT];
    typename Vec8<H>::type hn[VPT];
    int64_t row = (int64_t)blockIdx.x * kRows + (W == 1 ? wv : 0);
    const auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            gn[i] = load8_raw(g + r * p.ldg, c0 + i * (W * 512), n);
            hn[i] = load8_raw(h + r * p.ldh, c0 + i * (W * 512), n);
        }
    };
    if (row < p.T) fetch(row);
    for (int turn = 0; row < p.T; row += step, turn ^= 1) {
        f32x8 gv[VPT], hv[VPT];
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            gv[i] = widen(gn[i]);
            hv[i] = widen(hn[i]);
            const f32x8 w = load8_any(p.weight, p.w_dtype, c0 + i * (W * 512), n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sq += hv[i][j] * hv[i][j];
                dot += gv[i][j] * w[j] * hv[i][j];
            }
        }
        if (row + step < p.T) fetch(row + step);
        sq = wave_sum(sq);
        dot = wave_sum(dot);
        if (W > 1) {
            if (lane == 0) lds[turn][wave] = make_float2(sq, dot);
            __syncthreads();  // two arrays in turn: a wave is at most one barrier ahead
            sq = dot = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                sq += lds[turn][i].x;
                dot += lds[turn][i].y;
            }
        }
        const float r = 1.0f / sqrtf(sq / (float)n + p.eps);
        const float mean = dot * r / (float)n;
        G *gi = static_cast<G *>(p.gi) + row * p.ldgi;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t c = c0 + i * (W * 512);
            const f32x8 nv = hv[i] * r;
            gw[i] += gv[i] * nv;
            f32x8 d = (gv[i] * load8_any(p.weight, p.w_dtype, c, n) - nv * mean) * r;
            if (p.gh) {
                const char *gh = static_cast<const char *>(p.gh) + row * p.ldgh * (p.gh_dtype == EMU_DT_FP32 ? 4 : 2);
                d += load8_any(gh, p.gh_dtype, c, n);
            }
            if (c < n) store8_row(gi, c, n, d);
        }
    }
    if (W == 1) {  // the four waves' sums, in the order of the waves
        if (wv) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) share[(wv - 1) * VPT * 512 + (i * 8 + j) * 64 + lane] = gw[i][j];
        }
        __syncthreads();
        if (wv) return;
        for (int o = 0; o < 3; ++o)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) gw[i][j] += share[o * VPT * 512 + (i * 8 + j) * 64 + lane];
    }
    float *part = p.part + (int64_t)blockIdx.x * n;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (c0 + i * (W * 512) < n) store8_row(part, c0 + i * (W * 512), n, gw[i]);
}

// Rows too long for registers: the row is read twice, and the workgroup's own
// part in the workspace takes the place of the sums in registers.
template <typename G, typename H>
__global__ __launch_bounds__(1024) void norm_grad_long_rows(NormGradParams p, int64_t parts)
{
    __shared__ float lds[2][2][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = p.n;
    float *part = p.part + (int64_t)blockIdx.x * n;
    int turn = 0;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.T; row += parts, turn ^= 1, first = false) {
        const G *g = static_cast<const G *>(p.g) + row * p.ldg;
        const H *h = static_cast<const H *>(p.h) + row * p.ldh;
        float sq = 0.0f, dot = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
            const f32x8 gv = load8_row(g, c, n), hv = load8_row(h, c, n), w = load8_any(p.weight, p.w_dtype, c, n);
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
        for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
            const f32x8 gv = load8_row(g, c, n), nv = load8_row(h, c, n) * r;
            f32x8 d = (gv * load8_any(p.weight, p.w_dtype, c, n) - nv * mean) * r;
            if (p.gh) {
                const char *gh = static_cast<const char *>(p.gh) + row * p.ldgh * (p.gh_dtype == EMU_DT_FP32 ? 4 : 2);
                d += load8_any(gh, p.gh_dtype, c, n);
            }
            f32x8 t = gv * nv;
            if (!first) t += load8_row(part, c, n);
            store8_row(part, c, n, t);
            store8_row(static_cast<G *>(p.gi) + row * p.ldgi, c, n, d);
        }
    }
}

// grad_weight: 64 columns a workgroup, 16 waves that each add every 16th
// part, joined in the order of the waves.
__global__ __launch_bounds__(1024) void grad_weight_kernel(NormGradParams p, int64_t parts)
{
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < p.n)
        for (int64_t i = wave; i < parts; i += 16) s += p.part[i * p.n + c];
    lds[wave][lane] = s;
    __syncthreads();
    if (wave || c >= p.n) return;
    for (int i = 1; i < 16; ++i) s += lds[i][lane];
    if (p.w_dtype == EMU_DT_BF16)
        static_cast<__bf16 *>(p.gw)[c] = (__bf16)s;
    else if (p.w_dtype == EMU_DT_FP16)
        static_cast<_Float16 *>(p.gw)[c] = (_Float16)s;
    else
        static_cast<float *>(p.gw)[c] = s;
}

template <typename G, typename H>
void launch_norm_grad_of(const NormGradParams &p, int64_t parts, hipStream_t stream)
{
    const int64_t n = p.n;
    const dim3 grid((unsigned)parts);
    if (n <= 512)
        hipLaunchKernelGGL((norm_grad_rows<G, H, 1, 1>), grid, dim3(256), 0, stream, p, parts);
    else if (n <= 1024)
        hipLaunchKernelGGL((norm_grad_rows<G, H, 1, 2>), grid, dim3(256), 0, stream, p, parts);
    else if (n <= 2048)
        hipLaunchKernelGGL((norm_grad_rows<G, H, 4, 1>), grid, dim3(256), 0, stream, p, parts);
    else if (n <= 4096)
        hipLaunchKernelGGL((norm_grad_rows<G, H, 8, 1>), grid, dim3(512), 0, stream, p, parts);
    else if (n <= 8192)
        hipLaunchKernelGGL((norm_grad_rows<G, H, 8, 2>), grid, dim3(512), 0, stream, p, parts);
    else if (n <= 16384)
        hipLaunchKernelGGL((norm_grad_rows<G, H, 16, 2>), grid, dim3(1024), 0, stream, p, parts);
    else
        hipLaunchKernelGGL((norm_grad_long_rows<G, H>), grid, dim3(1024), 0, stream, p, parts);
}

}  // namespace

// Workgroups of the gradient, each with a part of grad_weight in the
// workspace: at most two for each CU, and one for each row (or four rows of
// up to 1,024 values, a row to a wave).
int64_t norm_grad_parts(int64_t T, int64_t n)
{
    const int64_t most = n <= 1024 ? (T + 3) / 4 : T;
    return most < 512 ? most : 512;
}

hipError_t launch_norm_grad(int g_dtype, int h_dtype, const NormGradParams &p, hipStream_t stream)
{
    const int64_t parts = norm_grad_parts(p.T, p.n);
    if (parts > 0) {
        if (g_dtype == EMU_DT_FP32)
            launch_norm_grad_of<float, float>(p, parts, stream);
        else if (g_dtype == EMU_DT_BF16 && h_dtype == EMU_DT_FP32)
            launch_norm_grad_of<__bf16, float>(p, parts, stream);
        else if (g_dtype == EMU_DT_BF16)
            launch_norm_grad_of<__bf16, __bf16>(p, parts, stream);
        else if (h_dtype == EMU_DT_FP32)
            launch_norm_grad_of<_Float16, float>(p, parts, stream);
        else
            launch_norm_grad_of<_Float16, _Float16>(p, parts, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(grad_weight_kernel, dim3((unsigned)((p.n + 63) / 64)), dim3(1024), 0, stream, p, parts);
    return hipGetLastError();
}

hipError_t launch_norm(int x_dtype, int res_dtype, const NormParams &p, hipStream_t stream)
{
    if (x_dtype == EMU_DT_BF16) return launch_norm_x<__bf16>(res_dtype, p, stream);
    if (x_dtype == EMU_DT_FP16) return launch_norm_x<_Float16>(res_dtype, p, stream);
    return launch_norm_x<float>(res_dtype, p, stream);
}

}  // namespace emu
