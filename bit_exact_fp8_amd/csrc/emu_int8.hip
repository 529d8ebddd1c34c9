// emu_int8.hip -- emu_int8_scaled_mm: out = (a @ w.T) * scale_a * scale_w + bias.
//
// The products are v_mfma_i32_16x16x64_i8's and their sums exact in int32, so
// neither tiles nor a split of K change a bit of the result.  The matrix
// instruction takes w's rows as its first operand: a lane then ends with four
// consecutive outputs of one row.
#include <hip/hip_runtime.h>

#include "ops_device.h"
#include "ops_internal.h"

namespace emu {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_u __attribute__((aligned(1)));

// 16 codes of a row from k, zeros past K.
__device__ __forceinline__ i32x4 load16(const int8_t *row, int64_t k, int64_t K)
{
    if (k + 16 <= K) return *reinterpret_cast<const i32x4_u *>(row + k);
    i32x4 r = {0, 0, 0, 0};
    for (int i = 0; i < 16; ++i)
        if (k + i < K) r[i >> 2] |= (int)((uint32_t)(uint8_t)row[k + i] << (8 * (i & 3)));
    return r;
}

__device__ __forceinline__ float bias_at(const Int8Params &p, int64_t n)
{
    if (p.bias_f32 || p.out_dtype == EMU_DT_FP32) return static_cast<const float *>(p.bias)[n];
    if (p.out_dtype == EMU_DT_BF16) return (float)static_cast<const __bf16 *>(p.bias)[n];
    return (float)static_cast<const _Float16 *>(p.bias)[n];
}

// Outputs (m, n .. n + 3) of the sums `acc`.
__device__ __forceinline__ void store4(const Int8Params &p, int64_t m, int64_t n, const i32x4 &acc)
{
    if (m >= p.M) return;
    const float sa = p.sa[p.a_per_row ? m : 0];
    float y[4];
    const int valid = p.N - n < 4 ? (int)(p.N - n) : 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = 0.0f;
        if (i < valid) {
            y[i] = (float)acc[i] * sa * p.sw[p.w_per_row ? n + i : 0];
            if (p.bias) y[i] += bias_at(p, n + i);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= valid) break;
        if (p.out_dtype == EMU_DT_BF16)
            static_cast<__bf16 *>(p.out)[m * p.ldo + n + i] = (__bf16)y[i];
        else if (p.out_dtype == EMU_DT_FP16)
            static_cast<_Float16 *>(p.out)[m * p.ldo + n + i] = (_Float16)y[i];
        else
            static_cast<float *>(p.out)[m * p.ldo + n + i] = y[i];
    }
}

// 64 x 64 outputs a workgroup, 32 x 32 a wave, 64 codes of K at a time
// through LDS.  Rows of LDS are padded to 80 bytes.
__global__ __launch_bounds__(256) void int8_tile(Int8Params p)
{
    __shared__ __attribute__((aligned(16))) int8_t as[64][80], ws[64][80];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    const int row = t >> 2, part = (t & 3) * 16;
    const int64_t am = m0 + row < p.M ? m0 + row : p.M - 1, wn = n0 + row < p.N ? n0 + row : p.N - 1;
    const int8_t *ar = p.a + am * p.lda, *wr = p.w + wn * p.ldw;
    i32x4 acc[2][2] = {};
    const int wm = (wave >> 1) * 32, wn0 = (wave & 1) * 32;
    for (int64_t k = 0; k < p.K; k += 64) {
        const i32x4 av = load16(ar, k + part, p.K), wv = load16(wr, k + part, p.K);
        __syncthreads();
        *reinterpret_cast<i32x4 *>(&as[row][part]) = av;
        *reinterpret_cast<i32x4 *>(&ws[row][part]) = wv;
        __syncthreads();
        i32x4 a[2], w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = *reinterpret_cast<const i32x4 *>(&as[wm + i * 16 + (lane & 15)][(lane >> 4) * 16]);
            w[i] = *reinterpret_cast<const i32x4 *>(&ws[wn0 + i * 16 + (lane & 15)][(lane >> 4) * 16]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], a[i], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            store4(p, m0 + wm + i * 16 + (lane & 15), n0 + wn0 + j * 16 + (lane >> 4) * 4, acc[i][j]);
}

}  // namespace

int64_t int8_mm_workspace(int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_int8_mm(const Int8Params &p, bool, hipStream_t stream)
{
    constexpr int64_t kRows = 64 * 32768;
    for (int64_t m = 0; m < p.M; m += kRows) {
        Int8Params q = p;
        q.M = p.M - m < kRows ? p.M - m : kRows;
        q.a = p.a + m * p.lda;
        if (p.a_per_row) q.sa = p.sa + m;
        q.out = static_cast<char *>(p.out) + m * p.ldo * (p.out_dtype == EMU_DT_FP32 ? 4 : 2);
        hipLaunchKernelGGL(int8_tile, dim3((unsigned)((q.N + 63) / 64), (unsigned)((q.M + 63) / 64)), dim3(256), 0,
                           stream, q);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace emu
