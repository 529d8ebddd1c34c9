// ops_block.h -- codes of 8-bit floating point with a scale for each block of
// 128: launch parameters and what the kernels of them share.
#pragma once

#include "../../include/emu_block_operators.h"
#include "ops_device.h"
#include "ops_internal.h"

namespace emu {

constexpr int kBlock = EMU_BLOCK;

__host__ __device__ constexpr int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

struct BlockQuantParams {
    const void *x;
    int64_t ldx, x_stride;
    int64_t E, T, n;
    void *q;
    void *scales;
    bool once;  // nothing of this size stays in a cache
};
hipError_t launch_block_quant(int x_dtype, int q_dtype, bool e8m0, int block_rows, const BlockQuantParams &p, hipStream_t stream);

struct SwigluParams {
    const void *gate, *up;
    int64_t ldgate, ldup;
    int64_t T, F;
    void *q, *scales;
    void *kept, *kept_scales;  // null, or both
    bool once;
};
hipError_t launch_swiglu(int dtype, int q_dtype, bool e8m0, const SwigluParams &p, hipStream_t stream);

struct SwigluGradParams {
    const void *g;
    int64_t ldg;
    const void *kept, *kept_scales;
    int64_t T, F;
    void *grad;
    int64_t ldgrad;
    bool once;
};
hipError_t launch_swiglu_grad(int g_dtype, int q_dtype, bool e8m0, const SwigluGradParams &p, hipStream_t stream);

// The product, dense or by groups of rows (ends not null).  Strides are in
// elements, those of scales between rows (of w: blocks of 128 of them) and
// between blocks of K.
struct BlockMMParams {
    const int8_t *a, *w;
    int64_t lda, ldw, w_stride;
    int64_t M, N, K;
    const void *sa, *sw;
    int64_t sa_row, sa_block, sw_row, sw_block, sw_stride;
    int e8m0;
    const void *bias;
    int bias_f32;          // the bias is binary32 (else of out's type)
    void *out;
    int out_dtype;
    int64_t ldo;
    const void *ends;      // of each group's rows, or null
    int ends64;            // they are int64 (else int32)
    int E;
    int zero_rest;         // rows behind the last group's become 0
    void *ws;
};
// Leading dimensions and row strides of scales whose offsets within a tile stay below 2^31.
constexpr int64_t kMaxTileLd = EMU_BLOCK_MAX_ALIGNED_LD, kMaxScaleLd = int64_t(1) << 20;
int64_t block_mm_workspace(int64_t M, int64_t N, int64_t K, int E, bool grouped, bool fp32_out, bool a_aligned, bool w_aligned);
hipError_t launch_block_mm(int a_dtype, int w_dtype, const BlockMMParams &p, bool a_aligned, bool w_aligned, hipStream_t stream);

// The weights' gradient, of all rows (E = 0) or of each of E groups.  g is
// bf16 in `planes` planes, whose sum it stands for.
struct WeightGradParams {
    const uint16_t *g;
    int64_t ldg, plane_stride;
    int planes;
    const int8_t *codes;
    int64_t ldc;
    const uint8_t *scales;
    int64_t s_row, s_block;
    int64_t T, N, K;
    const void *ends;
    int ends64;
    int E;
    void *out;
    int out_dtype;
    int64_t ldo, out_stride;
};
int64_t weight_grad_workspace(int64_t T, int E, int64_t N, int64_t K, int g_dtype, bool g_aligned, bool c_aligned);
// p.g: of g_dtype
hipError_t launch_weight_grad(int g_dtype, int c_dtype, const WeightGradParams &p, bool g_aligned, bool c_aligned, void *ws,
                              hipStream_t stream);

// Rows laid out anew (ops_tiles.h), both jobs in one launch: 3 us less than in two.
struct RepackRows;
RepackRows repack_job(const int8_t *in, int64_t ld, int64_t stride, int64_t per, int64_t total, int64_t K, int8_t *out, int64_t ldo);
void launch_repack(const RepackRows &a, const RepackRows &b, hipStream_t stream);

// The kernels of one pair of codes' types (emu_block_mm.hip).
enum BlockMode {
    kHardware,  // e8m0 scales go into the matrix instruction
    kScaled,    // each block's sum is multiplied by its scales
    kExact      // the same, the products summed in binary32
};
struct BlockPlan {
    int mode;        // BlockMode
    int tile;        // of the plan's tiles, or -1: few rows
    int rows;        // few rows: fragments of 16 of them
    int waves;       // few rows: waves of a workgroup
    bool words;      // few rows: the operands' rows are aligned to 4 bytes
    int S, stages;   // splits of K, stages of each
};
template <int AF, int WF>
void launch_block_kernel(const BlockMMParams &p, const BlockPlan &plan, float *part, hipStream_t stream);

#ifdef __HIPCC__

// Rows of tiles that an XCD's run is high: with 4 its 32 tiles at a time read 12
// tiles' worth of operands, with 2 18 (the product of 16384 x 8192 x 4096: 408 us
// and 425, in 8 groups 495 and 529, its weights' gradient 986 and 1003; with 8 469,
// 500 and 986).
constexpr int kHigh = 4;

// The value of a scale byte: 2^(b - 127) (a subnormal number for 0), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b)
{
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

// Two of four codes (F: 0 e4m3fn, 1 e5m2) times a power of two, in bf16.
template <int F>
__device__ __forceinline__ uint32_t two_bf16(uint32_t codes, bool high, float scale)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x2 v;
    if (F == 0)
        v = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true)
                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false);
    else
        v = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, scale, true)
                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, scale, false);
    return __builtin_bit_cast(uint32_t, v);
}

#endif

}  // namespace emu
