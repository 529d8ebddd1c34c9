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

#ifdef __HIPCC__

// The value of a scale byte: 2^(b - 127) (a subnormal number for 0), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b)
{
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

#endif

}  // namespace emu
