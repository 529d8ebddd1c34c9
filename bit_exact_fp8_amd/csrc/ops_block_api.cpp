// ops_block_api.cpp -- the C ABI of include/emu_block_operators.h: argument
// checks and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ops_block.h"

using emu::blocks_of;
using emu::set_error;

namespace {

emu_status invalid(const char *text) { return set_error(EMU_ERR_INVALID_ARG, text); }
emu_status unsupported(const char *text) { return set_error(EMU_ERR_UNSUPPORTED, text); }
emu_status done(hipError_t e)
{
    return e == hipSuccess ? set_error(EMU_OK, "") : set_error(EMU_ERR_DEVICE, hipGetErrorString(e));
}

bool is_float(int d) { return d == EMU_DT_BF16 || d == EMU_DT_FP16 || d == EMU_DT_FP32; }
bool is_code(int d) { return d == EMU_DT_E4M3FN || d == EMU_DT_E5M2; }
bool is_scale(int s) { return s == EMU_SCALE_FP32 || s == EMU_SCALE_E8M0; }
size_t size_of(int d) { return d == EMU_DT_FP32 ? 4 : d == EMU_DT_BF16 || d == EMU_DT_FP16 ? 2 : 1; }
size_t scale_size(int s) { return s == EMU_SCALE_FP32 ? 4 : 1; }
bool aligned_to(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Offsets of `count` steps of `ld` stay within 63 bits of bytes.
bool far(int64_t ld, int64_t count) { return count > 1 && ld > (INT64_MAX / 16) / count; }
bool bad_ld(int64_t ld, int64_t cols, int64_t rows) { return ld < cols || far(ld, rows); }

constexpr int64_t kMaxRows = INT32_MAX, kMaxCols = int64_t(1) << 30;

}  // namespace

extern "C" {

emu_status emu_block_quant(const void *x, emu_dtype x_dtype, int64_t ldx, int64_t x_stride, int64_t E, int64_t T,
                           int64_t n, int block_rows, void *q, emu_dtype q_dtype, void *scales, emu_scale_type s_type,
                           hipStream_t stream)
{
    if (E < 0 || T < 0 || n < 0) return invalid("negative size");
    if (!is_float(x_dtype)) return invalid("x must be bf16, fp16 or fp32");
    if (!is_code(q_dtype)) return invalid("q must be e4m3fn or e5m2");
    if (!is_scale(s_type)) return invalid("scales must be fp32 or e8m0");
    if (block_rows != 1 && block_rows != EMU_BLOCK) return invalid("a block has 1 or 128 rows");
    if (E > kMaxRows || T > kMaxRows || n > kMaxCols) return unsupported("E or T above 2^31-1, or n above 2^30");
    if (E == 0 || T == 0 || n == 0) return set_error(EMU_OK, "");
    if (T > (INT64_MAX / 16) / n || E > (INT64_MAX / 16) / (T * n)) return unsupported("more than 2^59 values");
    if (!x || !q || !scales) return invalid("null pointer");
    if (bad_ld(ldx, n, T) || x_stride < 0 || far(x_stride, E)) return invalid("leading dimension smaller than n, or a bad stride");
    if (!aligned_to(x, size_of(x_dtype)) || !aligned_to(scales, scale_size(s_type)))
        return invalid("a pointer is not aligned to its element");
    emu::BlockQuantParams p{};
    p.x = x;
    p.ldx = ldx;
    p.x_stride = x_stride;
    p.E = E;
    p.T = T;
    p.n = n;
    p.q = q;
    p.scales = scales;
    return done(emu::launch_block_quant(x_dtype, q_dtype, s_type == EMU_SCALE_E8M0, block_rows, p, stream));
}

emu_status emu_swiglu_block_quant(const void *gate, int64_t ldgate, const void *up, int64_t ldup, emu_dtype dtype,
                                  int64_t T, int64_t F, void *q, emu_dtype q_dtype, void *scales,
                                  emu_scale_type s_type, void *kept, void *kept_scales, hipStream_t stream)
{
    if (T < 0 || F < 0) return invalid("negative size");
    if (!is_float(dtype)) return invalid("gate and up must be bf16, fp16 or fp32");
    if (!is_code(q_dtype)) return invalid("q must be e4m3fn or e5m2");
    if (!is_scale(s_type)) return invalid("scales must be fp32 or e8m0");
    if ((kept == nullptr) != (kept_scales == nullptr) && T > 0 && F > 0) return invalid("kept and kept_scales go together");
    if (T > kMaxRows || F > kMaxCols) return unsupported("T above 2^31-1 or F above 2^30");
    if (T == 0 || F == 0) return set_error(EMU_OK, "");
    if (!gate || !up || !q || !scales) return invalid("null pointer");
    if (bad_ld(ldgate, F, T) || bad_ld(ldup, F, T)) return invalid("leading dimension smaller than F");
    if (!aligned_to(gate, size_of(dtype)) || !aligned_to(up, size_of(dtype)) || !aligned_to(scales, scale_size(s_type)) ||
        !aligned_to(kept_scales, scale_size(s_type)))
        return invalid("a pointer is not aligned to its element");
    emu::SwigluParams p{};
    p.gate = gate;
    p.up = up;
    p.ldgate = ldgate;
    p.ldup = ldup;
    p.T = T;
    p.F = F;
    p.q = q;
    p.scales = scales;
    p.kept = kept;
    p.kept_scales = kept_scales;
    return done(emu::launch_swiglu(dtype, q_dtype, s_type == EMU_SCALE_E8M0, p, stream));
}

emu_status emu_swiglu_block_backward(const void *g, emu_dtype g_dtype, int64_t ldg, const void *kept, emu_dtype q_dtype,
                                     const void *kept_scales, emu_scale_type s_type, int64_t T, int64_t F, void *grad,
                                     int64_t ldgrad, hipStream_t stream)
{
    if (T < 0 || F < 0) return invalid("negative size");
    if (!is_float(g_dtype)) return invalid("g must be bf16, fp16 or fp32");
    if (!is_code(q_dtype)) return invalid("kept must be e4m3fn or e5m2");
    if (!is_scale(s_type)) return invalid("scales must be fp32 or e8m0");
    if (T > kMaxRows || F > kMaxCols) return unsupported("T above 2^31-1 or F above 2^30");
    if (T == 0 || F == 0) return set_error(EMU_OK, "");
    if (!g || !kept || !kept_scales || !grad) return invalid("null pointer");
    if (bad_ld(ldg, F, T) || bad_ld(ldgrad, 2 * F, T)) return invalid("leading dimension smaller than a row");
    if (!aligned_to(g, size_of(g_dtype)) || !aligned_to(grad, size_of(g_dtype)) || !aligned_to(kept_scales, scale_size(s_type)))
        return invalid("a pointer is not aligned to its element");
    emu::SwigluGradParams p{};
    p.g = g;
    p.ldg = ldg;
    p.kept = kept;
    p.kept_scales = kept_scales;
    p.T = T;
    p.F = F;
    p.grad = grad;
    p.ldgrad = ldgrad;
    return done(emu::launch_swiglu_grad(g_dtype, q_dtype, s_type == EMU_SCALE_E8M0, p, stream));
}

}  // extern "C"
