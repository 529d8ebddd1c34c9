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
constexpr int64_t kMaxGroupedRows = int64_t(1) << 24, kMaxGroups = 65536;

// What both products ask of their operands; null where all is well.
struct Operand {
    const void *p;
    int64_t ld, stride;
    bool aligned() const
    {
        return aligned_to(p, 16) && ld % 16 == 0 && stride % 16 == 0 && ld <= emu::kMaxTileLd;
    }
};
const char *refused(const emu::BlockMMParams &p, int a_dtype, int w_dtype, int s_type, emu_dtype bias_dtype)
{
    if (p.M < 0 || p.N < 0 || p.K < 0 || p.E < 0) return "negative size";
    if (!is_code(a_dtype) || !is_code(w_dtype)) return "a and w must be e4m3fn or e5m2";
    if (!is_scale(s_type)) return "scales must be fp32 or e8m0";
    if (!is_float(p.out_dtype)) return "out must be bf16, fp16 or fp32";
    if (p.bias && bias_dtype != p.out_dtype && bias_dtype != EMU_DT_FP32) return "the bias must be of out's type or fp32";
    return nullptr;
}
const char *refused_pointers(const emu::BlockMMParams &p, int s_type, emu_dtype bias_dtype)
{
    const int64_t blocks = blocks_of(p.K), wide = blocks_of(p.N);
    if (!p.out || (p.K > 0 && (!p.a || !p.w || !p.sa || !p.sw))) return "null pointer";
    if (bad_ld(p.ldo, p.N, p.M)) return "leading dimension smaller than a row";
    if (p.K > 0) {
        if (bad_ld(p.lda, p.K, p.M) || bad_ld(p.ldw, p.K, p.N)) return "leading dimension smaller than a row";
        if (p.w_stride < 0 || p.sw_stride < 0 || far(p.w_stride, p.E) || far(p.sw_stride, p.E) || p.sa_row < 0 || p.sa_block < 0 ||
            p.sw_row < 0 || p.sw_block < 0 || far(p.sa_row, p.M) || far(p.sa_block, blocks) || far(p.sw_row, wide) ||
            far(p.sw_block, blocks))
            return "a negative stride, or one too large";
        if (!aligned_to(p.sa, scale_size(s_type)) || !aligned_to(p.sw, scale_size(s_type)))
            return "a pointer is not aligned to its element";
    }
    if (!aligned_to(p.out, size_of(p.out_dtype)) || (p.bias && !aligned_to(p.bias, size_of(bias_dtype))))
        return "a pointer is not aligned to its element";
    return nullptr;
}
const char *too_large(const emu::BlockMMParams &p)
{
    if (p.M > kMaxRows || p.N > kMaxRows) return "more than 2^31-1 rows";
    if (p.K > emu::kMaxTileLd) return "K above 2^22";
    if ((p.M > 1 && p.sa_row > emu::kMaxScaleLd) || (p.N > EMU_BLOCK && p.sw_row > emu::kMaxScaleLd))
        return "scales' rows more than 2^20 apart";
    return nullptr;
}
// Whether E matrices of N rows of K overlap, which have to lie one after the
// other or with their rows among each other: workgroups would write over each other.
bool overlapping(int64_t ld, int64_t stride, int64_t E, int64_t N, int64_t K)
{
    if (E <= 1) return false;
    if (N == 1 || stride >= ld) return stride < (N - 1) * ld + K;
    return stride < K || ld < (E - 1) * stride + K;
}
const char *grad_too_large(int64_t T, int64_t E, int64_t N, int64_t K)
{
    if (T > int64_t(1) << 30 || E > kMaxGroups) return "T above 2^30 or E above 65536";
    if (N > emu::kMaxTileLd || K > emu::kMaxTileLd) return "N or K above 2^22";
    if (blocks_of(N) * blocks_of(K) > (int64_t(1) << 23) / (E ? E : 1)) return "more than 2^23 tiles of 128 x 128";
    return nullptr;
}
emu_status block_mm(const emu::BlockMMParams &p, int a_dtype, int w_dtype, const void *ws, size_t bytes, hipStream_t stream)
{
    const bool a = Operand{p.a, p.lda, 0}.aligned(), w = Operand{p.w, p.ldw, p.w_stride}.aligned();
    const int64_t need = emu::block_mm_workspace(p.M, p.N, p.K, p.E, p.ends != nullptr, p.out_dtype == EMU_DT_FP32, a, w);
    if ((int64_t)bytes < need || (need > 0 && !ws)) return set_error(EMU_ERR_WORKSPACE, "workspace smaller than is needed");
    if (!aligned_to(ws, 16)) return invalid("the workspace is not 16-byte aligned");
    return done(emu::launch_block_mm(a_dtype, w_dtype, p, a, w, stream));
}

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

size_t emu_block_scaled_mm_workspace(int64_t M, int64_t N, int64_t K, emu_dtype out_dtype, int a_aligned, int w_aligned)
{
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxRows || N > kMaxRows || K > emu::kMaxTileLd || !is_float(out_dtype)) return 0;
    return (size_t)emu::block_mm_workspace(M, N, K, 1, false, out_dtype == EMU_DT_FP32, a_aligned != 0, w_aligned != 0);
}

emu_status emu_block_scaled_mm(const void *a, emu_dtype a_dtype, int64_t lda, const void *w, emu_dtype w_dtype, int64_t ldw,
                               int64_t M, int64_t N, int64_t K, const void *scale_a, int64_t sa_row, int64_t sa_block,
                               const void *scale_w, int64_t sw_row, int64_t sw_block, emu_scale_type s_type, const void *bias,
                               emu_dtype bias_dtype, void *out, emu_dtype out_dtype, int64_t ldo, void *workspace,
                               size_t workspace_bytes, hipStream_t stream)
{
    emu::BlockMMParams p{};
    p.a = static_cast<const int8_t *>(a);
    p.w = static_cast<const int8_t *>(w);
    p.lda = lda;
    p.ldw = ldw;
    p.M = M;
    p.N = N;
    p.K = K;
    p.sa = scale_a;
    p.sw = scale_w;
    p.sa_row = sa_row;
    p.sa_block = sa_block;
    p.sw_row = sw_row;
    p.sw_block = sw_block;
    p.e8m0 = s_type == EMU_SCALE_E8M0;
    p.bias = bias;
    p.bias_f32 = bias_dtype == EMU_DT_FP32;
    p.out = out;
    p.out_dtype = out_dtype;
    p.ldo = ldo;
    p.E = 1;
    p.ws = workspace;
    if (const char *text = refused(p, a_dtype, w_dtype, s_type, bias_dtype)) return invalid(text);
    if (const char *text = too_large(p)) return unsupported(text);
    if (M == 0 || N == 0) return set_error(EMU_OK, "");
    if (const char *text = refused_pointers(p, s_type, bias_dtype)) return invalid(text);
    return block_mm(p, a_dtype, w_dtype, workspace, workspace_bytes, stream);
}

size_t emu_grouped_block_scaled_mm_workspace(int64_t T, int64_t E, int64_t N, int64_t K, emu_dtype out_dtype, int a_aligned,
                                             int w_aligned)
{
    if (T <= 0 || E <= 0 || N <= 0 || K <= 0 || T > kMaxGroupedRows || E > kMaxGroups || N > kMaxRows || K > emu::kMaxTileLd ||
        !is_float(out_dtype))
        return 0;
    return (size_t)emu::block_mm_workspace(T, N, K, (int)E, true, out_dtype == EMU_DT_FP32, a_aligned != 0, w_aligned != 0);
}

emu_status emu_grouped_block_scaled_mm(const void *a, emu_dtype a_dtype, int64_t lda, const void *w, emu_dtype w_dtype,
                                       int64_t ldw, int64_t w_stride, int64_t T, int64_t E, int64_t N, int64_t K,
                                       const void *scale_a, int64_t sa_row, int64_t sa_block, const void *scale_w,
                                       int64_t sw_row, int64_t sw_block, int64_t sw_stride, emu_scale_type s_type,
                                       const void *ends, int ends_bits, int zero_rest, void *out, emu_dtype out_dtype,
                                       int64_t ldo, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    emu::BlockMMParams p{};
    p.a = static_cast<const int8_t *>(a);
    p.w = static_cast<const int8_t *>(w);
    p.lda = lda;
    p.ldw = ldw;
    p.w_stride = E > 1 ? w_stride : 0;
    p.M = T;
    p.N = N;
    p.K = K;
    p.sa = scale_a;
    p.sw = scale_w;
    p.sa_row = sa_row;
    p.sa_block = sa_block;
    p.sw_row = sw_row;
    p.sw_block = sw_block;
    p.sw_stride = E > 1 ? sw_stride : 0;
    p.e8m0 = s_type == EMU_SCALE_E8M0;
    p.out = out;
    p.out_dtype = out_dtype;
    p.ldo = ldo;
    p.ends = ends;
    p.ends64 = ends_bits == 64;
    p.E = E < 0 ? -1 : E > kMaxGroups ? (int)kMaxGroups : (int)E;
    p.zero_rest = zero_rest != 0;
    p.ws = workspace;
    if (const char *text = refused(p, a_dtype, w_dtype, s_type, EMU_DT_FP32)) return invalid(text);
    if (ends_bits != 32 && ends_bits != 64) return invalid("ends must be int32 or int64");
    if (T > kMaxGroupedRows || E > kMaxGroups) return unsupported("T above 2^24 or E above 65536");
    if (const char *text = too_large(p)) return unsupported(text);
    if (T == 0 || N == 0 || (E == 0 && !zero_rest)) return set_error(EMU_OK, "");
    if (E == 0) p.K = 0;  // (no sum: zeros behind no group's rows, for which no operand is read or laid out)
    if (!ends && E > 0) return invalid("null pointer");
    if (!aligned_to(ends, ends_bits / 8)) return invalid("a pointer is not aligned to its element");
    if (const char *text = refused_pointers(p, s_type, EMU_DT_FP32)) return invalid(text);
    if (!ends) p.ends = out;  // (no group: never read, but the call is one by groups)
    return block_mm(p, a_dtype, w_dtype, workspace, workspace_bytes, stream);
}

size_t emu_block_weight_grad_workspace(int64_t T, int64_t E, int64_t N, int64_t K, emu_dtype g_dtype, int g_aligned,
                                       int c_aligned)
{
    if (T < 0 || E < 0 || N <= 0 || K <= 0 || !is_float(g_dtype) || grad_too_large(T, E, N, K)) return 0;
    return (size_t)emu::weight_grad_workspace(T, (int)E, N, K, g_dtype, g_aligned != 0, c_aligned != 0);
}

emu_status emu_block_weight_grad(const void *g, emu_dtype g_dtype, int64_t ldg, const void *codes, emu_dtype c_dtype,
                                 int64_t ldc, const void *scales, int64_t s_row, int64_t s_block, int64_t T, int64_t N,
                                 int64_t K, const void *ends, int ends_bits, int64_t E, void *out, emu_dtype out_dtype,
                                 int64_t ldo, int64_t out_stride, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream)
{
    if (T < 0 || N < 0 || K < 0 || E < 0) return invalid("negative size");
    if (!is_float(g_dtype)) return invalid("g must be bf16, fp16 or fp32");
    if (!is_code(c_dtype)) return invalid("codes must be e4m3fn or e5m2");
    if (!is_float(out_dtype)) return invalid("out must be bf16, fp16 or fp32");
    if (ends ? ends_bits != 32 && ends_bits != 64 : E != 0) return invalid("ends must be int32 or int64, and null without groups");
    if (ends && E == 0) return set_error(EMU_OK, "");
    if (const char *text = grad_too_large(T, E, N, K)) return unsupported(text);
    if (N == 0 || K == 0) return set_error(EMU_OK, "");
    if (!out || (T > 0 && (!g || !codes || !scales))) return invalid("null pointer");
    if (bad_ld(ldo, K, N) || out_stride < 0 || (E > 1 && (out_stride < 1 || far(out_stride, E))))
        return invalid("leading dimension smaller than a row, or a bad stride");
    if (overlapping(ldo, out_stride, E, N, K)) return invalid("the output's matrices overlap");
    if (T > 0 && (bad_ld(ldg, N, T) || bad_ld(ldc, K, T))) return invalid("leading dimension smaller than a row");
    if (T > 0 && (s_row < 0 || s_block < 0 || far(s_row, T) || far(s_block, blocks_of(K)))) return invalid("a negative stride, or one too large");
    const size_t size = size_of(g_dtype);
    if (!aligned_to(g, size) || !aligned_to(out, size_of(out_dtype)) || (ends && !aligned_to(ends, ends_bits / 8)))
        return invalid("a pointer is not aligned to its element");
    const bool ga = aligned_to(g, 16) && ldg % (int64_t)(16 / size) == 0 && ldg <= emu::kMaxTileLd;
    const bool ca = aligned_to(codes, 16) && ldc % 16 == 0 && ldc <= emu::kMaxTileLd;
    const int64_t need = emu::weight_grad_workspace(T, (int)E, N, K, g_dtype, ga, ca);
    if ((int64_t)workspace_bytes < need || (need > 0 && !workspace))
        return set_error(EMU_ERR_WORKSPACE, "workspace smaller than emu_block_weight_grad_workspace");
    if (!aligned_to(workspace, 16)) return invalid("the workspace is not 16-byte aligned");
    emu::WeightGradParams p{};
    p.g = static_cast<const uint16_t *>(g);
    p.ldg = ldg;
    p.codes = static_cast<const int8_t *>(codes);
    p.ldc = ldc;
    p.scales = static_cast<const uint8_t *>(scales);
    p.s_row = s_row;
    p.s_block = s_block;
    p.T = T;
    p.N = N;
    p.K = K;
    p.ends = ends;
    p.ends64 = ends_bits == 64;
    p.E = (int)E;
    p.out = out;
    p.out_dtype = out_dtype;
    p.ldo = ldo;
    p.out_stride = out_stride;
    return done(emu::launch_weight_grad(g_dtype, c_dtype, p, ga, ca, workspace, stream));
}

}  // extern "C"
