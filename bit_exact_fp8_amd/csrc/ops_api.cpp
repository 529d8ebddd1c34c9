// ops_api.cpp -- the C ABI of include/emu_operators.h: argument checks and
// launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ops_internal.h"

using emu::set_error;

namespace {

emu_status invalid(const char *text) { return set_error(EMU_ERR_INVALID_ARG, text); }
emu_status unsupported(const char *text) { return set_error(EMU_ERR_UNSUPPORTED, text); }
emu_status done(hipError_t e)
{
    return e == hipSuccess ? set_error(EMU_OK, "") : set_error(EMU_ERR_DEVICE, hipGetErrorString(e));
}

bool is_float(int d) { return d == EMU_DT_BF16 || d == EMU_DT_FP16 || d == EMU_DT_FP32; }
size_t size_of(int d) { return d == EMU_DT_FP32 ? 4 : d == EMU_DT_BF16 || d == EMU_DT_FP16 ? 2 : 1; }
bool aligned_to(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
// An element type that may stand beside `d`: the same, or binary32.
bool beside(int e, int d) { return e == d || e == EMU_DT_FP32; }

// A leading dimension whose offsets stay within 63 bits.
bool bad_ld(int64_t ld, int64_t cols, int64_t rows)
{
    return ld < cols || (rows > 1 && ld > (INT64_MAX / 8) / rows);
}

constexpr int64_t kMaxRows = INT32_MAX, kMaxCols = int64_t(1) << 30;

}  // namespace

extern "C" {

emu_status emu_add_rms_norm_quant(const void *x, emu_dtype x_dtype, int64_t ldx, const void *weight,
                                  emu_dtype w_dtype, const void *residual, emu_dtype res_dtype, int64_t ldres,
                                  int64_t T, int64_t n, float eps, void *q, emu_dtype q_dtype, int64_t ldq,
                                  const float *scale, float *row_scales, void *h_out, int64_t ldh,
                                  hipStream_t stream)
{
    if (T < 0 || n < 0) return invalid("negative size");
    if (!is_float(x_dtype)) return invalid("x must be bf16, fp16 or fp32");
    if (!beside(w_dtype, x_dtype)) return invalid("the weight must be of x's type or fp32");
    if (residual && !beside(res_dtype, x_dtype)) return invalid("the residual must be of x's type or fp32");
    if (q_dtype != EMU_DT_E4M3FN && q_dtype != EMU_DT_E5M2 && q_dtype != EMU_DT_INT8)
        return invalid("q must be e4m3fn, e5m2 or int8");
    if (h_out && !residual) return invalid("h_out needs a residual");
    if (!(eps >= 0.0f)) return invalid("eps must be 0 or more");
    if (T > kMaxRows || n > kMaxCols) return unsupported("T above 2^31-1 or n above 2^30");
    if (T == 0) return set_error(EMU_OK, "");
    if (n == 0) return invalid("a norm of no values");
    if (!x || !weight || !q) return invalid("null pointer");
    if (!scale && !row_scales) return invalid("row_scales is null and no scale is given");
    if (bad_ld(ldx, n, T) || bad_ld(ldq, n, T) || (residual && bad_ld(ldres, n, T)) || (h_out && bad_ld(ldh, n, T)))
        return invalid("leading dimension smaller than n");
    const size_t xs = size_of(x_dtype), rs = residual ? size_of(res_dtype) : 1;
    if (!aligned_to(x, xs) || !aligned_to(weight, size_of(w_dtype)) || !aligned_to(residual, rs) ||
        !aligned_to(h_out, rs) || !aligned_to(scale, 4) || !aligned_to(row_scales, 4))
        return invalid("a pointer is not aligned to its element");
    emu::NormParams p{};
    p.weight = weight;
    p.w_dtype = w_dtype;
    p.ldx = ldx;
    p.ldres = ldres;
    p.n = n;
    p.eps = eps;
    p.q_dtype = q_dtype;
    p.ldq = ldq;
    p.scale = scale;
    p.ldh = ldh;
    constexpr int64_t kRows = 1 << 20;  // a launch's rows: grid x threads stays below 2^32
    for (int64_t r = 0; r < T; r += kRows) {
        p.T = T - r < kRows ? T - r : kRows;
        p.x = static_cast<const char *>(x) + r * ldx * (int64_t)xs;
        p.res = residual ? static_cast<const char *>(residual) + r * ldres * (int64_t)rs : nullptr;
        p.h = h_out ? static_cast<char *>(h_out) + r * ldh * (int64_t)rs : nullptr;
        p.q = static_cast<char *>(q) + r * ldq;
        p.row_scales = row_scales ? row_scales + r : nullptr;
        const hipError_t e = emu::launch_norm(x_dtype, res_dtype, p, stream);
        if (e != hipSuccess) return done(e);
    }
    return done(hipSuccess);
}

size_t emu_add_rms_norm_backward_workspace(int64_t T, int64_t n)
{
    if (T < 0 || n < 0 || T > kMaxRows || n > kMaxCols) return 0;
    return (size_t)(emu::norm_grad_parts(T, n) * emu::norm_grad_part_ld(n)) * 4;
}

emu_status emu_add_rms_norm_backward(const void *g, emu_dtype g_dtype, int64_t ldg, const void *h, emu_dtype h_dtype,
                                     int64_t ldh, const void *weight, emu_dtype w_dtype, const void *grad_h,
                                     emu_dtype gh_dtype, int64_t ldgh, int64_t T, int64_t n, float eps, void *grad_in,
                                     int64_t ldgi, void *grad_weight, void *workspace, size_t workspace_bytes,
                                     hipStream_t stream)
{
    if (T < 0 || n < 0) return invalid("negative size");
    if (!is_float(g_dtype)) return invalid("g must be bf16, fp16 or fp32");
    if (!beside(h_dtype, g_dtype)) return invalid("h must be of g's type or fp32");
    if (!beside(w_dtype, g_dtype)) return invalid("the weight must be of g's type or fp32");
    if (grad_h && !beside(gh_dtype, g_dtype)) return invalid("grad_h must be of g's type or fp32");
    if (!(eps >= 0.0f)) return invalid("eps must be 0 or more");
    if (T > kMaxRows || n > kMaxCols) return unsupported("T above 2^31-1 or n above 2^30");
    if (n == 0) return invalid("a norm of no values");
    if (!weight || !grad_weight || (T > 0 && (!g || !h || !grad_in))) return invalid("null pointer");
    if (T > 0 && (bad_ld(ldg, n, T) || bad_ld(ldh, n, T) || bad_ld(ldgi, n, T) || (grad_h && bad_ld(ldgh, n, T))))
        return invalid("leading dimension smaller than n");
    if (!aligned_to(g, size_of(g_dtype)) || !aligned_to(grad_in, size_of(g_dtype)) ||
        !aligned_to(h, size_of(h_dtype)) || !aligned_to(weight, size_of(w_dtype)) ||
        !aligned_to(grad_weight, size_of(w_dtype)) || (grad_h && !aligned_to(grad_h, size_of(gh_dtype))))
        return invalid("a pointer is not aligned to its element");
    if (workspace_bytes < emu_add_rms_norm_backward_workspace(T, n) || (T > 0 && !workspace))
        return set_error(EMU_ERR_WORKSPACE, "workspace smaller than emu_add_rms_norm_backward_workspace");
    if (!aligned_to(workspace, 16)) return invalid("the workspace is not 16-byte aligned");
    emu::NormGradParams p{};
    p.g = g;
    p.h = h;
    p.weight = weight;
    p.gh = grad_h;
    p.ldg = ldg;
    p.ldh = ldh;
    p.ldgh = ldgh;
    p.T = T;
    p.n = n;
    p.eps = eps;
    p.w_dtype = w_dtype;
    p.gh_dtype = gh_dtype;
    p.gi = grad_in;
    p.ldgi = ldgi;
    p.gw = grad_weight;
    p.part = static_cast<float *>(workspace);
    return done(emu::launch_norm_grad(g_dtype, h_dtype, p, stream));
}

size_t emu_int8_scaled_mm_workspace(int64_t M, int64_t N, int64_t K, int aligned)
{
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxRows || N > kMaxRows || K > 131071) return 0;
    return (size_t)emu::int8_mm_workspace(M, N, K, aligned != 0);
}

emu_status emu_int8_scaled_mm(const int8_t *a, int64_t lda, const int8_t *w, int64_t ldw, int64_t M, int64_t N,
                              int64_t K, const float *scale_a, int a_per_row, const float *scale_w, int w_per_row,
                              const void *bias, emu_dtype bias_dtype, void *out, emu_dtype out_dtype, int64_t ldo,
                              void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (M < 0 || N < 0 || K < 0) return invalid("negative size");
    if (!is_float(out_dtype)) return invalid("out must be bf16, fp16 or fp32");
    if (bias && !beside(bias_dtype, out_dtype)) return invalid("the bias must be of out's type or fp32");
    if (M > kMaxRows || N > kMaxRows) return unsupported("M or N above 2^31-1");
    if (K > 131071) return unsupported("K above 131071: the sum could pass int32");
    if (M == 0 || N == 0) return set_error(EMU_OK, "");
    if (!out || !scale_a || !scale_w || (K > 0 && (!a || !w))) return invalid("null pointer");
    if (bad_ld(ldo, N, M) || (K > 0 && (bad_ld(lda, K, M) || bad_ld(ldw, K, N))))
        return invalid("leading dimension smaller than a row");
    if (!aligned_to(out, size_of(out_dtype)) || !aligned_to(scale_a, 4) || !aligned_to(scale_w, 4) ||
        (bias && !aligned_to(bias, size_of(bias_dtype))))
        return invalid("a pointer is not aligned to its element");
    // (a tile's offsets from its first row have to stay within 31 bits)
    const bool aligned = aligned_to(a, 16) && aligned_to(w, 16) && lda % 16 == 0 && ldw % 16 == 0 &&
                         lda <= EMU_INT8_MAX_ALIGNED_LD && ldw <= EMU_INT8_MAX_ALIGNED_LD;
    const int64_t need = emu::int8_mm_workspace(M, N, K, aligned);
    if ((int64_t)workspace_bytes < need || (need > 0 && !workspace))
        return set_error(EMU_ERR_WORKSPACE, "workspace smaller than emu_int8_scaled_mm_workspace");
    if (!aligned_to(workspace, 16)) return invalid("the workspace is not 16-byte aligned");
    emu::Int8Params p{};
    p.a = a;
    p.w = w;
    p.lda = lda;
    p.ldw = ldw;
    p.M = M;
    p.N = N;
    p.K = K;
    p.sa = scale_a;
    p.sw = scale_w;
    p.a_per_row = a_per_row;
    p.w_per_row = w_per_row;
    p.bias = bias;
    p.bias_f32 = bias_dtype == EMU_DT_FP32;
    p.out = out;
    p.out_dtype = out_dtype;
    p.ldo = ldo;
    p.ws = workspace;
    return done(emu::launch_int8_mm(p, aligned, stream));
}

size_t emu_token_logprobs_workspace(int64_t T, int64_t V, int64_t top_k)
{
    if (T <= 0 || V <= 0 || T > kMaxRows || V > INT32_MAX - 4096 || top_k < 0 || top_k > EMU_MAX_TOP_TOKENS) return 0;
    return (size_t)emu::logp_workspace(T, V, (int)top_k);
}

emu_status emu_token_logprobs(const void *logits, emu_dtype z_dtype, int64_t ldz, int64_t T, int64_t V,
                              const int64_t *tokens, int64_t C, int64_t top_k, float *logprobs, float *entropy,
                              float *lse, float *top_logprobs, int64_t *top_tokens, void *workspace,
                              size_t workspace_bytes, hipStream_t stream)
{
    if (T < 0 || V < 0 || C < 0 || top_k < 0) return invalid("negative size");
    if (!is_float(z_dtype)) return invalid("the logits must be bf16, fp16 or fp32");
    if (T > kMaxRows || V > INT32_MAX - 4096) return unsupported("T above 2^31-1 or V above 2^31-4097");
    if (top_k > EMU_MAX_TOP_TOKENS) return unsupported("top_k above 64");
    if (T == 0) return set_error(EMU_OK, "");
    if (V == 0) return invalid("an empty vocabulary");
    if (top_k > V) return invalid("top_k above V");
    if (C > (INT64_MAX / 8) / T) return invalid("C too large");
    if (!logits || !entropy || !lse || (C > 0 && (!tokens || !logprobs)) || (top_k > 0 && (!top_logprobs || !top_tokens)))
        return invalid("null pointer");
    if (bad_ld(ldz, V, T)) return invalid("leading dimension smaller than V");
    if (!aligned_to(logits, size_of(z_dtype)) || !aligned_to(tokens, 8) || !aligned_to(logprobs, 4) ||
        !aligned_to(entropy, 4) || !aligned_to(lse, 4) || !aligned_to(top_logprobs, 4) || !aligned_to(top_tokens, 8))
        return invalid("a pointer is not aligned to its element");
    const int64_t need = emu::logp_workspace(T, V, (int)top_k);
    if ((int64_t)workspace_bytes < need || (need > 0 && !workspace))
        return set_error(EMU_ERR_WORKSPACE, "workspace smaller than emu_token_logprobs_workspace");
    if (!aligned_to(workspace, 16)) return invalid("the workspace is not 16-byte aligned");
    emu::LogpParams p{};
    p.z = logits;
    p.ldz = ldz;
    p.T = T;
    p.V = V;
    p.tokens = tokens;
    p.C = C;
    p.k = (int)top_k;
    p.logprobs = logprobs;
    p.entropy = entropy;
    p.lse = lse;
    p.top_lp = top_logprobs;
    p.top_tok = top_tokens;
    p.ws = workspace;
    return done(emu::launch_logp(z_dtype, p, stream));
}

emu_status emu_token_logprobs_backward(const void *logits, emu_dtype z_dtype, int64_t ldz, int64_t T, int64_t V,
                                       const int64_t *tokens, int64_t C, const float *lse, const float *entropy,
                                       const float *g, const float *g_entropy, const int64_t *top_tokens,
                                       const float *g_top, int64_t top_k, void *grad, int64_t ldgrad,
                                       hipStream_t stream)
{
    if (T < 0 || V < 0 || C < 0 || top_k < 0) return invalid("negative size");
    if (!is_float(z_dtype)) return invalid("the logits must be bf16, fp16 or fp32");
    if (T > kMaxRows || V > INT32_MAX - 4096) return unsupported("T above 2^31-1 or V above 2^31-4097");
    if (!g) C = 0;
    if (!g_top) top_k = 0;
    if (C > emu::kMaxGradTokens || top_k > emu::kMaxGradTokens - C) return unsupported("C + top_k above EMU_MAX_GRAD_TOKENS (1024)");
    if (T == 0 || V == 0) return set_error(EMU_OK, "");
    if (!logits || !lse || !grad || (C > 0 && !tokens) || (top_k > 0 && !top_tokens) || (g_entropy && !entropy))
        return invalid("null pointer");
    if (bad_ld(ldz, V, T) || bad_ld(ldgrad, V, T)) return invalid("leading dimension smaller than V");
    if (!aligned_to(logits, size_of(z_dtype)) || !aligned_to(grad, size_of(z_dtype)) || !aligned_to(tokens, 8) ||
        !aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(g, 4) || !aligned_to(g_entropy, 4) ||
        !aligned_to(top_tokens, 8) || !aligned_to(g_top, 4))
        return invalid("a pointer is not aligned to its element");
    emu::LogpGradParams p{};
    p.z = logits;
    p.ldz = ldz;
    p.T = T;
    p.V = V;
    p.tokens = tokens;
    p.C = C;
    p.lse = lse;
    p.entropy = entropy;
    p.g = g;
    p.ge = g_entropy;
    p.top_tok = top_tokens;
    p.gtop = g_top;
    p.k = (int)top_k;
    p.grad = grad;
    p.ldgrad = ldgrad;
    return done(emu::launch_logp_grad(z_dtype, p, stream));
}

}  // extern "C"
