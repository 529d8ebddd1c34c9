// ops_internal.h -- launch parameters of the operators of include/emu_operators.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/emu_operators.h"

namespace emu {

// Bytes read and written beyond which a launch passes by the last-level cache
// (256 MiB, of which it then finds little that its producer has left there).
constexpr int64_t kOnceBytes = int64_t(192) << 20;

struct NormParams {
    const void *x, *weight, *res;
    int64_t ldx, ldres;
    int64_t T, n;
    float eps;
    int w_dtype, q_dtype;
    void *q;
    int64_t ldq;
    const float *scale;   // one for all rows, or null: row_scales is written
    float *row_scales;
    void *h;              // null, or of the residual's type
    int64_t ldh;
    bool once;            // nothing of this size stays in a cache
};
// x_dtype: EMU_DT_BF16 .. FP32; res_dtype likewise (x's or FP32), ignored without a residual.
hipError_t launch_norm(int x_dtype, int res_dtype, const NormParams &p, hipStream_t stream);

struct NormGradParams {
    const void *g, *h, *weight, *gh;
    int64_t ldg, ldh, ldgh;
    int64_t T, n;
    float eps;
    int w_dtype, gh_dtype;
    void *gi;
    int64_t ldgi;
    void *gw;
    float *part;          // [norm_grad_parts(T, n), norm_grad_part_ld(n)]
    bool once;            // nothing of this size stays in a cache
};
int64_t norm_grad_parts(int64_t T, int64_t n);
int64_t norm_grad_part_ld(int64_t n);
hipError_t launch_norm_grad(int g_dtype, int h_dtype, const NormGradParams &p, hipStream_t stream);

struct Int8Params {
    const int8_t *a, *w;
    int64_t lda, ldw;
    int64_t M, N, K;
    const float *sa, *sw;
    int a_per_row, w_per_row;
    const void *bias;
    int bias_f32;         // the bias is binary32 (else of out's type)
    void *out;
    int out_dtype;
    int64_t ldo;
    void *ws;
};
int64_t int8_mm_workspace(int64_t M, int64_t N, int64_t K, bool aligned);
hipError_t launch_int8_mm(const Int8Params &p, bool aligned, hipStream_t stream);

struct LogpParams {
    const void *z;
    int64_t ldz, T, V;
    const int64_t *tokens;
    int64_t C;
    int k;
    float *logprobs, *entropy, *lse, *top_lp;
    int64_t *top_tok;
    void *ws;
};
int64_t logp_workspace(int64_t T, int64_t V, int k);
hipError_t launch_logp(int z_dtype, const LogpParams &p, hipStream_t stream);

struct LogpGradParams {
    const void *z;
    int64_t ldz, T, V;
    const int64_t *tokens;
    int64_t C;
    const float *lse, *entropy, *g, *ge;
    const int64_t *top_tok;
    const float *gtop;
    int k;
    void *grad;
    int64_t ldgrad;
};
constexpr int64_t kMaxGradTokens = EMU_MAX_GRAD_TOKENS;  // C + top_k: their tokens and values are kept in LDS
hipError_t launch_logp_grad(int z_dtype, const LogpGradParams &p, hipStream_t stream);

// Sets this thread's error text (emu_last_error_message) and returns s.
// Nothing is thrown: where the text cannot be stored it is left empty.
emu_status set_error(emu_status s, const char *text) noexcept;

}  // namespace emu
