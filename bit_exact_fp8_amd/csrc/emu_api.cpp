// emu_api.cpp -- the C ABI of include/emu_fp8gemm.h: argument checks, launch
// planning and kernel launches on the caller's stream.  No device memory is
// allocated here and the stream is never synchronised.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <string>

#include "../../include/emu_fp8gemm.h"
#include "emu_internal.h"
#include "fp_round.h"
#include "ops_internal.h"

namespace {

thread_local std::string g_last_error;

emu_status fail(emu_status s, const std::string &msg)
{
    g_last_error = msg;
    return s;
}

emu_status ok()
{
    g_last_error.clear();
    return EMU_OK;
}

constexpr int kMaxSplits = 65535;    // one grid dimension
constexpr int64_t kMaxGridY = 65535;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The profile's block width and split layout.
//  hopper (validation page, scope table rows "Hopper preset" and "Split-K on
//    the H100 PCIe"): 32-product blocks; nt = ceil(K/128) k-tiles,
//    tps = ceil(nt/S) per split, split s owns tiles [s*tps, (s+1)*tps)
//    (trailing splits may be empty); serial combination.
//  ada (validation page, scope table rows "Ada instruction model" and
//    "Split-K", claims table; limitations page, corrections table):
//    16-product blocks; 64-wide k-tiles dealt round-robin (tile t to split
//    t mod S); serial or pairwise combination.
struct Plan {
    int block;
    int tile_shift;
    int round_robin;
    int pairwise;
    int64_t tps;
    // slow accumulation with stored chunk results (see make_plan)
    int chunked;
    int chunk_groups;
    int chunks_per_group;
    int cps;
    // infinities resolved after the main kernel (see make_plan)
    int defer;
    // workspace layout: [split partials or chunk results][infinity lists];
    // the first part is required, the lists optional
    int64_t part_bytes, defer_bytes;
    int64_t required_bytes() const { return part_bytes; }
};

constexpr int64_t kChunk = 128;                          // slow-accumulation restart
constexpr int64_t kChunkWaveTarget = 4096;               // 4 waves on each SIMD
constexpr int64_t kMaxChunkWorkspace = int64_t(1) << 30; // bytes of stored chunk results
constexpr int64_t kResidentWgs = 256 * 3;                // 64x64 workgroups resident at once
constexpr double kDeferMinWork = 68719476736.0;          // M * N * K = 2^36
constexpr int64_t kDeferMaxK = emu::kDeferLdsBytes - 16; // one staged B row fits

static_assert(EMU_TILE_COUNT == emu::TILE_COUNT, "tile configurations of the header and the kernels");

// The plan options of a call: the caller's, or all automatic.
emu_plan_options options_of(const emu_plan_options *plan)
{
    if (plan) return *plan;
    emu_plan_options o;
    o.tile = EMU_TILE_AUTO;
    o.defer = -1;
    return o;
}

bool options_valid(const emu_plan_options &o)
{
    return o.tile >= EMU_TILE_AUTO && o.tile < EMU_TILE_COUNT && o.defer >= -1 && o.defer <= 1;
}

// The number of 128-chunks per group, from cps down to 1, whose workgroup
// count (tiles per group times groups) best fills whole rounds of `resident`
// workgroups, at least two rounds (one round leaves CUs idle while the last
// workgroups finish).
int64_t fill_groups(int64_t cps, int64_t tiles, int S, int64_t resident)
{
    int64_t best_cpg = cps;
    double best_fill = -1.0;
    for (int64_t cpg = cps; cpg >= 1; --cpg) {
        const int64_t groups = (cps + cpg - 1) / cpg;
        if (groups * S > kMaxSplits) break;
        const int64_t wgs = tiles * groups;
        const int64_t rounds = (wgs + resident - 1) / resident;
        const double fill = (double)wgs / (double)(rounds * resident) * (rounds >= 2 ? 1.0 : 0.5);
        if (fill > best_fill + 1e-9) {
            best_fill = fill;
            best_cpg = cpg;
        }
    }
    return best_cpg;
}

Plan make_plan(emu_profile profile, int64_t M, int64_t N, int64_t K, int S, int fast, const emu_plan_options &opt,
               int64_t chunk_limit)
{
    Plan p{};
    const bool ada = profile == EMU_PROFILE_ADA_SERIAL || profile == EMU_PROFILE_ADA_PAIRWISE;
    p.block = ada ? 16 : 32;
    p.tile_shift = ada ? 6 : 7;
    p.round_robin = ada ? 1 : 0;
    p.pairwise = profile == EMU_PROFILE_ADA_PAIRWISE ? 1 : 0;
    const int64_t W = int64_t(1) << p.tile_shift;
    const int64_t nt = (K + W - 1) / W;
    p.tps = (nt + S - 1) / S;
    p.chunked = 0;
    p.chunk_groups = 1;
    p.chunks_per_group = 1;
    p.cps = 1;
    // Slow accumulation restarts the chain every 128 positions of a split's
    // k-list (validation page, H100 claims table; scope table row "Slow
    // accumulation"), so its chunks are independent chains and only their
    // in-order binary32 additions are sequential.  When the output tiles
    // alone would leave the GPU under-occupied (fewer than 4,096 waves of
    // 64x64 tiles), the chunks are spread over the grid too and their
    // results stored for the combine kernel to add in order, as long as that
    // array stays within 1 GiB of workspace.  The chunks per group are chosen
    // so that the workgroup count fills whole rounds of the GPU's resident
    // 64x64 workgroups (3 per CU), at least two of them: one round leaves
    // CUs idle while the last workgroups finish (measured on the
    // 256 x 4096 x 4096 slow workload: 0.514 ms with one round of 768
    // workgroups, 0.482 ms with two).
    if (!fast && nt > 0) {
        const int64_t tiles_max = p.round_robin ? (nt + S - 1) / S : p.tps;
        const int64_t max_len = (tiles_max * W < K) ? tiles_max * W : K;
        const int64_t cps = (max_len + kChunk - 1) / kChunk;
        const int64_t tiles64 = ((M + 63) / 64) * ((N + 63) / 64) * (int64_t)S;
        const int64_t bytes = (int64_t)S * cps * M * N * 4;
        const int64_t limit = (chunk_limit >= 0 && chunk_limit < kMaxChunkWorkspace) ? chunk_limit : kMaxChunkWorkspace;
        if (cps >= 2 && tiles64 * 4 < kChunkWaveTarget && bytes <= limit) {
            const int64_t best_cpg = fill_groups(cps, tiles64, S, kResidentWgs);
            const int64_t groups = (cps + best_cpg - 1) / best_cpg;
            if (groups >= 2) {
                p.chunked = 1;
                p.chunks_per_group = (int)best_cpg;
                p.chunk_groups = (int)groups;
                p.cps = (int)cps;
            }
        }
    }
    p.part_bytes = (p.chunked ? (int64_t)S * p.cps : (S > 1 ? (int64_t)S : 0)) * M * N * 4;
    // An output whose e5m2 row holds an infinity is non-finite whatever the
    // chain computes; in the main kernel each such output reads its rows
    // once more, which on large problems with infinities in many rows can
    // double the run time (8192^3 with one e5m2 code in 1,000 infinite:
    // 88.8 ms against 45.0 ms).  On problems of 2^36 multiply-adds and more
    // the main kernel leaves those outputs alone; a pass over the e5m2 rows
    // lists their infinities (about 10 us per 64 MiB of codes, the only cost
    // when there are none) and a fix-up kernel resolves each affected output
    // from the lists.  The lists take (kDeferCap + 1) 32-bit words per row of
    // the larger operand, from the optional end of the workspace; stored
    // chunk results keep the main kernel's own handling.
    p.defer = 0;
    p.defer_bytes = 0;
    const int forced_defer = opt.defer;
    const bool big = (double)M * (double)N * (double)K >= kDeferMinWork;
    if (!p.chunked && M > 0 && N > 0 && K > 0 && K <= kDeferMaxK && forced_defer != 0 &&
        (big || forced_defer == 1)) {
        p.defer = 1;
        p.defer_bytes = (M > N ? M : N) * (int64_t)(emu::kDeferCap + 1) * 4;
    }
    return p;
}

// Pick the tile configuration with the best expected throughput: its
// measured steady-state efficiency on MI355X (fraction of the integer-VALU
// roofline on a full machine) scaled down by how far the launch falls short
// of 2 waves on each of the 1,024 SIMDs and of one workgroup on each of the
// 256 CUs.
int choose_tile(int64_t M, int64_t N, int S, const emu_plan_options &opt)
{
    if (opt.tile >= 0) return opt.tile;
    struct Cand {
        int cfg;
        double eff;
    };
    const Cand cands[] = {{emu::TILE_64x64_MX, 1.16}, {emu::TILE_64x128_MX, 1.07}, {emu::TILE_64x64, 0.90},
                          {emu::TILE_64x128, 0.87}, {emu::TILE_32x64, 0.60}, {emu::TILE_32x32, 0.60},
                          {emu::TILE_16x16_G2, 0.30}, {emu::TILE_16x16_G4, 0.24}, {emu::TILE_16x8_G4, 0.24}};
    int best = emu::TILE_16x8_G4;
    double best_est = -1.0;
    for (const Cand &c : cands) {
        const emu::TileShape t = emu::tile_shape(c.cfg);
        const double wgs = (double)((M + t.bm - 1) / t.bm) * (double)((N + t.bn - 1) / t.bn) * S;
        const double waves = wgs * (t.threads / 64);
        const double est = c.eff * (waves >= 2048.0 ? 1.0 : waves / 2048.0) * (wgs >= 256.0 ? 1.0 : wgs / 256.0);
        if (est > best_est) {
            best_est = est;
            best = c.cfg;
        }
    }
    // The 32x32 tile staging 4 K-blocks per barrier with the block maxima on
    // the matrix cores issues a sixth fewer VALU instructions than the VALU
    // maxima and hides more load latency than 2 K-blocks per barrier; its 72
    // KB of LDS leave room for two workgroups per CU.  Measured on MI355X (A/B
    // in one session) it wins up to 720 workgroups: 64 x 5760 x 1920 (360)
    // 0.1445 ms against 0.1588 ms for the 4-stage VALU form; 256 x 2048 x 4096
    // (512) 0.307 against 0.339 ms; 128 x 5760 x 1920 (720) 0.224 against
    // 0.228 ms for the 2-stage VALU form, which stays the choice beyond.
    // (Reading every matrix-instruction result since costs it about 3%:
    // 0.315 and 0.232 ms on the last two.)
    // Between 257 and 384 such workgroups, the CUs that hold two of them set
    // the time while the others idle for half of it; the 32x16 form of the
    // same tile (2x1 thread tiles, 5 K-blocks per barrier, three workgroups
    // per CU) splits the work finer: 64 x 5760 x 1920 (360 32x32 workgroups)
    // 0.130 against 0.144 ms (with 2, 3 and 4 K-blocks per barrier 0.136,
    // 0.134 and 0.132 ms; 6 would leave room for two workgroups per CU only).
    // With whole rounds of 32x32 workgroups it only costs (256 x 2048 x 4096,
    // 512: 0.378 against 0.305 ms with 3 K-blocks per barrier).
    if (best == emu::TILE_32x32) {
        const int64_t wgs = ((M + 31) / 32) * ((N + 31) / 32) * (int64_t)S;
        if (wgs > 256 && wgs <= 384)
            best = emu::TILE_32x16_MX_S5;
        else if (wgs <= 3 * 256)
            best = emu::TILE_32x32_MX_S4;
    }
    return best;
}

emu_status check_common(const uint8_t *x, emu_fp8_format xf, int64_t ldx, const uint8_t *w,
                        emu_fp8_format wf, int64_t ldw, int64_t M, int64_t N, int64_t K, int split_S,
                        emu_profile profile)
{
    if (M < 0 || N < 0 || K < 0) return fail(EMU_ERR_INVALID_ARG, "negative dimension");
    if ((xf != EMU_FP8_E4M3FN && xf != EMU_FP8_E5M2) || (wf != EMU_FP8_E4M3FN && wf != EMU_FP8_E5M2))
        return fail(EMU_ERR_INVALID_ARG, "unknown FP8 format");
    if (split_S < 1) return fail(EMU_ERR_INVALID_ARG, "split_S must be >= 1");
    if (profile != EMU_PROFILE_HOPPER && profile != EMU_PROFILE_ADA_SERIAL && profile != EMU_PROFILE_ADA_PAIRWISE)
        return fail(EMU_ERR_INVALID_ARG, "unknown profile");
    if (split_S > kMaxSplits) return fail(EMU_ERR_UNSUPPORTED, "split_S above 65535");
    if (ldx < K || ldw < K) return fail(EMU_ERR_INVALID_ARG, "leading dimension smaller than K");
    if (xf == EMU_FP8_E5M2 && wf == EMU_FP8_E5M2)
        return fail(EMU_ERR_REJECTED, "e5m2 x e5m2 is rejected (as torch does)");
    if (K % 16 || N % 16) return fail(EMU_ERR_REJECTED, "K and N must be multiples of 16");
    if (ldx % 16 || ldw % 16) return fail(EMU_ERR_REJECTED, "ldx and ldw must be multiples of 16");
    if (M > 0 && N > 0 && K > 0) {
        if (!x || !w) return fail(EMU_ERR_INVALID_ARG, "null operand pointer");
        if (!aligned16(x) || !aligned16(w)) return fail(EMU_ERR_REJECTED, "operands must be 16-byte aligned");
    }
    if (M > INT32_MAX || N > INT32_MAX) return fail(EMU_ERR_UNSUPPORTED, "M or N above 2^31-1");
    return EMU_OK;
}

// The combine kernel over S split partials (or chunk results) in `part`.
emu_status launch_combine_of(const Plan &plan, float *part, int S, int64_t M, int64_t N, int out_kind,
                             void *out, int64_t ldo, const float *sx, const float *sw, const float *sr,
                             hipStream_t stream)
{
    emu::CombineParams c{};
    c.part = part;
    c.S = S;
    c.cps = plan.cps;
    c.pairwise = plan.pairwise;
    c.M = (int)M;
    c.N = (int)N;
    c.out_kind = out_kind;
    c.out = out;
    c.ldo = ldo;
    c.scale_x = sx;
    c.scale_w = sw;
    c.scale_result = sr;
    hipError_t e = emu::launch_combine(c, stream);
    if (e != hipSuccess) return fail(EMU_ERR_DEVICE, std::string("combine kernel launch: ") + hipGetErrorString(e));
    return EMU_OK;
}

emu_status run(const Plan &plan, const uint8_t *x, emu_fp8_format xf, int64_t ldx, const uint8_t *w,
               emu_fp8_format wf, int64_t ldw, int64_t M, int64_t N, int64_t K, const float *sx, const float *sw,
               const float *sr, void *out, int out_kind, size_t out_elem, int64_t ldo, int fast, int S,
               void *workspace, size_t workspace_bytes, hipStream_t stream, const emu_plan_options &opt)
{
    const int Z = S * plan.chunk_groups;  // grid z: splits, times chunk groups
    const int cfg = choose_tile(M, N, Z, opt);
    const emu::TileShape ts = emu::tile_shape(cfg);
    const int64_t rows_per_launch = kMaxGridY * ts.bm;

    emu::MainParams p{};
    p.ldx = ldx;
    p.ldw = ldw;
    p.N = (int)N;
    p.K = K;
    p.tile_shift = plan.tile_shift;
    p.round_robin = plan.round_robin;
    p.tps = plan.tps;
    p.S = S;
    p.fast = fast ? 1 : 0;
    p.chunked = plan.chunked;
    p.chunk_groups = plan.chunk_groups;
    p.chunks_per_group = plan.chunks_per_group;
    p.cps = plan.cps;
    const bool partials = S > 1 || plan.chunked;  // the combine kernel finishes the job
    p.scale_x = sx;
    p.scale_w = sw;
    p.scale_result = sr;
    p.w = w;
    // deferred infinities: only where a format has them and the workspace
    // holds the lists
    const int64_t required = plan.required_bytes();
    emu::DeferParams d{};
    const bool defer = plan.defer && (xf == EMU_FP8_E5M2 || wf == EMU_FP8_E5M2) && workspace &&
                       (reinterpret_cast<uintptr_t>(workspace) & 3u) == 0 &&
                       (int64_t)workspace_bytes >= required + plan.defer_bytes;
    if (defer) {
        const bool a_is_w = wf == EMU_FP8_E5M2;
        d.a = a_is_w ? w : x;
        d.lda = a_is_w ? ldw : ldx;
        d.b = a_is_w ? x : w;
        d.ldb = a_is_w ? ldx : ldw;
        d.ra = (int)(a_is_w ? N : M);
        d.rb = (int)(a_is_w ? M : N);
        d.K = K;
        d.a_is_w = a_is_w ? 1 : 0;
        d.info = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + required);
        d.pos = d.info + (M > N ? M : N);
        const int64_t br = emu::kDeferLdsBytes / (K + 16);
        d.b_rows = (int)(br < 16 ? br : 16);
        const int64_t ar = (d.ra + kMaxGridY - 1) / kMaxGridY;
        d.a_rows = (int)(ar > 2048 ? ar : 2048);
        d.out_kind = out_kind;
        d.out = out;
        d.ldo = ldo;
        d.scale_x = sx;
        d.scale_w = sw;
        d.scale_result = sr;
        hipError_t e = emu::launch_inf_rows(d, stream);
        if (e != hipSuccess)
            return fail(EMU_ERR_DEVICE, std::string("infinity row kernel launch: ") + hipGetErrorString(e));
        p.defer_specials = 1;
    }
    if (!partials) {
        p.out_kind = out_kind;
        p.ldo = ldo;
        p.split_stride = 0;
    } else {
        p.out_kind = emu::OUT_ACC_F32;
        p.ldo = N;
        p.split_stride = M * N;
    }
    for (int64_t m_start = 0; m_start < M; m_start += rows_per_launch) {
        const int64_t rows = (M - m_start < rows_per_launch) ? M - m_start : rows_per_launch;
        p.x = x ? x + m_start * ldx : nullptr;
        p.M = (int)rows;
        if (!partials)
            p.out = static_cast<char *>(out) + m_start * ldo * (int64_t)out_elem;
        else
            p.out = static_cast<char *>(workspace) + m_start * N * 4;
        hipError_t e = emu::launch_main(cfg, plan.block, xf, wf, p, Z, stream);
        if (e != hipSuccess) return fail(EMU_ERR_DEVICE, std::string("main kernel launch: ") + hipGetErrorString(e));
    }
    if (partials) {
        emu_status st = launch_combine_of(plan, static_cast<float *>(workspace), S, M, N, out_kind, out, ldo,
                                          sx, sw, sr, stream);
        if (st != EMU_OK) return st;
    }
    if (defer) {
        hipError_t e = emu::launch_inf_fixup(d, stream);
        if (e != hipSuccess)
            return fail(EMU_ERR_DEVICE, std::string("infinity fix-up kernel launch: ") + hipGetErrorString(e));
    }
    return ok();
}

// emu_scaled_mm's checks, then its launches.  out_dtype < 0 asks for the
// accumulator (emu_accumulate: acc in `out`, leading dimension ldo, scales
// not read).  chunk_limit caps the bytes of stored slow-mode chunk results
// the plan may use (the no-allocation entry point's scratch size; -1: no
// cap beyond the plan's own).
emu_status scaled_mm_call(const uint8_t *x, emu_fp8_format x_fmt, int64_t ldx, const uint8_t *w,
                          emu_fp8_format w_fmt, int64_t ldw, int64_t M, int64_t N, int64_t K, const float *scale_x,
                          const float *scale_w, const float *scale_result, void *out, int out_dtype, int64_t ldo,
                          int fast_accum, int split_S, emu_profile profile, void *workspace, size_t workspace_bytes,
                          hipStream_t stream, const emu_plan_options *plan, int64_t chunk_limit)
{
    emu_status s = check_common(x, x_fmt, ldx, w, w_fmt, ldw, M, N, K, split_S, profile);
    if (s != EMU_OK) return s;
    const emu_plan_options opt = options_of(plan);
    if (!options_valid(opt)) return fail(EMU_ERR_INVALID_ARG, "plan options out of range");
    const bool acc_only = out_dtype < 0;
    int kind = emu::OUT_ACC_F32;
    size_t elem = 4;
    if (!acc_only) {
        switch (out_dtype) {
        case EMU_OUT_BF16: kind = emu::OUT_BF16; elem = 2; break;
        case EMU_OUT_FP16: kind = emu::OUT_F16; elem = 2; break;
        case EMU_OUT_FP32: kind = emu::OUT_F32; elem = 4; break;
        case EMU_OUT_E4M3FN: kind = emu::OUT_E4M3; elem = 1; break;
        case EMU_OUT_E5M2: kind = emu::OUT_E5M2; elem = 1; break;
        default: return fail(EMU_ERR_INVALID_ARG, "unknown output dtype");
        }
        const bool fp8_out = kind == emu::OUT_E4M3 || kind == emu::OUT_E5M2;
        if (scale_result && !fp8_out) return fail(EMU_ERR_UNSUPPORTED, "scale_result is for FP8 outputs only");
        if (out_dtype == EMU_OUT_E5M2 && x_fmt == EMU_FP8_E4M3FN && w_fmt == EMU_FP8_E4M3FN)
            return fail(EMU_ERR_REJECTED, "e4m3fn x e4m3fn -> e5m2 is rejected (as cuBLASLt does)");
    }
    if (ldo < N) return fail(EMU_ERR_INVALID_ARG, acc_only ? "ldacc smaller than N" : "ldo smaller than N");
    if (M == 0 || N == 0) return ok();
    if (acc_only) {
        if (!out) return fail(EMU_ERR_INVALID_ARG, "null accumulator pointer");
        if (reinterpret_cast<uintptr_t>(out) & 3u) return fail(EMU_ERR_INVALID_ARG, "acc must be 4-byte aligned");
    } else {
        if (!out || !scale_x || !scale_w) return fail(EMU_ERR_INVALID_ARG, "null output or scale pointer");
        if (!aligned16(out)) return fail(EMU_ERR_REJECTED, "out must be 16-byte aligned");
    }
    const Plan pl = make_plan(profile, M, N, K, split_S, fast_accum, opt, chunk_limit);
    const size_t need = (size_t)pl.required_bytes();
    if (workspace_bytes < need || (need && !workspace))
        return fail(EMU_ERR_WORKSPACE, "workspace smaller than the split partials need");
    if (need && (reinterpret_cast<uintptr_t>(workspace) & 3u))
        return fail(EMU_ERR_INVALID_ARG, "workspace must be 4-byte aligned");
    // The accumulator's call does not read the scale pointers.
    return run(pl, x, x_fmt, ldx, w, w_fmt, ldw, M, N, K, acc_only ? nullptr : scale_x,
               acc_only ? nullptr : scale_w, acc_only ? nullptr : scale_result, out, kind, elem, ldo, fast_accum,
               split_S, workspace, workspace_bytes, stream, opt);
}

}  // namespace

namespace emu {

emu_status scaled_mm_in_scratch(const uint8_t *x, emu_fp8_format x_fmt, int64_t ldx, const uint8_t *w,
                                emu_fp8_format w_fmt, int64_t ldw, int64_t M, int64_t N, int64_t K,
                                const float *scale_x, const float *scale_w, const float *scale_result, void *out,
                                emu_out_dtype out_dtype, int64_t ldo, int fast_accum, int split_S,
                                emu_profile profile, void *(*scratch)(size_t *bytes, std::string *err),
                                size_t scratch_bytes, hipStream_t stream, const emu_plan_options *plan)
{
    // the same checks as emu_scaled_mm, then the required part of the plan
    // (stored chunk results capped at the scratch size) against the scratch,
    // before the scratch is looked up
    emu_status s = check_common(x, x_fmt, ldx, w, w_fmt, ldw, M, N, K, split_S, profile);
    if (s != EMU_OK) return s;
    const emu_plan_options opt = options_of(plan);
    if (!options_valid(opt)) return fail(EMU_ERR_INVALID_ARG, "plan options out of range");
    if (M > 0 && N > 0) {
        const Plan pl = make_plan(profile, M, N, K, split_S, fast_accum, opt, (int64_t)scratch_bytes);
        if ((size_t)pl.required_bytes() > scratch_bytes)
            return fail(EMU_ERR_WORKSPACE, "the split partials need " + std::to_string(pl.required_bytes()) +
                                               " bytes, more than the " + std::to_string(scratch_bytes) +
                                               "-byte scratch of the no-allocation entry point");
    }
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (M > 0 && N > 0) {
        std::string err;
        ws = scratch(&ws_bytes, &err);
        if (!ws) return fail(EMU_ERR_DEVICE, err);
    }
    return scaled_mm_call(x, x_fmt, ldx, w, w_fmt, ldw, M, N, K, scale_x, scale_w, scale_result, out,
                          (int)out_dtype < 0 ? 1000 : (int)out_dtype, ldo, fast_accum, split_S, profile, ws,
                          ws_bytes, stream, plan, (int64_t)scratch_bytes);
}

}  // namespace emu

namespace emu {

emu_status set_error(emu_status s, const char *text) noexcept
{
    try {
        g_last_error = text;
    } catch (...) {
        g_last_error.clear();
    }
    return s;
}

}  // namespace emu

extern "C" {

size_t emu_workspace_bytes(int64_t M, int64_t N, int64_t K, int split_S, int fast_accum, emu_profile profile,
                           const emu_plan_options *plan)
{
    if (M < 0 || N < 0 || K < 0 || split_S < 1 || split_S > kMaxSplits) return 0;
    const emu_plan_options opt = options_of(plan);
    if (!options_valid(opt)) return 0;
    const Plan pl = make_plan(profile, M, N, K, split_S, fast_accum, opt, -1);
    return (size_t)(pl.required_bytes() + pl.defer_bytes);
}

emu_status emu_scaled_mm(const uint8_t *x, emu_fp8_format x_fmt, int64_t ldx, const uint8_t *w,
                         emu_fp8_format w_fmt, int64_t ldw, int64_t M, int64_t N, int64_t K,
                         const float *scale_x, const float *scale_w, const float *scale_result, void *out,
                         emu_out_dtype out_dtype, int64_t ldo, int fast_accum, int split_S, emu_profile profile,
                         void *workspace, size_t workspace_bytes, hipStream_t stream, const emu_plan_options *plan)
{
    // an out-of-range enum value is passed on as is and refused there
    return scaled_mm_call(x, x_fmt, ldx, w, w_fmt, ldw, M, N, K, scale_x, scale_w, scale_result, out,
                          (int)out_dtype < 0 ? 1000 : (int)out_dtype, ldo, fast_accum, split_S, profile, workspace,
                          workspace_bytes, stream, plan, -1);
}

emu_status emu_accumulate(const uint8_t *x, emu_fp8_format x_fmt, int64_t ldx, const uint8_t *w,
                          emu_fp8_format w_fmt, int64_t ldw, int64_t M, int64_t N, int64_t K, float *acc,
                          int64_t ldacc, int fast_accum, int split_S, emu_profile profile, void *workspace,
                          size_t workspace_bytes, hipStream_t stream, const emu_plan_options *plan)
{
    return scaled_mm_call(x, x_fmt, ldx, w, w_fmt, ldw, M, N, K, nullptr, nullptr, nullptr, acc, -1, ldacc,
                          fast_accum, split_S, profile, workspace, workspace_bytes, stream, plan, -1);
}

emu_status emu_accumulate_c(const uint8_t *x, emu_fp8_format x_fmt, int64_t ldx, const uint8_t *w,
                            emu_fp8_format w_fmt, int64_t ldw, int64_t M, int64_t N, int64_t K, const float *c_in,
                            int64_t ldc, float *acc, int64_t ldacc, emu_profile profile, hipStream_t stream,
                            const emu_plan_options *plan)
{
    emu_status s = check_common(x, x_fmt, ldx, w, w_fmt, ldw, M, N, K, 1, profile);
    if (s != EMU_OK) return s;
    const emu_plan_options opt = options_of(plan);
    if (!options_valid(opt)) return fail(EMU_ERR_INVALID_ARG, "plan options out of range");
    if (ldacc < N || ldc < N) return fail(EMU_ERR_INVALID_ARG, "ldacc or ldc smaller than N");
    if (M == 0 || N == 0) return ok();
    if (!acc || !c_in) return fail(EMU_ERR_INVALID_ARG, "null accumulator pointer");
    if ((reinterpret_cast<uintptr_t>(acc) & 3u) || (reinterpret_cast<uintptr_t>(c_in) & 3u))
        return fail(EMU_ERR_INVALID_ARG, "acc and c_in must be 4-byte aligned");
    const Plan pl = make_plan(profile, M, N, K, 1, 1, opt, -1);
    const int cfg = choose_tile(M, N, 1, opt);
    const emu::TileShape ts = emu::tile_shape(cfg);
    const int64_t rows_per_launch = kMaxGridY * ts.bm;
    emu::MainParams p{};
    p.ldx = ldx;
    p.ldw = ldw;
    p.N = (int)N;
    p.K = K;
    p.tile_shift = pl.tile_shift;
    p.round_robin = pl.round_robin;
    p.tps = pl.tps;
    p.S = 1;
    p.fast = 1;
    p.chunk_groups = 1;
    p.chunks_per_group = 1;
    p.cps = 1;
    p.out_kind = emu::OUT_ACC_F32;
    p.ldo = ldacc;
    p.w = w;
    p.ldc = ldc;
    for (int64_t m_start = 0; m_start < M; m_start += rows_per_launch) {
        const int64_t rows = (M - m_start < rows_per_launch) ? M - m_start : rows_per_launch;
        p.x = x ? x + m_start * ldx : nullptr;
        p.M = (int)rows;
        p.c_in = c_in + m_start * ldc;
        p.out = acc + m_start * ldacc;
        hipError_t e = emu::launch_main_cin(cfg, pl.block, x_fmt, w_fmt, p, stream);
        if (e != hipSuccess) return fail(EMU_ERR_DEVICE, std::string("main kernel launch: ") + hipGetErrorString(e));
    }
    return ok();
}

const char *emu_status_string(emu_status status)
{
    switch (status) {
    case EMU_OK: return "ok";
    case EMU_ERR_INVALID_ARG: return "invalid argument";
    case EMU_ERR_REJECTED: return "rejected (a call torch / cuBLASLt would refuse)";
    case EMU_ERR_UNSUPPORTED: return "unsupported feature";
    case EMU_ERR_WORKSPACE: return "workspace too small";
    case EMU_ERR_DEVICE: return "device error";
    }
    return "unknown status";
}

const char *emu_last_error_message(void) { return g_last_error.c_str(); }

int emu_abi_version(void) { return EMU_ABI_VERSION; }

uint32_t emu_host_mul_f32(uint32_t a, uint32_t b) { return emu::mul_f32(a, b); }
uint32_t emu_host_epilogue_f32(uint32_t acc, uint32_t alpha) { return emu::canon_f32(emu::epilogue_f32(acc, alpha)); }
uint16_t emu_host_f32_to_bf16(uint32_t f) { return emu::f32_to_bf16(f); }
uint16_t emu_host_f32_to_f16(uint32_t f) { return emu::f32_to_f16(f); }
uint8_t emu_host_f32_to_e4m3fn(uint32_t f) { return emu::f32_to_fp8_sat<true>(f); }
uint8_t emu_host_f32_to_e5m2(uint32_t f) { return emu::f32_to_fp8_sat<false>(f); }

}  // extern "C"
