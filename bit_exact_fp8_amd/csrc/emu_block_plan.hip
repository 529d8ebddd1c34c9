// emu_block_plan.hip -- emu_block_scaled_mm and its form by groups of rows:
// which kernel of emu_block_mm.hip runs, operands laid out anew where their
// rows are not aligned to 16 bytes, and the sums of a split K.
#include <hip/hip_runtime.h>

#include "ops_block.h"
#include "ops_tiles.h"

namespace emu {

extern template void launch_block_kernel<0, 0>(const BlockMMParams &, const BlockPlan &, float *, hipStream_t);
extern template void launch_block_kernel<0, 1>(const BlockMMParams &, const BlockPlan &, float *, hipStream_t);
extern template void launch_block_kernel<1, 0>(const BlockMMParams &, const BlockPlan &, float *, hipStream_t);
extern template void launch_block_kernel<1, 1>(const BlockMMParams &, const BlockPlan &, float *, hipStream_t);

namespace {

__global__ __launch_bounds__(256) void block_repack(RepackRows a, RepackRows b, int64_t of_a, int64_t base)
{
    const int64_t group = base + blockIdx.x;
    if (group < of_a)
        repack_rows(a, group);
    else
        repack_rows(b, group - of_a);
}

// The sums of S splits and the epilogue, four outputs a thread.
__global__ __launch_bounds__(256) void block_join(BlockMMParams p, const float *part, int S)
{
    const int64_t quads = (p.N + 3) / 4, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = id / quads, n = id % quads * 4;
    if (m >= p.M) return;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    typedef f32x4 words __attribute__((aligned(4)));
    const float *at = part + m * p.N + n;
    for (int s = 0; s < S; ++s, at += p.M * p.N) {
        if (n + 4 <= p.N) {
            sum += *reinterpret_cast<const words *>(at);
        } else {
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) sum[e] += at[e];
        }
    }
    with_type(p.out_dtype, [&](auto *type) {
        typedef std::remove_pointer_t<decltype(type)> E;
        if (p.bias) {
            for (int e = 0; e < 4; ++e) {
                const int64_t c = n + e < p.N ? n + e : p.N - 1;
                sum[e] += p.bias_f32 ? static_cast<const float *>(p.bias)[c] : (float)static_cast<const E *>(p.bias)[c];
            }
        }
        store_valid(static_cast<E *>(p.out) + m * p.ldo + n, __builtin_convertvector(sum, Four<E>), p.N - n);
    });
}

// The tiles, with what the CUs take for a round of one tile each or (where LDS
// has room for two) of two: microseconds to begin and end, and for each stage in
// kHardware.  Measured at 4096 x 4096 of K with 128 to 2048 rows and at 8192^3.
struct Tile {
    int bm, bn, per_cu;
    double ends, stage, stage2;
};
constexpr Tile kTiles[] = {{64, 64, 2, 3.0, 0.28, 0.45}, {128, 128, 2, 4.0, 0.80, 1.15}, {64, 128, 2, 3.5, 0.42, 0.70},
                           {256, 128, 1, 6.0, 0.92, 0}, {256, 256, 1, 12.0, 1.45, 0}};
constexpr double kStageOf[] = {1.0, 1.2, 2.0};  // of each mode, relative to kHardware

double tiles_us(const Tile &t, int64_t tiles, int64_t stages, int mode)
{
    const double one = t.ends + (double)stages * t.stage * kStageOf[mode], two = t.ends + (double)stages * t.stage2 * kStageOf[mode];
    const int64_t round = 256 * t.per_cu, left = tiles % round;
    return (double)(tiles / round) * (t.per_cu == 2 ? two : one) + (left == 0 ? 0.0 : left > 256 ? two : one);
}

struct Plan {
    BlockPlan kernel;
    bool repack_a, repack_w;
    int64_t ld;                  // of repacked operands
    int64_t a_bytes, w_bytes, part_bytes;
};

bool needs_repack(int64_t K, bool aligned) { return K > 0 && (!aligned || K % 16 != 0); }

int64_t mean_rows(int64_t M, int E, bool grouped) { return grouped && E > 0 ? ceil_div(M, E) : M; }

Plan make_plan(int64_t M, int64_t N, int64_t K, int E, bool grouped, int mode, bool a_aligned, bool w_aligned)
{
    Plan p{};
    BlockPlan &k = p.kernel;
    k.mode = mode;
    k.S = 1;
    k.tile = -1;
    const int64_t total = blocks_of(K);
    k.stages = total ? (int)total : 1;
    const bool ra = needs_repack(K, a_aligned), rw = needs_repack(K, w_aligned);
    // Operands that are not aligned are laid out anew for tiles, which for up to
    // 64 rows (of each group, in the mean) takes longer than to read them in words.
    // More waves for a longer K: 1 x 4096 x 4099 takes 6.7 us with 16 of them and 8.2
    // with 4, 32 x 4096 x 4099 11.7 with 8 and 12.8 with 4; up to K = 4096 they are
    // within 0.6 us (1921: 5.2 and 5.8, 8.9 and 9.0).  64 rows, K = 4099: 17.8 with 8,
    // 20.8 with 4, 28.5 with 16.
    const int64_t mean = mean_rows(M, E, grouped);
    if ((mean <= 64 && (ra || rw)) || K == 0) {
        k.rows = mean <= 16 || K == 0 ? 1 : mean <= 32 ? 2 : 4;
        k.waves = k.rows == 4 ? 8 : K > 4096 ? (k.rows == 1 ? 16 : 8) : 4;
        return p;
    }
    p.repack_a = ra;
    p.repack_w = rw;
    p.ld = total * kStage;
    p.a_bytes = ra ? M * p.ld : 0;
    p.w_bytes = rw ? (int64_t)E * N * p.ld : 0;
    // The fastest estimate; a split of K takes 5 us more and its sums at 4 TB/s,
    // there and back.  Each group's last tile is half full in the mean.
    double best = 0.0;
    for (int i = 0; i < (mode == kExact ? 2 : 5); ++i)
        for (int S = 1; S <= (grouped ? 1 : 8); S *= 2) {
            const int64_t stages = ceil_div(total, S);
            if (S > 1 && stages < 4) break;
            const int64_t tm = grouped ? ceil_div(M, kTiles[i].bm) + (E < M ? E : M) / 2 : ceil_div(M, kTiles[i].bm);
            double us = tiles_us(kTiles[i], tm * ceil_div(N, kTiles[i].bn) * S, stages, mode);
            if (S > 1) us += 5.0 + (double)S * (double)M * (double)N * 8.0 / 4e6;
            if (k.tile >= 0 && us >= best) continue;
            best = us;
            k.tile = i;
            k.S = S;
        }
    // Up to 16 rows read w once, straight into registers, and wait for nothing,
    // but read a again for every 16 columns (16 x 4096 x 4096: 10.0 us, in tiles
    // 11.2; 16 x 8192 x 8192: 24.2 and 16.7).  Groups take tiles in any case: 32 x
    // 4096 x 2048 over 16 of them 29.9 us, in tiles 24.2.  With 4 waves 1 x 5760 x
    // 1920 takes 4.9 us, with 16 6.0; x 8192 11.9 and 12.8, which on 4096 columns
    // (x 8195, in words) is 12.4 and 9.8.
    if (!grouped && M <= 16 && 2.5 + (double)N * (double)K * (1.0 + (double)M / 16.0) / 7.5e6 < best) {
        k.tile = -1;
        k.S = k.rows = 1;
        k.waves = K > 4096 ? 16 : 4;
        return p;
    }
    k.stages = total ? (int)ceil_div(total, k.S) : 1;
    k.S = total ? (int)ceil_div(total, k.stages) : 1;
    p.part_bytes = k.S > 1 ? k.S * M * N * 4 : 0;
    return p;
}

int mode_of(bool fp32_out, bool e8m0) { return fp32_out ? kExact : e8m0 ? kHardware : kScaled; }

// A launch's rows (dense) and columns, so that its grid stays below 2^32
// threads: of groups, whose rows one launch has to hold, fewer columns at a time.
// Without K block_join alone makes the outputs, four a thread: at most 2^33 of them.
constexpr int64_t kSliceM = 1 << 18, kSliceN = 1 << 17;
int64_t slice_m(int64_t M, int64_t K, bool grouped) { return grouped ? M : K ? kSliceM : (int64_t(1) << 33) / kSliceN; }
int64_t slice_n(int64_t M, int64_t K, int E, bool grouped)
{
    if (!grouped) return kSliceN;
    // at most 2^21 workgroups, of the few rows' kernel or of the smallest tile
    const int64_t unit = mean_rows(M, E, grouped) <= 64 || K == 0 ? 16 : 64;
    const int64_t n = (int64_t(1) << 21) / (ceil_div(M, unit) + E + 1) * unit / kBlock * kBlock;
    return n < kBlock ? kBlock : n > kSliceN ? kSliceN : n;
}

bool in_words(const BlockMMParams &p)
{
    return ((reinterpret_cast<uintptr_t>(p.a) | reinterpret_cast<uintptr_t>(p.w) | p.lda | p.ldw | p.w_stride) & 3) == 0;
}

void launch_slice(int a_dtype, int w_dtype, BlockMMParams p, bool a_aligned, bool w_aligned, hipStream_t stream)
{
    const dim3 quads((unsigned)ceil_div(p.M * ceil_div(p.N, 4), 256));
    if (p.K == 0 && !p.ends) {
        hipLaunchKernelGGL(block_join, quads, dim3(256), 0, stream, p, nullptr, 0);
        return;
    }
    const Plan plan = make_plan(p.M, p.N, p.K, p.E, p.ends != nullptr, mode_of(p.out_dtype == EMU_DT_FP32, p.e8m0), a_aligned, w_aligned);
    BlockPlan k = plan.kernel;
    k.words = in_words(p);
    char *ws = static_cast<char *>(p.ws);
    RepackRows a{}, w{};
    if (plan.repack_a) {
        a = repack_job(p.a, p.lda, 0, p.M, p.M, p.K, reinterpret_cast<int8_t *>(ws), plan.ld);
        p.a = a.out;
        p.lda = plan.ld;
    }
    if (plan.repack_w) {
        w = repack_job(p.w, p.ldw, p.w_stride, p.N, p.E * p.N, p.K, reinterpret_cast<int8_t *>(ws + plan.a_bytes), plan.ld);
        p.w = w.out;
        p.ldw = plan.ld;
        p.w_stride = p.N * plan.ld;
    }
    launch_repack(a, w, stream);
    if (plan.repack_a && plan.repack_w) p.K = plan.ld;
    float *part = k.S > 1 ? reinterpret_cast<float *>(ws + plan.a_bytes + plan.w_bytes) : nullptr;
    const bool a5 = a_dtype == EMU_DT_E5M2, w5 = w_dtype == EMU_DT_E5M2;
    (a5 ? w5 ? launch_block_kernel<1, 1> : launch_block_kernel<1, 0> : w5 ? launch_block_kernel<0, 1> : launch_block_kernel<0, 0>)(
        p, k, part, stream);
    if (part)
        hipLaunchKernelGGL(block_join, quads, dim3(256), 0, stream, p, part, k.S);
}

}  // namespace

RepackRows repack_job(const int8_t *in, int64_t ld, int64_t stride, int64_t per, int64_t total, int64_t K, int8_t *out, int64_t ldo)
{
    const bool words = ((reinterpret_cast<uintptr_t>(in) | ld | stride) & 3) == 0;
    return {in, ld, stride, per, total, K, out, ldo, (int)ceil_div(512, ldo / 16), words};  // (some two chunks a thread)
}
void launch_repack(const RepackRows &a, const RepackRows &b, hipStream_t stream)
{
    constexpr int64_t most = int64_t(1) << 22;  // workgroups of a launch
    const int64_t of_a = repack_groups(a), all = of_a + repack_groups(b);
    for (int64_t base = 0; base < all; base += most)
        hipLaunchKernelGGL(block_repack, dim3((unsigned)(all - base < most ? all - base : most)), dim3(256), 0, stream, a, b, of_a, base);
}

int64_t block_mm_workspace(int64_t M, int64_t N, int64_t K, int E, bool grouped, bool fp32_out, bool a_aligned, bool w_aligned)
{
    if (K == 0) return 0;
    int64_t most = 0;
    const int64_t step = slice_n(M, K, E, grouped), high = slice_m(M, K, grouped);
    for (int64_t m : {M < high ? M : high, M % high})
        for (int64_t n : {N < step ? N : step, N % step}) {
            if (!m || !n) continue;
            for (bool e8m0 : {false, true}) {
                const Plan p = make_plan(m, n, K, E, grouped, mode_of(fp32_out, e8m0), a_aligned, w_aligned);
                const int64_t need = p.a_bytes + p.w_bytes + p.part_bytes;
                if (need > most) most = need;
            }
        }
    return most;
}

hipError_t launch_block_mm(int a_dtype, int w_dtype, const BlockMMParams &p, bool a_aligned, bool w_aligned, hipStream_t stream)
{
    const int64_t size = p.out_dtype == EMU_DT_FP32 ? 4 : 2, unit = p.e8m0 ? 1 : 4;
    const bool grouped = p.ends != nullptr;
    const int64_t step = slice_n(p.M, p.K, p.E, grouped), high = slice_m(p.M, p.K, grouped);
    for (int64_t m = 0; m < p.M; m += high)
        for (int64_t n = 0; n < p.N; n += step) {
            BlockMMParams q = p;
            q.M = p.M - m < high ? p.M - m : high;
            q.N = p.N - n < step ? p.N - n : step;
            if (p.K) {
                q.a = p.a + m * p.lda;
                q.w = p.w + n * p.ldw;
                q.sa = static_cast<const char *>(p.sa) + m * p.sa_row * unit;
                q.sw = static_cast<const char *>(p.sw) + n / kBlock * p.sw_row * unit;
            }
            if (p.bias) q.bias = static_cast<const char *>(p.bias) + n * (p.bias_f32 ? 4 : size);
            q.out = static_cast<char *>(p.out) + (m * p.ldo + n) * size;
            launch_slice(a_dtype, w_dtype, q, a_aligned, w_aligned, stream);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

}  // namespace emu
