// emu_weight_grad.hip -- emu_block_weight_grad: the gradient of a product's
// weights, out[n, k] = sum over rows t of g[t, n] x[t, k], from the codes that
// x was kept in.
//
// The sum runs over rows, along which scales differ, so x is made whole again:
// with scales that are powers of two bf16 holds code times scale exactly, and
// v_mfma_f32_16x16x32_bf16 adds in binary32 (1.95 PFLOP/s of instructions alone).  g
// in fp16 or fp32 is split into the two or three bf16 numbers whose sum it is, and
// the product of each is added.  For outputs of 16 bits two stand for an fp32 g
// too: what they leave of it, at most 2^-17, is little beside the output's rounding
// (2^-9 or 2^-12), and the third costs as much as each of them.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops_block.h"
#include "ops_tiles.h"

namespace emu {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// ---- g in planes of bf16 -------------------------------------------------

// Eight values a thread, cut to 8 significant bits, then what that left, and
// what that left: each cut is exact, and no part is larger than the value.  Two
// parts of an fp32 value are its nearest one (or cut, where that were an infinity)
// and the nearest of what that left.
// Workgroups from `groups` on lay out rows of codes.
template <typename G, int PLANES>
__global__ __launch_bounds__(256) void split_planes(const G *g, int64_t ldg, int64_t T, int64_t N, uint16_t *out, int64_t ldo,
                                                    int64_t plane, unsigned groups, RepackRows codes)
{
    if (blockIdx.x >= groups) {
        repack_rows(codes, blockIdx.x - groups);
        return;
    }
    const uint32_t chunks = (uint32_t)(ldo / 8), id = blockIdx.x * 256 + threadIdx.x, row = id / chunks;
    const int64_t t = row;
    const int c = (int)(id - row * chunks) * 8, n = (int)N;
    if (t >= T) return;
    f32x8 v = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (c < n) v = settle8<G>(fetch8(g + t * ldg, c, n), c, n);
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
        Raw8<uint16_t> r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = __float_as_uint(v[i]);
            const bool finite = (bits & 0x7F800000u) != 0x7F800000u, nan = v[i] != v[i];
            uint32_t part = bits >> 16 | (nan ? 0x40u : 0u);
            if (sizeof(G) == 4 && PLANES == 2) {
                const uint32_t near = (bits + 0x7FFFu + (bits >> 16 & 1u)) >> 16;
                part = finite && (near & 0x7F80u) != 0x7F80u ? near : part;
            }
            r[i] = (uint16_t)part;
            v[i] = finite ? v[i] - __uint_as_float(part << 16) : 0.0f;
        }
        *reinterpret_cast<Raw8<uint16_t> *>(out + p * plane + t * ldo + c) = r;
    }
}

// ---- tiles ---------------------------------------------------------------
//
// A workgroup of WN x WK waves makes BN x BK outputs, a stage of 64 rows at a
// time, in two halves of 32, what one instruction takes.  g and codes come into
// registers, codes are widened with their rows' scales, and both are written to
// LDS as bf16, two stages deep.  They lie there as they do in memory, row by row,
// and ds_read_b64_tr_b16 turns 4 rows by 16 columns as it reads them, so that a
// lane gets consecutive rows of its column.  While a half is multiplied out of
// registers the next is read:
//   (s, 0): multiply; read the fragments of (s, 1), write the codes of s + 1 into
//           the other buffer and load those of s + 2 (or of s + 3, AHEAD 2);
//   wait until every wave has written s + 1 and read buffer s (one barrier a stage);
//   (s, 1): multiply; read the fragments of (s + 1, 0), write g of s + 2 into buffer
//           s and load that of s + 3 (s + 4).
// LDS bounds it: a stage of 64 rows writes 64 KiB and reads 192 to 2048 cycles of
// products, and 16384 x 8192 x 4096 in 8 groups (920 us) takes 750 without the
// writes and 820 without the reads.  With both operands' writes in one half, 936.
// (Loads straight into LDS would spare g its way through registers, but the
// compiler then waits for all of them before each read that turns: 2.4 ms for 1.2.)
// 16 rows' segments of 32 bytes meet in one read: row t's pair of chunks of 16
// bytes c stands at place c ^ ((t & 3) + 4 (t / 8 & 1)), which spreads them over all
// banks.  Of codes' pairs those of every other four stand with their second chunk
// first, so that 8 lanes that write a chunk of each meet all banks too (944 us, 935).

constexpr int kRows = 64;

__device__ __forceinline__ int turn(int t) { return (t & 3) | (t >> 1 & 4); }
__device__ __forceinline__ int half_of(int c) { return (c & 4) << 2; }

template <int BN, int BK>
constexpr int kGradLds = 2 * kRows * (BN + BK) * 2;

// (the conversions read a scale's exponent alone: a byte's 2^-127 and NaN are
// the exponents 0 and 255)
template <int CF>
__device__ __forceinline__ i32x4 widened(int lo, int hi, float scale)
{
    return i32x4{(int)two_bf16<CF>((uint32_t)lo, false, scale), (int)two_bf16<CF>((uint32_t)lo, true, scale),
                 (int)two_bf16<CF>((uint32_t)hi, false, scale), (int)two_bf16<CF>((uint32_t)hi, true, scale)};
}

// Infinities and NaN become 0: they have met g's first part, and its others
// may be 0 where g is not.
__device__ __forceinline__ i32x4 finite_parts(i32x4 v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (uint32_t)v[i];
        const uint32_t low = (w & 0x7F80u) == 0x7F80u ? 0u : 0xFFFFu, high = (w & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFF0000u;
        v[i] = (int)(w & (low | high));
    }
    return v;
}

// 16 bytes a lane from base + offset, zeros from `size` on.
__device__ __forceinline__ i32x4 load_within(const void *base, int size, int offset)
{
    const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, size, 0x00020000);
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0));
}
__device__ __forceinline__ s16x4 read_turned(const int8_t *lds)
{
    typedef __attribute__((address_space(3))) s16x4 *ptr;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_ptr)lds);
}

// part: null, or [S, E, N, K] sums of each split of a group's rows (grid y).
// AHEAD: the stages between the last one written and the last one loaded, in as
// many sets of registers (one of 256 x 256 has none to spare; 128 x 128: two take
// 18.9 us for 1024 x 1920 x 1920, one 20).
// PLANES: g may have more planes than one (without the test in the writes, one
// plane of 16384 x 8192 x 4096 in 8 groups takes 945 us for 976, 1024 x 1920 x
// 1920 21.0 for 23.0).
template <int CF, bool PLANES, int BN, int BK, int WN, int WK, int AHEAD>
__global__ __launch_bounds__(WN *WK * 64, 2) void grad_tiles(WeightGradParams p, int tn, int tk, int S,
                                                                                                float *part)
{
    constexpr int FN = BN / WN / 16, FK = BK / WK / 16, threads = WN * WK * 64, F = FN * FK;
    constexpr int GC = BN * 2 / 16, XC = BK / 16;                          // a row's chunks of g (LDS) and of codes (global)
    constexpr int GL = kRows * GC / threads, XL = kRows * XC / threads;    // a thread's loads a stage
    constexpr int GBUF = kRows * BN * 2, BUF = GBUF + kRows * BK * 2;
    static_assert(GL * threads == kRows * GC && XL * threads == kRows * XC && BK % kBlock == 0 && GC >= 16 && XC >= 8, "");
    __shared__ __attribute__((aligned(1024))) int8_t lds[kGradLds<BN, BK>];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // Groups one after the other, each one's tiles over all XCDs: groups differ
    // in rows, and with one to an XCD the largest would end last (16384 x 8192 x
    // 4096 in 8 groups as routers leave them: 1.99 ms).
    const int e = (int)blockIdx.x / (tn * tk);
    int ti, tj;
    tile_of<kHigh>((int)blockIdx.x - e * (tn * tk), tn, tk, ti, tj);
    // the group's rows: an end below one before counts as that one, one past T as T
    int first = 0, rows = (int)p.T;
    if (p.E) {
        int before = 0, upto = 0;
        for (int base = 0; base <= e; base += 64) {
            const int i = base + lane;
            int64_t v = 0;
            if (i <= e) v = p.ends64 ? static_cast<const int64_t *>(p.ends)[i] : static_cast<const int *>(p.ends)[i];
            const int c = v < 0 ? 0 : v > p.T ? (int)p.T : (int)v;
            upto = c > upto ? c : upto;
            before = i < e && c > before ? c : before;
        }
        const auto larger = [](int a, int b) { return a > b ? a : b; };
        first = uniform(wave_reduce(before, larger));
        rows = uniform(wave_reduce(upto, larger)) - first;
    }
    const int64_t n0 = (int64_t)ti * BN, k0 = (int64_t)tj * BK;
    const int cols_n = (int)(p.N - n0 < BN ? p.N - n0 : BN), cols_k = (int)(p.K - k0 < BK ? p.K - k0 : BK);
    // this split's stages: of all of the group's, plane after plane
    const int per_plane = (int)(((unsigned)rows + kRows - 1) / kRows), all = per_plane * (PLANES ? p.planes : 1), share = uniform((all + S - 1) / S);
    const int s0 = (int)blockIdx.y * share, count = all - s0 < share ? (all - s0 < 0 ? 0 : all - s0) : share;

    // where stage s lies: its plane, its first row of the group, how many are left of 64 (none past the last stage)
    struct Stage {
        int row, plane, left;
    };
    const auto stage_at = [&](int s) {
        Stage r;
        const int at = s0 + s;
        r.plane = 0;
        if (PLANES) {
            r.plane = at >= 2 * per_plane ? 2 : at >= per_plane ? 1 : 0;
            r.plane = r.plane < p.planes ? r.plane : p.planes - 1;
        }
        r.row = (at - r.plane * per_plane) * kRows;
        r.left = s < count ? (rows - r.row < kRows ? rows - r.row : kRows) : 0;
        return r;
    };
    // The bytes that may be read from a stage's first row on (whole words of the last row, which lie within its leading
    // dimension, a multiple of 16 bytes; none of no rows).
    const auto range = [&](int left, int ld, int width) {
        const int size = left * ld - (ld - ((width + 3) & ~3));
        return uniform(size > 0 ? size : 0);
    };

    // g: 16 bytes a lane, in the order of their places in LDS.  Load q of a wave
    // takes rows GROWS q .. of those it loads: which chunk a lane takes depends
    // on q in VARIANTS ways.
    constexpr int GROWS = 64 / GC, VARIANTS = GC == 32 ? 4 : 2;
    const auto variant = [](int q) { return GC == 32 ? (q & 1) | (q >> 2 & 1) << 1 : q >> 1 & 1; };
    const int ldg2 = (int)p.ldg * 2, grow = wave * GL * GROWS;
    int gfrom[VARIANTS];
#pragma unroll
    for (int q = 0; q < GL; ++q)
        gfrom[variant(q)] = lane / GC * ldg2 + ((lane % GC) ^ (turn(grow + GROWS * q + lane / GC) * 2)) * 16;
    i32x4 graw[AHEAD][GL];
    const auto load_g = [&](int set, int q, const Stage &s) {
        graw[set][q] = load_within(p.g + s.plane * p.plane_stride + (int64_t)(first + s.row) * p.ldg + n0, range(s.left, ldg2, cols_n * 2),
                              gfrom[variant(q)] + (grow + q * GROWS) * ldg2);
    };
    const auto write_g = [&](int set, int q, int buf) {
        *reinterpret_cast<i32x4 *>(lds + buf * BUF + (wave * GL + q) * 1024 + lane * 16) = graw[set][q];
    };
    // codes: 16 a lane, XROWS rows with each of a workgroup's loads
    constexpr int XROWS = threads / XC;
    static_assert(XROWS % 16 == 0 && (VARIANTS < 4 || GL <= 8), "a lane's places turn alike in all of its loads");
    const int xrow = (int)threadIdx.x / XC, xchunk = (int)threadIdx.x % XC, ldc = (int)p.ldc;
    const int xfrom = xrow * ldc + xchunk * 16, xto = GBUF + xrow * BK * 2 + (xchunk ^ turn(xrow)) * 32 + half_of(xchunk);
    const int last_block = (int)(blocks_of(p.K) - 1 - k0 / kBlock), xblock = xchunk * 16 / kBlock;
    const uint8_t *const xscale = p.scales + (k0 / kBlock + (xblock < last_block ? xblock : last_block)) * p.s_block;
    i32x4 codes[AHEAD][XL];
    int scale[AHEAD][XL];
    const auto load_x = [&](int set, int q, const Stage &s) {
        codes[set][q] = load_within(p.codes + (int64_t)(first + s.row) * p.ldc + k0, range(s.left, ldc, cols_k), xfrom + q * XROWS * ldc);
        // (rows past the group's last have the last one's: their codes are zeros, and a NaN is in its block anyway)
        const int t = s.row + xrow + q * XROWS;
        scale[set][q] = xscale[(int64_t)(first + (t < rows ? t : rows - 1)) * p.s_row];
    };
    const auto write_x = [&](int set, int q, int h, const Stage &s, int buf) {
        i32x4 v = widened<CF>(codes[set][q][2 * h], codes[set][q][2 * h + 1], __uint_as_float((uint32_t)scale[set][q] << 23));
        if (PLANES && s.plane) v = finite_parts(v);
        *reinterpret_cast<i32x4 *>(lds + buf * BUF + (h ? xto ^ 16 : xto) + q * XROWS * BK * 2) = v;
    };

    // fragments: this lane's place in rows 8 (lane / 16) + (lane / 4 & 3) of a half, and 4 below
    const int wn = (wave / WK) * (BN / WN), wk = (wave % WK) * (BK / WK);
    const int trow = (lane >> 4) * 8 + (lane >> 2 & 3);
    int gat[FN], xat[FK];
#pragma unroll
    for (int i = 0; i < FN; ++i) gat[i] = trow * BN * 2 + (((wn / 16 + i) ^ turn(trow)) * 32) + (lane & 3) * 8;
#pragma unroll
    for (int j = 0; j < FK; ++j) xat[j] = GBUF + trow * BK * 2 + (((wk / 16 + j) ^ turn(trow)) * 32) + ((lane & 3) * 8 ^ half_of(wk / 16 + j));
    const auto turned = [&](int at, int row_bytes) {
        const s16x4 a = read_turned(lds + at), b = read_turned(lds + at + 4 * row_bytes);
        return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    };
    const auto read_g = [&](int i, int half, int buf) { return turned(buf * BUF + gat[i] + half * 32 * BN * 2, BN * 2); };
    const auto read_x = [&](int j, int half, int buf) { return turned(buf * BUF + xat[j] + half * 32 * BK * 2, BK * 2); };

    f32x4 acc[FN][FK] = {};
    bf16x8 G[FN], X[2][FK];
    if (count) {
#pragma unroll
        for (int b = 0; b < AHEAD + 2; ++b) {
            // (what is not written stays in registers until its buffer is free)
            if (b == AHEAD) {
                const Stage s = stage_at(0);
#pragma unroll
                for (int q = 0; q < GL; ++q) write_g(0, q, 0);
#pragma unroll
                for (int q = 0; q < XL; ++q) write_x(0, q, 0, s, 0), write_x(0, q, 1, s, 0);
            }
            if (b == AHEAD + 1) {
#pragma unroll
                for (int q = 0; q < GL; ++q) write_g(1 % AHEAD, q, 1);
            }
            const Stage s = stage_at(b);
#pragma unroll
            for (int q = 0; q < GL; ++q) load_g(b % AHEAD, q, s);
            if (b == AHEAD + 1) break;
#pragma unroll
            for (int q = 0; q < XL; ++q) load_x(b % AHEAD, q, s);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FN; ++i) G[i] = read_g(i, 0, 0);
#pragma unroll
        for (int j = 0; j < FK; ++j) X[0][j] = read_x(j, 0, 0);
    }
    const auto half = [&](auto which, auto parity, const Stage &now, const Stage &then, int buf) {
        constexpr int h = decltype(which)::value, o = h ^ 1, set = (h + decltype(parity)::value + 1) % AHEAD;
        // what goes between the instructions: reads, and writes and loads of one of the operands
        constexpr int WORK = h ? 2 * GL : 3 * XL;
        const int from = h ? buf ^ 1 : buf;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < F; ++t) {
            const int i = t / FK, j = t % FK;
#pragma unroll
            for (int u = t * FK / (F / 2); u < FK && u < (t + 1) * FK / (F / 2); ++u) X[o][u] = read_x(u, o, from);
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(X[h][j], G[i], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (j == FK - 1) G[i] = read_g(i, o, from);
#pragma unroll
            for (int u = t * WORK / F; u < (t + 1) * WORK / F; ++u) {
                if (h && u % 2)
                    load_g(set, u / 2, then);
                else if (h)
                    write_g(set, u / 2, buf);
                else if (u % 3 == 2)
                    load_x(set, u / 3, then);
                else
                    write_x(set, u / 3, u % 3, now, buf ^ 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    typedef std::integral_constant<int, 0> First;
    typedef std::integral_constant<int, 1> Second;
    const auto stage = [&](auto parity, int s, int buf) {
        const Stage next = stage_at(s + 1), x = stage_at(s + 1 + AHEAD), g = stage_at(s + 2 + AHEAD);
        half(First{}, parity, next, x, buf);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave has read buffer s and written its part of s + 1
        __builtin_amdgcn_s_barrier();
        half(Second{}, parity, next, g, buf);
    };
    if constexpr (AHEAD == 1) {
        for (int s = 0, buf = 0; s < count; ++s, buf ^= 1) stage(First{}, s, buf);
    } else {
        int s = 0;
        for (; s + 1 < count; s += 2) stage(First{}, s, 0), stage(Second{}, s + 1, 1);
        if (s < count) stage(First{}, s, 0);
    }
    const int64_t n = n0 + wn + (lane & 15);
    const bool whole = cols_n == BN && cols_k == BK;
    const f32x4 none[FK] = {};
    if (part)
        store_tile(part + ((int64_t)blockIdx.y * (p.E ? p.E : 1) + e) * p.N * p.K, EMU_DT_FP32, p.K, acc, none, false, n, p.N, k0 + wk, p.K,
                   lane, whole);
    else
        store_tile(static_cast<char *>(p.out) + e * p.out_stride * (p.out_dtype == EMU_DT_FP32 ? 4 : 2), p.out_dtype, p.ldo, acc, none,
                   false, n, p.N, k0 + wk, p.K, lane, whole);
}

// The sums of S splits, four outputs a thread.
__global__ __launch_bounds__(256) void grad_join(WeightGradParams p, const float *part, int S)
{
    const int64_t quads = (p.K + 3) / 4, id = (int64_t)blockIdx.x * 256 + threadIdx.x, row = id / quads, k = id % quads * 4;
    const int64_t rows = (p.E ? p.E : 1) * p.N;
    if (row >= rows) return;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    typedef f32x4 words __attribute__((aligned(4)));
    const float *at = part + row * p.K + k;
    for (int s = 0; s < S; ++s, at += rows * p.K) {
        if (k + 4 <= p.K) {
            sum += *reinterpret_cast<const words *>(at);
        } else {
            for (int i = 0; i < 4; ++i)
                if (k + i < p.K) sum[i] += at[i];
        }
    }
    with_type(p.out_dtype, [&](auto *type) {
        typedef std::remove_pointer_t<decltype(type)> E;
        E *out = static_cast<E *>(p.out) + row / p.N * p.out_stride + row % p.N * p.ldo + k;
        store_valid(out, __builtin_convertvector(sum, Four<E>), p.K - k);
    });
}

// ---- the plan ----------------------------------------------------------

struct GradPlan {
    bool large;          // tiles of 256 x 256, else of 128 x 128
    int S;               // splits of a group's rows
    int planes;
    bool split_g, repack_c;
    int64_t ldg, ldc;    // of both where they are laid out anew
    int64_t g_bytes, c_bytes, part_bytes;
};

GradPlan make_plan(int64_t T, int E, int64_t N, int64_t K, int g_dtype, bool out16, bool g_aligned, bool c_aligned)
{
    GradPlan p{};
    const int64_t groups = E ? E : 1;
    p.planes = g_dtype == EMU_DT_BF16 ? 1 : g_dtype == EMU_DT_FP16 || out16 ? 2 : 3;
    p.split_g = p.planes > 1 || !g_aligned;
    p.repack_c = !c_aligned;
    p.ldg = ceil_div(N, 8) * 8;
    p.ldc = blocks_of(K) * kBlock;
    p.g_bytes = p.split_g ? (p.planes * T * p.ldg * 2 + 15) / 16 * 16 : 0;
    p.c_bytes = p.repack_c ? T * p.ldc : 0;
    // The fastest estimate, as for the products: a round of 256 large tiles, or of
    // 512 small ones, two to a CU, or a rest of up to 256, one to a CU, as measured
    // (4096 x 4096 of 1024 rows: 43 us large, 51 small; 2048 x 2048: 35 and 20); a
    // split of rows 5 us more and its sums at 4 TB/s, there and back.  (Stages of
    // later planes, whose codes are looked at for infinities, are priced like those
    // of one plane: 4096^3 takes 110 us in bf16, of fp32 g in two planes 257.)
    const int64_t stages = ceil_div(ceil_div(T, groups), kRows) * p.planes;
    double best = 0.0;
    p.S = 1;
    bool any = false;
    for (int large = 0; large < 2; ++large)
        for (int S = 1; S <= 16; S *= 2) {
            if (S > 1 && stages / S < 4) break;
            const int64_t side = large ? 256 : 128;
            const int64_t tiles = ceil_div(N, side) * ceil_div(K, side) * groups * S;
            const int64_t rest = large ? 0 : tiles % 512 <= 256 ? tiles % 512 : 0;
            const double each = (double)ceil_div(stages, S);
            double us = (double)ceil_div(tiles - rest, large ? 256 : 512) * (large ? 6.0 + each * 1.65 : 5.0 + each * 1.2);
            if (rest) us += 4.0 + each * 0.7;
            if (S > 1) us += 5.0 + (double)S * (double)groups * (double)N * (double)K * 8.0 / 4e6;
            if (any && us >= best) continue;
            any = true;
            best = us;
            p.large = large;
            p.S = S;
        }
    p.part_bytes = p.S > 1 ? p.S * groups * N * K * 4 : 0;
    return p;
}

template <int CF, bool PLANES>
void launch_tiles(const WeightGradParams &p, const GradPlan &plan, float *part, hipStream_t stream)
{
    const int64_t side = plan.large ? 256 : 128, tn = ceil_div(p.N, side), tk = ceil_div(p.K, side);
    const dim3 grid((unsigned)(tn * tk * (p.E ? p.E : 1)), (unsigned)plan.S);
    if (plan.large)
        hipLaunchKernelGGL((grad_tiles<CF, PLANES, 256, 256, 2, 4, 1>), grid, dim3(512), 0, stream, p, (int)tn, (int)tk, plan.S, part);
    else
        hipLaunchKernelGGL((grad_tiles<CF, PLANES, 128, 128, 2, 2, 2>), grid, dim3(256), 0, stream, p, (int)tn, (int)tk, plan.S, part);
}

// With the codes' rows in the first launch, where it has room for them.
template <typename G, int PLANES>
void launch_split(const WeightGradParams &p, uint16_t *out, int64_t ldo, RepackRows codes, hipStream_t stream)
{
    int64_t step = (int64_t(1) << 30) / (ldo / 8);  // a launch's rows
    step = step < 1 ? 1 : step;
    if (repack_groups(codes) > int64_t(1) << 22) {
        launch_repack(codes, RepackRows{}, stream);
        codes = RepackRows{};
    }
    for (int64_t t = 0; t < p.T; t += step) {
        const int64_t rows = p.T - t < step ? p.T - t : step;
        const unsigned groups = (unsigned)ceil_div(rows * (ldo / 8), 256);
        hipLaunchKernelGGL((split_planes<G, PLANES>), dim3(groups + (unsigned)repack_groups(codes)), dim3(256), 0, stream,
                           reinterpret_cast<const G *>(p.g) + t * p.ldg, p.ldg, rows, p.N, out + t * ldo, ldo, p.T * ldo, groups, codes);
        codes = RepackRows{};
    }
}

}  // namespace

int64_t weight_grad_workspace(int64_t T, int E, int64_t N, int64_t K, int g_dtype, bool g_aligned, bool c_aligned)
{
    int64_t most = 0;  // of either kind of output
    for (const bool out16 : {false, true}) {
        const GradPlan p = make_plan(T, E, N, K, g_dtype, out16, g_aligned, c_aligned);
        const int64_t bytes = p.g_bytes + p.c_bytes + p.part_bytes;
        most = bytes > most ? bytes : most;
    }
    return most;
}

hipError_t launch_weight_grad(int g_dtype, int c_dtype, const WeightGradParams &params, bool g_aligned, bool c_aligned, void *ws,
                              hipStream_t stream)
{
    WeightGradParams p = params;
    const GradPlan plan = make_plan(p.T, p.E, p.N, p.K, g_dtype, p.out_dtype != EMU_DT_FP32, g_aligned, c_aligned);
    char *at = static_cast<char *>(ws);
    p.planes = plan.planes;
    RepackRows codes{};
    if (plan.repack_c && p.T > 0) {
        codes = repack_job(p.codes, p.ldc, 0, p.T, p.T, p.K, reinterpret_cast<int8_t *>(at + plan.g_bytes), plan.ldc);
        p.codes = codes.out;
        p.ldc = plan.ldc;
    }
    if (plan.split_g && p.T > 0) {
        uint16_t *g = reinterpret_cast<uint16_t *>(at);
        if (g_dtype == EMU_DT_BF16)
            launch_split<__bf16, 1>(p, g, plan.ldg, codes, stream);
        else if (g_dtype == EMU_DT_FP16)
            launch_split<_Float16, 2>(p, g, plan.ldg, codes, stream);
        else if (plan.planes == 2)
            launch_split<float, 2>(p, g, plan.ldg, codes, stream);
        else
            launch_split<float, 3>(p, g, plan.ldg, codes, stream);
        p.g = g;
        p.ldg = plan.ldg;
        p.plane_stride = p.T * plan.ldg;
    } else {
        launch_repack(codes, RepackRows{}, stream);
    }
    at += plan.g_bytes + plan.c_bytes;
    float *part = plan.S > 1 ? reinterpret_cast<float *>(at) : nullptr;
    const bool e4 = c_dtype == EMU_DT_E4M3FN, planes = plan.planes > 1;
    (e4 ? planes ? launch_tiles<0, true> : launch_tiles<0, false> : planes ? launch_tiles<1, true> : launch_tiles<1, false>)(
        p, plan, part, stream);
    if (part)
        hipLaunchKernelGGL(grad_join, dim3((unsigned)ceil_div((p.E ? p.E : 1) * p.N * ceil_div(p.K, 4), 256)), dim3(256), 0, stream, p,
                           part, plan.S);
    return hipGetLastError();
}

}  // namespace emu
