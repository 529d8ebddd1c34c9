// emu_int8.hip -- emu_int8_scaled_mm: out = (a @ w.T) * scale_a * scale_w + bias.
//
// The products are v_mfma_i32_16x16x64_i8's and their sums exact in int32, so
// neither tiles nor a split of K change a bit of the result.  The matrix
// instruction takes w's rows as its first operand: a lane then ends with four
// consecutive outputs of one row.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops_device.h"
#include "ops_internal.h"

namespace emu {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_words __attribute__((aligned(4)));

// ---- the epilogue ------------------------------------------------------

__device__ __forceinline__ float bias_at(const Int8Params &p, int64_t n)
{
    if (p.bias_f32 || p.out_dtype == EMU_DT_FP32) return static_cast<const float *>(p.bias)[n];
    if (p.out_dtype == EMU_DT_BF16) return (float)static_cast<const __bf16 *>(p.bias)[n];
    return (float)static_cast<const _Float16 *>(p.bias)[n];
}
// The scale of a column and of a row; those past the end are the last one's.
__device__ __forceinline__ float column_scale(const Int8Params &p, int64_t n)
{
    return p.sw[p.w_per_row ? (n < p.N ? n : p.N - 1) : 0];
}
__device__ __forceinline__ float row_scale(const Int8Params &p, int64_t m)
{
    return p.sa[p.a_per_row ? (m < p.M ? m : p.M - 1) : 0];
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Four columns' scales and biases.
struct Columns {
    f32x4 sw, b;
};
__device__ __forceinline__ Columns columns_at(const Int8Params &p, int64_t n)
{
    Columns c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c.sw[i] = column_scale(p, n + i);
        c.b[i] = p.bias ? bias_at(p, n + i < p.N ? n + i : p.N - 1) : 0.0f;
    }
    return c;
}

// Four outputs of a row from their sums.  Each step is rounded as the
// definition has it: the sum to binary32, both products, the bias, the output.
template <typename E>
using Four = E __attribute__((ext_vector_type(4)));
template <typename E>
__device__ __forceinline__ Four<E> outputs4(const i32x4 &sum, float sa, const Columns &c, bool bias)
{
    f32x4 y = __builtin_convertvector(sum, f32x4) * sa * c.sw;
    if (bias) y += c.b;
    return __builtin_convertvector(y, Four<E>);
}
// The first `valid` of v's values.
template <typename V, typename E>
__device__ __forceinline__ void store_valid(E *o, const V &v, int64_t valid)
{
    constexpr int n = sizeof(V) / sizeof(E);
    typedef V mem __attribute__((aligned(sizeof(E))));
    if (valid >= n) {
        *reinterpret_cast<mem *>(o) = v;
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (i < valid) o[i] = v[i];
    }
}

// f(null pointer of out's element type)
template <typename F>
__device__ __forceinline__ void with_type(int dtype, F f)
{
    if (dtype == EMU_DT_BF16)
        f(static_cast<__bf16 *>(nullptr));
    else if (dtype == EMU_DT_FP16)
        f(static_cast<_Float16 *>(nullptr));
    else
        f(static_cast<float *>(nullptr));
}

// Outputs (m, n .. n + 3).
__device__ __forceinline__ void finish(const Int8Params &p, int64_t m, int64_t n, const i32x4 &sum, float sa,
                                       const Columns &c)
{
    if (m >= p.M || n >= p.N) return;
    with_type(p.out_dtype, [&](auto *type) {
        typedef std::remove_pointer_t<decltype(type)> E;
        store_valid(static_cast<E *>(p.out) + m * p.ldo + n, outputs4<E>(sum, sa, c, p.bias != nullptr), p.N - n);
    });
}

// ---- tiles -------------------------------------------------------------
//
// 8192^3 takes 415 us (2.65 POP/s; 370 to 445 as the card's power allows, against
// 4.4 POP/s of matrix instructions alone on such codes, also at the power
// limit, and 4.9 on zeros).
// A workgroup of WM x WN waves makes BM x BN outputs, a stage of 128 codes of
// K at a time.  Stages come from global memory straight into LDS (16 bytes a
// lane), NB buffers deep, whole 128-byte lines: a CU takes up to 115 GB/s of
// them from its L2, against 32 in pieces of 64 bytes of rows 8192 apart.  A
// stage is multiplied in two halves; the fragments of a half are read into
// registers while the half before it is multiplied:
//   (s, 0): multiply (s, 0); read the fragments of (s, 1).
//   (s, 1): wait until s + 1 has arrived and every wave has read buffer s
//           (one barrier a stage); then, between the matrix instructions,
//           load s + NB into buffer s and read the fragments of (s + 1, 0).
// The matrix instructions keep their second operand for a row of them: the
// other way round the same work takes 10% longer (the card is then at its
// power limit).
//
// LDS holds a stage's rows of 128 bytes as eight chunks of 16; row r's chunk c
// stands at place c ^ swizzle(r), which spreads the 16 rows that a
// ds_read_b128 meets over all banks.

constexpr int kStage = 128, kHalf = 64;

__device__ const i32x4 kZeros = {0, 0, 0, 0};

__device__ __forceinline__ int swizzle(int r)
{
    const int j = (r >> 1) & 7;
    return j ^ ((j >> 1 ^ j >> 2) & 1);
}

// s_waitcnt with only the vector memory counter
template <int N>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

typedef __attribute__((address_space(3))) void *lds_ptr;

// 16 bytes a lane from base + row + k into LDS.  A buffer load, since the
// compiler takes a global one to count as an LDS access too and then waits
// for every fragment in flight (250 x 4096 x 4096: 11.8 us against 11.3).
__device__ __forceinline__ void load_lds(const int8_t *base, int row, int k, int8_t *to)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, -1, 0x00020000), (lds_ptr)to, 16, row, k, 0, 0);
}

// Workgroups go round the 8 XCDs in turn; each XCD gets a run of
// neighbouring tiles, two rows of tiles high, whose operands its L2 then holds.
__device__ __forceinline__ void tile_of(int id, int tm, int tn, int &m, int &n)
{
    const int total = tm * tn, xcd = id & 7, each = total >> 3, rest = total & 7;
    id = xcd * each + (xcd < rest ? xcd : rest) + (id >> 3);
    const int pair = id / (2 * tn), high = tm - 2 * pair < 2 ? 1 : 2, in = id - pair * 2 * tn;
    m = 2 * pair + in % high;
    n = in / high;
}

// part: null, or [S, M, N] sums of each K split (grid y).  The launch bounds
// ask for the waves a SIMD that the stages in LDS leave room for, at most 2.
template <int BM, int BN, int WM, int WN, int NB>
__global__ __launch_bounds__(WM * WN * 64, NB * (BM + BN) * kStage * 2 <= 160 * 1024 || WM * WN > 4 ? 2 : 1) void int8_tiles(
    Int8Params p, int tm, int tn, int stages, int *part)
{
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;           // fragments of a wave, in a half
    constexpr int LPW = (BM + BN) / 8 / (WM * WN);                // its loads a stage, 8 rows each
    constexpr int BUF = (BM + BN) * kStage;
    constexpr int T = FM * FN;
    static_assert(LPW * WM * WN * 8 == BM + BN && BM % 16 == 0 && FN % 2 == 0, "");
    __shared__ __attribute__((aligned(1024))) int8_t lds[NB * BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ti, tj;
    tile_of(blockIdx.x, tm, tn, ti, tj);
    const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)tj * BN;
    const int64_t k0 = (int64_t)blockIdx.y * stages * kStage;     // this split's first code
    const int K = (int)(p.K - k0 < (int64_t)stages * kStage ? p.K - k0 : (int64_t)stages * kStage);
    const int8_t *abase = p.a + m0 * p.lda + k0, *wbase = p.w + n0 * p.ldw + k0;

    // a lane's row (of 8) and chunk in each load; rows past the end read the last one
    int src[LPW], chunk[2];
    chunk[0] = ((lane & 7) ^ swizzle(lane >> 3)) * 16;
    chunk[1] = ((lane & 7) ^ swizzle(8 + (lane >> 3))) * 16;
#pragma unroll
    for (int q = 0; q < LPW; ++q) {
        const int at = wave * LPW + q, row = at * 8 + (lane >> 3);
        if (row < BM)
            src[q] = (int)((m0 + row < p.M ? row : p.M - 1 - m0) * p.lda) + chunk[at & 1];
        else
            src[q] = (int)((n0 + row - BM < p.N ? row - BM : p.N - 1 - n0) * p.ldw) + chunk[at & 1];
    }
    int8_t *const dst = lds + wave * LPW * 1024;
    // `whole`: the stage lies within K; else the chunks past K (K % 16 == 0) are zeros
    const auto load = [&](int q, int s, int buf, bool whole) {
        const int at = wave * LPW + q;
        const int8_t *base = at * 8 < BM ? abase : wbase;
        int8_t *to = dst + buf * BUF + q * 1024;
        if (whole) {
            load_lds(base, src[q], s * kStage, to);
        } else {
            const int8_t *from = base + src[q] + s * kStage;
            if (s * kStage + chunk[at & 1] >= K) from = reinterpret_cast<const int8_t *>(&kZeros);
            __builtin_amdgcn_global_load_lds(
                reinterpret_cast<const __attribute__((address_space(1))) void *>(reinterpret_cast<uintptr_t>(from)),
                (lds_ptr)to, 16, 0, 0);
        }
    };

    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const int fr = lane & 15;
    const int8_t *fa[2], *fw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int place = ((h * 4 + (lane >> 4)) ^ swizzle(fr)) * 16;
        fa[h] = lds + (wm + fr) * kStage + place;
        fw[h] = lds + (BM + wn + fr) * kStage + place;
    }
    // a row's or a column's scale and bias, which go into LDS after the last stage
    static_assert(BM + BN <= WM * WN * 64, "");
    float scale = 0.0f, bias = 0.0f;
    if (!part) {
        const int t = threadIdx.x;
        if (t < BM) {
            scale = row_scale(p, m0 + t);
        } else if (t < BM + BN) {
            const int64_t n = n0 + t - BM;
            scale = column_scale(p, n);
            if (p.bias) bias = bias_at(p, n < p.N ? n : p.N - 1);
        }
    }
    i32x4 acc[FM][FN] = {};
    i32x4 A[FM], B[2][FN];

#pragma unroll
    for (int s = 0; s < NB; ++s)
#pragma unroll
        for (int q = 0; q < LPW; ++q) load(q, s, s, false);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // (the stages' loads may be global ones: see load_lds)
    wait_loads<(NB - 1) * LPW>();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int j = 0; j < FN; ++j) B[0][j] = *reinterpret_cast<const i32x4 *>(fw[0] + j * 16 * kStage);
#pragma unroll
    for (int i = 0; i < FM; ++i) A[i] = *reinterpret_cast<const i32x4 *>(fa[0] + i * 16 * kStage);

    // half h of the stage in buffer `buf`; `next`: the buffer of the half after it
    const auto half = [&](int s, auto which, int buf, int next, bool whole) {
        constexpr int h = decltype(which)::value, o = h ^ 1;
        __builtin_amdgcn_sched_barrier(0);
        constexpr int NW = (FN + FM - 1) / FM;       // fragments of w to read with a row
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (h && i == 0) {
                __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave has read buffer s
                wait_loads<(NB - 2) * LPW>();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int x = i * NW; x < (i + 1) * NW && x < FN; ++x)
                B[o][x] = *reinterpret_cast<const i32x4 *>(fw[o] + next * BUF + x * 16 * kStage);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int t = i * FN + j;
                if (h) {
#pragma unroll
                    for (int q = t * LPW / T; q < (t + 1) * LPW / T; ++q) load(q, s + NB, buf, whole);
                }
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(B[h][j], A[i], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            A[i] = *reinterpret_cast<const i32x4 *>(fa[o] + next * BUF + i * 16 * kStage);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    typedef std::integral_constant<int, 0> First;
    typedef std::integral_constant<int, 1> Second;
    __builtin_amdgcn_s_waitcnt(0xC07F);  // nothing else is pending when the loop counts its LDS reads
    __builtin_amdgcn_sched_barrier(0);
    int s = 0;
    for (const int last = K / kStage - 2 * NB; s <= last; s += NB) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            half(s + b, First{}, b, b, true);
            half(s + b, Second{}, b, b + 1 == NB ? 0 : b + 1, true);
        }
    }
    for (; s * kStage < K; ++s) {
        const int buf = s % NB;
        half(s, First{}, buf, buf, false);
        if (s * kStage + kHalf < K) half(s, Second{}, buf, buf + 1 == NB ? 0 : buf + 1, false);
    }
    wait_loads<0>();  // nothing may arrive in LDS after the workgroup has left it

    const int64_t m = m0 + wm + fr, n = n0 + wn + (lane >> 4) * 4;
    if (part) {
        int *out = part + (int64_t)blockIdx.y * p.M * p.N;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int64_t mm = m + i * 16, nn = n + j * 16;
                if (mm >= p.M || nn >= p.N) continue;
                int *o = out + mm * p.N + nn;
                if (nn + 4 <= p.N) {
                    *reinterpret_cast<i32x4_words *>(o) = acc[i][j];
                } else {
                    for (int e = 0; e < 4; ++e)
                        if (nn + e < p.N) o[e] = acc[i][j][e];
                }
            }
        return;
    }
    __syncthreads();
    float *const scales = reinterpret_cast<float *>(lds);  // BM of rows, BN of columns, BN biases
    if (threadIdx.x < BM + BN) scales[threadIdx.x] = scale;
    if (threadIdx.x >= BM && threadIdx.x < BM + BN) scales[BN + threadIdx.x] = bias;
    __syncthreads();
    const float *rows = scales + wm + fr, *cols = scales + BM + wn + (lane >> 4) * 4;
    const bool whole = m0 + BM <= p.M && n0 + BN <= p.N;
    Columns c[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        c[j].sw = *reinterpret_cast<const f32x4 *>(cols + j * 16);
        c[j].b = *reinterpret_cast<const f32x4 *>(cols + BN + j * 16);
    }
    // Outputs of 16 bits go out eight to a lane: the quarters of a wave swap
    // halves between two fragments, and a store then writes 64 bytes of each of
    // 16 rows, not 32 (8192 x 8192 x 64: 34 us, 48 without).
    with_type(p.out_dtype, [&](auto *type) {
        typedef std::remove_pointer_t<decltype(type)> E;
        const int quarter = lane >> 4;
        const int64_t n8 = n0 + wn + (quarter & 1) * 16 + (quarter >> 1) * 8;
        E *out = static_cast<E *>(p.out) + m * p.ldo;
#pragma unroll
        for (int i = 0; i < FM; ++i, out += 16 * p.ldo) {
            const float sa = rows[i * 16];
            const bool in = whole || m + i * 16 < p.M;
#pragma unroll
            for (int j = 0; j < FN; j += 2) {
                const Four<E> v = outputs4<E>(acc[i][j], sa, c[j], p.bias != nullptr),
                              w = outputs4<E>(acc[i][j + 1], sa, c[j + 1], p.bias != nullptr);
                if constexpr (sizeof(E) == 2) {
                    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
                    typedef E e8 __attribute__((ext_vector_type(8)));
                    const u32x2 a = __builtin_bit_cast(u32x2, v), b = __builtin_bit_cast(u32x2, w);
                    const auto x = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
                    const auto y = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
                    const u32x4 both = {x[0], y[0], x[1], y[1]};
                    const int64_t at = n8 + j * 16;
                    if (in) store_valid(out + at, __builtin_bit_cast(e8, both), whole ? 8 : p.N - at);
                } else if (in) {
                    const int64_t at = n + j * 16;
                    store_valid(out + at, v, whole ? 4 : p.N - at);
                    store_valid(out + at + 16, w, whole ? 4 : p.N - at - 16);
                }
            }
        }
    });
}

// The sums of S splits and the epilogue, four outputs a thread.
__global__ __launch_bounds__(256) void int8_join(Int8Params p, const int *part, int S)
{
    const int64_t quads = (p.N + 3) / 4, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = id / quads, n = id % quads * 4;
    if (m >= p.M) return;
    i32x4 sum = {0, 0, 0, 0};
    const int *at = part + m * p.N + n;
    for (int s = 0; s < S; ++s, at += p.M * p.N) {
        if (n + 4 <= p.N) {
            sum += *reinterpret_cast<const i32x4_words *>(at);
        } else {
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) sum[e] += at[e];
        }
    }
    finish(p, m, n, sum, row_scale(p, m), columns_at(p, n));
}

// ---- few rows ----------------------------------------------------------
//
// Up to 16 R rows of a: w is read once, from global memory straight into
// fragments.  A workgroup takes 16 columns, its W waves the steps of K in
// turn; their sums are joined in LDS.  Any alignment and any K.

// 16 codes from any address.  Loads of 16 bytes that are not aligned to 4 are
// slow, so where WORDS is false they are taken from the five aligned words
// that hold them (four where the address is aligned after all): no word is
// read that holds none.  32 x 5760 x 1921: 22.6 -> 11.3 us (with K = 1920
// 8.3), 1 x 5760 x 1921: 9.6 -> 6.7 (5.7).
template <bool WORDS>
struct Codes16 {
    i32x4 v;
    int last;
    __device__ __forceinline__ void read(const int8_t *p)
    {
        if (WORDS) {
            v = *reinterpret_cast<const i32x4_words *>(p);
        } else {
            const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 3);
            const int8_t *word = p - shift;
            v = *reinterpret_cast<const i32x4_words *>(word);
            last = *reinterpret_cast<const int *>(word + (shift ? 16 : 12));
        }
    }
    // p: the address read from
    __device__ __forceinline__ i32x4 codes(const int8_t *p) const
    {
        if (WORDS) return v;
        const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 3);
        return i32x4{(int)__builtin_amdgcn_alignbyte(v[1], v[0], shift), (int)__builtin_amdgcn_alignbyte(v[2], v[1], shift),
                     (int)__builtin_amdgcn_alignbyte(v[3], v[2], shift), (int)__builtin_amdgcn_alignbyte(last, v[3], shift)};
    }
};

// 16 codes of a row from k, zeros past K: where the row ends before, its last
// 16 are read and moved into place.
template <bool WORDS>
__device__ __forceinline__ i32x4 load16(const int8_t *row, int64_t k, int64_t K)
{
    if (K < 16) {
        i32x4 v = {0, 0, 0, 0};
        for (int i = 0; i < 16; ++i)
            if (k + i < K) v[i >> 2] |= (int)((uint32_t)(uint8_t)row[k + i] << (8 * (i & 3)));
        return v;
    }
    const int64_t over = k + 16 - K;
    const int8_t *at = row + (over <= 0 ? k : K - 16);
    i32x4 v;
    if (WORDS && over <= 0) {
        v = *reinterpret_cast<const i32x4_words *>(at);
    } else {
        Codes16<false> c;
        c.read(at);
        v = c.codes(at);
    }
    if (over <= 0) return v;
    const unsigned __int128 bits = __builtin_bit_cast(unsigned __int128, v);
    return over < 16 ? __builtin_bit_cast(i32x4, bits >> (8 * (int)over)) : i32x4{0, 0, 0, 0};
}

// WORDS: the operands' rows are aligned to 4 bytes.
template <int R, int W, bool WORDS>
__global__ __launch_bounds__(W * 64) void int8_rows(Int8Params p)
{
    __shared__ i32x4 sums[W > 1 ? W - 1 : 1][R][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t wrow = n0 + (lane & 15) < p.N ? n0 + (lane & 15) : p.N - 1;
    const int8_t *w = p.w + wrow * p.ldw;
    const int8_t *a[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t row = i * 16 + (lane & 15);
        a[i] = p.a + (row < p.M ? row : p.M - 1) * p.lda;
    }
    i32x4 acc[R] = {};
    const int64_t part = (lane >> 4) * 16;
    int64_t k = (int64_t)wave * kHalf;
    constexpr int64_t step = W * kHalf;
    constexpr int U = R == 1 ? 4 : 2;  // steps whose loads are in flight together
    for (; k + (U - 1) * step + kHalf <= p.K; k += U * step) {
        Codes16<WORDS> wv[U], av[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) wv[u].read(w + k + u * step + part);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < R; ++i) av[u][i].read(a[i] + k + u * step + part);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < R; ++i)
                acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u].codes(w + part), av[u][i].codes(a[i] + part), acc[i], 0, 0, 0);
    }
    for (; k < p.K; k += step) {
        const i32x4 wv = load16<WORDS>(w, k + part, p.K);
#pragma unroll
        for (int i = 0; i < R; ++i)
            acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, load16<WORDS>(a[i], k + part, p.K), acc[i], 0, 0, 0);
    }
    if (W > 1) {
        if (wave) {
#pragma unroll
            for (int i = 0; i < R; ++i) sums[wave - 1][i][lane] = acc[i];
        }
        __syncthreads();
        if (wave) return;
        for (int o = 0; o < W - 1; ++o)
#pragma unroll
            for (int i = 0; i < R; ++i) acc[i] += sums[o][i][lane];
    }
    const int64_t n = n0 + (lane >> 4) * 4;
    const Columns c = columns_at(p, n);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t m = i * 16 + (lane & 15);
        finish(p, m, n, acc[i], row_scale(p, m), c);
    }
}

// Both operands' rows laid out anew, a's and then w's, with the leading
// dimension `ldo`, a multiple of 128, and zeros past K.  A workgroup takes
// `rows` of them.
template <bool WORDS>
__global__ __launch_bounds__(256) void int8_repack(Int8Params p, int8_t *out, int64_t ldo, int rows)
{
    const int chunks = (int)(ldo / 16);
    const int64_t first = (int64_t)blockIdx.x * rows;
    for (int i = threadIdx.x; i < rows * chunks; i += 256) {
        const int64_t row = first + i / chunks, k = i % chunks * 16;
        if (row >= p.M + p.N) return;
        const int8_t *in = row < p.M ? p.a + row * p.lda : p.w + (row - p.M) * p.ldw;
        *reinterpret_cast<i32x4 *>(out + row * ldo + k) = load16<WORDS>(in, k, p.K);
    }
}

// ---- the plan ----------------------------------------------------------

// The tiles, with what one stage of a tile costs a CU in microseconds.
struct Tile {
    int bm, bn;
    double stage;
};
constexpr Tile kTiles[] = {{64, 64, 0.20}, {128, 64, 0.36}, {128, 128, 0.57}, {256, 128, 1.00}, {256, 256, 1.60}};

struct Plan {
    int tile;        // of kTiles, or -1: int8_rows
    int S;           // splits of K
    int stages;      // of each split
    bool repack;
    int64_t ld;      // of the repacked operands
    int64_t repack_bytes, part_bytes;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

Plan make_plan(int64_t M, int64_t N, int64_t K, bool aligned)
{
    Plan p{};
    p.S = 1;
    p.tile = -1;
    aligned = aligned && K % 16 == 0;
    // Few rows read w once and wait for nothing; from 33 rows on the smallest
    // tile is faster (48 x 4096 x 4096: 9.4 us against 10.5), but not if the
    // operands have to be laid out anew for it.
    if (M <= 32 || (M <= 64 && !aligned)) return p;
    const int64_t total = ceil_div(K, kStage);
    p.repack = K > 0 && !aligned;
    p.ld = total * kStage;
    p.repack_bytes = p.repack ? (M + N) * p.ld : 0;
    // The fastest estimate: 1 us and its stages for each round of 256 tiles
    // (one for a CU), and for a split of K 5 us and its sums at 4 TB/s, there
    // and back.
    double best = 0.0;
    for (int i = 0; i < 5; ++i)
        for (int S = 1; S <= 8; S *= 2) {
            const int64_t stages = ceil_div(total, S);
            if (S > 1 && stages < 4) break;
            const int64_t tiles = ceil_div(M, kTiles[i].bm) * ceil_div(N, kTiles[i].bn);
            const double rounds = (double)ceil_div(tiles * S, 256);
            double us = rounds * (1.0 + (double)stages * kTiles[i].stage);
            if (S > 1) us += 5.0 + (double)S * (double)M * (double)N * 8.0 / 4e6;
            if (p.tile >= 0 && us >= best) continue;
            best = us;
            p.tile = i;
            p.S = S;
        }
    p.stages = total ? (int)ceil_div(total, p.S) : 1;
    p.S = total ? (int)ceil_div(total, p.stages) : 1;
    p.part_bytes = p.S > 1 ? p.S * M * N * 4 : 0;
    return p;
}

template <int BM, int BN, int WM, int WN, int NB>
void launch_tiles(const Int8Params &p, const Plan &plan, int *part, hipStream_t stream)
{
    const int64_t tm = ceil_div(p.M, BM), tn = ceil_div(p.N, BN);
    hipLaunchKernelGGL((int8_tiles<BM, BN, WM, WN, NB>), dim3((unsigned)(tm * tn), (unsigned)plan.S), dim3(WM * WN * 64), 0,
                       stream, p, (int)tm, (int)tn, plan.stages, part);
}

bool in_words(const Int8Params &p)
{
    return ((reinterpret_cast<uintptr_t>(p.a) | reinterpret_cast<uintptr_t>(p.w) | p.lda | p.ldw) & 3) == 0;
}

template <int R, bool WORDS>
void launch_rows(const Int8Params &p, hipStream_t stream)
{
    const dim3 grid((unsigned)ceil_div(p.N, 16));
    constexpr int W = R == 1 ? 16 : 8;
    // 1 x 4096 x 16384: 15.7 us with 16 waves, 18.3 with 4; 1 x 5760 x 1920: 4.9 and 4.5
    if (p.K > 4096)
        hipLaunchKernelGGL((int8_rows<R, W, WORDS>), grid, dim3(W * 64), 0, stream, p);
    else
        hipLaunchKernelGGL((int8_rows<R, 4, WORDS>), grid, dim3(256), 0, stream, p);
}
template <int R>
void launch_rows(const Int8Params &p, hipStream_t stream)
{
    if (in_words(p))
        launch_rows<R, true>(p, stream);
    else
        launch_rows<R, false>(p, stream);
}

void run_tiles(Int8Params p, const Plan &plan, hipStream_t stream)
{
    char *ws = static_cast<char *>(p.ws);
    if (plan.repack) {
        int8_t *a = reinterpret_cast<int8_t *>(ws);
        const int rows = (int)ceil_div(512, plan.ld / 16);  // some two chunks a thread
        const dim3 grid((unsigned)ceil_div(p.M + p.N, rows));
        if (in_words(p))
            hipLaunchKernelGGL((int8_repack<true>), grid, dim3(256), 0, stream, p, a, plan.ld, rows);
        else
            hipLaunchKernelGGL((int8_repack<false>), grid, dim3(256), 0, stream, p, a, plan.ld, rows);
        p.a = a;
        p.w = a + p.M * plan.ld;
        p.lda = p.ldw = p.K = plan.ld;
    }
    int *part = plan.S > 1 ? reinterpret_cast<int *>(ws + plan.repack_bytes) : nullptr;
    const int64_t tiles = ceil_div(p.M, 128) * ceil_div(p.N, 128) * plan.S;
    switch (plan.tile) {
    case 0: launch_tiles<64, 64, 2, 2, 4>(p, plan, part, stream); break;
    case 1: launch_tiles<128, 64, 2, 2, 4>(p, plan, part, stream); break;
    case 2:
        // three buffers where a CU has one tile, else two and two tiles at once
        // (2048 x 2048 x 8192: 35.0 us against 46.7; 4096^3: 79 against 71)
        if (tiles <= 256)
            launch_tiles<128, 128, 2, 4, 3>(p, plan, part, stream);
        else
            launch_tiles<128, 128, 2, 4, 2>(p, plan, part, stream);
        break;
    case 3: launch_tiles<256, 128, 2, 4, 3>(p, plan, part, stream); break;
    default: launch_tiles<256, 256, 2, 4, 2>(p, plan, part, stream); break;
    }
    if (part)
        hipLaunchKernelGGL(int8_join, dim3((unsigned)ceil_div(p.M * ceil_div(p.N, 4), 256)), dim3(256), 0, stream, p, part,
                           plan.S);
}

void launch_slice(const Int8Params &p, bool aligned, hipStream_t stream)
{
    const Plan plan = make_plan(p.M, p.N, p.K, aligned);
    if (plan.tile >= 0)
        run_tiles(p, plan, stream);
    else if (p.M <= 16)
        launch_rows<1>(p, stream);
    else if (p.M <= 32)
        launch_rows<2>(p, stream);
    else
        launch_rows<4>(p, stream);
}

// A launch's rows and columns, so that its grid stays below 2^32 threads.
constexpr int64_t kSliceM = 1 << 18, kSliceN = 1 << 20;

}  // namespace

int64_t int8_mm_workspace(int64_t M, int64_t N, int64_t K, bool aligned)
{
    if (K == 0) return 0;
    int64_t most = 0;
    for (int64_t m : {M < kSliceM ? M : kSliceM, M % kSliceM})
        for (int64_t n : {N < kSliceN ? N : kSliceN, N % kSliceN}) {
            if (!m || !n) continue;
            const Plan p = make_plan(m, n, K, aligned);
            if (p.repack_bytes + p.part_bytes > most) most = p.repack_bytes + p.part_bytes;
        }
    return most;
}

hipError_t launch_int8_mm(const Int8Params &p, bool aligned, hipStream_t stream)
{
    const int64_t size = p.out_dtype == EMU_DT_FP32 ? 4 : 2;
    for (int64_t m = 0; m < p.M; m += kSliceM)
        for (int64_t n = 0; n < p.N; n += kSliceN) {
            Int8Params q = p;
            q.M = p.M - m < kSliceM ? p.M - m : kSliceM;
            q.N = p.N - n < kSliceN ? p.N - n : kSliceN;
            if (p.K) {
                q.a = p.a + m * p.lda;
                q.w = p.w + n * p.ldw;
            }
            if (p.a_per_row) q.sa = p.sa + m;
            if (p.w_per_row) q.sw = p.sw + n;
            if (p.bias) q.bias = static_cast<const char *>(p.bias) + n * (p.bias_f32 ? 4 : size);
            q.out = static_cast<char *>(p.out) + (m * p.ldo + n) * size;
            launch_slice(q, aligned, stream);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

}  // namespace emu
