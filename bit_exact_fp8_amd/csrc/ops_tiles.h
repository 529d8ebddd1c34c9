// ops_tiles.h -- what the products of 8-bit codes share: LDS places, waits,
// loads of codes from any address and stores of outputs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_device.h"

namespace emu {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_words __attribute__((aligned(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename E>
using Four = E __attribute__((ext_vector_type(4)));
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

constexpr int kStage = 128;  // codes of K at a time

// What is the same for all lanes, known to be so.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v));
}

// LDS holds a stage's rows of 128 bytes as eight chunks of 16; row r's chunk c
// stands at place c ^ swizzle(r), which spreads the 16 rows that a
// ds_read_b128 meets over all banks.
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

// Workgroups go round the 8 XCDs in turn; each XCD gets a run of neighbouring
// tiles, HIGH rows of tiles high, whose operands its L2 then holds.
template <int HIGH>
__device__ __forceinline__ void tile_of(int id, int tm, int tn, int &m, int &n)
{
    const int total = tm * tn, xcd = id & 7, each = total >> 3, rest = total & 7;
    id = xcd * each + (xcd < rest ? xcd : rest) + (id >> 3);
    const int band = id / (HIGH * tn), left = tm - HIGH * band, high = left < HIGH ? left : HIGH, in = id - band * HIGH * tn;
    m = HIGH * band + in % high;
    n = in / high;
}

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

// Rows of matrices of `per` rows each, `total` in all, laid out anew: 16-byte
// aligned, with the leading dimension `ldo`, a multiple of 128, and zeros past K.
// A workgroup takes `rows` of them.
struct RepackRows {
    const int8_t *in;
    int64_t ld, stride, per, total, K;
    int8_t *out;
    int64_t ldo;
    int rows;
    bool words;  // the rows are aligned to 4 bytes
};
inline int64_t repack_groups(const RepackRows &j) { return j.total ? ceil_div(j.total, j.rows) : 0; }
__device__ __forceinline__ void repack_rows(const RepackRows &j, int64_t group)
{
    const int chunks = (int)(j.ldo / 16);
    const int64_t first = group * j.rows, matrix = j.per < j.total ? first / j.per : 0, at = first - matrix * j.per;
    const int64_t left = j.total - first;
    const int rows = left < j.rows ? (int)left : j.rows;
    for (int i = threadIdx.x; i < rows * chunks; i += 256) {
        const int r = i / chunks, k = (i - r * chunks) * 16;
        int64_t m = matrix, row = at + r;
        while (row >= j.per) row -= j.per, ++m;
        const int8_t *from = j.in + m * j.stride + row * j.ld;
        *reinterpret_cast<i32x4 *>(j.out + (first + r) * j.ldo + k) = j.words ? load16<true>(from, k, j.K) : load16<false>(from, k, j.K);
    }
}

// A wave's outputs: fragment (i, j) holds the outputs of row m + 16 i from
// column n + 16 j + 4 (lane / 16) on, four to a lane; `whole`: all of them lie
// within the matrix; `add`: a bias for each column.  Outputs of 16 bits go out eight to a lane: the quarters of
// a wave swap halves between two fragments, and a store then writes 64 bytes
// of each of 16 rows, not 32.
template <int FM, int FN>
__device__ __forceinline__ void store_tile(void *to, int dtype, int64_t ld, const f32x4 (&acc)[FM][FN], const f32x4 (&bias)[FN], bool add,
                                           int64_t m, int64_t rows, int64_t n, int64_t cols, int lane, bool whole)
{
    with_type(dtype, [&](auto *type) {
        typedef std::remove_pointer_t<decltype(type)> E;
        const int quarter = lane >> 4;
        const int64_t n4 = n + quarter * 4, n8 = n + (quarter & 1) * 16 + (quarter >> 1) * 8;
        E *out = static_cast<E *>(to) + m * ld;
#pragma unroll
        for (int i = 0; i < FM; ++i, out += 16 * ld) {
            const bool in = whole || m + i * 16 < rows;
#pragma unroll
            for (int j = 0; j < FN; j += 2) {
                f32x4 x = acc[i][j], y = acc[i][j + 1];
                if (add) x += bias[j], y += bias[j + 1];
                const Four<E> v = __builtin_convertvector(x, Four<E>), w = __builtin_convertvector(y, Four<E>);
                if constexpr (sizeof(E) == 2) {
                    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
                    typedef E e8 __attribute__((ext_vector_type(8)));
                    const u32x2 a = __builtin_bit_cast(u32x2, v), b = __builtin_bit_cast(u32x2, w);
                    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
                    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
                    const u32x4 both = {c[0], d[0], c[1], d[1]};
                    const int64_t at = n8 + j * 16;
                    if (in) store_valid(out + at, __builtin_bit_cast(e8, both), whole ? 8 : cols - at);
                } else if (in) {
                    const int64_t at = n4 + j * 16;
                    store_valid(out + at, v, whole ? 4 : cols - at);
                    store_valid(out + at + 16, w, whole ? 4 : cols - at - 16);
                }
            }
        }
    });
}

}  // namespace emu
