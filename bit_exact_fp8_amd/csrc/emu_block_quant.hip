// emu_block_quant.hip -- codes of blocks of 128 and the gated activation
// between two products of such codes, forward and back.
//
// All of them stream: a value is read once and is in registers until its code
// is stored, since a block's largest magnitude is met within 16 lanes (8
// values each) or, for 128 x 128 values, within one workgroup.
#include <hip/hip_runtime.h>

#include "ops_block.h"

namespace emu {

namespace {

constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126

template <int Q>
constexpr float kLargest = Q == EMU_DT_E4M3FN ? 448.0f : 57344.0f;

// A block's scale and what makes codes of it.
struct BlockScale {
    float value;      // the scale
    float by;         // its reciprocal: exact (e8m0), or within 2^-23
    uint32_t byte;    // e8m0
};

// From the block's largest magnitude, NaN where it holds one.
template <int Q, bool E8M0>
__device__ __forceinline__ BlockScale scale_of(float most)
{
    BlockScale s;
    const uint32_t bits = __float_as_uint(most);
    const bool finite = bits < 0x7F800000u;
    if (E8M0) {
        // Both largest values are 7/8 of a power of two (2^9, 2^16): the least
        // 2^k that brings m 2^e, 1 <= m < 2, within is e - 8 or e - 15, and one
        // more where m is over 1.75.
        const int e = (int)(bits >> 23) + ((bits & 0x7FFFFFu) > 0x600000u) - (Q == EMU_DT_E4M3FN ? 8 : 15);
        const uint32_t b = (uint32_t)(e < 1 ? 1 : e);
        s.byte = finite ? b : 255;
        s.value = finite ? __uint_as_float(b << 23) : NAN;
        s.by = finite ? __uint_as_float((254u - b) << 23) : NAN;
    } else {
        const float v = most / kLargest<Q>;
        s.value = finite ? (v > kLeastScale ? v : kLeastScale) : NAN;
        s.by = __builtin_amdgcn_rcpf(s.value);
        s.byte = 0;
    }
    return s;
}

// x / s on a border between two codes: its neighbour with an odd last digit on
// the side where the quotient lies, so that the code's rounding is that of the
// whole quotient.
__device__ __forceinline__ float quotient_to_odd(float x, float s)
{
    const float y = x / s;
    const float off = __builtin_fmaf(-y, s, x);  // the sign of the quotient less y
    const uint32_t bits = __float_as_uint(y);
    const bool plain = off != 0.0f && __builtin_fabsf(y) > 1e-30f && __builtin_fabsf(y) < INFINITY;
    return plain ? __uint_as_float((bits - ((__float_as_uint(off) ^ bits) >> 31)) | 1) : y;
}

template <int Q>
__device__ __forceinline__ uint2 nearest_codes(const f32x8 &y)
{
    uint32_t r[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (Q == EMU_DT_E4M3FN) {
            const int b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j], y[4 * j + 1], 0, false);
            r[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j + 2], y[4 * j + 3], b, true);
        } else {
            const int b = __builtin_amdgcn_cvt_pk_bf8_f32(y[4 * j], y[4 * j + 1], 0, false);
            r[j] = (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(y[4 * j + 2], y[4 * j + 3], b, true);
        }
    }
    return make_uint2(r[0], r[1]);
}

// 8 codes of v.  Binary32 scales: v times the reciprocal is the quotient to
// within 2^-22, so that 2^-21 less and more enclose it, and where both have one
// code it is the quotient's; else all are divided.  Values past the type's largest
// (by the scale's own rounding) become it.
template <int Q, bool E8M0>
__device__ __forceinline__ uint2 codes_of(const f32x8 &v, const BlockScale &s)
{
    if (E8M0) return nearest_codes<Q>(v * s.by);
    constexpr float most = kLargest<Q>;
    f32x8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(v[i] * s.by, -most, most);
    uint2 codes = nearest_codes<Q>(y * 0.99999952f);
    const uint2 above = nearest_codes<Q>(y * 1.00000048f);
    if (__any(codes.x != above.x || codes.y != above.y)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(quotient_to_odd(v[i], s.value), -most, most);
        codes = nearest_codes<Q>(y);
    }
    const bool nan = s.value != s.value;
    return nan ? make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu) : codes;
}

template <typename T>
struct Bytes {
    T v;
} __attribute__((packed, aligned(1)));

// Codes c .. c + 7 of a row of n, those past its end not stored.
__device__ __forceinline__ void store_codes(uint8_t *row, int c, int n, const uint2 &r, bool once)
{
    uint64_t v = (uint64_t)r.y << 32 | r.x;
    uint8_t *p = row + c;
    if (c + 8 <= n) {
        if (once)
            __builtin_nontemporal_store(v, &reinterpret_cast<Bytes<uint64_t> *>(p)->v);
        else
            reinterpret_cast<Bytes<uint64_t> *>(p)->v = v;
        return;
    }
    for (int left = c < n ? n - c : 0; left > 0; --left, v >>= 8) *p++ = (uint8_t)v;
}
__device__ __forceinline__ uint2 load_codes(const uint8_t *row, int c, int n)
{
    uint64_t v = 0;
    if (c + 8 <= n) {
        v = reinterpret_cast<const Bytes<uint64_t> *>(row + c)->v;
    } else {
        for (int i = n - 1; i >= c; --i) v = v << 8 | row[i];
    }
    return make_uint2((uint32_t)v, (uint32_t)(v >> 32));
}
// What 8 codes stand for but for their scale.
template <int Q>
__device__ __forceinline__ f32x8 values_of(const uint2 &r)
{
    f32x8 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int w = (int)(j < 2 ? r.x : r.y);
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        f32x2 t;
        if (Q == EMU_DT_E4M3FN)
            t = j & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true) : __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
        else
            t = j & 1 ? __builtin_amdgcn_cvt_pk_f32_bf8(w, true) : __builtin_amdgcn_cvt_pk_f32_bf8(w, false);
        v[2 * j] = t[0];
        v[2 * j + 1] = t[1];
    }
    return v;
}

template <bool E8M0>
__device__ __forceinline__ void store_scale(void *scales, int64_t at, const BlockScale &s)
{
    if (E8M0)
        static_cast<uint8_t *>(scales)[at] = (uint8_t)s.byte;
    else
        static_cast<float *>(scales)[at] = s.value;
}
template <bool E8M0>
__device__ __forceinline__ float load_scale(const void *scales, int64_t at)
{
    if (E8M0) return e8m0_value(static_cast<const uint8_t *>(scales)[at]);
    return static_cast<const float *>(scales)[at];
}

__device__ __forceinline__ float most_of(const f32x8 &v)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __builtin_elementwise_maximum(m, __builtin_fabsf(v[i]));
    return m;
}
// Over 16 lanes: those of a block (the mirrors stand for lanes 4 and 8 apart).
__device__ __forceinline__ float most_of_16(float m)
{
    m = __builtin_elementwise_maximum(m, by_dpp<0xB1>(m));
    m = __builtin_elementwise_maximum(m, by_dpp<0x4E>(m));
    m = __builtin_elementwise_maximum(m, by_dpp<0x141>(m));
    return __builtin_elementwise_maximum(m, by_dpp<0x140>(m));
}

// Where a group of 16 lanes finds its blocks: a workgroup of 256 threads has
// ITEMS * 16 blocks one after the other along the rows, a group every 16th.
struct Place {
    int64_t row;
    int block;
    int c;       // this lane's first column
    bool in;     // (a group past the last block goes along with it)
};
__device__ __forceinline__ Place place_of(int item, int64_t items, int per_row, int lane16)
{
    Place p;
    p.in = item < items;
    const uint32_t at = p.in ? (uint32_t)item : (uint32_t)(items - 1);
    const uint32_t row = at / (uint32_t)per_row;
    p.row = row;
    p.block = (int)(at - row * (uint32_t)per_row);
    p.c = p.block * kBlock + lane16 * 8;
    return p;
}

// ---- blocks of 1 x 128 ---------------------------------------------------

// 16 lanes a block, two blocks a lane, whose loads are under way together: bf16
// with e8m0 scales take 3.8 us at 2047 x 1920, 16 at 4096 x 8192 and 62 at 16384 x
// 8192, with one block 4.2, 19 and 78 (64 x 4096: 2.7 and 2.5).  14001 x 8057, past
// the cache, runs at the memory's rate.
template <typename X, int Q, bool E8M0, int ITEMS>
__global__ __launch_bounds__(256) void quant_rows(BlockQuantParams p, int per_row)
{
    const int lane16 = threadIdx.x & 15, n = (int)p.n;
    const int64_t items = p.T * per_row;
    const int first = (int)blockIdx.x * (16 * ITEMS) + (int)(threadIdx.x >> 4);
    Place at[ITEMS];
    Raw8<X> raw[ITEMS];
    with_bool(p.once, [&](auto once) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            at[i] = place_of(first + 16 * i, items, per_row, lane16);
            raw[i] = fetch8<once()>(static_cast<const X *>(p.x) + at[i].row * p.ldx, at[i].c, n);
        }
    });
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const f32x8 v = settle8<X>(raw[i], at[i].c, n);
        const BlockScale s = scale_of<Q, E8M0>(most_of_16(most_of(v)));
        if (!at[i].in) continue;
        store_codes(static_cast<uint8_t *>(p.q) + at[i].row * p.n, at[i].c, n, codes_of<Q, E8M0>(v, s), p.once);
        if (lane16 == 0) store_scale<E8M0>(p.scales, at[i].row * per_row + at[i].block, s);
    }
}

// ---- blocks of 128 x 128 -------------------------------------------------

// A workgroup of 256 has a block: 16 lanes a row, 8 rows a thread (8 matrices of
// 4096 x 4096 fp32: 112 us, 6.0 TB/s; 115 to 121 one call after the other).
template <typename X, int Q, bool E8M0>
__global__ __launch_bounds__(256) void quant_squares(BlockQuantParams p)
{
    __shared__ float lds[4];
    const int lane = threadIdx.x & 63, wave = wave_index(), n = (int)p.n;
    const int c = (int)blockIdx.x * kBlock + (threadIdx.x & 15) * 8;
    const int64_t r0 = (int64_t)blockIdx.y * kBlock + (threadIdx.x >> 4);
    const X *x = static_cast<const X *>(p.x) + (int64_t)blockIdx.z * p.x_stride;
    Raw8<X> raw[8];
    with_bool(p.once, [&](auto once) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 16 * i;
            raw[i] = fetch8<once()>(x + (r < p.T ? r : p.T - 1) * p.ldx, c, n);
        }
    });
    float m = 0.0f;  // (a row past the end is the last one again)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __builtin_elementwise_maximum(m, most_of(settle8<X>(raw[i], c, n)));
    m = row_max<4>(m, lds, wave, lane);
    const BlockScale s = scale_of<Q, E8M0>(m);
    uint8_t *q = static_cast<uint8_t *>(p.q) + (int64_t)blockIdx.z * p.T * p.n;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r < p.T) store_codes(q + r * p.n, c, n, codes_of<Q, E8M0>(settle8<X>(raw[i], c, n), s), p.once);
    }
    if (threadIdx.x == 0)
        store_scale<E8M0>(p.scales, ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x, s);
}

// ---- the gated activation ------------------------------------------------

// p = 1 / (1 + exp(-a)) of 8 values, and exp(-a), which is 2^t with what t's
// rounding cut off put back; where it overflows p is 0.  The reciprocal is the
// hardware's with one step of Newton's, within a unit of the last place, unless
// a value is so far out that p is all but subnormal.
__device__ __forceinline__ f32x8 sigmoid(const f32x8 &a, f32x8 &e)
{
    constexpr float log2e = 1.44269502f, rest = 1.92596299e-8f, ln2 = 0.693147181f;
    float most = 0.0f;
    f32x8 p;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = -a[i] * log2e;
        const float cut = __builtin_fmaf(-a[i], log2e, -t) - a[i] * rest;
        const float x = __builtin_amdgcn_exp2f(t);
        e[i] = __builtin_fabsf(t) < 126.0f ? __builtin_fmaf(x, cut * ln2, x) : x;
        most = __builtin_elementwise_maximum(most, e[i]);
        const float d = 1.0f + e[i], near = __builtin_amdgcn_rcpf(d);
        p[i] = __builtin_fmaf(__builtin_fmaf(-d, near, 1.0f), near, near);
    }
    if (__any(!(most < 1.2676506e30f))) {  // 2^100, or a NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = 1.0f / (1.0f + e[i]);
    }
    return p;
}

// KEEP: gate's and up's own codes are stored too.  Two blocks a lane: 8192 x 8192
// bf16 with e8m0 scales takes 65 us, with all three codes 87 (with one block 80 and
// 97).  For few rows, where twice the waves hide the instructions' latencies, one
// would take less: 5.4 us for 6.0 at 1023 x 1925 with binary32 scales, 3.0 for 3.6
// at 64 x 4096; at 2240 x 10163 fp16 with all three it makes no difference (50).
template <typename X, int Q, bool E8M0, bool KEEP, int ITEMS>
__global__ __launch_bounds__(256) void swiglu_rows(SwigluParams p, int per_row)
{
    const int lane16 = threadIdx.x & 15, n = (int)p.F;
    const int64_t items = p.T * per_row;
    const int first = (int)blockIdx.x * (16 * ITEMS) + (int)(threadIdx.x >> 4);
    Place at[ITEMS];
    Raw8<X> raw[ITEMS][2];
    with_bool(p.once, [&](auto once) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            at[i] = place_of(first + 16 * i, items, per_row, lane16);
            raw[i][0] = fetch8<once()>(static_cast<const X *>(p.gate) + at[i].row * p.ldgate, at[i].c, n);
            raw[i][1] = fetch8<once()>(static_cast<const X *>(p.up) + at[i].row * p.ldup, at[i].c, n);
        }
    });
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const f32x8 g = settle8<X>(raw[i][0], at[i].c, n), u = settle8<X>(raw[i][1], at[i].c, n);
        f32x8 e;
        const f32x8 h = g * sigmoid(g, e) * u;
        const BlockScale s = scale_of<Q, E8M0>(most_of_16(most_of(h)));
        BlockScale sg, su;
        if (KEEP) {
            sg = scale_of<Q, E8M0>(most_of_16(most_of(g)));
            su = scale_of<Q, E8M0>(most_of_16(most_of(u)));
        }
        if (!at[i].in) continue;
        store_codes(static_cast<uint8_t *>(p.q) + at[i].row * p.F, at[i].c, n, codes_of<Q, E8M0>(h, s), p.once);
        if (lane16 == 0) store_scale<E8M0>(p.scales, at[i].row * per_row + at[i].block, s);
        if (KEEP) {
            uint8_t *kept = static_cast<uint8_t *>(p.kept) + at[i].row * 2 * p.F;
            store_codes(kept, at[i].c, n, codes_of<Q, E8M0>(g, sg), p.once);
            store_codes(kept + p.F, at[i].c, n, codes_of<Q, E8M0>(u, su), p.once);
            if (lane16 == 0) {
                const int64_t b = at[i].row * 2 * per_row + at[i].block;
                store_scale<E8M0>(p.kept_scales, b, sg);
                store_scale<E8M0>(p.kept_scales, b + per_row, su);
            }
        }
    }
}

// (8192 x 8192 bf16: 89 us, 6.0 TB/s; one call after the other 81 in the first
// 2 ms and 92 to 101 in the next 8.  With one block a lane as much; 1023 x 1925
// 7.8 us, with one 5.9)
template <typename G, int Q, bool E8M0, int ITEMS>
__global__ __launch_bounds__(256) void swiglu_grad_rows(SwigluGradParams p, int per_row)
{
    const int lane16 = threadIdx.x & 15, n = (int)p.F;
    const int64_t items = p.T * per_row;
    const int first = (int)blockIdx.x * (16 * ITEMS) + (int)(threadIdx.x >> 4);
    Place at[ITEMS];
    Raw8<G> raw[ITEMS];
    uint2 codes[ITEMS][2];
    float s[ITEMS][2];
    with_bool(p.once, [&](auto once) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            at[i] = place_of(first + 16 * i, items, per_row, lane16);
            const uint8_t *kept = static_cast<const uint8_t *>(p.kept) + at[i].row * 2 * p.F;
            const int64_t b = at[i].row * 2 * per_row + at[i].block;
            raw[i] = fetch8<once()>(static_cast<const G *>(p.g) + at[i].row * p.ldg, at[i].c, n);
            codes[i][0] = load_codes(kept, at[i].c, n);
            codes[i][1] = load_codes(kept + p.F, at[i].c, n);
            s[i][0] = load_scale<E8M0>(p.kept_scales, b);
            s[i][1] = load_scale<E8M0>(p.kept_scales, b + per_row);
        }
    });
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        if (!at[i].in) continue;
        const f32x8 g = settle8<G>(raw[i], at[i].c, n), a = values_of<Q>(codes[i][0]) * s[i][0],
                    b = values_of<Q>(codes[i][1]) * s[i][1];
        f32x8 da, db, e;
        const f32x8 s = sigmoid(a, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float rest = e[j] > 1.0f ? 1.0f - s[j] : e[j] * s[j];  // (no infinity meets a zero)
            da[j] = g[j] * b[j] * (s[j] * __builtin_fmaf(a[j], rest, 1.0f));
            db[j] = g[j] * (a[j] * s[j]);
        }
        G *out = static_cast<G *>(p.grad) + at[i].row * p.ldgrad;
        with_bool(p.once, [&](auto once) {
            store8_row<once()>(out, at[i].c, n, da);
            store8_row<once()>(out + p.F, at[i].c, n, db);
        });
    }
}

// ---- launches ------------------------------------------------------------

// f(null pointer of the element type, the codes' type, whether scales are e8m0)
template <typename F>
void with_types(int x_dtype, int q_dtype, bool e8m0, F f)
{
    const auto with_x = [&](auto q, auto e) {
        if (x_dtype == EMU_DT_BF16)
            f(static_cast<__bf16 *>(nullptr), q, e);
        else if (x_dtype == EMU_DT_FP16)
            f(static_cast<_Float16 *>(nullptr), q, e);
        else
            f(static_cast<float *>(nullptr), q, e);
    };
    const auto with_q = [&](auto e) {
        if (q_dtype == EMU_DT_E4M3FN)
            with_x(std::integral_constant<int, EMU_DT_E4M3FN>{}, e);
        else
            with_x(std::integral_constant<int, EMU_DT_E5M2>{}, e);
    };
    if (e8m0)
        with_q(std::true_type{});
    else
        with_q(std::false_type{});
}

// Rows of a launch: 2^28 blocks, of 8 threads each where a lane has two, so that
// its grid stays below 2^32 threads (and blocks are counted in 31 bits).
int64_t rows_of_launch(int64_t T, int64_t per_row)
{
    const int64_t most = (int64_t(1) << 28) / per_row;
    return T < most ? T : most < 1 ? 1 : most;
}
// Blocks of a group of 16 lanes.
constexpr int kItems = 2;
unsigned groups_of(int64_t items) { return (unsigned)((items + 16 * kItems - 1) / (16 * kItems)); }

}  // namespace

hipError_t launch_block_quant(int x_dtype, int q_dtype, bool e8m0, int block_rows, const BlockQuantParams &p, hipStream_t stream)
{
    const int64_t size = x_dtype == EMU_DT_FP32 ? 4 : 2, per_row = blocks_of(p.n);
    BlockQuantParams o = p;
    o.once = p.E * p.T * p.n * (size + 1) > kOnceBytes;
    hipError_t status = hipSuccess;
    with_types(x_dtype, q_dtype, e8m0, [&](auto *type, auto q, auto e) {
        typedef std::remove_pointer_t<decltype(type)> X;
        constexpr int Q = q();
        constexpr bool E8 = e();
        const auto scales = [&](int64_t at) { return static_cast<char *>(p.scales) + at * (E8 ? 1 : 4); };
        if (block_rows == 1) {
            for (int64_t m = 0; m < p.E; ++m)
                for (int64_t r = 0; r < p.T; r += rows_of_launch(p.T, per_row)) {
                    o.T = rows_of_launch(p.T - r, per_row);
                    o.x = static_cast<const X *>(p.x) + m * p.x_stride + r * p.ldx;
                    o.q = static_cast<char *>(p.q) + (m * p.T + r) * p.n;
                    o.scales = scales((m * p.T + r) * per_row);
                    hipLaunchKernelGGL((quant_rows<X, Q, E8, kItems>), dim3(groups_of(o.T * per_row)), dim3(256), 0, stream, o,
                                       (int)per_row);
                    if (status == hipSuccess) status = hipGetLastError();
                }
            return;
        }
        // Whole matrices where a launch holds one, else parts of one: its grid
        // stays below 2^32 threads and within its axes' limits.
        const int64_t tall = blocks_of(p.T);
        int64_t step = (int64_t(1) << 23) / per_row;
        step = step < 1 ? 1 : step > 32768 ? 32768 : step;
        const int64_t high = tall < step ? tall : step, deep = high < tall ? 1 : step / high;
        for (int64_t m = 0; m < p.E; m += deep)
            for (int64_t r = 0; r < tall; r += high) {
                const int64_t h = tall - r < high ? tall - r : high, d = p.E - m < deep ? p.E - m : deep;
                o.T = r + h < tall ? h * kBlock : p.T - r * kBlock;
                o.x = static_cast<const X *>(p.x) + m * p.x_stride + r * kBlock * p.ldx;
                o.q = static_cast<char *>(p.q) + (m * p.T + r * kBlock) * p.n;
                o.scales = scales((m * tall + r) * per_row);
                hipLaunchKernelGGL((quant_squares<X, Q, E8>), dim3((unsigned)per_row, (unsigned)h, (unsigned)d), dim3(256), 0,
                                   stream, o);
                if (status == hipSuccess) status = hipGetLastError();
            }
    });
    return status;
}

hipError_t launch_swiglu(int dtype, int q_dtype, bool e8m0, const SwigluParams &p, hipStream_t stream)
{
    const int64_t size = dtype == EMU_DT_FP32 ? 4 : 2, per_row = blocks_of(p.F), unit = e8m0 ? 1 : 4;
    SwigluParams o = p;
    o.once = p.T * p.F * (2 * size + (p.kept ? 3 : 1)) > kOnceBytes;
    hipError_t status = hipSuccess;
    with_types(dtype, q_dtype, e8m0, [&](auto *type, auto q, auto e) {
        typedef std::remove_pointer_t<decltype(type)> X;
        for (int64_t r = 0; r < p.T; r += rows_of_launch(p.T, per_row)) {
            o.T = rows_of_launch(p.T - r, per_row);
            o.gate = static_cast<const X *>(p.gate) + r * p.ldgate;
            o.up = static_cast<const X *>(p.up) + r * p.ldup;
            o.q = static_cast<char *>(p.q) + r * p.F;
            o.scales = static_cast<char *>(p.scales) + r * per_row * unit;
            const dim3 grid(groups_of(o.T * per_row));
            if (p.kept) {
                o.kept = static_cast<char *>(p.kept) + r * 2 * p.F;
                o.kept_scales = static_cast<char *>(p.kept_scales) + r * 2 * per_row * unit;
                hipLaunchKernelGGL((swiglu_rows<X, q(), e(), true, kItems>), grid, dim3(256), 0, stream, o, (int)per_row);
            } else {
                hipLaunchKernelGGL((swiglu_rows<X, q(), e(), false, kItems>), grid, dim3(256), 0, stream, o, (int)per_row);
            }
            if (status == hipSuccess) status = hipGetLastError();
        }
    });
    return status;
}

hipError_t launch_swiglu_grad(int g_dtype, int q_dtype, bool e8m0, const SwigluGradParams &p, hipStream_t stream)
{
    const int64_t size = g_dtype == EMU_DT_FP32 ? 4 : 2, per_row = blocks_of(p.F), unit = e8m0 ? 1 : 4;
    SwigluGradParams o = p;
    o.once = p.T * p.F * (3 * size + 2) > kOnceBytes;
    hipError_t status = hipSuccess;
    with_types(g_dtype, q_dtype, e8m0, [&](auto *type, auto q, auto e) {
        typedef std::remove_pointer_t<decltype(type)> G;
        for (int64_t r = 0; r < p.T; r += rows_of_launch(p.T, per_row)) {
            o.T = rows_of_launch(p.T - r, per_row);
            o.g = static_cast<const G *>(p.g) + r * p.ldg;
            o.kept = static_cast<const char *>(p.kept) + r * 2 * p.F;
            o.kept_scales = static_cast<const char *>(p.kept_scales) + r * 2 * per_row * unit;
            o.grad = static_cast<G *>(p.grad) + r * p.ldgrad;
            hipLaunchKernelGGL((swiglu_grad_rows<G, q(), e(), kItems>), dim3(groups_of(o.T * per_row)), dim3(256), 0, stream, o,
                               (int)per_row);
            if (status == hipSuccess) status = hipGetLastError();
        }
    });
    return status;
}

}  // namespace emu
