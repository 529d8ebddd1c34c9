// emu_logprobs.hip -- emu_token_logprobs and its gradient.
//
// Forward, one pass over a row: with m the largest logit, S = sum e^(z-m) and
// U = sum e^(z-m) (z-m),
//   lse = m + log S,   entropy = log S - U / S.
// Every thread runs the three numbers over its own logits with a running
// maximum (S and U are scaled when it grows); they are joined over lanes, waves
// and, where a row is split over workgroups, segments.
//
// Top tokens, in the order of 64-bit keys (the logit's bits made monotone,
// then the complement of its index: all keys differ, ties go to the lower
// index): the k-th largest of the threads' own maxima is a lower bound for
// the k-th largest logit, so only the k threads that reach it hold answers.
// Their logits are read again, those that pass the bound collected, and ranked.
#include <hip/hip_runtime.h>

#include "ops_device.h"
#include "ops_internal.h"

namespace emu {

namespace {

template <typename Z>
__device__ __forceinline__ f32x8 load8_fill(const Z *p, int64_t c, int64_t end, float fill)
{
    if (c + 8 <= end) return widen<Z>(load8(p + c));
    f32x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = c + i < end ? (float)p[c + i] : fill;
    return r;
}

constexpr int kThreads = 256;
constexpr int kTile = kThreads * 8;          // logits that a workgroup reads at once
constexpr float kLowest = -3.402823466e+38f;
constexpr float kLog2e = 1.44269504088896341f;
// e^-104 < 2^-150 rounds to 0 in binary32: differences are cut there, which
// keeps e^d d at 0 for a logit of -inf.
constexpr float kFar = -104.0f;

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

struct Stats {
    float m, s, u;
};

__device__ __forceinline__ void scale_to(Stats &a, float m)
{
    const float d = fmaxf(a.m - m, kFar);
    const float f = exp_of(d);
    a.u = f * (a.u + a.s * d);
    a.s *= f;
    a.m = m;
}

__device__ __forceinline__ Stats join(Stats a, Stats b)
{
    const float m = __builtin_elementwise_maximum(a.m, b.m);
    scale_to(a, m);
    scale_to(b, m);
    a.s += b.s;
    a.u += b.u;
    return a;
}

__device__ __forceinline__ Stats wave_join(Stats a)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        Stats b{__shfl_xor(a.m, o), __shfl_xor(a.s, o), __shfl_xor(a.u, o)};
        a = join(a, b);
    }
    return a;
}

__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 counts as 0
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o)
{
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index)
{
    return ((uint64_t)ordered(v) << 32) | (uint32_t)~index;
}

// What a row's joined numbers say.  bad: it holds a NaN or +inf.
struct Row {
    float lse, entropy;
    bool nan;
};
__device__ __forceinline__ Row row_of(const Stats &a)
{
    Row r;
    const float nan = __uint_as_float(0x7FC00000u);
    r.nan = a.m != a.m;
    if (r.nan || a.m > 3.402823466e+38f) {
        r.lse = r.entropy = nan;
    } else if (a.s == 0.0f) {
        r.lse = -INFINITY;
        r.entropy = 0.0f;
    } else {
        const float l = logf(a.s);
        r.lse = a.m + l;
        r.entropy = l - a.u / a.s;
    }
    return r;
}

__device__ __forceinline__ float logprob(float z, float lse) { return lse == -INFINITY ? lse : z - lse; }

template <typename Z>
__device__ __forceinline__ void write_tokens(const LogpParams &p, const Z *z, int64_t t, float lse)
{
    for (int64_t c = threadIdx.x; c < p.C; c += kThreads) {
        const int64_t v = p.tokens[t * p.C + c];
        p.logprobs[t * p.C + c] = v < 0 ? 0.0f : v >= p.V ? __uint_as_float(0x7FC00000u) : logprob((float)z[v], lse);
    }
}

__device__ __forceinline__ void write_top(const LogpParams &p, int64_t t, int i, uint64_t key, float lse)
{
    p.top_lp[t * p.k + i] = logprob(unordered((uint32_t)(key >> 32)), lse);
    p.top_tok[t * p.k + i] = (int64_t)(uint32_t)~(uint32_t)key;
}
__device__ __forceinline__ void write_no_top(const LogpParams &p, int64_t t)
{
    for (int i = threadIdx.x; i < p.k; i += kThreads) {
        p.top_lp[t * p.k + i] = __uint_as_float(0x7FC00000u);
        p.top_tok[t * p.k + i] = -1;
    }
}

constexpr int kMaxCandidates = 1024;

struct TopShared {
    uint64_t cand[kMaxCandidates];  // first the threads' keys, then the candidates
    uint64_t bound;
    uint64_t wave_best[4];
    uint16_t winner[EMU_MAX_TOP_TOKENS];
    int count;
};

// The k largest keys of the segment [s0, s1), in falling order; fewer where
// it has fewer logits.  emit(i, key).  `mine`: this thread's largest, or 0.
template <typename Z, typename Emit>
__device__ void top_of_segment(const Z *z, int64_t s0, int64_t s1, int k, uint64_t mine, TopShared &sh, Emit emit)
{
    const int t = threadIdx.x;
    const int iters = (int)((s1 - s0 + kTile - 1) / kTile);
    sh.cand[t] = mine;
    if (t == 0) {
        sh.bound = 0;
        sh.count = 0;
    }
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < kThreads; ++i) rank += sh.cand[i] > mine ? 1 : 0;
    const int full = __syncthreads_count(mine != 0);
    const int winners = full < k ? full : k;
    if (mine != 0 && rank < k) {
        sh.winner[rank] = (uint16_t)t;
        if (rank == k - 1) sh.bound = mine;
    }
    __syncthreads();
    const uint64_t bound = sh.bound;
    const float least = bound ? unordered((uint32_t)(bound >> 32)) : -INFINITY;
    const auto each = [&](auto f) {  // every key of the winners' logits that passes the bound
        for (int j = t; j < winners * iters; j += kThreads) {
            const int64_t c = s0 + (int64_t)(j / winners) * kTile + (int)sh.winner[j % winners] * 8;
            if (c >= s1) continue;
            const f32x8 v = load8_fill(z, c, s1, -INFINITY);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (v[e] >= least && c + e < s1) {
                    const uint64_t key = key_of(v[e], (uint32_t)(c + e));
                    if (key >= bound) f(key);
                }
        }
    };
    each([&](uint64_t key) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kMaxCandidates) sh.cand[at] = key;
    });
    __syncthreads();
    const int count = sh.count;
    if (count <= kMaxCandidates) {
        for (int i = t; i < count; i += kThreads) {
            const uint64_t key = sh.cand[i];
            int r = 0;
            for (int j = 0; j < count; ++j) r += sh.cand[j] > key ? 1 : 0;
            if (r < k) emit(r, key);
        }
        if (t >= count && t < k) emit(t, 0);
        return;
    }
    // More logits pass than there is room for (the row's largest are crowded
    // into few threads): one after the other, the largest below the last.
    uint64_t last = ~0ull;
    for (int i = 0; i < k; ++i) {
        uint64_t best = 0;
        each([&](uint64_t key) {
            if (key < last && key > best) best = key;
        });
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const uint64_t other = __shfl_xor(best, o);
            best = other > best ? other : best;
        }
        if ((t & 63) == 0) sh.wave_best[t >> 6] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 4; ++w) best = sh.wave_best[w] > best ? sh.wave_best[w] : best;
        __syncthreads();
        if (t == 0) emit(i, best);
        last = best;
    }
}

// Workgroup (t, seg) of a grid of T * P: `span` logits of row t from seg * span.
// With P = 1 it finishes the row; else logp_join does.
template <typename Z, bool TOP>
__global__ __launch_bounds__(kThreads) void logp_rows(LogpParams p, int64_t first_row, int P, int64_t span)
{
    __shared__ Stats waves[4];
    __shared__ TopShared sh;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = first_row + blockIdx.x / P;
    const int seg = blockIdx.x % P;
    const Z *z = static_cast<const Z *>(p.z) + t * p.ldz;
    const int64_t s0 = seg * span, s1 = s0 + span < p.V ? s0 + span : p.V;

    Stats a{kLowest, 0.0f, 0.0f};
    int64_t at = -1;  // where this thread's largest logit was first met
    const int64_t c0 = s0 + threadIdx.x * 8;
    const auto take = [&](const f32x8 &x, const f32x8 &y, int64_t c) {
        float cx = x[0], cy = y[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            cx = __builtin_elementwise_maximum(cx, x[j]);
            cy = __builtin_elementwise_maximum(cy, y[j]);
        }
        const float most = __builtin_elementwise_maximum(cx, cy);
        const float m = __builtin_elementwise_maximum(a.m, most);
        // (the running maximum starts at the lowest finite value, which a logit may be)
        if (TOP && (most > a.m || (at < 0 && most == a.m))) at = cx == most ? c : c + kTile;
        scale_to(a, m);
        float s[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float dx = fmaxf(x[j] - m, kFar), dy = fmaxf(y[j] - m, kFar);
            const float ex = exp_of(dx), ey = exp_of(dy);
            s[0] += ex;
            s[1] += ey;
            u[0] = __builtin_fmaf(ex, dx, u[0]);
            u[1] = __builtin_fmaf(ey, dy, u[1]);
        }
        a.s += s[0] + s[1];
        a.u += u[0] + u[1];
    };
    int64_t c = c0;
    for (; c + kTile + 8 <= s1; c += 2 * kTile) take(widen<Z>(load8(z + c)), widen<Z>(load8(z + c + kTile)), c);
    if (c < s1) take(load8_fill(z, c, s1, -INFINITY), load8_fill(z, c + kTile, s1, -INFINITY), c);

    uint64_t mine = 0;
    if (TOP && c0 < s1) {
        // a lower bound for the key of this thread's largest logit: its vector's last index
        const int64_t from = at < 0 ? c0 : at;
        mine = key_of(at < 0 ? -INFINITY : a.m, (uint32_t)(from + 7));
    }
    a = wave_join(a);
    if (lane == 0) waves[wave] = a;
    __syncthreads();
    a = join(join(waves[0], waves[1]), join(waves[2], waves[3]));

    if (P == 1) {
        const Row r = row_of(a);
        if (threadIdx.x == 0) {
            p.lse[t] = r.lse;
            p.entropy[t] = r.entropy;
        }
        write_tokens(p, z, t, r.lse);
        if (TOP) {
            if (r.nan)
                write_no_top(p, t);
            else
                top_of_segment(z, s0, s1, p.k, mine, sh, [&](int i, uint64_t key) { write_top(p, t, i, key, r.lse); });
        }
        return;
    }
    float4 *stats = static_cast<float4 *>(p.ws);
    if (threadIdx.x == 0) stats[t * P + seg] = make_float4(a.m, a.s, a.u, 0.0f);
    if (TOP && a.m == a.m) {
        uint64_t *keys = reinterpret_cast<uint64_t *>(stats + p.T * P) + (t * P + seg) * p.k;
        top_of_segment(z, s0, s1, p.k, mine, sh, [&](int i, uint64_t key) { keys[i] = key; });
    }
}

// One workgroup a row: joins its P <= 64 segments.  Their top keys (P k <=
// kMaxCandidates) are ranked by counting the larger ones.
template <typename Z>
__global__ __launch_bounds__(kThreads) void logp_join(LogpParams p, int64_t first_row, int P)
{
    __shared__ uint64_t cand[kMaxCandidates];
    const int64_t t = first_row + blockIdx.x;
    const int lane = threadIdx.x & 63;
    const float4 *stats = static_cast<const float4 *>(p.ws);
    const uint64_t *keys = reinterpret_cast<const uint64_t *>(stats + p.T * P) + t * P * p.k;
    const int count = P * p.k;
    for (int i = threadIdx.x; i < count; i += kThreads) cand[i] = keys[i];
    Stats a{kLowest, 0.0f, 0.0f};
    if (lane < P) {
        const float4 v = stats[t * P + lane];
        a = Stats{v.x, v.y, v.z};
    }
    const Row r = row_of(wave_join(a));
    if (threadIdx.x == 0) {
        p.lse[t] = r.lse;
        p.entropy[t] = r.entropy;
    }
    write_tokens(p, static_cast<const Z *>(p.z) + t * p.ldz, t, r.lse);
    if (!p.k) return;
    if (r.nan) {
        write_no_top(p, t);
        return;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t key = cand[i];
        if (!key) continue;
        int rank = 0;
        for (int j = 0; j < count; ++j) rank += cand[j] > key ? 1 : 0;
        if (rank < p.k) write_top(p, t, rank, key, r.lse);
    }
}

// Segments a row: enough for some 1,024 workgroups, of at least two tiles,
// at most 64 (16 with top tokens, whose keys the join ranks).
struct Split {
    int P;
    int64_t span;  // logits in a segment, whole tiles
};
Split split_of(int64_t T, int64_t V, int k)
{
    if (T <= 0 || T >= 512) return Split{1, V};
    int64_t P = (1024 + T - 1) / T;
    const int64_t most = (V + 2 * kTile - 1) / (2 * kTile);
    if (P > most) P = most;
    if (P > (k ? 16 : 64)) P = k ? 16 : 64;
    const int64_t span = ((V + P - 1) / P + kTile - 1) / kTile * kTile;
    return Split{(int)((V + span - 1) / span), span};
}

constexpr int64_t kRowsPerLaunch = 1 << 20;  // grid x threads stays below 2^32

template <typename Z>
hipError_t launch_logp_of(const LogpParams &p, hipStream_t stream)
{
    const auto [P, span] = split_of(p.T, p.V, p.k);
    for (int64_t r = 0; r < p.T; r += kRowsPerLaunch) {
        const int64_t rows = p.T - r < kRowsPerLaunch ? p.T - r : kRowsPerLaunch;
        const dim3 grid((unsigned)(rows * P));
        if (p.k)
            hipLaunchKernelGGL((logp_rows<Z, true>), grid, dim3(kThreads), 0, stream, p, r, P, span);
        else
            hipLaunchKernelGGL((logp_rows<Z, false>), grid, dim3(kThreads), 0, stream, p, r, P, span);
        if (P > 1) hipLaunchKernelGGL((logp_join<Z>), dim3((unsigned)rows), dim3(kThreads), 0, stream, p, r, P);
    }
    return hipGetLastError();
}

// ---- the gradient ------------------------------------------------------
//
// Elementwise but for the tokens named: with total = sum g + sum g_top and
// A = -(total + g_entropy entropy), grad = p (A - g_entropy lp), and the
// tokens' own gradients are added before the rounding.  A workgroup reads its
// tokens' logits before it writes (grad may be the logits), and writes those
// elements again at the end, each by the thread of the token's first mention.
template <typename Z>
__global__ __launch_bounds__(kThreads) void logp_grad_rows(LogpGradParams p, int64_t first_row, int64_t P, int64_t span)
{
    extern __shared__ char dyn[];
    const int H = (int)p.C + p.k;
    int *tok = reinterpret_cast<int *>(dyn);               // relative to the segment, -1 outside
    float *val = reinterpret_cast<float *>(tok + H), *logit = val + H;
    const int64_t t = first_row + blockIdx.x / P;
    const int64_t s0 = blockIdx.x % P * span, s1 = s0 + span < p.V ? s0 + span : p.V;
    const Z *z = static_cast<const Z *>(p.z) + t * p.ldz;
    Z *grad = static_cast<Z *>(p.grad) + t * p.ldgrad;
    const float lse = p.lse[t];
    const float ge = p.ge ? p.ge[t] : 0.0f;

    float part = 0.0f;
    for (int j = threadIdx.x & 63; j < H; j += 64) {  // every wave adds all of them, in the same order
        const bool given = j < p.C;
        const int64_t v = given ? p.tokens[t * p.C + j] : p.top_tok[t * p.k + (j - p.C)];
        float x = given ? (p.g ? p.g[t * p.C + j] : 0.0f) : p.gtop[t * p.k + (j - p.C)];
        if (v < 0) x = 0.0f;
        if (v >= p.V) x = __uint_as_float(0x7FC00000u);
        part += x;
        if (threadIdx.x < 64) {
            const bool here = v >= s0 && v < s1;
            tok[j] = here ? (int)(v - s0) : -1;
            val[j] = x;
            logit[j] = here ? (float)z[v] : 0.0f;
        }
    }
    const float total = wave_sum(part);
    float A = -total;
    if (p.ge) A -= ge * p.entropy[t];
    if (lse != lse) A = lse;
    const bool empty = lse == -INFINITY;
    const auto value = [&](float x) {
        const float d = fmaxf(x - lse, kFar);
        return exp_of(d) * __builtin_fmaf(-ge, d, A);
    };
    if (H) __syncthreads();
    for (int64_t c = s0 + threadIdx.x * 8; c < s1; c += kTile) {
        const f32x8 x = load8_fill(z, c, s1, 0.0f);
        f32x8 r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = empty ? 0.0f : value(x[j]);
        store8_row(grad + s0, (int)(c - s0), (int)(s1 - s0), r);
    }
    if (!H || empty) return;
    __syncthreads();
    for (int j = threadIdx.x; j < H; j += kThreads) {
        const int v = tok[j];
        if (v < 0) continue;
        bool again = false;
        for (int i = 0; i < j; ++i) again |= tok[i] == v;
        if (again) continue;
        float r = value(logit[j]);
        for (int i = j; i < H; ++i)
            if (tok[i] == v) r += val[i];
        grad[s0 + v] = (Z)r;
    }
}

template <typename Z>
hipError_t launch_logp_grad_of(const LogpGradParams &p, hipStream_t stream)
{
    const int64_t span = 4 * kTile;
    const int64_t P = (p.V + span - 1) / span;
    const size_t lds = (size_t)(p.C + p.k) * 12;
    const int64_t at_once = (int64_t(1) << 23) / P > 0 ? (int64_t(1) << 23) / P : 1;
    for (int64_t r = 0; r < p.T; r += at_once) {
        const int64_t rows = p.T - r < at_once ? p.T - r : at_once;
        hipLaunchKernelGGL((logp_grad_rows<Z>), dim3((unsigned)(rows * P)), dim3(kThreads), lds, stream, p, r, P, span);
    }
    return hipGetLastError();
}

}  // namespace

int64_t logp_workspace(int64_t T, int64_t V, int k)
{
    const int P = split_of(T, V, k).P;
    return P > 1 ? T * P * (16 + 8 * (int64_t)k) : 0;
}

hipError_t launch_logp(int z_dtype, const LogpParams &p, hipStream_t stream)
{
    if (z_dtype == EMU_DT_BF16) return launch_logp_of<__bf16>(p, stream);
    if (z_dtype == EMU_DT_FP16) return launch_logp_of<_Float16>(p, stream);
    return launch_logp_of<float>(p, stream);
}

hipError_t launch_logp_grad(int z_dtype, const LogpGradParams &p, hipStream_t stream)
{
    if (z_dtype == EMU_DT_BF16) return launch_logp_grad_of<__bf16>(p, stream);
    if (z_dtype == EMU_DT_FP16) return launch_logp_grad_of<_Float16>(p, stream);
    return launch_logp_grad_of<float>(p, stream);
}

}  // namespace emu
