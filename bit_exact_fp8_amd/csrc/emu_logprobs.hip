// emu_logprobs.hip -- emu_token_logprobs and its gradient.
//
// Forward, one pass over a row: with m the largest logit, S = sum e^(z-m) and
// U = sum e^(z-m) (z-m),
//   lse = m + log S,   entropy = log S - U / S.
// Every thread runs S and U over its own logits against a reference that
// follows its maximum; they are joined over lanes, waves and, where a row is
// split over workgroups, segments.
//
// Top tokens, in the order of 64-bit keys (the logit's bits made monotone,
// then the complement of its index: all keys differ, ties go to the lower
// index): the k-th largest of the threads' own maxima is a lower bound for
// the k-th largest logit, so only the k threads that reach it hold answers.
// Their logits that pass the bound are collected, and ranked.
#include <hip/hip_runtime.h>

#include "ops_device.h"
#include "ops_internal.h"

namespace emu {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = kThreads * 8;          // logits that a workgroup reads at once
constexpr float kLowest = -3.402823466e+38f;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kLog2eRest = (float)(1.44269504088896341 - (double)kLog2e);
// e^-104 < 2^-150 rounds to 0 in binary32: differences are cut there, which
// keeps e^d d at 0 for a logit of -inf.
constexpr float kFar = -104.0f;

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// 8 logits from c, -inf past n (fetch8's loads: any c, n >= 1).
template <typename Z>
__device__ __forceinline__ f32x8 logits8(const Z *z, int c, int n)
{
    const f32x8 v = widen<Z>(fetch8(z, c, n));
    if (c + 8 <= n) return v;
    if (n >= 8) return moved(v, c + 8 - n < 8 ? c + 8 - n : 8, -INFINITY);
    f32x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = c + i < n ? v[i] : -INFINITY;
    return r;
}

struct Stats {
    float m, s, u;
};

// A thread's sums, in base 2: s = sum 2^d and u = sum 2^d d with d = z log2(e) - r.
// r is a whole number near most log2(e), so that d is rounded once (one fma),
// and is moved only when the maximum has left it by 6 (s stays below 2^7 a
// logit).  Logits below kClamp count as kClamp, whose 2^d is 0; a row whose
// largest lies beyond kWide is summed again (wide_stats), since r would
// not be near enough there.
constexpr float kClamp = -1048576.0f, kWide = 524288.0f;
struct Run {
    float most, r, s, u;  // most: the largest logit, NaN once there was one
};
__device__ __forceinline__ Run empty_run() { return Run{-INFINITY, kClamp * kLog2e, 0.0f, 0.0f}; }

__device__ __forceinline__ void move_to(Run &a, float r)
{
    const float d = a.r - r, f = __builtin_amdgcn_exp2f(d);
    a.u = f * __builtin_fmaf(a.s, d, a.u);
    a.s *= f;
    a.r = r;
}

// 16 logits more.
__device__ __forceinline__ void take16(Run &a, f32x8 x, f32x8 y, float most)
{
    a.most = __builtin_elementwise_maximum(a.most, most);
    float least = __builtin_elementwise_minimum(x[0], y[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) least = __builtin_elementwise_minimum(__builtin_elementwise_minimum(least, x[j]), y[j]);
    if (__any(least < kClamp)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = __builtin_elementwise_maximum(x[j], kClamp);
            y[j] = __builtin_elementwise_maximum(y[j], kClamp);
        }
    }
    const float top = a.most * kLog2e;
    if (top > a.r + 6.0f) move_to(a, ceilf(top));
    float s[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float dx = __builtin_fmaf(x[j], kLog2e, -a.r), dy = __builtin_fmaf(y[j], kLog2e, -a.r);
        const float ex = __builtin_amdgcn_exp2f(dx), ey = __builtin_amdgcn_exp2f(dy);
        s[0] += ex;
        s[1] += ey;
        u[0] = __builtin_fmaf(ex, dx, u[0]);
        u[1] = __builtin_fmaf(ey, dy, u[1]);
    }
    a.s += s[0] + s[1];
    a.u += u[0] + u[1];
}

__device__ __forceinline__ float most8(const f32x8 &x)
{
    float m = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = __builtin_elementwise_maximum(m, x[j]);
    return m;
}

// The runs of a workgroup's threads in one, the same in each.
__device__ __forceinline__ Run block_join(Run a, Run *waves)
{
    const float r = wave_max(a.r);
    move_to(a, r);
    a = Run{wave_max(a.most), r, wave_sum(a.s), wave_sum(a.u)};
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = a;
    __syncthreads();
    Run w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = waves[i];
    const float top = fmaxf(fmaxf(w[0].r, w[1].r), fmaxf(w[2].r, w[3].r));
    Run b{w[0].most, top, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        move_to(w[i], top);
        b.most = __builtin_elementwise_maximum(b.most, w[i].most);
        b.s += w[i].s;
        b.u += w[i].u;
    }
    return b;
}

// Against the largest logit itself, and in base e.
__device__ __forceinline__ Stats stats_of(const Run &a)
{
    const float d = __builtin_fmaf(a.most, kLog2e, -a.r), f = __builtin_amdgcn_exp2f(-d);
    return Stats{a.most, a.s * f, kLn2 * f * __builtin_fmaf(-d, a.s, a.u)};
}

// The same of [s0, s1) where the largest logit m is finite but far from 0.
template <typename Z>
__device__ Stats wide_stats(const Z *z, int s0, int s1, float m, Stats *waves)
{
    Stats a{m, 0.0f, 0.0f};
    for (int c = s0 + (int)threadIdx.x * 8; c < s1; c += kTile) {
        const f32x8 x = logits8(z, c, s1);
        float s = 0.0f, u = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = fmaxf(x[j] - m, kFar), e = exp_of(d);
            s += e;
            u = __builtin_fmaf(e, d, u);
        }
        a.s += s;
        a.u += u;
    }
    a.s = wave_sum(a.s);
    a.u = wave_sum(a.u);
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = a;
    __syncthreads();
    return Stats{m, waves[0].s + waves[1].s + (waves[2].s + waves[3].s), waves[0].u + waves[1].u + (waves[2].u + waves[3].u)};
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

// A given token's logit, read before the row's sums are there; and what it gives.
template <typename Z>
__device__ __forceinline__ float token_logit(const LogpParams &p, const Z *z, int64_t t, int64_t c, int64_t &v)
{
    v = c < p.C ? p.tokens[t * p.C + c] : -1;
    return v >= 0 && v < p.V ? (float)z[v] : 0.0f;
}
__device__ __forceinline__ void write_token(const LogpParams &p, int64_t t, int64_t c, int64_t v, float logit, float lse)
{
    if (c < p.C) p.logprobs[t * p.C + c] = v < 0 ? 0.0f : v >= p.V ? __uint_as_float(0x7FC00000u) : logprob(logit, lse);
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

// Leading bits of ordered() in which two values of a type can differ (the
// rest are all 0 or, below 0, all 1).
template <typename Z>
constexpr int kOrderBits = sizeof(Z) == 4 ? 32 : __is_same(Z, __bf16) ? 16 : 19;

// A key that at least k of a wave's 64 R keys reach; 0 if there are not k (0
// is no key).  Only keys of the same value as the k-th largest can make them
// more, and where those are more than kSpare too many, none but such of a
// lower index does.  Bit by bit, the lanes counted by ballots.  Loops and not
// straight code here and below: in a kernel this short what was never run
// before has to be fetched (1 x 4096, one top token: 6.2 us unrolled, 4.9).
constexpr int kSpare = 64;

template <int R, typename F>
__device__ __forceinline__ int wave_count(F pred)
{
    int n = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) n += __popcll(__ballot(pred(r)));
    return n;
}
template <int BITS, int R>
__device__ __forceinline__ uint64_t kth_key(const uint64_t (&key)[R], int k)
{
    uint32_t high[R], index[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        high[r] = (uint32_t)(key[r] >> 32);
        index[r] = (uint32_t)key[r];
        asm("" : "+v"(high[r]), "+v"(index[r]));  // (compared in 32 bits, not as halves of 64)
    }
    uint32_t b = 0;
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit >= 1u << (32 - BITS) && bit; bit >>= 1)
        if (wave_count<R>([&](int r) { return high[r] >= (b | bit); }) >= k) b |= bit;
    if (!b) return 0;
    if (BITS < 32 && !(b >> 31)) b |= (uint32_t)((1ull << (32 - BITS)) - 1);
    const int over = wave_count<R>([&](int r) { return high[r] > b; });
    const int same = wave_count<R>([&](int r) { return high[r] == b; });
    uint32_t low = 0;
    if (over + same > k + kSpare) {
#pragma unroll 1
        for (uint32_t bit = 1u << 31; bit; bit >>= 1)
            if (wave_count<R>([&](int r) { return high[r] == b && index[r] >= (low | bit); }) >= k - over) low |= bit;
    }
    return (uint64_t)b << 32 | low;
}

constexpr int kMaxCandidates = 1024;

constexpr int kVectors = 256;

struct TopShared {
    float logit[kVectors][8];       // vectors that hold a logit that passes
    int index[kVectors];            // of their first logits
    uint64_t cand[kMaxCandidates];  // keys that pass, zeros after the last
    uint64_t key[kThreads];         // the threads' own
    uint64_t wave_best[4];
    uint16_t winner[kThreads];
    int count, vectors, winners;
};
__device__ __forceinline__ void clear(TopShared &sh)
{
#pragma unroll
    for (int i = 0; i < kMaxCandidates; i += kThreads) sh.cand[i + threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.count = sh.vectors = sh.winners = 0;
}
__device__ __forceinline__ void collect(TopShared &sh, uint64_t key)
{
    const int at = atomicAdd(&sh.count, 1);
    if (at < kMaxCandidates) sh.cand[at] = key;
}

// emit(rank, key) of the k largest candidates.
template <typename Emit>
__device__ __forceinline__ void rank_candidates(const TopShared &sh, int count, int k, Emit emit)
{
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t key = sh.cand[i];
        int r = 0;
        for (int j = 0; j < count; j += 8) {
            uint64_t other[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) other[e] = sh.cand[j + e];
#pragma unroll
            for (int e = 0; e < 8; ++e) r += other[e] > key ? 1 : 0;
        }
        if (r < k) emit(r, key);
    }
}

// What a thread knows of its logits.
struct Own {
    uint64_t key;  // a lower bound for its largest key (that of its vector's last index), or 0
    int at;        // that vector's first index
    float second;  // the largest logit of its other vectors
};

// The k largest keys of the segment [s0, s1), in falling order; fewer where
// it has fewer logits, and zeros for the rest.  emit(i, key).  HELD: the
// segment's logits are x (from s0 + 8 threadIdx.x) and y (a tile further);
// else a thread whose key passes reads its vector again, and where its others
// may hold a logit that passes, all threads read those.
template <bool HELD, typename Z, typename Emit>
__device__ __forceinline__ void top_of_segment(const Z *z, int s0, int s1, const f32x8 &x, const f32x8 &y, int k,
                                               const Own &own, TopShared &sh, Emit emit)
{
    const int t = threadIdx.x;
    sh.key[t] = own.key;
    clear(sh);
    __syncthreads();
    uint64_t all[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) all[i] = sh.key[i * 64 + (t & 63)];
    const uint64_t bound = kth_key<kOrderBits<Z>>(all, k);  // the same in every wave
    const bool wins = own.key && own.key >= bound;
    const float least = bound ? unordered((uint32_t)(bound >> 32)) : -INFINITY;
    const bool others = wins && own.second >= least;
    if (!HELD) {
        if (others) sh.winner[atomicAdd(&sh.winners, 1)] = (uint16_t)t;
        __syncthreads();
    }
    const auto each = [&](auto f) {  // f(vector, its first index), of all that may hold a logit that passes
        if constexpr (HELD) {
            if (!wins) return;
            f(x, s0 + t * 8);
            f(y, s0 + t * 8 + kTile);
        } else {
            if (wins && !others) f(logits8(z, own.at, s1), own.at);
            const int winners = sh.winners, iters = (s1 - s0 + kTile - 1) / kTile;
            for (int j = t; j < winners * iters; j += kThreads) {
                const int c = s0 + j / winners * kTile + (int)sh.winner[j % winners] * 8;
                if (c < s1) f(logits8(z, c, s1), c);
            }
        }
    };
    each([&](const f32x8 &v, int c) {
        if (most8(v) < least || c >= s1) return;
        const int at = atomicAdd(&sh.vectors, 1);
        if (at >= kVectors) return;
        *reinterpret_cast<f32x8 *>(sh.logit[at]) = v;
        sh.index[at] = c;
    });
    __syncthreads();
    const int vectors = sh.vectors;
    for (int i = t; i < vectors * 8 && vectors <= kVectors; i += kThreads) {
        const int c = sh.index[i >> 3] + (i & 7);
        if (c >= s1) continue;
        const uint64_t key = key_of(sh.logit[i >> 3][i & 7], (uint32_t)c);
        if (key >= bound) collect(sh, key);
    }
    __syncthreads();
    const int count = sh.count;
    if (vectors <= kVectors && count <= kMaxCandidates) {
        rank_candidates(sh, count, k, emit);
        if (t >= count && t < k) emit(t, 0);
        return;
    }
    // More logits pass than there is room for (the row's largest are crowded
    // into few threads): one after the other, the largest below the last.
    uint64_t last = ~0ull;
    for (int i = 0; i < k; ++i) {
        uint64_t best = 0;
        each([&](const f32x8 &v, int c) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t key = c + e < s1 ? key_of(v[e], (uint32_t)(c + e)) : 0;
                best = key < last && key > best ? key : best;
            }
        });
        best = wave_reduce(best, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
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
// With P = 1 it finishes the row; else logp_join does.  HELD: span is at
// most two tiles, which stay in registers.
template <typename Z, bool TOP, bool HELD, bool ONCE>
__global__ __launch_bounds__(kThreads, HELD ? 6 : 8) void logp_rows(LogpParams p, int64_t first_row, int P, int span)
{
    __shared__ Run waves[4];
    __shared__ Stats wide[4];
    __shared__ TopShared sh;
    const int64_t t = first_row + blockIdx.x / P;
    const int seg = blockIdx.x % P;
    const Z *z = static_cast<const Z *>(p.z) + t * p.ldz;
    const int s0 = seg * span, s1 = span < p.V - s0 ? s0 + span : (int)p.V;
    int64_t token = -1;
    float logit = 0.0f;
    if (P == 1) logit = token_logit(p, z, t, threadIdx.x, token);

    Run a = empty_run();
    int at = -1;  // the vector where this thread's largest logit was first met
    float second = -INFINITY;  // the largest logit of its other vectors
    const int c0 = s0 + (int)threadIdx.x * 8;
    const auto take = [&](const f32x8 &x, const f32x8 &y, int c) {
        const float mx = most8(x), my = most8(y), most = __builtin_elementwise_maximum(mx, my);
        if (TOP) {
            second = fmaxf(second, fmaxf(fminf(mx, my), fminf(most, a.most)));
            if (most > a.most) at = mx == most ? c : c + kTile;
        }
        take16(a, x, y, most);
    };
    f32x8 x{}, y{};  // (only HELD uses them)
    if constexpr (HELD) {
        x = logits8(z, c0, s1);
        y = logits8(z, c0 + kTile, s1);
        take(x, y, c0);
    } else {
        int c = c0;
        for (; c + kTile + 8 <= s1; c += 2 * kTile) take(widen<Z>(load8<ONCE>(z + c)), widen<Z>(load8<ONCE>(z + c + kTile)), c);
        if (c < s1) take(logits8(z, c, s1), logits8(z, c + kTile, s1), c);
    }

    Own own{0, at < 0 ? c0 : at, second};
    if (TOP && c0 < s1) own.key = key_of(a.most, (uint32_t)(own.at + 7));
    a = block_join(a, waves);
    Stats st{a.most, 0.0f, 0.0f};
    if (a.most == -INFINITY)
        st.m = kLowest;
    else if (__builtin_fabsf(a.most) <= kWide)
        st = stats_of(a);
    else if (__builtin_fabsf(a.most) <= 3.402823466e+38f)
        st = wide_stats(z, s0, s1, a.most, wide);

    if (P == 1) {
        const Row r = row_of(st);
        if (threadIdx.x == 0) {
            p.lse[t] = r.lse;
            p.entropy[t] = r.entropy;
        }
        write_token(p, t, threadIdx.x, token, logit, r.lse);
        for (int64_t c = threadIdx.x + kThreads; c < p.C; c += kThreads) {
            logit = token_logit(p, z, t, c, token);
            write_token(p, t, c, token, logit, r.lse);
        }
        if (TOP) {
            if (r.nan)
                write_no_top(p, t);
            else
                top_of_segment<HELD>(z, s0, s1, x, y, p.k, own, sh,
                                     [&](int i, uint64_t key) { write_top(p, t, i, key, r.lse); });
        }
        return;
    }
    float4 *stats = static_cast<float4 *>(p.ws);
    if (threadIdx.x == 0) stats[t * P + seg] = make_float4(st.m, st.s, st.u, 0.0f);
    if (TOP && st.m == st.m) {
        uint64_t *keys = reinterpret_cast<uint64_t *>(stats + p.T * P) + (t * P + seg) * p.k;
        top_of_segment<HELD>(z, s0, s1, x, y, p.k, own, sh, [&](int i, uint64_t key) { keys[i] = key; });
    }
}

// One workgroup a row: joins its P <= 64 segments.  Each wave finds a bound
// for its quarter of the P k <= kMaxCandidates top keys; those that pass the
// highest bound are ranked.
template <typename Z>
__global__ __launch_bounds__(kThreads) void logp_join(LogpParams p, int64_t first_row, int P)
{
    __shared__ TopShared sh;
    const int64_t t = first_row + blockIdx.x;
    const int lane = threadIdx.x & 63, wave = wave_index();
    const Z *z = static_cast<const Z *>(p.z) + t * p.ldz;
    const float4 *stats = static_cast<const float4 *>(p.ws);
    const uint64_t *keys = reinterpret_cast<const uint64_t *>(stats + p.T * P) + t * P * p.k;
    const int count = P * p.k;
    int64_t token;
    float logit = token_logit(p, z, t, threadIdx.x, token);
    uint64_t key[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = i * kThreads + (int)threadIdx.x;
        if (j < count) key[i] = keys[j];
    }
    Stats a{kLowest, 0.0f, 0.0f};
    if (lane < P) {
        const float4 v = stats[t * P + lane];
        a = Stats{v.x, v.y, v.z};
    }
    const float m = wave_max(a.m);
    const float d = fmaxf(a.m - m, kFar), f = exp_of(d);
    const Row r = row_of(Stats{m, wave_sum(a.s * f), wave_sum(f * __builtin_fmaf(a.s, d, a.u))});
    if (threadIdx.x == 0) {
        p.lse[t] = r.lse;
        p.entropy[t] = r.entropy;
    }
    write_token(p, t, threadIdx.x, token, logit, r.lse);
    for (int64_t c = threadIdx.x + kThreads; c < p.C; c += kThreads) {
        logit = token_logit(p, z, t, c, token);
        write_token(p, t, c, token, logit, r.lse);
    }
    if (!p.k) return;
    if (r.nan) {  // (a segment with a NaN has written no keys)
        write_no_top(p, t);
        return;
    }
    uint64_t bound = kth_key<kOrderBits<Z>>(key, p.k);
    if (lane == 0) sh.wave_best[wave] = bound;
    clear(sh);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) bound = sh.wave_best[w] > bound ? sh.wave_best[w] : bound;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (key[i] && key[i] >= bound) collect(sh, key[i]);
    __syncthreads();
    rank_candidates(sh, sh.count, p.k, [&](int i, uint64_t top) { write_top(p, t, i, top, r.lse); });
}

// Segments a row.  Up to 512 rows: two tiles each, which a workgroup holds in
// registers, but at most 64, as many as a join can rank the top keys of, and
// some 1,024 workgroups in all.
struct Split {
    int P;
    int span;  // logits in a segment
};
Split split_of(int64_t T, int64_t V, int k)
{
    int64_t P = 1;
    if (T > 0 && T < 512) {
        P = (1024 + T - 1) / T;
        const int64_t most = (V + 2 * kTile - 1) / (2 * kTile), ranked = k ? kMaxCandidates / k : 64;
        if (P > most) P = most;
        if (P > ranked) P = ranked;
        if (P > 64) P = 64;
    }
    int64_t span = V;
    if (P > 1) {
        span = ((V + P - 1) / P + kTile - 1) / kTile * kTile;
        P = (V + span - 1) / span;
    }
    return Split{(int)P, (int)span};
}

constexpr int64_t kRowsPerLaunch = 1 << 20;  // grid x threads stays below 2^32

template <typename Z, bool TOP, bool HELD, bool ONCE>
void launch_rows(const LogpParams &p, int64_t r, int64_t rows, const Split &s, hipStream_t stream)
{
    hipLaunchKernelGGL((logp_rows<Z, TOP, HELD, ONCE>), dim3((unsigned)(rows * s.P)), dim3(kThreads), 0, stream, p, r, s.P, s.span);
}

template <typename Z>
hipError_t launch_logp_of(const LogpParams &p, hipStream_t stream)
{
    const Split s = split_of(p.T, p.V, p.k);
    const bool held = s.span <= 2 * kTile;
    // After their producer has written them, 4096 x 65536 bf16 take 96 us past
    // the cache and 126 through it, 1000 x 32000, which fit it, 16 and 14.
    const bool once = p.T * p.V * (int64_t)sizeof(Z) > kOnceBytes;
    for (int64_t r = 0; r < p.T; r += kRowsPerLaunch) {
        const int64_t rows = p.T - r < kRowsPerLaunch ? p.T - r : kRowsPerLaunch;
        if (p.k && held)
            launch_rows<Z, true, true, false>(p, r, rows, s, stream);
        else if (p.k && once)
            launch_rows<Z, true, false, true>(p, r, rows, s, stream);
        else if (p.k)
            launch_rows<Z, true, false, false>(p, r, rows, s, stream);
        else if (held)
            launch_rows<Z, false, true, false>(p, r, rows, s, stream);
        else if (once)
            launch_rows<Z, false, false, true>(p, r, rows, s, stream);
        else
            launch_rows<Z, false, false, false>(p, r, rows, s, stream);
        if (s.P > 1) hipLaunchKernelGGL((logp_join<Z>), dim3((unsigned)rows), dim3(kThreads), 0, stream, p, r, s.P);
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
template <typename Z, bool ONCE>
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
    bool beyond = false;
    for (int j = threadIdx.x & 63; j < H; j += 64) {  // every wave adds all of them, in the same order
        const bool given = j < p.C;
        const int64_t v = given ? p.tokens[t * p.C + j] : p.top_tok[t * p.k + (j - p.C)];
        float x = given ? (p.g ? p.g[t * p.C + j] : 0.0f) : p.gtop[t * p.k + (j - p.C)];
        if (v < 0) x = 0.0f;
        if (v >= p.V) x = __uint_as_float(0x7FC00000u);
        beyond |= v >= p.V;
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
    const bool empty = lse == -INFINITY && !__any(beyond);
    const auto value = [&](float x) {
        const float d = fmaxf(x - lse, kFar);
        float e = exp_of(d);
        if (sizeof(Z) == 4) {  // what d log2(e) was rounded by, up to 2^-24 |d| of the result
            const float rest = __builtin_fmaf(d, kLog2eRest, __builtin_fmaf(d, kLog2e, -(d * kLog2e)));
            e = __builtin_fmaf(e, rest * kLn2, e);
        }
        return e * __builtin_fmaf(-ge, d, A);
    };
    if (H) __syncthreads();
    for (int64_t c = s0 + threadIdx.x * 8; c < s1; c += kTile) {
        const f32x8 x = settle8<Z>(fetch8<ONCE>(z, (int)c, (int)s1), (int)c, (int)s1);
        f32x8 r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = empty ? 0.0f : value(x[j]);
        store8_row<ONCE>(grad + s0, (int)(c - s0), (int)(s1 - s0), r);
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
    // four tiles to a workgroup, fewer where there would not be 8 workgroups for
    // each CU (2 x 38336: 4.0 us with one, 5.4 with four)
    int64_t span = 4 * kTile;
    while (span > kTile && p.T * ((p.V + span - 1) / span) < 2048) span /= 2;
    const int64_t P = (p.V + span - 1) / span;
    const size_t lds = (size_t)(p.C + p.k) * 12;
    // (as in launch_logp_of: 4096 x 65536 bf16 163 us past the cache and 187
    // through it, 1000 x 32000 both 22)
    const bool once = 2 * p.T * p.V * (int64_t)sizeof(Z) > kOnceBytes;
    const int64_t at_once = (int64_t(1) << 23) / P > 0 ? (int64_t(1) << 23) / P : 1;
    for (int64_t r = 0; r < p.T; r += at_once) {
        const int64_t rows = p.T - r < at_once ? p.T - r : at_once;
        const dim3 grid((unsigned)(rows * P));
        if (once)
            hipLaunchKernelGGL((logp_grad_rows<Z, true>), grid, dim3(kThreads), lds, stream, p, r, P, span);
        else
            hipLaunchKernelGGL((logp_grad_rows<Z, false>), grid, dim3(kThreads), lds, stream, p, r, P, span);
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
