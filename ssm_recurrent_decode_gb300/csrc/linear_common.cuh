// linear_common.cuh -- segments and decays of linear attention (internal to libgdn_decode.so).
#pragma once

#include "gdn_common.cuh"
#include "linear_launch.h"

namespace gdn {

// A segment of a sequence: rows [begin, begin + n) of the packed tokens.
struct LinearItem {
    int seq;            // -1: none
    int begin, n;
    int seq_begin, seq_end;
    int state;          // row in the state buffers; -1: a bad index (no states, outputs zeroed)
    int index;          // of the segment in the sequence
    int id;             // of the segment among all
    int slot;           // its place in local and total
};

// rows of sequence s; a sequence whose borders leave 0 .. T or decrease has none (bad)
__device__ __forceinline__ void linear_rows(const LinearLaunch &P, int s, int &b, int &e, bool &bad)
{
    if (P.a.cu_seqlens) {
        b = P.a.cu_seqlens[s];
        e = P.a.cu_seqlens[s + 1];
        bad = b < 0 || e > P.a.T || e < b;
        if (bad) b = e = 0;
    } else {
        b = s * P.Ls;
        e = b + P.Ls;
        bad = false;
    }
}

// row of sequence s in the state buffers; -1: a bad index
__device__ __forceinline__ int linear_state(const LinearLaunch &P, int s, bool report)
{
    if (!P.states) return s;
    const int state = P.a.state_indices ? P.a.state_indices[s] : s;
    if (state >= 0 && state < P.a.num_states) return state;
    if (report) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
    return -1;
}

__device__ __forceinline__ int linear_segments(const LinearLaunch &P, int rows)
{
    return rows <= P.seg ? 1 : (rows + P.seg - 1) / P.seg;
}

// whether a block looks for its segment, not a warp
__device__ __forceinline__ bool linear_many(const LinearLaunch &P) { return P.a.cu_seqlens && P.a.S > kLinearSorted; }

// The first segment of sequence s; all 32 lanes of a warp call it.
__device__ __forceinline__ int linear_first_item(const LinearLaunch &P, int s)
{
    if (!P.a.cu_seqlens) return s * linear_segments(P, P.Ls);
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int s0 = lane; s0 < s; s0 += 32) {
        int b, e;
        bool bad;
        linear_rows(P, s0, b, e, bad);
        before += linear_segments(P, e - b);
    }
    return __reduce_add_sync(0xFFFFFFFFu, before);
}

// The segment that item i stands for; all 32 lanes of a warp call it and get the same answer. With cu_seqlens the
// sequences' segments are counted 32 sequences at a time.
__device__ __forceinline__ LinearItem linear_item(const LinearLaunch &P, int i, bool report)
{
    LinearItem it;
    it.seq = -1;
    it.begin = it.n = it.seq_begin = it.seq_end = it.state = it.index = 0;
    it.id = it.slot = i;
    const int lane = threadIdx.x & 31;
    if (!P.a.cu_seqlens) {
        const int per = linear_segments(P, P.Ls);
        const int s = i / per;
        if (s >= P.a.S) return it;
        it.seq = s;
        it.index = i - s * per;
        it.seq_begin = s * P.Ls;
        it.seq_end = it.seq_begin + P.Ls;
    } else {
        int before = 0;
        for (int s0 = 0; s0 < P.a.S; s0 += 32) {
            const int s = s0 + lane;
            int b = 0, e = 0, m = 0;
            bool bad = false;
            if (s < P.a.S) {
                linear_rows(P, s, b, e, bad);
                m = linear_segments(P, e - b);
            }
            int sum = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += v;
            }
            const bool mine = s < P.a.S && i >= before + sum - m && i < before + sum;
            const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
            if (who) {
                const int src = __ffs(who) - 1;
                it.seq = s0 + src;
                const int first = before + __shfl_sync(0xFFFFFFFFu, sum - m, src);
                it.index = i - first;
                it.seq_begin = __shfl_sync(0xFFFFFFFFu, b, src);
                it.seq_end = __shfl_sync(0xFFFFFFFFu, e, src);
                // (only borders that decrease can make more segments than there is room for)
                const int wrong = __shfl_sync(0xFFFFFFFFu, (int)bad, src);
                if (wrong || first + linear_segments(P, it.seq_end - it.seq_begin) > P.items) {
                    if (report && lane == 0) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
                    it.seq = -1;
                    return it;
                }
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (it.seq < 0) return it;
    }
    it.begin = it.seq_begin + it.index * P.seg;
    it.n = min(P.seg, it.seq_end - it.begin);
    it.state = linear_state(P, it.seq, report && lane == 0);
    return it;
}

// The segment that is i-th when the longest sequences come first: CTAs start in about that order, and the last ones to start
// are then short (24 sequences of 0 to 2000 tokens, 32 heads: 147 us, 183 in the order given; the gradients of ten, 16 heads: 234 and 265). Up to kLinearSorted sequences, two a
// lane; more of them fill the SMs in any order. All 32 lanes of a warp call it.
__device__ __forceinline__ int linear_turn(const LinearLaunch &P, int i)
{
    const int S = P.a.S, lane = threadIdx.x & 31;
    if (!P.a.cu_seqlens || S > kLinearSorted) return i;
    static_assert(kLinearSorted <= 64, "two sequences a lane");
    int n[2], m[2], first[2] = {0, 0}, at[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int b = 0, e = 0;
        bool bad;
        if (lane + 32 * h < S) linear_rows(P, lane + 32 * h, b, e, bad);
        n[h] = e - b;
        m[h] = linear_segments(P, n[h]);
    }
    for (int j = 0; j < S; ++j) {
        const int nj = __shfl_sync(0xFFFFFFFFu, j < 32 ? n[0] : n[1], j & 31), mj = __shfl_sync(0xFFFFFFFFu, j < 32 ? m[0] : m[1], j & 31);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool before = j < lane + 32 * h;
            if (before) first[h] += mj;
            if (nj > n[h] || (nj == n[h] && before)) at[h] += mj;
        }
    }
    int item = i;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const unsigned who = __ballot_sync(0xFFFFFFFFu, lane + 32 * h < S && i >= at[h] && i < at[h] + m[h]);
        if (who) item = __shfl_sync(0xFFFFFFFFu, first[h] + i - at[h], __ffs(who) - 1);
    }
    return item;
}

// What a block of threads adds up over many sequences: every warp's segments, and those of sequences that have several.
struct LinearScan {
    long long all[32], cut[32];
};

// Calls f(s, b, e, bad, first, cut) for all sequences: each thread for a range of its own, in order. first: segments of the
// sequences before; cut: of those among them that have several. bad: no rows, or segments that there is no room for (which
// only borders that decrease can make). All NT threads of a block call it; `w` is free again behind the caller's next barrier.
template <int NT, typename F> __device__ __forceinline__ void linear_each(const LinearLaunch &P, LinearScan &w, F &&f)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t per = ((int64_t)P.a.S + NT - 1) / NT;
    const int s0 = (int)min((int64_t)P.a.S, per * threadIdx.x), s1 = (int)min((int64_t)P.a.S, per * (threadIdx.x + 1));
    long long own[2] = {0, 0};
    for (int s = s0; s < s1; ++s) {
        int b, e;
        bool bad;
        linear_rows(P, s, b, e, bad);
        const int m = linear_segments(P, e - b);
        own[0] += m;
        if (m > 1) own[1] += m;
    }
    long long sum[2] = {own[0], own[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, sum[k], o);
            if (lane >= o) sum[k] += v;
        }
    if (lane == 31) w.all[warp] = sum[0], w.cut[warp] = sum[1];
    __syncthreads();
    long long first = sum[0] - own[0], cut = sum[1] - own[1];
    for (int i = 0; i < warp; ++i) first += w.all[i], cut += w.cut[i];
    for (int s = s0; s < s1; ++s) {
        int b, e;
        bool bad;
        linear_rows(P, s, b, e, bad);
        const int m = linear_segments(P, e - b);
        f(s, b, e, bad || first + m > P.items || (m > 1 && cut + m > P.cut_items), first, cut);
        first += m;
        if (m > 1) cut += m;
    }
}

// The search of linear_find among many sequences (apart, so that the others' kernels do not carry its code between theirs).
template <int NT>
__device__ __noinline__ void linear_find_block(const LinearLaunch &P, int i, bool cut, bool report, LinearScan &w, LinearItem *to)
{
    if (threadIdx.x == 0) to->seq = -1, to->begin = to->n = 0;      // (linear_each has a barrier before it calls)
    linear_each<NT>(P, w, [&](int s, int b, int e, bool bad, long long first, long long before) {
        const int m = linear_segments(P, e - b);
        const long long j = i - (cut ? before : first);
        if (j < 0 || j >= m || (cut && m == 1)) return;
        if (bad) {
            if (report) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
            return;
        }
        LinearItem it;
        it.seq = s;
        it.index = (int)j;
        it.seq_begin = b;
        it.seq_end = e;
        it.begin = b + it.index * P.seg;
        it.n = min(P.seg, e - it.begin);
        it.state = linear_state(P, s, report);
        it.id = (int)(first + j);
        it.slot = (int)(before + j);
        *to = it;
    });
}

// linear_item for a block of NT threads, into *to in shared memory; up to kLinearSorted sequences by warp `by` alone. `i` counts
// the segments of sequences with several where only those are asked for (`cut`; not up to kLinearSorted sequences). Ends with a
// barrier. (A warp that counts 2048 sequences takes 64 steps, one behind the other.)
template <int NT>
__device__ __forceinline__ void linear_find(const LinearLaunch &P, int i, bool cut, bool report, int by, LinearScan &w, LinearItem *to)
{
    const int lane = threadIdx.x & 31;
    if (!linear_many(P)) {
        if ((int)(threadIdx.x >> 5) == by) {
            const LinearItem it = linear_item(P, i, report);
            if (lane == 0) *to = it;
        }
    } else {
        linear_find_block<NT>(P, i, cut, report, w, to);
    }
    __syncthreads();
}

// ---- decays ------------------------------------------------------------------------------------
// Log decays are summed in 64 bits as powers of two and turned into factors whole: a product of a thousand rounded
// factors near one would be off by a thousand times their common rounding error.
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr double kLog2e = 1.4426950408889634;

__device__ __forceinline__ double linear_log2(float g)
{
    return (g < -200.f ? -200.0 : (double)g) * kLog2e;     // (a NaN stays one)
}

// 2^a to fp32 accuracy for any a
__device__ __forceinline__ float exp2_wide(double a)
{
    if (a < -160.0) return 0.f;
    const double n = rint(a < 200.0 ? a : 200.0);
    return ldexpf(exp2f((float)(a - n)), (int)n);
}

// The same sums as 64-bit integers in steps of 2^-40, for the kernels whose path they are on (fp64 runs at two operations
// a clock and SM). A NaN is kept apart.
__device__ __forceinline__ long long linear_fixed(float g, bool &nan)
{
    nan = !(g < INFINITY);
    const float x = nan ? 0.f : fminf(fmaxf(g, -200.f), 200.f);
    // x log2(e) as the sum of two fp32 numbers
    const float q = x * 1.44269502f, e = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -q));
    return __float2ll_rn(q * 0x1p40f) + __float2ll_rn(e * 0x1p40f);
}
// such a sum as hi + lo, hi in steps of 1/256; and 2 to its power
__device__ __forceinline__ void linear_parts(long long G, float &hi, float &lo)
{
    const long long h = (G + (1ll << 31)) >> 32;
    hi = (float)(int)h * 0x1p-8f;
    lo = (float)(int)(G - (h << 32)) * 0x1p-40f;
}
__device__ __forceinline__ float linear_exp2(long long G)
{
    float hi, lo;
    linear_parts(G, hi, lo);
    return exp2f(hi) * exp2f(lo);
}

// such a sum in fp64 as the same two numbers (a NaN stays one)
__device__ __forceinline__ float2 linear_parts(double G)
{
    const double hi = rint(G * 256.0) / 256.0;
    return make_float2((float)hi, (float)(G - hi));
}
// 2^(hi + lo) as the factor of a state, chunk by chunk or segment by segment. Near one, where many of them are multiplied, by its series:
// the hardware's 2^x is low by 2e-8 there on average, 3e-7 after the sixteen chunks of 2048 tokens (and 5e-7 after 31
// segments of 48).
__device__ __forceinline__ float linear_decay_factor(float hi, float lo)
{
    const float x = hi + lo, y = x * 0.693147182f;
    float p = fmaf(y, 1.f / 720, 1.f / 120);
    p = fmaf(p, y, 1.f / 24);
    p = fmaf(p, y, 1.f / 6);
    p = fmaf(p, y, 0.5f);
    p = fmaf(p, y, 1.f);
    return fabsf(x) < 0.25f ? fmaf(p, y, 1.f) : exp2f(hi) * exp2f(lo);      // (0.17^7 / 5040 < 2^-29)
}

// decay that a sweep applies before it takes token t (in its own direction)
__device__ __forceinline__ double linear_decay(const LinearLaunch &P, int hv, int t, int seq_end, int reverse)
{
    const int at = reverse ? t + 1 : t;
    return at < seq_end ? linear_log2(P.a.g[at * P.a.g_stride + hv]) : 0.0;
}

// debug build: a segment's rows, state and workspace lie inside their buffers
__device__ __forceinline__ bool linear_in(const LinearLaunch &P, const LinearItem &it)
{
    return GDN_IN(P.a.err_flags, it.begin, (int64_t)P.a.T + 1) && GDN_IN(P.a.err_flags, it.n, (int64_t)P.a.T - it.begin + 1) &&
           GDN_IN(P.a.err_flags, it.id, P.items) && (it.seq_end - it.seq_begin <= P.seg || GDN_IN(P.a.err_flags, it.slot, P.cut_items)) &&
           (!P.states || it.state < 0 || GDN_IN(P.a.err_flags, it.state, P.a.num_states));
}
// token row t of value head hv
__device__ __forceinline__ bool linear_in(const LinearLaunch &P, int t, int head, int heads)
{
    return GDN_IN(P.a.err_flags, t, P.a.T) && GDN_IN(P.a.err_flags, head, heads);
}

}  // namespace gdn
