// beam_select.cu -- one beam-search selection (gdn_beam_select).
//
// Launch 1 reads the logits once: a CTA takes a segment of one beam's row, keeps the running maximum
// and sum of exponentials, and the segment's K best logits. Candidates are found by a threshold:
// after the first chunk of the segment, the smallest over the eight warps of the warp's
// ceil(K / 8)-th largest per-lane maximum is a value that at least K elements reach, and only a few
// more do; after that the K-th best so far, which hardly any element passes. Only those elements are
// ranked. Launch 2, one CTA per batch entry, joins the segments of each row (a warp per beam), then
// the beams.
// Bound by reading the logits: 5 instructions per element stay below the memory time.
#include <cmath>
#include <cstdint>

#include "gdn_beam.h"
#include "gdn_chain.cuh"
#include "gdn_common.cuh"
#include "scan_common.cuh"

namespace gdn {

namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelVecs = 4;                 // 16-byte loads per thread and chunk, all in flight
#ifndef KSEL
#define KSEL 4
#endif
constexpr int kSelCtas = KSEL;                 // resident CTAs per SM
constexpr int kSelCap = 1024;               // candidates kept before they are ranked
constexpr int kSelMaxSegs = 32;             // segments per row: a lane each in the join
constexpr unsigned kFullMask = 0xFFFFFFFFu;

struct SelectLaunch {
    gdn_beam_select_args a;
    int segs;             // segments per row
    int chunks;           // chunks per segment
    unsigned long long *keys;   // [batch * beams, segs, K] best first, 0: none
    float2 *stats;              // [batch * beams, segs] maximum, sum of exp(logit - maximum)
};

// Logits in ascending order as unsigned integers; with the inverted token below, keys in
// ascending order are candidates from worst to best. -0 counts as +0.
__device__ __forceinline__ unsigned ordered(float x)
{
    const unsigned b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(unsigned u)
{
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ unsigned long long make_key(float x, int token)
{
    return (unsigned long long)ordered(x) << 32 | (0xFFFFFFFFu - (unsigned)token);
}

template <typename T> struct Vec16 {
    static constexpr int E = 16 / (int)sizeof(T);
};

// a 16-byte vector as pairs of fp32
__device__ __forceinline__ void unpack16(uint4 v, float2 (&x)[2])
{
    x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void unpack16(uint4 v, float2 (&x)[4])
{
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// The elements i .. i + E - 1 (i a multiple of E) of a row of V elements; those outside are -inf. In a
// row that starts `shift` elements behind a 16-byte boundary they lie in two aligned vectors and are
// shifted out of them: which thread adds up which elements depends on their index alone, so that equal
// rows give bit-equal sums wherever they lie.
template <typename T, bool SHIFTED> __device__ __forceinline__ uint4 load_vec(const T *row, int64_t i, int V, int shift)
{
    constexpr int E = Vec16<T>::E;
    if (!SHIFTED && i + E <= V) return __ldcs(reinterpret_cast<const uint4 *>(row + i));
    if (SHIFTED && i >= shift && i - shift + 2 * E <= V) {
        const uint4 lo = *reinterpret_cast<const uint4 *>(row + i - shift), hi = *reinterpret_cast<const uint4 *>(row + i - shift + E);
        unsigned w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const int words = shift * (int)sizeof(T) / 4;
        if (words & 2) {
#pragma unroll
            for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
        }
        if (words & 1) {
#pragma unroll
            for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
        }
        if (sizeof(T) == 2 && (shift & 1)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    unsigned w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (sizeof(T) == 4) {
            w[k] = i + k < V ? *reinterpret_cast<const unsigned *>(row + i + k) : 0xFF800000u;
        } else {
            const unsigned short *p = reinterpret_cast<const unsigned short *>(row);
            const unsigned lo = i + 2 * k < V ? p[i + 2 * k] : 0xFF80u, hi = i + 2 * k + 1 < V ? p[i + 2 * k + 1] : 0xFF80u;
            w[k] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// the largest of a vector's elements (NaN only if all are)
__device__ __forceinline__ float vec_max(const uint4 (&v)[kSelVecs], float)
{
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kSelVecs; ++k)
        m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v[k].x)), fmaxf(__uint_as_float(v[k].y), __uint_as_float(v[k].z))), __uint_as_float(v[k].w));
    return m;
}
__device__ __forceinline__ float vec_max(const uint4 (&v)[kSelVecs], bf16)
{
    __nv_bfloat162 m = __float2bfloat162_rn(-INFINITY);
#pragma unroll
    for (int k = 0; k < kSelVecs; ++k) {
        const unsigned w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
    }
    return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ float exp_fast(float d)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * 1.4426950408889634f));
    return r;
}

// Sum of exp(x - m) over a thread's elements, on pairs (the difference first, in its own rounding: it is
// exact near the maximum). An element that is NaN counts nothing; an infinite maximum counts its elements.
template <typename T> __device__ __forceinline__ float exp_sum(const uint4 (&v)[kSelVecs], float m)
{
    constexpr int E = Vec16<T>::E;
    if (m == -INFINITY) return 0.f;
    f2 total = 0ull;
    const f2 minus = pack2(-m, -m), log2e = pack2(1.4426950408889634f, 1.4426950408889634f);
#pragma unroll
    for (int k = 0; k < kSelVecs; ++k) {
        float2 x[E / 2];
        unpack16(v[k], x);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            const float2 d = unpack2(mul2(add2(pack2(x[j].x, x[j].y), minus), log2e));
            total = add2(total, pack2(ex2_approx(d.x), ex2_approx(d.y)));
        }
    }
    const float2 both = unpack2(total);
    const bool finite = m < INFINITY;
    float s = both.x + both.y;
    if (finite && s == s) return s;
    s = 0.f;
#pragma unroll 1
    for (int k = 0; k < kSelVecs * E; ++k) {
        float y = 0.f;
#pragma unroll
        for (int q = 0; q < kSelVecs; ++q) {       // no dynamic index into registers
            float2 x[E / 2];
            unpack16(v[q], x);
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (q * E + j == k) y = j & 1 ? x[j / 2].y : x[j / 2].x;
        }
        s += y == m ? 1.f : y == y && finite ? exp_fast(y - m) : 0.f;
    }
    return s;
}

// (m, s) of two parts joined
__device__ __forceinline__ void join_stats(float &m, float &s, float m2, float s2)
{
    const float top = fmaxf(m, m2);
    if (top == -INFINITY) return;
    s = (m == top ? s : s * exp_fast(m - top)) + (m2 == top ? s2 : s2 * exp_fast(m2 - top));
    m = top;
}

// Ranks list[0 .. n) (all different) and leaves its best min(n, K) in order at its front. Contains
// barriers; every thread calls it. `sorted` holds K keys.
__device__ __forceinline__ void rank_list(unsigned long long *list, int n, int K, unsigned long long *sorted, int tid)
{
    for (int i = tid; i < n; i += kSelThreads) {
        const unsigned long long k = list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += list[j] > k;
        if (rank < K) sorted[rank] = k;
    }
    __syncthreads();
    for (int i = tid; i < min(n, K); i += kSelThreads) list[i] = sorted[i];
    __syncthreads();
}

// Every warp's k-th largest of its lanes' values (-inf where it has fewer): the largest or the smallest
// of them over the warps. Contains barriers.
__device__ __forceinline__ float kth_top(float top, int k, int lane, int warp, float *wthr, bool largest)
{
    unsigned mine = top > -INFINITY ? ordered(top) : 0, best = 0;
    for (int i = 0; i < k; ++i) {
        best = __reduce_max_sync(kFullMask, mine);
        const unsigned at = __ballot_sync(kFullMask, mine == best);
        if (lane == __ffs(at) - 1) mine = 0;
    }
    __syncthreads();
    if (lane == 0) wthr[warp] = best ? unordered(best) : -INFINITY;
    __syncthreads();
    float t = wthr[0];
#pragma unroll
    for (int w = 1; w < kSelWarps; ++w) t = largest ? fmaxf(t, wthr[w]) : fminf(t, wthr[w]);
    return t;
}

template <typename T, bool SHIFTED>
__global__ void __launch_bounds__(kSelThreads, kSelCtas) beam_segment_kernel(const __grid_constant__ SelectLaunch P)
{
    constexpr int E = Vec16<T>::E;
    constexpr int64_t CHUNK = (int64_t)kSelThreads * kSelVecs * E;
    __shared__ unsigned long long list[kSelCap], sorted[GDN_BEAM_MAX_SELECT];
    __shared__ float wthr[kSelWarps], wm[kSelWarps], ws[kSelWarps];
    __shared__ unsigned long long wkey[kSelWarps];
    __shared__ int count;
    ordinary_launch_start();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int beam = (int)(blockIdx.x / (unsigned)P.segs), seg = (int)(blockIdx.x % (unsigned)P.segs);
    const int V = P.a.vocab, K = P.a.K;
    unsigned long long *out = P.keys + ((int64_t)beam * P.segs + seg) * K;
    const int64_t r = P.a.rows ? (int64_t)P.a.rows[beam] : beam;
    if (r < 0 || r >= P.a.num_rows) {
        if (tid == 0 && seg == 0) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
        return;                                   // the join does not look at this beam
    }
    if (!(P.a.scores[beam] > -INFINITY) || (P.a.finished && P.a.finished[beam])) return;

    const T *row = static_cast<const T *>(P.a.logits) + r * P.a.row_stride;
    const int shift = SHIFTED ? (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T)) : 0;
    const int64_t first = (int64_t)seg * P.chunks * CHUNK;
    const int64_t last = min((int64_t)V, first + P.chunks * CHUNK);     // the segment: elements first .. last - 1

    float m = -INFINITY, s = 0.f;
    float thr = -INFINITY;       // candidates are above it (full) or reach it (not yet K found)
    bool full = false, overflow = false;
    if (tid == 0) count = 0;
    __syncthreads();
    uint4 ahead[kSelVecs];
#pragma unroll
    for (int v = 0; v < kSelVecs; ++v) ahead[v] = load_vec<T, SHIFTED>(row, first + ((int64_t)v * kSelThreads + tid) * E, V, shift);
    for (int64_t base = first; base < last; base += CHUNK) {
        uint4 x[kSelVecs];
#pragma unroll
        for (int v = 0; v < kSelVecs; ++v) x[v] = ahead[v];
        if (base + CHUNK < last) {
#pragma unroll
            for (int v = 0; v < kSelVecs; ++v)
                ahead[v] = load_vec<T, SHIFTED>(row, base + CHUNK + ((int64_t)v * kSelThreads + tid) * E, V, shift);
        }
        const float top = vec_max(x, T());
        join_stats(m, s, top, exp_sum<T>(x, top));

        if (base == first) {
            // a value that at least K elements reach, if there are as many: from every warp its share,
            // or, where warps have too few values, K from one of them
            thr = kth_top(top, (K + kSelWarps - 1) / kSelWarps, lane, warp, wthr, false);
            if (thr == -INFINITY && K <= 32) thr = kth_top(top, K, lane, warp, wthr, true);
        }
        if (full ? top > thr : top >= thr) {
#pragma unroll
            for (int v = 0; v < kSelVecs; ++v) {
                const int64_t i = base + ((int64_t)v * kSelThreads + tid) * E;
                float2 e[E / 2];
                unpack16(x[v], e);
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const float y = k & 1 ? e[k / 2].y : e[k / 2].x;
                    if ((full ? y > thr : y >= thr) && y > -INFINITY) {
                        const int at = atomicAdd(&count, 1);
                        if (at < kSelCap) list[at] = make_key(y, (int)(i + k));
                    }
                }
            }
        }
        __syncthreads();
        const int n = count;
        __syncthreads();             // nobody adds to the next chunk's count before all have read this one
        if (n > kSelCap) {
            overflow = true;
            break;
        }
        if (n >= K && n > (full ? K : 0) && base + CHUNK < last) {
            rank_list(list, n, K, sorted, tid);
            if (tid == 0) count = K;
            thr = unordered((unsigned)(list[K - 1] >> 32));
            full = true;
            __syncthreads();
        }
    }
    if (overflow) {
        // Many equal values, or an adversarial order: exactly, one candidate at a time.
        m = -INFINITY;
        s = 0.f;
        unsigned long long before = ~0ull;
        for (int k = 0; k < K; ++k) {
            unsigned long long best = 0;
            for (int64_t i = first + tid; i < last; i += kSelThreads) {
                const float y = to_f32(row[i]);
                if (!(y > -INFINITY)) continue;
                const unsigned long long key = make_key(y, (int)i);
                if (key < before && key > best) best = key;
                if (k == 0) join_stats(m, s, y, 1.f);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const unsigned long long o = __shfl_xor_sync(kFullMask, best, off);
                best = o > best ? o : best;
            }
            __syncthreads();
            if (lane == 0) wkey[warp] = best;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kSelWarps; ++w) best = wkey[w] > best ? wkey[w] : best;
            if (tid == 0) out[k] = best;
            before = best;                        // 0 once there are none left
        }
    } else {
        const int n = count;
        __syncthreads();
        for (int i = tid; i < n; i += kSelThreads) {
            const unsigned long long k = list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += list[j] > k;
            if (rank < K) out[rank] = k;
        }
        for (int i = n + tid; i < K; i += kSelThreads) out[i] = 0;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        join_stats(m, s, __shfl_xor_sync(kFullMask, m, off), __shfl_xor_sync(kFullMask, s, off));
    if (lane == 0) {
        wm[warp] = m;
        ws[warp] = s;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kSelWarps; ++w) join_stats(m, s, wm[w], ws[w]);
        P.stats[(int64_t)beam * P.segs + seg] = make_float2(m, s);
    }
}

// scores as unsigned 64-bit integers in the same order; -inf is the lowest that occurs
__device__ __forceinline__ unsigned long long ordered64(double x)
{
    const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// largest key over the warp
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k)
{
    const unsigned hi = __reduce_max_sync(kFullMask, (unsigned)(k >> 32));
    const unsigned lo = __reduce_max_sync(kFullMask, (unsigned)(k >> 32) == hi ? (unsigned)k : 0u);
    return (unsigned long long)hi << 32 | lo;
}

// log(x) for a normal x > 0 in fp64, to about 1e-15: x = 2^e f with f in [sqrt(1/2), sqrt(2)), and
// log f = 2 atanh(q) = 2 (q + q^3/3 + ...) at q = (f - 1) / (f + 1), |q| <= 0.1716 (11 terms)
__device__ __forceinline__ double log64(double x)
{
    long long b = __double_as_longlong(x);
    int e = (int)(b >> 52) - 1023;
    double f = __longlong_as_double((b & 0x000FFFFFFFFFFFFFll) | 0x3FF0000000000000ll);
    if (f > 1.4142135623730951) {
        f *= 0.5;
        ++e;
    }
    const double q = (f - 1.0) / (f + 1.0), q2 = q * q;
    // even and odd terms side by side, to halve the chain
    const double q4 = q2 * q2;
    double even = 1.0 / 21, odd = 1.0 / 19;
    even = fma(even, q4, 1.0 / 17);
    odd = fma(odd, q4, 1.0 / 15);
    even = fma(even, q4, 1.0 / 13);
    odd = fma(odd, q4, 1.0 / 11);
    even = fma(even, q4, 1.0 / 9);
    odd = fma(odd, q4, 1.0 / 7);
    even = fma(even, q4, 1.0 / 5);
    odd = fma(odd, q4, 1.0 / 3);
    even = fma(even, q4, 1.0);
    return fma((double)e, 0.69314718055994530942, 2.0 * q * fma(odd, q2, even));
}

// One CTA per batch entry, a warp per beam.
__global__ void __launch_bounds__(32 * GDN_BEAM_MAX_BEAMS) beam_join_kernel(const __grid_constant__ SelectLaunch P)
{
    // fp64 runs at two lanes a clock, so each fp64 step is taken once for all beams (or candidates) side
    // by side, not in every beam's warp
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ double row_sum[GDN_BEAM_MAX_BEAMS];
    __shared__ float row_top[GDN_BEAM_MAX_BEAMS];
    const int lane = threadIdx.x & 31, j = threadIdx.x >> 5;
    const int K = P.a.K, beams = P.a.beams;
    double *score = reinterpret_cast<double *>(smem);                       // [beams, K]
    float *logit = reinterpret_cast<float *>(score + beams * K);            // [beams, K]
    int *token = reinterpret_cast<int *>(logit + beams * K);                // [beams, K]
    const int64_t beam = (int64_t)blockIdx.x * beams + j;

    // The call's inputs may be read before the wait: this kernel's CTAs start when every CTA of the
    // segment kernel has let them, which each does after its own wait for the kernels before it.
    const float cum = P.a.scores[beam];
    const int64_t r = P.a.rows ? (int64_t)P.a.rows[beam] : beam;
    const bool live = cum > -INFINITY && r >= 0 && r < P.a.num_rows;
    const bool done = P.a.finished && P.a.finished[beam] && cum > -INFINITY;
    for (int k = lane; k < K; k += 32) {
        logit[j * K + k] = done && k == 0 ? 0.f : -INFINITY;
        token[j * K + k] = done && k == 0 ? P.a.eos_token : -1;
    }
    if (lane == 0) {
        row_sum[j] = 1.0;            // an ended beam: score + 0 - log 1
        row_top[j] = 0.f;
    }
    __syncwarp();
    ordinary_launch_start();
    if (live && !done) {
        // the segments' lists, best first: a lane's two next keys are at hand
        const bool on = lane < P.segs;
        const unsigned long long *mine = P.keys + (beam * P.segs + lane) * K;
        const float2 st = on ? P.stats[beam * P.segs + lane] : make_float2(-INFINITY, 0.f);
        unsigned long long head = on ? mine[0] : 0, next = on && K > 1 ? mine[1] : 0;
        // the row's maximum and sum
        float top = st.x;
        int lanes = 1;
        while (lanes < P.segs) lanes *= 2;
        for (int off = lanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
        top = __shfl_sync(kFullMask, top, 0);
        if (top > -INFINITY) {
            double sum = st.x == -INFINITY ? 0.0 : st.x == top ? (double)st.y : (double)(st.y * exp_fast(st.x - top));
            for (int off = lanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(kFullMask, sum, off);
            if (lane == 0) {
                row_sum[j] = sum;
                row_top[j] = top;
            }
            int at = 2;
            for (int k = 0; k < K; ++k) {
                const unsigned long long best = warp_max(head);
                if (best == 0) break;
                if (head == best) {
                    head = next;
                    next = on && at < K ? mine[at] : 0;
                    ++at;
                }
                if (lane == 0) {
                    logit[j * K + k] = unordered((unsigned)(best >> 32));
                    token[j * K + k] = (int)(0xFFFFFFFFu - (unsigned)best);
                }
            }
        }
    }
    __syncthreads();
    if (j == 0 && lane < beams) row_sum[lane] = log64(row_sum[lane]);
    __syncthreads();
    for (int i = threadIdx.x; i < beams * K; i += 32 * beams) {
        const int q = i / K;
        const float x = logit[i], top = row_top[q];
        const double base = (double)P.a.scores[(int64_t)blockIdx.x * beams + q];
        score[i] = x == -INFINITY ? -INFINITY : base + ((x == top ? 0.0 : (double)x - (double)top) - row_sum[q]);
    }
    __syncthreads();
    if (j != 0) return;
    // the beams' lists: a lane per beam; the lowest lane wins a tie
    int at = 0;
    const bool on = lane < beams;
    const unsigned long long none = ordered64(-INFINITY);
    unsigned long long head = on ? ordered64(score[lane * K]) : none;
    for (int k = 0; k < K; ++k) {
        const unsigned long long best = warp_max(head);
        const bool any = best > none;
        const int who = __ffs(__ballot_sync(kFullMask, on && head == best)) - 1;
        const int64_t o = (int64_t)blockIdx.x * K + k;
        if (any && lane == who) {
            const int t = token[lane * K + at];
            P.a.out_scores[o] = (float)score[lane * K + at];
            P.a.out_parents[o] = lane;
            P.a.out_tokens[o] = t;
            if (P.a.out_finished) P.a.out_finished[o] = t == P.a.eos_token;
            ++at;
            head = at < K ? ordered64(score[lane * K + at]) : none;
        } else if (!any && lane == 0) {
            P.a.out_scores[o] = -INFINITY;
            P.a.out_parents[o] = -1;
            P.a.out_tokens[o] = -1;
            if (P.a.out_finished) P.a.out_finished[o] = 0;
        }
    }
}

// Segments per row and chunks per segment: the split whose CTAs take the fewest rounds of chunks, with a
// CTA's own work (threshold, ranking) counted as one and a half chunks.
void segment_plan(int64_t rows, int vocab, int elem_bytes, int &segs, int &chunks)
{
    constexpr int64_t kSlots = 152 * kSelCtas;
    const int64_t chunk = (int64_t)kSelThreads * kSelVecs * (16 / elem_bytes);
    const int64_t all = (vocab + chunk - 1) / chunk;
    double best = 0;
    segs = 0;
    for (int64_t n = 1; n <= kSelMaxSegs && n <= all; ++n) {
        const int64_t c = (all + n - 1) / n, used = (all + c - 1) / c;
        const double cost = (double)((rows * used + kSlots - 1) / kSlots) * (c + 1.5);
        if (segs == 0 || cost < best) {
            best = cost;
            segs = (int)used;
            chunks = (int)c;
        }
    }
}

bool select_sizes_ok(int32_t batch, int32_t beams, int32_t vocab, int32_t K)
{
    return batch >= 0 && beams >= 1 && beams <= GDN_BEAM_MAX_BEAMS && vocab >= 1 && K >= 1 && K <= GDN_BEAM_MAX_SELECT &&
           (int64_t)batch * beams <= INT32_MAX / kSelMaxSegs;
}

size_t round16(size_t v) { return (v + 15) / 16 * 16; }
bool aligned_to(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }

}  // namespace

}  // namespace gdn

extern "C" {

size_t gdn_beam_select_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t K)
{
    if (!gdn::select_sizes_ok(batch, beams, vocab, K)) return 0;
    // the larger of both types' segment counts
    int segs = 1;
    for (int es : {2, 4}) {
        int s, c;
        gdn::segment_plan((int64_t)batch * beams > 0 ? (int64_t)batch * beams : 1, vocab, es, s, c);
        segs = s > segs ? s : segs;
    }
    const size_t rows = (size_t)batch * beams;
    return gdn::round16(rows * segs * K * 8) + gdn::round16(rows * segs * 8);
}

int gdn_beam_select(const gdn_beam_select_args *a, gdn_stream_t stream)
{
    using namespace gdn;
    if (!a) return GDN_ERR_NULL;
    if (!select_sizes_ok(a->batch, a->beams, a->vocab, a->K)) return GDN_ERR_SHAPE;
    if (a->logits_dtype != GDN_F32 && a->logits_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if ((a->finished || a->out_finished) && (a->eos_token < 0 || a->eos_token >= a->vocab)) return GDN_ERR_ARG;
    if (a->batch == 0) return GDN_OK;
    if (!a->logits || !a->scores || !a->out_scores || !a->out_parents || !a->out_tokens || !a->workspace) return GDN_ERR_NULL;
    if (a->row_stride < a->vocab || a->num_rows < 1 || (!a->rows && a->num_rows < (int64_t)a->batch * a->beams))
        return GDN_ERR_SHAPE;
    if (a->workspace_bytes < gdn_beam_select_workspace_bytes(a->batch, a->beams, a->vocab, a->K)) return GDN_ERR_SHAPE;
    const int es = a->logits_dtype == GDN_BF16 ? 2 : 4;
    if (!aligned_to(a->logits, es) || !aligned_to(a->rows, 4) || !aligned_to(a->scores, 4) || !aligned_to(a->out_scores, 4) ||
        !aligned_to(a->out_parents, 4) || !aligned_to(a->out_tokens, 4) || !aligned_to(a->workspace, 16))
        return GDN_ERR_ALIGN;
    SelectLaunch P;
    P.a = *a;
    const int64_t rows = (int64_t)a->batch * a->beams;
    segment_plan(rows, a->vocab, es, P.segs, P.chunks);
    P.keys = static_cast<unsigned long long *>(a->workspace);
    P.stats = reinterpret_cast<float2 *>(static_cast<unsigned char *>(a->workspace) + round16((size_t)rows * P.segs * a->K * 8));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)(rows * P.segs));
    const bool shifted = !aligned_to(a->logits, 16) || (a->row_stride * es) % 16 != 0;
    const auto kern = es == 2 ? (shifted ? beam_segment_kernel<bf16, true> : beam_segment_kernel<bf16, false>)
                              : (shifted ? beam_segment_kernel<float, true> : beam_segment_kernel<float, false>);
    if (launch_ordinary(kern, grid, dim3(kSelThreads), 0, s, P) != cudaSuccess) return GDN_ERR_LAUNCH;
    const size_t smem = (size_t)a->beams * a->K * 16;
    return launch_ordinary(beam_join_kernel, dim3((unsigned)a->batch), dim3(32u * a->beams), smem, s, P) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_LAUNCH;
}

}  // extern "C"
