// beam_select.cu -- one beam-search selection (gdn_beam_select).
//
// Launch 1 reads the logits once: a CTA takes a segment of one beam's row, keeps the running maximum
// and sum of exponentials, and the segment's K best logits. Only elements that reach a threshold
// become candidates. In the segment's first chunk it is the smallest over the eight warps of the warp's
// ceil(K / 8)-th largest per-lane maximum: at least K elements reach it, and only a few more do. After
// that chunk it is the K-th best found there, and the warps go on without barriers, each appending what
// passes to a list of its own (a full list is cut to its K best). All lists are ranked at the end.
// Launch 2, one CTA per batch entry, joins the segments of each row (a warp per beam), then the beams.
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
constexpr int kSelCtas = 3;                 // resident CTAs per SM
constexpr int kSelCap = 128;                // candidates of a warp
constexpr int kSelMaxSegs = 32;             // segments per row: a lane each in the join
constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr float kLowest = -3.402823466e38f;  // every finite logit reaches it

struct SelectLaunch {
    gdn_beam_select_args a;
    int segs;             // segments per row
    int chunks;           // chunks per segment
    int staged;           // the join copies the segments' keys to shared memory
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
template <typename T, bool SHIFTED> __device__ __forceinline__ uint4 load_vec(const T *row, unsigned i, unsigned V, unsigned shift)
{
    constexpr unsigned E = Vec16<T>::E;
    if (!SHIFTED && i + E <= V) return __ldcs(reinterpret_cast<const uint4 *>(row + i));
    if (SHIFTED && i >= shift && i - shift + 2 * E <= V) {
        const uint4 lo = *reinterpret_cast<const uint4 *>(row + i - shift), hi = *reinterpret_cast<const uint4 *>(row + i - shift + E);
        unsigned w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const unsigned words = shift * (unsigned)sizeof(T) / 4;
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

// the largest of a vector's elements; NaN counts as -inf
__device__ __forceinline__ float vec_max(uint4 v, float)
{
    return fmaxf(fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))), -INFINITY);
}
__device__ __forceinline__ float vec_max(uint4 v, bf16)
{
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162 *>(&w[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);
}

__device__ __forceinline__ float exp_fast(float d)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * 1.4426950408889634f));
    return r;
}

// Sum of exp(x - m) over a thread's elements for a finite m, on pairs: 2^(x L - c) with L = log2(e) in fp32
// and c = m L rounded. The product is exact inside the multiply-add, so each exponent is (x - m) L plus the
// rounding error r = m L - c, the same for all: 2^-r takes it out of the sum. NaN where an element is, and where
// |r| is so large (|m| above 1.5e9) that 2^r, a sum of up to 32 of them or 2^-r could leave the normal numbers:
// up to 96 they stay within 2^-96 .. 2^101.
template <typename T> __device__ __forceinline__ float exp_sum(const uint4 (&v)[kSelVecs], float m)
{
    constexpr int E = Vec16<T>::E;
    constexpr float L = 1.4426950408889634f;
    f2 total = 0ull;
    const float c = m * L;
    const f2 minus = pack2(-c, -c), log2e = pack2(L, L);
#pragma unroll
    for (int k = 0; k < kSelVecs; ++k) {
        float2 x[E / 2];
        unpack16(v[k], x);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            const float2 d = unpack2(fma2(pack2(x[j].x, x[j].y), log2e, minus));
            total = add2(total, pack2(ex2_approx(d.x), ex2_approx(d.y)));
        }
    }
    const float2 both = unpack2(total);
    const float r = fmaf(m, L, -c);
    return fabsf(r) <= 96.f ? (both.x + both.y) * ex2_approx(-r) : NAN;
}

// The same for any m, element by element from memory: NaN counts nothing, an infinite maximum counts its
// elements. Rare, and kept out of the loop's code.
template <typename T> __device__ __noinline__ float exp_sum_careful(const T *row, unsigned base, unsigned V, float m)
{
    constexpr unsigned E = Vec16<T>::E;
    float s = 0.f;
    for (unsigned k = 0; k < kSelVecs * E; ++k) {
        const unsigned i = base + (k / E * kSelThreads + threadIdx.x) * E + k % E;
        const float y = i < V ? to_f32(row[i]) : -INFINITY;
        s += y == m ? 1.f : y == y && m < INFINITY ? exp_fast(y - m) : 0.f;
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

// How many of n keys (all different) are larger than k.
__device__ __forceinline__ int rank_of(unsigned long long k, const unsigned long long *keys, int n)
{
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += keys[j] > k;
    return rank;
}

// A warp cuts its list of n candidates to the K best, in order; returns how many are left.
__device__ __noinline__ int cut_list(unsigned long long *list, int n, int K, int lane)
{
    unsigned long long k[kSelCap / 32];
    int rank[kSelCap / 32];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSelCap / 32; ++i) {
        k[i] = i * 32 + lane < n ? list[i * 32 + lane] : 0;
        rank[i] = k[i] ? 0 : K;
    }
    for (int j = 0; j < n; ++j) {
        const unsigned long long o = list[j];
#pragma unroll
        for (int i = 0; i < kSelCap / 32; ++i) rank[i] += o > k[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSelCap / 32; ++i)
        if (rank[i] < K) list[rank[i]] = k[i];
    __syncwarp();
    return min(n, K);
}

// Every warp's k-th largest of its lanes' values (the lowest finite value where it has fewer): the largest or the smallest
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
    if (lane == 0) wthr[warp] = best ? unordered(best) : kLowest;
    __syncthreads();
    float t = wthr[0];
#pragma unroll
    for (int w = 1; w < kSelWarps; ++w) t = largest ? fmaxf(t, wthr[w]) : fminf(t, wthr[w]);
    return t;
}

template <typename T, bool SHIFTED>
__global__ void __launch_bounds__(kSelThreads, kSelCtas) beam_segment_kernel(const __grid_constant__ SelectLaunch P)
{
    constexpr unsigned E = Vec16<T>::E, CHUNK = kSelThreads * kSelVecs * E;
    __shared__ unsigned long long lists[kSelWarps][kSelCap];
    __shared__ unsigned long long all[kSelWarps * kSelCap];
    __shared__ float wthr[kSelWarps], wm[kSelWarps], ws[kSelWarps];
    __shared__ int wcount[kSelWarps];
    __shared__ float kth;
    ordinary_launch_start();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int beam = (int)(blockIdx.x / (unsigned)P.segs), seg = (int)(blockIdx.x % (unsigned)P.segs);
    const unsigned V = (unsigned)P.a.vocab;
    const int K = P.a.K;
    unsigned long long *out = P.keys + ((int64_t)beam * P.segs + seg) * K;
    const int64_t r = P.a.rows ? (int64_t)P.a.rows[beam] : beam;
    const float cum = P.a.scores[beam];
    const bool ended = P.a.finished && P.a.finished[beam];
    if (!(cum > -INFINITY) || ended) return;      // its row is not read, whatever it is
    if (r < 0 || r >= P.a.num_rows) {
        if (tid == 0 && seg == 0) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
        return;                                   // the join does not look at this beam
    }

    const T *row = static_cast<const T *>(P.a.logits) + r * P.a.row_stride;
    const unsigned shift = SHIFTED ? (unsigned)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T)) : 0;
    // the segment: elements first .. last - 1 (below 2^32: vocab fits 31 bits)
    const unsigned first = (unsigned)seg * P.chunks * CHUNK, last = min(V, first + P.chunks * CHUNK);

    float m = -INFINITY, s = 0.f;
    float thr = kLowest;         // candidates reach it (strict: are above it); -inf and NaN never do
    bool strict = false;
    unsigned long long *list = lists[warp];
    int n = 0;                   // candidates in this warp's list
    uint4 ahead[kSelVecs];
#pragma unroll
    for (int v = 0; v < kSelVecs; ++v) ahead[v] = load_vec<T, SHIFTED>(row, first + (v * kSelThreads + tid) * E, V, shift);
    for (unsigned base = first; base < last; base += CHUNK) {
        uint4 x[kSelVecs];
        float vtop[kSelVecs], top = m;
#pragma unroll
        for (int v = 0; v < kSelVecs; ++v) {
            x[v] = ahead[v];
            vtop[v] = vec_max(x[v], T());
            top = fmaxf(top, vtop[v]);
        }
        if (base + CHUNK < last) {
#pragma unroll
            for (int v = 0; v < kSelVecs; ++v)
                ahead[v] = load_vec<T, SHIFTED>(row, base + CHUNK + (v * kSelThreads + tid) * E, V, shift);
        }
        if (top > -INFINITY) {
            float more = exp_sum<T>(x, top);
            if (!(top < INFINITY && more == more)) more = exp_sum_careful(row, base, V, top);
            s = more + (m == top ? s : s * exp_fast(m - top));
            m = top;
        }
        if (base == first) {
            // a value that at least K elements reach, if there are as many: from every warp its share,
            // or, where warps have too few values, K from one of them
            thr = kth_top(top, (K + kSelWarps - 1) / kSelWarps, lane, warp, wthr, false);
            if (thr == kLowest && K <= 32) thr = kth_top(top, K, lane, warp, wthr, true);
        }
#pragma unroll
        for (int v = 0; v < kSelVecs; ++v) {
            if (!__any_sync(kFullMask, strict ? vtop[v] > thr : vtop[v] >= thr)) continue;
            unsigned bits = 0;       // which of the vector's elements pass
            float2 e[E / 2];
            unpack16(x[v], e);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float y = k & 1 ? e[k / 2].y : e[k / 2].x;
                if (strict ? y > thr : y >= thr) bits |= 1u << k;
            }
            const unsigned i = base + (v * kSelThreads + tid) * E;
            unsigned lanes;
            while ((lanes = __ballot_sync(kFullMask, bits != 0)) != 0) {
                if (n + 32 > kSelCap) {
                    n = cut_list(list, n, K, lane);
                    const float own = unordered((unsigned)(list[K - 1] >> 32));     // more than K were there
                    if (own > thr) {
                        thr = own;
                        strict = false;          // an equal one in this chunk may have a lower token
                    }
                }
                if (bits) {
                    const int at = __ffs(bits) - 1;
                    bits &= bits - 1;
                    float y = e[0].x;
#pragma unroll
                    for (int k = 1; k < E; ++k)
                        if (at == k) y = k & 1 ? e[k / 2].y : e[k / 2].x;
                    list[n + __popc(lanes & ((1u << lane) - 1))] = make_key(y, (int)(i + at));
                }
                n += __popc(lanes);
            }
        }
        if (base + CHUNK >= last) break;
        if (base == first) {
            // the K-th best so far: later elements that only equal it have higher tokens
            if (n > K) n = cut_list(list, n, K, lane);
            if (lane == 0) wcount[warp] = n;
            if (tid == 0) kth = kLowest;
            __syncthreads();
            int total = 0, before = 0;
#pragma unroll
            for (int w = 0; w < kSelWarps; ++w) {
                before += w < warp ? wcount[w] : 0;
                total += wcount[w];
            }
            for (int j = lane; j < n; j += 32) all[before + j] = list[j];
            __syncthreads();
            for (int j = tid; j < total; j += kSelThreads)
                if (rank_of(all[j], all, total) == K - 1) kth = unordered((unsigned)(all[j] >> 32));
            __syncthreads();
            if (total >= K) {
                thr = kth;
                strict = true;
            }
        } else if (n >= 2 * K + 16) {
            n = cut_list(list, n, K, lane);
            const float own = unordered((unsigned)(list[K - 1] >> 32));
            if (own >= thr) {
                thr = own;
                strict = true;
            }
        }
    }
    {
        if (n > K) n = cut_list(list, n, K, lane);
        __syncthreads();             // wcount and all may still be read
        if (lane == 0) wcount[warp] = n;
        __syncthreads();
        int total = 0, before = 0;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            before += w < warp ? wcount[w] : 0;
            total += wcount[w];
        }
        for (int j = lane; j < n; j += 32) all[before + j] = list[j];
        __syncthreads();
        for (int j = tid; j < total; j += kSelThreads) {
            const int rank = rank_of(all[j], all, total);
            if (rank < K) out[rank] = all[j];
        }
        for (int j = total + tid; j < K; j += kSelThreads) out[j] = 0;
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

// log(x) for a normal x > 0 in fp64, to about 1e-9: x = 2^e f with f in [sqrt(1/2), sqrt(2)), and
// log f = 2 atanh(q) = 2 (q + q^3/3 + ... + q^9/9) at q = (f - 1) / (f + 1), |q| <= 0.1716 (the next term
// is below 7e-10). The division is a fp32 reciprocal with one Newton step.
__device__ __forceinline__ double log64(double x)
{
    const long long b = __double_as_longlong(x);
    int e = (int)(b >> 52) - 1023;
    double f = __longlong_as_double((b & 0x000FFFFFFFFFFFFFll) | 0x3FF0000000000000ll);
    if (f > 1.4142135623730951) {
        f *= 0.5;
        ++e;
    }
    const double den = f + 1.0, r0 = (double)(1.0f / (float)den);
    const double r = fma(r0, fma(-den, r0, 1.0), r0), q = (f - 1.0) * r, q2 = q * q;
    const double p = fma(fma(fma(fma(1.0 / 9, q2, 1.0 / 7), q2, 1.0 / 5), q2, 1.0 / 3), q2, 1.0);
    return fma((double)e, 0.69314718055994530942, 2.0 * q * p);
}

// The best K of one row's segments by rounds: a lane per segment holds its list's two next keys. For rows
// with more keys than are ranked against each other (or fit shared memory).
__device__ __noinline__ void join_row(const unsigned long long *keys, int segs, int K, int lane, float *logit, int *token)
{
    const bool on = lane < segs;
    const unsigned long long *mine = keys + lane * K;
    unsigned long long head = on ? mine[0] : 0, next = on && K > 1 ? mine[1] : 0;
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
            logit[k] = unordered((unsigned)(best >> 32));
            token[k] = (int)(0xFFFFFFFFu - (unsigned)best);
        }
    }
}

// One CTA per batch entry. fp64 runs at two lanes a clock, so each fp64 step is taken once for all beams (or
// candidates) side by side. Few keys are ranked each against all, which beats rounds of warp-wide maxima
// (each some 120 cycles) up to the counts below.
constexpr int kJoinThreads = 256;
constexpr int kRankKeys = 128;             // keys of a row
constexpr int kRankCandidates = 256;       // of a batch entry

__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const __grid_constant__ SelectLaunch P)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ double row_sum[GDN_BEAM_MAX_BEAMS];
    __shared__ float row_top[GDN_BEAM_MAX_BEAMS], row_cum[GDN_BEAM_MAX_BEAMS];
    __shared__ int row_state[GDN_BEAM_MAX_BEAMS];        // 0: no beam, 1: ended, 2: has a row
    constexpr int kWarps = kJoinThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = P.a.K, beams = P.a.beams, n = beams * K, per_row = P.segs * K;
    unsigned long long *order = reinterpret_cast<unsigned long long *>(smem);               // [beams, K] the scores, as integers
    float *logit = reinterpret_cast<float *>(order + n);                                    // [beams, K]
    int *token = reinterpret_cast<int *>(logit + n);                                        // [beams, K]
    unsigned long long *keys = reinterpret_cast<unsigned long long *>(token + n);           // [beams, segs, K] where they fit
    const int64_t beam0 = (int64_t)blockIdx.x * beams;

    // The call's inputs may be read before the wait: this kernel's CTAs start when every CTA of the
    // segment kernel has let them, which each does after its own wait for the kernels before it.
    if (tid < beams) {
        const float cum = P.a.scores[beam0 + tid];
        const int64_t r = P.a.rows ? (int64_t)P.a.rows[beam0 + tid] : beam0 + tid;
        const bool ended = P.a.finished && P.a.finished[beam0 + tid];
        row_state[tid] = !(cum > -INFINITY) ? 0 : ended ? 1 : r >= 0 && r < P.a.num_rows ? 2 : 0;
        row_cum[tid] = cum;
        row_sum[tid] = 1.0;              // an ended beam: score + 0 - log 1
        row_top[tid] = 0.f;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kJoinThreads) {
        const bool itself = row_state[i / K] == 1 && i % K == 0;
        logit[i] = itself ? 0.f : -INFINITY;
        token[i] = itself ? P.a.eos_token : -1;
    }
    ordinary_launch_start();

    if (P.staged) {
        for (int i = tid; i < beams * per_row; i += kJoinThreads) keys[i] = P.keys[beam0 * per_row + i];
    }
    for (int j = warp; j < beams; j += kWarps) {
        if (row_state[j] != 2) continue;
        // the row's maximum and sum
        const float2 st = lane < P.segs ? P.stats[(beam0 + j) * P.segs + lane] : make_float2(-INFINITY, 0.f);
        float top = st.x;
        int lanes = 1;
        while (lanes < P.segs) lanes *= 2;
        for (int off = lanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
        top = __shfl_sync(kFullMask, top, 0);
        if (top == -INFINITY) continue;
        double sum = st.x == -INFINITY ? 0.0 : st.x == top ? (double)st.y : (double)(st.y * exp_fast(st.x - top));
        for (int off = lanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(kFullMask, sum, off);
        if (lane == 0) {
            row_sum[j] = sum;
            row_top[j] = top;
        }
    }
    __syncthreads();                     // the keys and sums are there, and the lists are cleared
    if (warp == kWarps - 1 && lane < beams) row_sum[lane] = log64(row_sum[lane]);
    if (P.staged && per_row <= kRankKeys) {
        for (int i = tid; i < beams * per_row; i += kJoinThreads) {
            const int j = i / per_row;
            if (row_state[j] != 2) continue;
            const unsigned long long key = keys[i];
            const int rank = rank_of(key, keys + j * per_row, per_row);
            if (key != 0 && rank < K) {
                logit[j * K + rank] = unordered((unsigned)(key >> 32));
                token[j * K + rank] = (int)(0xFFFFFFFFu - (unsigned)key);
            }
        }
    } else {
        for (int j = warp; j < beams; j += kWarps)
            if (row_state[j] == 2)
                join_row(P.staged ? keys + j * per_row : P.keys + (beam0 + j) * per_row, P.segs, K, lane, logit + j * K, token + j * K);
    }
    __syncthreads();
    const unsigned long long none = ordered64(-INFINITY);
    for (int i = tid; i < n; i += kJoinThreads) {
        const int j = i / K;
        const float x = logit[i], top = row_top[j];
        const double v = (double)row_cum[j] + ((x == top ? 0.0 : (double)x - (double)top) - row_sum[j]);
        logit[i] = (float)v;
        order[i] = x == -INFINITY ? none : ordered64(v);
    }
    __syncthreads();

    const int64_t out = (int64_t)blockIdx.x * K;
    const auto put = [&](int k, int i) {
        const int t = token[i];
        if (!GDN_IN(P.a.err_flags, t, P.a.vocab) || !GDN_IN(P.a.err_flags, k, K)) return;
        P.a.out_scores[out + k] = logit[i];
        P.a.out_parents[out + k] = i / K;
        P.a.out_tokens[out + k] = t;
        if (P.a.out_finished) P.a.out_finished[out + k] = t == P.a.eos_token;
    };
    const auto put_none = [&](int k) {
        P.a.out_scores[out + k] = -INFINITY;
        P.a.out_parents[out + k] = -1;
        P.a.out_tokens[out + k] = -1;
        if (P.a.out_finished) P.a.out_finished[out + k] = 0;
    };
    if (n <= kRankCandidates) {
        // a candidate a thread; equal ones by beam (a row's own are in order already)
        int rank = K;
        bool any = false;
        if (tid < n) {
            const unsigned long long v = order[tid];
            any = v > none;
            rank = 0;
#pragma unroll 4
            for (int o = 0; o < n; ++o) rank += order[o] > v || (order[o] == v && o < tid);
            if (any && rank < K) put(rank, tid);
        }
        const int count = __syncthreads_count(any);
        for (int k = count + tid; k < K; k += kJoinThreads) put_none(k);
        return;
    }
    if (warp != 0) return;
    // the beams' lists: a lane per beam; the lowest lane wins a tie
    int at = 0;
    const bool on = lane < beams;
    unsigned long long head = on ? order[lane * K] : none;
    for (int k = 0; k < K; ++k) {
        const unsigned long long best = warp_max(head);
        const int who = __ffs(__ballot_sync(kFullMask, on && head == best)) - 1;
        if (best > none && lane == who) {
            put(k, lane * K + at);
            ++at;
            head = at < K ? order[lane * K + at] : none;
        } else if (best <= none && lane == 0) {
            put_none(k);
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
bool overlap(const void *p, size_t pn, const void *q, size_t qn)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + qn && b < a + pn;
}

// Whether an output lies over memory that the join still reads: its CTAs run in no order, and each reads its entry's
// part of the tables before it writes its own results. So with several entries only a table of the very same layout
// may be an output.
bool outputs_overlap(const gdn_beam_select_args &a, size_t workspace)
{
    const size_t in = (size_t)a.batch * a.beams, out = (size_t)a.batch * a.K;
    const struct { const void *p; size_t es; } tables[] = {{a.rows, 4}, {a.scores, 4}, {a.finished, 1}},
                                               outputs[] = {{a.out_scores, 4}, {a.out_parents, 4}, {a.out_tokens, 4}, {a.out_finished, 1}};
    for (const auto &o : outputs) {
        if (overlap(o.p, out * o.es, a.workspace, workspace)) return true;
        for (const auto &t : tables)
            if (a.batch > 1 && overlap(o.p, out * o.es, t.p, in * t.es) && !(o.p == t.p && o.es == t.es && a.K == a.beams)) return true;
    }
    return false;
}

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
    const size_t need = gdn_beam_select_workspace_bytes(a->batch, a->beams, a->vocab, a->K);
    if (a->workspace_bytes < need) return GDN_ERR_SHAPE;
    const int es = a->logits_dtype == GDN_BF16 ? 2 : 4;
    if (!aligned_to(a->logits, es) || !aligned_to(a->rows, 4) || !aligned_to(a->scores, 4) || !aligned_to(a->out_scores, 4) ||
        !aligned_to(a->out_parents, 4) || !aligned_to(a->out_tokens, 4) || !aligned_to(a->workspace, 16))
        return GDN_ERR_ALIGN;
    if (outputs_overlap(*a, need)) return GDN_ERR_ARG;
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
    size_t smem = (size_t)a->beams * a->K * 16;
    const size_t keys = (size_t)a->beams * P.segs * a->K * 8;
    P.staged = smem + keys <= 40 * 1024;
    if (P.staged) smem += keys;
    return launch_ordinary(beam_join_kernel, dim3((unsigned)a->batch), dim3(kJoinThreads), smem, s, P) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_LAUNCH;
}

}  // extern "C"
