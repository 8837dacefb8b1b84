// scan_common.cuh -- what the selective scan's forward and backward kernels share (internal to
// libgdn_decode.so): fp32-pair arithmetic, staging of token tiles, the walk over a chunk's sequences.
//
// Work split. The packed token rows are cut into chunks of C rows, the channels into tiles of
// ScanShape::CB; one CTA of four warps owns a (chunk, channel tile) and walks its rows in order, each
// thread keeping CPT channels x 4 state entries in registers. A chunk may hold pieces of several
// sequences: the state is set anew where one begins, so ragged prompts cost what their tokens cost.
// States cross chunk borders through a summary pass (the state each chunk would end with from zero,
// and the sum of its dt: its decay is exp(A sum dt), one exp per entry and chunk) and a carry pass
// over the chunks. The summary costs a second exp per state entry, so it is skipped where the
// sequences alone fill the GPU (plan in scan_api.cu).
#pragma once

#include <cmath>
#include <cstdint>

#include "gdn_chain.cuh"
#include "gdn_common.cuh"
#include "gdn_pipe.cuh"
#include "mamba_scan.h"
#include "scan_launch.h"

namespace gdn {

constexpr int kScanThreads = 128;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanTile = 16;               // token rows staged at a time
constexpr unsigned kScanFull = 0xFFFFFFFFu;

// Lanes along the state: NL lanes x 4 entries cover a row of up to 4 NL entries (missing ones are
// zeros); the other lanes and the warps lie along the channels, CPT consecutive ones a thread. What
// bounds the kernels besides the arithmetic is shared memory's 128 bytes a clock: a thread loads CPT
// dt and x and 4 B and C per token for its 4 CPT entries, so a square 4 x 4 tile of entries per thread
// loads least, and the operands stay in their own type until they are in registers.
template <int NL_, int CPT_> struct ScanShape {
    static constexpr int NL = NL_, CPT = CPT_, P = CPT_ / 2;   // P pairs of channels
    static constexpr int NP = 4 * NL;                     // padded state size
    static constexpr int CLN = 32 / NL;                   // channel lanes of a warp
    static constexpr int CW = CLN * CPT;                  // channels of a warp
    static constexpr int CB = CW * kScanWarps;            // channels of a CTA
    static constexpr int YP = CW + 8;                     // row pitch of a warp's per-channel sums (no bank conflicts)
};

// ---------------------------------------------------------------------------------------------
// fp32 pairs (fma.rn.f32x2: half the issue slots of the scalar instructions at the same rate, each
// element rounded alike)
// ---------------------------------------------------------------------------------------------
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(f2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Decays close to one are multiplied over thousands of tokens, so a bias of their rounding grows
// with the length of the memory. exp(-x) by ex2.approx measured a mean relative error of -0.5e-8 for x below
// 0.002, -1e-8 to -3e-8 from there to 0.03 and about -2e-8 up to 0.6 (GB300, 2^18 arguments a bin). An exponent
// larger by this constant takes part of it out at no cost (the product dt A becomes a multiply-add): more would
// hurt the longest memories, less the others. Against 64 bits, in relative L2 norm, the worst of nine cases (states
// of 4 to 128 entries, 300 to 8000 tokens, step sizes from 0.001 to 0.1), constants of 0, 0.9, 1.3 and 2.2e-8: final states off by 20, 6.4,
// 7.0 and 21e-7, dA by 14, 9.8, 7.9 and 6.3e-7, outputs in fp32 by 12, 7.0, 5.8 and 7.7e-7.
constexpr float kDecayBias = 1.3e-8f;

// exp(dt A) of a pair of entries, A2 = A log2(e)
__device__ __forceinline__ f2 decay2(f2 dtdt, f2 A2)
{
    const float2 y = unpack2(fma2(dtdt, A2, pack2(kDecayBias, kDecayBias)));
    return pack2(ex2_approx(y.x), ex2_approx(y.y));
}

// sigmoid of a pair on the fast reciprocal and exponential (relative error of a few 2^-23; exactly 0 where
// exp(-z) overflows)
__device__ __forceinline__ f2 sigmoid2(f2 z)
{
    const float2 t = unpack2(mul2(z, pack2(-kLog2e, -kLog2e)));
    const float2 d = unpack2(add2(pack2(ex2_approx(t.x), ex2_approx(t.y)), pack2(1.f, 1.f)));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    return pack2(r.x, r.y);
}

// Sums v[0 .. M) over the NL lanes of a group, M values at once: each halving of the lanes halves
// the values a lane keeps. Lane nl ends with values nl M / NL .. (M >= NL), or with value
// nl / (NL / M) (M < NL, the same one in NL / M lanes).
template <int M, int NL> __device__ __forceinline__ void group_reduce(float (&v)[M], int nl, int lane_step = 1)
{
    int m = M;
#pragma unroll
    for (int off = NL / 2; off > 0; off >>= 1) {
        const bool hi = (nl & off) != 0;
        if (m > 1) {
            m /= 2;
#pragma unroll
            for (int i = 0; i < M / 2; ++i) {
                if (i < m) {
                    const float send = hi ? v[i] : v[i + m];
                    const float keep = hi ? v[i + m] : v[i];
                    v[i] = keep + __shfl_xor_sync(kScanFull, send, off * lane_step);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(kScanFull, v[0], off * lane_step);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// staging: R rows x W elements of a row-strided tensor into shared memory
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void cp_async4(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

// Where a staged tile lies in its tensor: rows t0 .. of T, columns c0 .. of `width`.
template <typename T> struct TileSource {
    const T *base;
    int64_t stride;
    int t0, rows, c0, width;
    int mode;            // kRows16, kRows4 or kRowsAny
};

// eight bf16 elements from p on, which may lie across 16-byte boundaries: shifted out of two aligned vectors
__device__ __forceinline__ uint4 load_across(const bf16 *p)
{
    const int shift = (int)((reinterpret_cast<uintptr_t>(p) & 15) / 2);
    const uint4 lo = *reinterpret_cast<const uint4 *>(p - shift), hi = *reinterpret_cast<const uint4 *>(p - shift + 8);
    unsigned w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (shift & 4) {
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
    }
    if (shift & 2) {
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
    }
    if (shift & 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// bf16 rows of any alignment, through registers. A vector is read whole where both aligned vectors lie in the
// tensor: in its row, or between rows that it has.
template <int W, int R, bool LAST, typename T>
__device__ __forceinline__ void stage_across(T *, const T *, const TileSource<T> &, int, int, int)
{
}
template <int W, int R, bool LAST>
__device__ __forceinline__ void stage_across(bf16 *dst, const bf16 *src, const TileSource<bf16> &s, int n, int ncols, int tid)
{
    constexpr int VPR = W / 8;
    const int lead = LAST ? R - n : 0;
    const bf16 *at = src - lead * s.stride;       // where row 0 of the tile would be
#pragma unroll 2
    for (int i = tid; i < R * VPR; i += kScanThreads) {
        const int r = i / VPR, v = i % VPR, c = s.c0 + v * 8, left = ncols - v * 8;
        uint4 q = make_uint4(0, 0, 0, 0);
        if ((LAST ? r >= lead : r < n) && left > 0) {
            const bf16 *p = at + r * s.stride + v * 8;
            const int row = s.t0 + r - lead;
            if (left >= 8 && (c >= 7 || row > 0) && (c + 16 <= s.width || row + 1 < s.rows)) {
                q = load_across(p);
            } else {
                const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
                unsigned w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = (2 * k < left ? u[2 * k] : 0u) | (2 * k + 1 < left ? (unsigned)u[2 * k + 1] << 16 : 0u);
                q = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        *reinterpret_cast<uint4 *>(dst + r * W + v * 8) = q;
    }
}

template <typename T, int W, int R, bool LAST> __device__ __noinline__ void stage_unaligned(T *dst, TileSource<T> s, int n, int tid)
{
    const T *src = s.base + (int64_t)s.t0 * s.stride + s.c0;
    const int ncols = min(W, s.width - s.c0);
    if (sizeof(T) == 4 || s.mode == kRows4) {
        constexpr int E = 4 / (int)sizeof(T), PR = W / E;
        const int lead = LAST ? R - n : 0;
        const T *at = src - lead * s.stride;
#pragma unroll 4
        for (int i = tid; i < R * PR; i += kScanThreads) {
            const int r = i / PR, v = i % PR;
            int left = (LAST ? r >= lead : r < n) ? (ncols - v * E) * (int)sizeof(T) : 0;
            left = left < 0 ? 0 : left > 4 ? 4 : left;
            cp_async4(dst + r * W + v * E, left ? at + r * s.stride + v * E : src, left);
        }
    } else {
        stage_across<W, R, LAST>(dst, src, s, n, ncols, tid);
    }
}

// The n rows from t0 on become the tile's first ones or, with LAST, its last ones; its other rows and columns >= the
// tensor's width are filled with zeros. Aligned rows are copied asynchronously
// in 16 bytes, rows on 4-byte boundaries in 4; bf16 rows that begin between those (odd strides) go through
// registers in 16 bytes (4 x 2000 rows, N = 16, bf16: 777 channels 106 us against 84 for 776; gradients 341
// against 261).
template <typename T, int W, int R = kScanTile, bool LAST = false>
__device__ __forceinline__ void stage_rows(T *dst, const TileSource<T> &s, int n, int tid)
{
    constexpr int VE = 16 / (int)sizeof(T), VPR = W / VE;
    static_assert(W % VE == 0, "a staged row is whole 16-byte vectors");
    const T *src = s.base + (int64_t)s.t0 * s.stride + s.c0;
    const int ncols = min(W, s.width - s.c0);
    if (s.mode == kRows16) {
        const int lead = LAST ? R - n : 0;
        const T *at = src - lead * s.stride;
#pragma unroll
        for (int k = 0; k < (R * VPR + kScanThreads - 1) / kScanThreads; ++k) {
            const int i = k * kScanThreads + tid;
            const int r = i / VPR, v = i % VPR;
            if (R * VPR % kScanThreads == 0 || r < R) {
                int left = (LAST ? r >= lead : r < n) ? (ncols - v * VE) * (int)sizeof(T) : 0;
                left = left < 0 ? 0 : left > 16 ? 16 : left;
                cp_async16(dst + r * W + v * VE, left ? at + r * s.stride + v * VE : src, left);
            }
        }
    } else {
        stage_unaligned<T, W, R, LAST>(dst, s, n, tid);
    }
}

// ---------------------------------------------------------------------------------------------
// sequences
// ---------------------------------------------------------------------------------------------
// first row of sequence s (s = S: the end of the last one)
__device__ __forceinline__ int seq_bound(const ScanLaunch &P, int s)
{
    return P.a.cu_seqlens ? P.a.cu_seqlens[s] : s * P.L;
}

// The last sequence that begins at or before row pos (-1: none; S: pos lies behind the last one),
// found by the whole CTA. Contains two barriers with cu_seqlens.
__device__ __forceinline__ int find_seq(const ScanLaunch &P, int pos, int *scratch, int tid)
{
    if (!P.a.cu_seqlens) return P.L ? pos / P.L : 0;
    int c = 0;
    for (int i = tid; i <= P.a.S; i += kScanThreads) c += P.a.cu_seqlens[i] <= pos;
    c = __reduce_add_sync(kScanFull, c);
    __syncthreads();
    if ((tid & 31) == 0) scratch[tid >> 5] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) c += scratch[w];
    return c - 1;
}

// A staged tile: rows t0 .. t0 + n - 1 of one sequence (seq -1: rows of no sequence, or of one whose
// state index is out of range: their outputs are zeros).
struct ScanTile {
    int t0, n;
    int seq;
    int64_t slot;     // its row in the state buffers
    bool fresh;       // first tile of this sequence in the chunk
    bool starts;      // holds the sequence's first row
    bool ends;        // holds the sequence's last row
};

// Walks rows pos .. end - 1 in tiles that never span two sequences.
struct ScanIter {
    int pos, end, s, run_begin, run_end;
    int64_t slot;
    bool live;

    __device__ __forceinline__ void init(int first, int last, int seq)
    {
        pos = first;
        end = last;
        s = seq;
        run_end = first;
        live = false;
    }

    __device__ __forceinline__ bool next(const ScanLaunch &P, ScanTile &t)
    {
        if (pos >= end) return false;
        t.fresh = pos >= run_end;
        if (t.fresh) {
            if (s < 0 && seq_bound(P, 0) <= pos) s = 0;
            while (s >= 0 && s < P.a.S && seq_bound(P, s + 1) <= pos) ++s;
            live = s >= 0 && s < P.a.S;
            run_begin = live ? seq_bound(P, s) : pos;
            run_end = live ? seq_bound(P, s + 1) : s < 0 ? min(seq_bound(P, 0), end) : end;
            if (live) {
                slot = P.a.state_indices ? (int64_t)P.a.state_indices[s] : s;
                if (P.has_states && (slot < 0 || slot >= P.a.num_states)) live = false;
            }
            if (!live) raise_flag(threadIdx.x == 0 ? P.a.err_flags : nullptr, GDN_DEVERR_BAD_INDEX);
        }
        t.t0 = pos;
        t.n = min(kScanTile, min(run_end, end) - pos);
        t.seq = live ? s : -1;
        t.slot = slot;
        t.starts = live && pos == run_begin;
        t.ends = live && pos + t.n == run_end;
        pos += t.n;
        return true;
    }
};

// ---------------------------------------------------------------------------------------------
// operands in shared memory
// ---------------------------------------------------------------------------------------------
// CPT consecutive channels of a staged row as pairs
__device__ __forceinline__ void load_pairs(const float *p, f2 (&v)[1]) { v[0] = *reinterpret_cast<const f2 *>(p); }
__device__ __forceinline__ void load_pairs(const float *p, f2 (&v)[2])
{
    const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(p);
    v[0] = q.x;
    v[1] = q.y;
}
__device__ __forceinline__ f2 widen2(uint32_t w) { return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ void load_pairs(const bf16 *p, f2 (&v)[1]) { v[0] = widen2(*reinterpret_cast<const uint32_t *>(p)); }
__device__ __forceinline__ void load_pairs(const bf16 *p, f2 (&v)[2])
{
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    v[0] = widen2(q.x);
    v[1] = widen2(q.y);
}
__device__ __forceinline__ void store_pairs(float *p, const f2 (&v)[1]) { *reinterpret_cast<f2 *>(p) = v[0]; }
__device__ __forceinline__ void store_pairs(float *p, const f2 (&v)[2]) { *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v[0], v[1]); }
// four consecutive state entries of a staged B or C row, each in both halves of a pair
template <typename T> __device__ __forceinline__ void load_twice(const T *p, f2 (&v)[4])
{
    const float4 q = load4(p);
    v[0] = pack2(q.x, q.x);
    v[1] = pack2(q.y, q.y);
    v[2] = pack2(q.z, q.z);
    v[3] = pack2(q.w, q.w);
}

// ---------------------------------------------------------------------------------------------
// a thread's entries of a [D, N] fp32 state row: v[n][p] holds entry n0 + n of channels d + 2 p, d + 2 p + 1
// ---------------------------------------------------------------------------------------------
template <int P> __device__ __forceinline__ void load_entries(const float *row, int d, int D, int n0, int N, bool vec, f2 (&v)[4][P])
{
#pragma unroll
    for (int p = 0; p < P; ++p) {
        float e[2][4] = {};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (d + 2 * p + c < D) {
                const float *q = row + (int64_t)(d + 2 * p + c) * N + n0;
                if (vec && n0 < N) {
                    const float4 f = *reinterpret_cast<const float4 *>(q);
                    e[c][0] = f.x; e[c][1] = f.y; e[c][2] = f.z; e[c][3] = f.w;
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        if (n0 + n < N) e[c][n] = q[n];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) v[n][p] = pack2(e[0][n], e[1][n]);
    }
}
template <int P> __device__ __forceinline__ void store_entries(float *row, int d, int D, int n0, int N, bool vec, const f2 (&v)[4][P])
{
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const float2 e[4] = {unpack2(v[0][p]), unpack2(v[1][p]), unpack2(v[2][p]), unpack2(v[3][p])};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (d + 2 * p + c < D) {
                float *q = row + (int64_t)(d + 2 * p + c) * N + n0;
                const float f[4] = {c ? e[0].y : e[0].x, c ? e[1].y : e[1].x, c ? e[2].y : e[2].x, c ? e[3].y : e[3].x};
                if (vec && n0 < N) {
                    *reinterpret_cast<float4 *>(q) = make_float4(f[0], f[1], f[2], f[3]);
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        if (n0 + n < N) q[n] = f[n];
                }
            }
        }
    }
}
template <int P> __device__ __forceinline__ void zero_entries(f2 (&v)[4][P])
{
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int p = 0; p < P; ++p) v[n][p] = 0ull;
}

// A log2(e) of a thread's entries. An A of minus infinity (forget everything) becomes the lowest
// finite value: the same decay of zero for every dt of a token, and still one for the dt of zero that
// fills up a tile's missing rows.
__device__ __forceinline__ float finite_rate(float a) { return a == -INFINITY ? -3.402823466e38f : a; }
template <int P> __device__ __forceinline__ void load_rates(const float *A, int d, int D, int n0, int N, bool vec, f2 (&v)[4][P])
{
    load_entries(A, d, D, n0, N, vec, v);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float2 a = unpack2(v[n][p]);
            v[n][p] = pack2(finite_rate(a.x * kLog2e), finite_rate(a.y * kLog2e));
        }
}

// a thread's consecutive elements of a row-strided output, as one access where the row allows it
__device__ __forceinline__ void store_whole(float *p, const f2 (&v)[1]) { *reinterpret_cast<f2 *>(p) = v[0]; }
__device__ __forceinline__ void store_whole(float *p, const f2 (&v)[2]) { store_pairs(p, v); }
__device__ __forceinline__ uint32_t narrow2(f2 v)
{
    const float2 f = unpack2(v);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ void store_whole(bf16 *p, const f2 (&v)[1]) { *reinterpret_cast<uint32_t *>(p) = narrow2(v[0]); }
__device__ __forceinline__ void store_whole(bf16 *p, const f2 (&v)[2])
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(narrow2(v[0]), narrow2(v[1]));
}
// whole: the access is aligned and within the row
template <typename T, int P> __device__ __forceinline__ void store_row(T *p, const f2 (&v)[P], int left, bool whole)
{
    if (whole) {
        store_whole(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float2 f = unpack2(v[j]);
            if (2 * j < left) p[2 * j] = from_f32<T>(f.x);
            if (2 * j + 1 < left) p[2 * j + 1] = from_f32<T>(f.y);
        }
    }
}

}  // namespace gdn
