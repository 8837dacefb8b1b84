// linear_carry.cu -- what linear attention does between and behind its sweeps: states across segments, sums over
// value heads that share a head, gradients of the log decays.
#include "linear_common.cuh"

namespace gdn {

namespace {

// local[j]: from the state segment j ends with, starting from zero, to the state it starts with. One thread takes four
// entries of a sequence's states over all its segments; memory-bound, 8 K V bytes a segment and head.
__global__ void __launch_bounds__(256) linear_carry_kernel(const __grid_constant__ LinearLaunch P, const __grid_constant__ LinearSweep p)
{
    const int hv = blockIdx.y;
    int state, item0, segs;
    if (linear_many(P)) {                            // CTAs for the segments of sequences that are cut; the first one's work
        __shared__ LinearItem s_item;
        __shared__ LinearScan s_scan;
        linear_find<256>(P, blockIdx.x, true, false, 0, s_scan, &s_item);
        const LinearItem it = s_item;
        if (it.seq < 0 || it.index > 0 || it.state < 0) return;
        state = it.state;
        item0 = it.slot;
        segs = linear_segments(P, it.seq_end - it.seq_begin);
    } else {
        const int s = blockIdx.x;
        int b, e;
        bool bad;
        linear_rows(P, s, b, e, bad);
        segs = linear_segments(P, e - b);
        if (bad || segs == 1) return;
        state = linear_state(P, s, false);
        item0 = linear_first_item(P, s);
        if (state < 0 || item0 + segs > P.items) return;     // (left out, as in linear_item)
    }
    const int KV = P.a.K * P.a.V, at = (blockIdx.z * 256 + threadIdx.x) * 4;
    if (at >= KV || !GDN_IN(P.a.err_flags, item0 + segs - 1, P.cut_items)) return;
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.start) run = *reinterpret_cast<const float4 *>(p.start + ((size_t)state * P.a.HV + hv) * KV + at);
    // four segments' states at a time on their way
    for (int j0 = 0; j0 < segs; j0 += 4) {
        float4 own[4];
        float2 f[4];
        float4 *l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = min(j0 + j, segs - 1);
            const size_t item = (size_t)(item0 + (p.reverse ? segs - 1 - k : k)) * P.a.HV + hv;
            l[j] = reinterpret_cast<float4 *>(P.local + item * KV + at);
            own[j] = *l[j];
            f[j] = P.total[item];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j0 + j >= segs) break;
            const float g = linear_decay_factor(f[j].x, f[j].y);
            *l[j] = run;
            run = make_float4(fmaf(g, run.x, own[j].x), fmaf(g, run.y, own[j].y), fmaf(g, run.z, own[j].z), fmaf(g, run.w, own[j].w));
        }
    }
}

// A warp per token and q/k head: the sum over the value heads that share it, and each one's product with `with`. A CTA takes
// kFoldRows token rows, those among them that some sequence has. (A grid of segments x the longest segment's rows, whose CTAs each
// count all sequences, grows with the square of their number: gradients of 2048 documents of 256 tokens, 32 heads of 128 x 128,
// took 1757 ms, 34 so; of 64 documents 1.39 and 1.30.)
constexpr int kFoldRows = 64;
template <typename Tin>
__global__ void __launch_bounds__(256) linear_fold_kernel(const __grid_constant__ LinearLaunch P, const __grid_constant__ LinearFold f)
{
    const int lane = threadIdx.x & 31, h = blockIdx.y, K = P.a.K, G = P.a.HV / P.a.H;
    const int64_t t0 = (int64_t)blockIdx.x * kFoldRows;
    __shared__ unsigned long long s_mine;
    __shared__ LinearScan s_scan;
    unsigned long long mine = ~0ull;
    static_assert(kFoldRows == 64, "a bit a row");
    if (P.a.cu_seqlens) {
        if (threadIdx.x == 0) s_mine = 0;
        __syncthreads();
        linear_each<256>(P, s_scan, [&](int, int b, int e, bool bad, long long, long long) {
            const int from = (int)max((int64_t)0, b - t0), to = (int)min((int64_t)kFoldRows, e - t0);
            if (!bad && from < to) atomicOr(&s_mine, (~0ull >> (64 - (to - from))) << from);
        });
        __syncthreads();
        mine = s_mine;
    }
    const int last = (int)min((int64_t)kFoldRows, P.a.T - t0);
    for (int r = threadIdx.x >> 5; r < last; r += 8) {
        const int64_t t = t0 + r;
        if (!(mine >> r & 1) || !GDN_IN(P.a.err_flags, t, P.a.T)) continue;
        float sum[4] = {0.f, 0.f, 0.f, 0.f}, y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lane + 32 * i;
            y[i] = c < K ? to_f32(static_cast<const Tin *>(f.with)[t * f.with_stride + (int64_t)h * f.with_head + c]) : 0.f;
        }
        for (int g = 0; g < G; ++g) {
            const int hv = h * G + g;
            const float *part = f.part + ((size_t)t * P.a.HV + hv) * K;
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = lane + 32 * i;
                const float v = c < K ? part[c] : 0.f;
                sum[i] += v;
                d = fmaf(v, y[i], d);
            }
            if (f.dot) {
                d = group_sum<32>(d);
                if (lane == 0) f.dot[(size_t)t * P.a.HV + hv] = d;
            }
        }
        if (f.out)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = lane + 32 * i;
                if (c < K) static_cast<Tin *>(f.out)[t * f.out_stride + (int64_t)h * f.out_head + c] = from_f32<Tin>(sum[i]);
            }
    }
}

// Sums of many terms whose difference counts: kept as a pair of fp32 numbers (the rounding error of each addition is
// added to the second), since fp64 runs at two operations a clock and SM.
struct Pair {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x)
    {
        const float s = hi + x, b = s - hi;
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
    __device__ __forceinline__ float value() const { return hi + lo; }
};

// A CTA per segment and eight heads; 64 ranges of tokens, each summed, then taken again from behind with the sum of the
// ranges behind it.
constexpr int kDgHeads = 8, kDgRanges = 64;
__global__ void __launch_bounds__(kDgHeads *kDgRanges) linear_dg_kernel(const __grid_constant__ LinearLaunch P, const float *qdq,
                                                                     const float *kdk, const float *segment_dot, int parts,
                                                                     float *dg, int64_t dg_stride, float *part)
{
    const int i = threadIdx.x % kDgHeads, range = threadIdx.x / kDgHeads;
    const int hv = blockIdx.y * kDgHeads + i, HV = P.a.HV;
    __shared__ float hi[kDgRanges][kDgHeads], lo[kDgRanges][kDgHeads];
    __shared__ LinearItem s_item;
    __shared__ LinearScan s_scan;
    linear_find<kDgHeads * kDgRanges>(P, blockIdx.x, false, false, 0, s_scan, &s_item);
    const LinearItem it = s_item;
    if (it.seq >= 0 && !linear_in(P, it)) return;
    const bool skip = it.seq < 0 || it.state < 0;
    const int b = it.begin, e = it.seq < 0 ? b : b + it.n;
    const int per = (e - b + kDgRanges - 1) / kDgRanges;
    const int first = b + range * per, last = min(e, first + per);
    const bool mine = hv < HV;
    Pair sum;
    if (mine && !skip)
        for (int t = first; t < last; ++t) {
            sum.add(qdq[(size_t)t * HV + hv]);
            sum.add(-kdk[(size_t)t * HV + hv]);
        }
    hi[range][i] = sum.hi;
    lo[range][i] = sum.lo;
    __syncthreads();
    if (!mine) return;
    Pair run, total;
    if (!skip)
        for (int k = 0; k < parts; ++k) run.add(segment_dot[((size_t)blockIdx.x * HV + hv) * parts + k]);
    for (int r = kDgRanges - 1; r > range; --r) {
        run.add(hi[r][i]);
        run.add(lo[r][i]);
    }
    const bool fixed = P.a.g_stride == 0;
    for (int t = last - 1; t >= first; --t) {
        if (!skip) {
            run.add(qdq[(size_t)t * HV + hv]);
            run.add(-kdk[(size_t)t * HV + hv]);
        }
        const float v = skip ? 0.f : run.value();
        if (fixed) total.add(v);
        else dg[t * dg_stride + hv] = v;
    }
    if (fixed) part[((size_t)blockIdx.x * kDgRanges + range) * HV + hv] = total.value();
}

// dg of one decay a head: the ranges' sums of every segment (eight of every chunk), in order
__global__ void __launch_bounds__(256) linear_dg_fixed_kernel(const float *part, int64_t rows, int HV, float *dg)
{
    const int hv = blockIdx.x;
    __shared__ double sums[8];
    double s = 0.0;
    for (int64_t r = threadIdx.x; r < rows; r += 256) s += part[(size_t)r * HV + hv];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) s += sums[w];
        dg[hv] = (float)s;
    }
}

// Of the tensor-core kernel: no sum is longer than a chunk. A CTA per chunk and 32 heads, eight ranges of 16 rows.
struct DgChunk {
    int seq, at, rows;
};
__global__ void __launch_bounds__(256) linear_dg_chunk_kernel(const __grid_constant__ LinearLaunch P, const float *qdq, const float *kdk,
                                                           const float *chunk_dot, float *dg, int64_t dg_stride, float *part)
{
    const int i = threadIdx.x & 31, range = threadIdx.x >> 5, hv = blockIdx.y * 32 + i, HV = P.a.HV;
    const int id = blockIdx.x;                        // first row / 128 + sequence
    __shared__ float sums[8][32];
    __shared__ DgChunk s_chunk;
    __shared__ LinearScan s_scan;
    if (threadIdx.x == 0) s_chunk.seq = -1;
    __syncthreads();
    const auto take = [&](int s, int b, int e) {
        const int j = id - s - b / kLinearChunk;
        if (j < 0 || (int64_t)j * kLinearChunk >= e - b) return;
        const int at = b + j * kLinearChunk;
        s_chunk = {s, at, min(kLinearChunk, e - at)};
    };
    if (P.a.cu_seqlens) {
        linear_each<256>(P, s_scan, [&](int s, int b, int e, bool bad, long long, long long) {
            if (!bad) take(s, b, e);                  // (one sequence, or of borders that decrease any of them)
        });
    } else if (threadIdx.x < 2) {
        // s L / 128 + s <= id, the last such s: 128 id / (L + 128), or the one behind it
        const int64_t s = (int64_t)id * kLinearChunk / (P.Ls + kLinearChunk) + threadIdx.x;
        if (s < P.a.S) take((int)s, (int)s * P.Ls, (int)s * P.Ls + P.Ls);
    }
    __syncthreads();
    const DgChunk it = s_chunk;
    const int at = it.at, rows = it.seq < 0 ? 0 : it.rows;
    const bool fixed = P.a.g_stride == 0;
    if (it.seq < 0) {                                 // nobody's
        if (fixed && hv < HV) part[((size_t)id * 8 + range) * HV + hv] = 0.f;
        return;
    }
    if (!GDN_IN(P.a.err_flags, at, P.a.T) || !GDN_IN(P.a.err_flags, rows, P.a.T - at + 1)) return;
    const bool mine = hv < HV && linear_state(P, it.seq, false) >= 0;
    const int first = 16 * range, last = min(rows, first + 16);
    float d[16], sum = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const size_t t = (size_t)(at + first + k) * HV + hv;
        d[k] = mine && first + k < last ? qdq[t] - kdk[t] : 0.f;
    }
#pragma unroll
    for (int k = 15; k >= 0; --k) sum += d[k];
    sums[range][i] = sum;
    __syncthreads();
    if (hv >= HV) return;
    float run = 0.f, total = 0.f;
    if (mine)
        for (int k = 0; k < 8; ++k) run += chunk_dot[((size_t)id * HV + hv) * 8 + k];
    for (int r = 7; r > range; --r) run += sums[r][i];
#pragma unroll
    for (int k = 15; k >= 0; --k) {
        run += d[k];
        if (first + k >= last) continue;
        if (fixed) total += run;
        else dg[(int64_t)(at + first + k) * dg_stride + hv] = run;
    }
    if (fixed) {
        __syncwarp();
        part[((size_t)id * 8 + range) * HV + hv] = total;
    }
}

// A thread per eight values.
__global__ void __launch_bounds__(256) linear_pack_kernel(const uint16_t *from, int64_t stride, int64_t head, int64_t count, int heads,
                                                       int n, int vectors, uint4 *to)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= count) return;
    const int c = (int)(i % vectors) * 8;
    const int64_t th = i / vectors, t = th / heads;
    const uint16_t *p = from + t * stride + (th - t * heads) * head;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = (c + 2 * j < n ? p[c + 2 * j] : 0u) | (c + 2 * j + 1 < n ? (uint32_t)p[c + 2 * j + 1] << 16 : 0u);
    to[i] = make_uint4(w[0], w[1], w[2], w[3]);
}

int status() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

}  // namespace

size_t linear_dg_part_floats(int items, int HV) { return (size_t)items * kDgRanges * HV; }

int launch_linear_pack(const void *from, int64_t stride, int64_t head, int T, int heads, int n, void *to, cudaStream_t stream)
{
    const int vectors = (n + 7) / 8;
    const int64_t count = (int64_t)T * heads * vectors, grid = (count + 255) / 256;
    if (grid > INT32_MAX) return GDN_ERR_SHAPE;
    linear_pack_kernel<<<(unsigned)grid, 256, 0, stream>>>(static_cast<const uint16_t *>(from), stride, head, count, heads, n, vectors,
                                                         static_cast<uint4 *>(to));
    return status();
}

int launch_linear_carry(const LinearLaunch &P, const LinearSweep &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)(P.a.cu_seqlens && P.a.S > kLinearSorted ? P.cut_items : P.a.S), (unsigned)P.a.HV, (unsigned)((P.a.K * P.a.V + 1023) / 1024));
    linear_carry_kernel<<<grid, 256, 0, stream>>>(P, p);
    return status();
}

int launch_linear_fold(const LinearLaunch &P, const LinearFold &f, cudaStream_t stream)
{
    if (P.a.T == 0) return GDN_OK;
    const dim3 grid((unsigned)(((int64_t)P.a.T + kFoldRows - 1) / kFoldRows), (unsigned)P.a.H);
    if (P.a.in_dtype == GDN_BF16) linear_fold_kernel<bf16><<<grid, 256, 0, stream>>>(P, f);
    else linear_fold_kernel<float><<<grid, 256, 0, stream>>>(P, f);
    return status();
}

int launch_linear_dg(const LinearLaunch &P, const float *qdq, const float *kdk, const float *segment_dot, int parts, float *dg,
                     int64_t dg_stride, float *part, cudaStream_t stream)
{
    const dim3 grid((unsigned)P.items, (unsigned)((P.a.HV + kDgHeads - 1) / kDgHeads));
    linear_dg_kernel<<<grid, kDgHeads * kDgRanges, 0, stream>>>(P, qdq, kdk, segment_dot, parts, dg, dg_stride, part);
    if (P.a.g_stride == 0) linear_dg_fixed_kernel<<<P.a.HV, 256, 0, stream>>>(part, (int64_t)P.items * kDgRanges, P.a.HV, dg);
    return status();
}

int launch_linear_dg_chunks(const LinearLaunch &P, const float *qdq, const float *kdk, const float *chunk_dot, float *dg,
                            int64_t dg_stride, float *part, cudaStream_t stream)
{
    const int ids = P.a.T / kLinearChunk + P.a.S;
    linear_dg_chunk_kernel<<<dim3((unsigned)ids, (unsigned)((P.a.HV + 31) / 32)), 256, 0, stream>>>(P, qdq, kdk, chunk_dot, dg, dg_stride, part);
    if (P.a.g_stride == 0) linear_dg_fixed_kernel<<<P.a.HV, 256, 0, stream>>>(part, (int64_t)ids * 8, P.a.HV, dg);
    return status();
}

}  // namespace gdn
