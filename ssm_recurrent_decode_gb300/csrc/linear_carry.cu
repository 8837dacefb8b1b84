// linear_carry.cu -- what linear attention does between and behind its sweeps: states across segments, sums over
// value heads that share a head, gradients of the log decays.
#include "linear_common.cuh"

namespace gdn {

namespace {

// local[j]: from the state segment j ends with, starting from zero, to the state it starts with. One thread takes four
// entries of a sequence's states over all its segments; memory-bound, 8 K V bytes a segment and head.
__global__ void __launch_bounds__(256) linear_carry_kernel(const __grid_constant__ LinearLaunch P, const __grid_constant__ LinearSweep p)
{
    const int s = blockIdx.x, hv = blockIdx.y;
    int b, e;
    bool bad;
    linear_rows(P, s, b, e, bad);
    const int segs = linear_segments(P, e - b);
    if (bad || segs == 1) return;
    int state = s;
    if (P.states) {
        if (P.a.state_indices) state = P.a.state_indices[s];
        if (state < 0 || state >= P.a.num_states) return;
    }
    const int item0 = linear_first_item(P, s);
    if (item0 + segs > P.items) return;              // (left out, as in linear_item)
    const int KV = P.a.K * P.a.V, at = (blockIdx.z * 256 + threadIdx.x) * 4;
    if (at >= KV) return;
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.start) run = *reinterpret_cast<const float4 *>(p.start + ((size_t)state * P.a.HV + hv) * KV + at);
    // four segments' states at a time on their way
    for (int j0 = 0; j0 < segs; j0 += 4) {
        float4 own[4];
        float f[4];
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
            const float g = exp2f(f[j]);
            *l[j] = run;
            run = make_float4(fmaf(g, run.x, own[j].x), fmaf(g, run.y, own[j].y), fmaf(g, run.z, own[j].z), fmaf(g, run.w, own[j].w));
        }
    }
}

// A warp per token and q/k head: the sum over the value heads that share it, and each one's product with `with`.
constexpr int kFoldRows = 64;          // token rows of a segment per CTA
template <typename Tin>
__global__ void __launch_bounds__(256) linear_fold_kernel(const __grid_constant__ LinearLaunch P, const __grid_constant__ LinearFold f)
{
    const int lane = threadIdx.x & 31, h = blockIdx.y, K = P.a.K, G = P.a.HV / P.a.H;
    const LinearItem it = linear_item(P, blockIdx.x, false);
    if (it.seq < 0) return;
    const int last = min(it.n, ((int)blockIdx.z + 1) * kFoldRows);
    for (int r = blockIdx.z * kFoldRows + (threadIdx.x >> 5); r < last; r += 8) {
        const int64_t t = it.begin + r;
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
    const LinearItem it = linear_item(P, blockIdx.x, false);
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

// dg of one decay a head: the ranges' sums of every segment, in order
__global__ void __launch_bounds__(256) linear_dg_fixed_kernel(const float *part, int rows, int HV, float *dg)
{
    const int hv = blockIdx.x;
    __shared__ double sums[8];
    double s = 0.0;
    for (int r = threadIdx.x; r < rows; r += 256) s += part[(size_t)r * HV + hv];
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
__global__ void __launch_bounds__(256) linear_dg_chunk_kernel(const __grid_constant__ LinearLaunch P, const float *qdq, const float *kdk,
                                                           const float *chunk_dot, float *dg, int64_t dg_stride, float *part)
{
    const int i = threadIdx.x & 31, range = threadIdx.x >> 5, hv = blockIdx.z * 32 + i, HV = P.a.HV;
    __shared__ float sums[8][32];
    const LinearItem it = linear_item(P, blockIdx.x, false);
    const int at = it.begin + blockIdx.y * kLinearChunk, rows = min(kLinearChunk, it.begin + it.n - at);
    if (it.seq < 0 || rows <= 0) return;
    const bool mine = hv < HV && it.state >= 0;
    const int first = 16 * range, last = min(rows, first + 16);
    const size_t chunk = (size_t)(at / kLinearChunk + it.seq) * HV + hv;
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
        for (int k = 0; k < 8; ++k) run += chunk_dot[chunk * 8 + k];
    for (int r = 7; r > range; --r) run += sums[r][i];
    const bool fixed = P.a.g_stride == 0;
#pragma unroll
    for (int k = 15; k >= 0; --k) {
        run += d[k];
        if (first + k >= last) continue;
        if (fixed) total += run;
        else dg[(int64_t)(at + first + k) * dg_stride + hv] = run;
    }
    if (fixed) {
        __syncwarp();
        part[chunk * 8 + range] = total;
    }
}

// dg of one decay a head: every chunk's parts, in order
__global__ void __launch_bounds__(256) linear_dg_chunk_fixed_kernel(const __grid_constant__ LinearLaunch P, const float *part, float *dg)
{
    const int hv = blockIdx.x;
    __shared__ double sums[8];
    double sum = 0.0;
    for (int s = 0; s < P.a.S; ++s) {
        int b, e;
        bool bad;
        linear_rows(P, s, b, e, bad);
        for (int k = threadIdx.x; k < (e - b + kLinearChunk - 1) / kLinearChunk * 8; k += 256)
            sum += part[((size_t)((b + (k >> 3) * kLinearChunk) / kLinearChunk + s) * P.a.HV + hv) * 8 + (k & 7)];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) sum += sums[w];
        dg[hv] = (float)sum;
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
    const dim3 grid((unsigned)P.a.S, (unsigned)P.a.HV, (unsigned)((P.a.K * P.a.V + 1023) / 1024));
    linear_carry_kernel<<<grid, 256, 0, stream>>>(P, p);
    return status();
}

int launch_linear_fold(const LinearLaunch &P, const LinearFold &f, cudaStream_t stream)
{
    const dim3 grid((unsigned)P.items, (unsigned)P.a.H, (unsigned)((P.seg + kFoldRows - 1) / kFoldRows));
    if (P.a.in_dtype == GDN_BF16) linear_fold_kernel<bf16><<<grid, 256, 0, stream>>>(P, f);
    else linear_fold_kernel<float><<<grid, 256, 0, stream>>>(P, f);
    return status();
}

int launch_linear_dg(const LinearLaunch &P, const float *qdq, const float *kdk, const float *segment_dot, int parts, float *dg,
                     int64_t dg_stride, float *part, cudaStream_t stream)
{
    const dim3 grid((unsigned)P.items, (unsigned)((P.a.HV + kDgHeads - 1) / kDgHeads));
    linear_dg_kernel<<<grid, kDgHeads * kDgRanges, 0, stream>>>(P, qdq, kdk, segment_dot, parts, dg, dg_stride, part);
    if (P.a.g_stride == 0) linear_dg_fixed_kernel<<<P.a.HV, 256, 0, stream>>>(part, P.items * kDgRanges, P.a.HV, dg);
    return status();
}

int launch_linear_dg_chunks(const LinearLaunch &P, const float *qdq, const float *kdk, const float *chunk_dot, float *dg,
                            int64_t dg_stride, float *part, cudaStream_t stream)
{
    const dim3 grid((unsigned)P.items, (unsigned)((P.seg + kLinearChunk - 1) / kLinearChunk), (unsigned)((P.a.HV + 31) / 32));
    linear_dg_chunk_kernel<<<grid, 256, 0, stream>>>(P, qdq, kdk, chunk_dot, dg, dg_stride, part);
    if (P.a.g_stride == 0) linear_dg_chunk_fixed_kernel<<<P.a.HV, 256, 0, stream>>>(P, part, dg);
    return status();
}

}  // namespace gdn
