// linear_recurrent.cu -- linear attention of fp32 inputs on the CUDA cores, token by token.
//
// A CTA owns one segment of a sequence, one value head and 64 columns of z; a thread keeps 16 x 2 entries of the state
// State[y, z] in registers: DY / 16 lanes side by side share two columns. A token costs every entry two multiply-adds,
// State += y z and out += State x; the decay costs none: the state is kept times the decay up to a reference token ahead
// (2^-held, held >= 0), z is multiplied by it as it is staged and out divided. So what is kept is never above the state itself, and
// below it by no more than 2^40, in a block of 16 tokens that decays by less than 16 octaves no more than 2^21: neither end of
// fp32's range comes nearer than that. (Kept divided by the decay since a token behind, products above 2^48 overflowed.)
// The reference moves by whole octaves, which is exact, and a block that decays by more than 28 octaves in itself, or grows by
// more than five, is taken with one more product an entry and token instead. Log decays are summed in 64 bits, so a
// long memory loses nothing to rounded factors near one.
// x, y (broadcast within a column pair's lanes) and z come from shared memory, 16 tokens at a time, the next 16
// already on their way in registers.
//
// 2 K V multiply-adds a token and head (33 k at K = V = 128) against 128 a clock and SM, 80 TFLOP/s in all. 64 x 4096 tokens of 16 heads,
// which fill the machine, reach 16 of them: 4.1 ms, the multiply-add pipe active 32% of the time, half of the issue slots used, two CTAs of
// eight warps an SM by their registers; a token's operands come from shared memory with little to cover their latency. Short calls
// (3 x 777 tokens of 12 heads: 69 us, 5 TFLOP/s) are bound by the latency of some 50 tokens one after the other, twice.
#include "gdn_chain.cuh"
#include "linear_common.cuh"

namespace gdn {

namespace {

constexpr int kBlock = 16;             // tokens staged together

template <int NY> struct Geometry {
    static constexpr int kLanes = NY / 16;                     // lanes that share two columns
    static constexpr int kThreads = 32 * kLanes;               // kLinearZ columns, two a lane group
};

template <int NY, bool OUT>
__global__ void __launch_bounds__(Geometry<NY>::kThreads) linear_recurrent_kernel(const __grid_constant__ LinearLaunch P,
                                                                                 const __grid_constant__ LinearSweep p)
{
    using G = Geometry<NY>;
    constexpr int YS = G::kLanes, NT = G::kThreads;
    constexpr int EX = kBlock * NY / NT, EZ = kBlock * kLinearZ / NT;          // elements staged by a thread
    __shared__ __align__(16) float sx[2][kBlock][NY], sy[2][kBlock][NY], sz[2][kBlock][kLinearZ];
    __shared__ float so[OUT ? kBlock : 1][kLinearZ];
    __shared__ float s_in[2][kBlock], s_out[2][kBlock], s_first[2], s_z[2];
    __shared__ int s_each[2];
    __shared__ LinearItem s_item;
    __shared__ LinearScan s_scan;
    __shared__ float s_last;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hv = blockIdx.y, zpart = blockIdx.z, z0 = zpart * kLinearZ;
    linear_find<NT>(P, blockIdx.x, !OUT, OUT && hv == 0 && zpart == 0, 0, s_scan, &s_item);
    const LinearItem it = s_item;
    if (it.seq < 0 || !linear_in(P, it)) return;
    const bool whole = it.seq_end - it.seq_begin <= P.seg;                     // the sequence's only segment
    if (!OUT && (whole || it.state < 0)) return;
    const size_t item_state = ((size_t)it.slot * P.a.HV + hv) * ((size_t)P.a.K * P.a.V);
    const int n = it.n;
    const bool skip = it.state < 0;                                            // a bad state index: outputs zeroed

    const int sub = tid % YS, col = (tid / YS) * 2;                            // this thread's columns col, col + 1
    const auto y_of = [&](int i) { return (i >> 2) * (4 * YS) + sub * 4 + (i & 3); };
    float S[16][2];
    {
        const float *from = nullptr;
        if (OUT && !skip) {
            if (!whole) from = P.local + item_state;
            else if (p.start) from = p.start + ((size_t)it.state * P.a.HV + hv) * ((size_t)P.a.K * P.a.V);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int y = y_of(i), z = z0 + col + j;
                S[i][j] = from && y < p.DY && z < p.DZ ? from[y * p.sy + z * p.sz] : 0.f;
            }
    }

    // dg's boundary terms: the product of the state's gradient, as it reaches the segment's last row, and the state behind it
    const size_t kept = (((size_t)blockIdx.x * P.a.HV + hv) * gridDim.z + zpart) * (32 * NT) + tid;
    if (OUT && p.chunk_dot) {
        float d = 0.f;
        if (!skip)
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) d = fmaf(S[i][j], p.chunk_states[kept + (2 * i + j) * NT], d);
        d = group_sum<32>(d);
        if (lane == 0) so[0][warp] = d;
        __syncthreads();
        if (tid == 0) {
            float sum = 0.f;
            for (int w = 0; w < NT / 32; ++w) sum += so[0][w];
            bool nan = false;
            const int next = it.begin + n;
            const float g = next < it.seq_end ? linear_exp2(linear_fixed(P.a.g[next * P.a.g_stride + hv], nan)) : 1.f;
            p.chunk_dot[((size_t)blockIdx.x * P.a.HV + hv) * gridDim.z + zpart] = nan ? __int_as_float(0x7fc00000) : sum * g;
        }
        __syncthreads();
    }

    const float *xp = OUT ? static_cast<const float *>(p.x) + (int64_t)(hv / p.x_group) * p.x_head : nullptr;
    const float *yp = static_cast<const float *>(p.y) + (int64_t)(hv / p.y_group) * p.y_head;
    const float *zp = static_cast<const float *>(p.z) + (int64_t)(hv / p.z_group) * p.z_head;
    const int first = p.reverse ? it.begin + n - 1 : it.begin, dir = p.reverse ? -1 : 1;
    float rx[OUT ? EX : 1], ry[EX], rz[EZ];
    const auto fetch = [&](int block) {
#pragma unroll
        for (int i = 0; i < EX; ++i) {
            const int e = tid + i * NT, r = block * kBlock + e / NY, c = e % NY;
            const int64_t t = first + (int64_t)dir * r;
            const bool in = r < n && c < p.DY && linear_in(P, (int)t, hv, P.a.HV);
            ry[i] = in ? yp[t * p.y_stride + c] : 0.f;
            if (OUT) rx[i] = in ? xp[t * p.x_stride + c] * p.x_scale : 0.f;
        }
#pragma unroll
        for (int i = 0; i < EZ; ++i) {
            const int e = tid + i * NT, r = block * kBlock + e / kLinearZ, c = z0 + e % kLinearZ;
            const int64_t t = first + (int64_t)dir * r;
            rz[i] = r < n && c < p.DZ && linear_in(P, (int)t, hv, P.a.HV) ? zp[t * p.z_stride + c] * p.z_scale : 0.f;
        }
    };
    const auto put = [&](int b) {
#pragma unroll
        for (int i = 0; i < EX; ++i) {
            const int e = tid + i * NT;
            sy[b][e / NY][e % NY] = ry[i];
            if (OUT) sx[b][e / NY][e % NY] = rx[i];
        }
#pragma unroll
        for (int i = 0; i < EZ; ++i) {
            const int e = tid + i * NT;
            sz[b][e / kLinearZ][e % kLinearZ] = rz[i];
        }
    };
    // warp 0: the factors of a block's tokens; held: -log2 of the decay up to the reference token (steps of 2^-40)
    constexpr long long kOne = 1ll << 40;
    long long held = 0;
    double all = 0.0;                                                          // of the whole segment: its steps would pass 64 bits after 29000
                                                                               // tokens of the largest decay
    bool lost = false;                                                         // a NaN came
    const auto factors = [&](int block, int b) {
        const int r = block * kBlock + lane;
        bool nan = false;
        long long s = 0;
        if (lane < kBlock && r < n) {
            const int t = first + dir * r + (p.reverse ? 1 : 0);
            if (t < it.seq_end) s = linear_fixed(P.a.g[t * P.a.g_stride + hv], nan);
        }
        const long long own = s;
#pragma unroll
        for (int o = 1; o < kBlock; o <<= 1) {
            const long long v = __shfl_up_sync(kAll, s, o);
            if (lane >= o) s += v;
        }
        const unsigned nans = __ballot_sync(kAll, nan);
        const bool gone = lost || (nans & ((2u << lane) - 1));                  // (it leaves the tokens before it alone)
        const long long span = __shfl_sync(kAll, s, kBlock - 1);
        // the lowest and highest sum in octaves (the highest to the next one)
        const int octaves = lane < kBlock ? (int)(s >> 40) : 0;
        const int low = min(0, __reduce_min_sync(kAll, octaves)), high = max(0, __reduce_max_sync(kAll, octaves)) + 1;
        const bool each = low < -28 || high > 5;
        int move = 0;                                                          // of the reference, in octaves
        if (each) move = -(int)(held >> 40);
        else if (held + low * kOne < 0 || held + high * kOne > 40 * kOne) move = (int)(((4 - low) * kOne - held + kOne - 1) >> 40);
        held += move * kOne;
        const float none = __int_as_float(0x7fc00000);
        if (lane < kBlock) {
            s_in[b][lane] = gone ? none : linear_exp2(each ? own : -(held + s));
            s_out[b][lane] = linear_exp2(each ? held : held + s);
        }
        if (lane == 0) {
            s_first[b] = __int_as_float((127 - move) << 23);
            s_z[b] = linear_exp2(-held);
            s_each[b] = each;
        }
        if (!each) held += span;
        if (!OUT) all += (double)span * 0x1p-40;
        lost = lost || nans;
    };

    const int blocks = (n + kBlock - 1) / kBlock;
    if (blocks > 0) {
        fetch(0);
        if (warp == 0) factors(0, 0);
        put(0);
    }
    __syncthreads();
    for (int k = 0; k < blocks; ++k) {
        const int b = k & 1, rows = min(kBlock, n - k * kBlock);
        if (k + 1 < blocks) fetch(k + 1);
        const bool each = s_each[b];
        const float f = s_first[b], block_z = s_z[b];
        if (f != 1.f)
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i][0] *= f, S[i][1] *= f;
        for (int r = 0; r < rows; ++r) {
            const float fin = s_in[b][r];
            float2 z = *reinterpret_cast<const float2 *>(&sz[b][r][col]);
            if (each) {
#pragma unroll
                for (int i = 0; i < 16; ++i) S[i][0] *= fin, S[i][1] *= fin;
            }
            const float fz = each ? block_z : fin;
            z.x *= fz;
            z.y *= fz;
            float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 y4 = *reinterpret_cast<const float4 *>(&sy[b][r][q * (4 * YS) + sub * 4]);
                const float yy[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    S[4 * q + i][0] = fmaf(yy[i], z.x, S[4 * q + i][0]);
                    S[4 * q + i][1] = fmaf(yy[i], z.y, S[4 * q + i][1]);
                }
                if (OUT) {
                    const float4 x4 = *reinterpret_cast<const float4 *>(&sx[b][r][q * (4 * YS) + sub * 4]);
                    const float xx[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[0][i & 1] = fmaf(xx[i], S[4 * q + i][0], acc[0][i & 1]);
                        acc[1][i & 1] = fmaf(xx[i], S[4 * q + i][1], acc[1][i & 1]);
                    }
                }
            }
            if (OUT) {
                float o0 = acc[0][0] + acc[0][1], o1 = acc[1][0] + acc[1][1];
                const float d = s_out[b][r];
                if constexpr (YS > 1) {
                    // an even lane keeps the first column's sum, an odd one the second's
                    const bool odd = lane & 1;
                    const float give = odd ? o0 : o1;
                    float o = (odd ? o1 : o0) + __shfl_xor_sync(kAll, give, 1);
#pragma unroll
                    for (int m = 2; m < YS; m <<= 1) o += __shfl_xor_sync(kAll, o, m);
                    if (sub < 2) so[r][col + sub] = o * d;
                } else {
                    so[r][col] = o0 * d;
                    so[r][col + 1] = o1 * d;
                }
            }
        }
        if (k + 1 < blocks) {
            put(b ^ 1);
            if (warp == 0) factors(k + 1, b ^ 1);
        }
        __syncthreads();
        if (OUT) {
#pragma unroll
            for (int i = 0; i < EZ; ++i) {
                const int e = tid + i * NT, r = e / kLinearZ, c = e % kLinearZ;
                if (p.out && r < rows && z0 + c < p.DZ) {
                    const int64_t t = first + (int64_t)dir * (k * kBlock + r);
                    if (!linear_in(P, (int)t, hv, P.a.HV)) continue;
                    const int64_t at = t * p.out_stride + (int64_t)hv * p.out_head + z0 + c;
                    const float v = skip ? 0.f : so[r][c];
                    if (p.out_f32) static_cast<float *>(p.out)[at] = v;
                    else static_cast<bf16 *>(p.out)[at] = __float2bfloat16_rn(v);
                }
            }
            __syncthreads();
        }
    }

    // the state as it is: divided by the decay up to the reference token
    if (tid == 0) s_last = lost ? __int_as_float(0x7fc00000) : linear_exp2(held);
    __syncthreads();
    float f = s_last;
    const bool ends = p.reverse ? it.index == 0 : it.begin + n == it.seq_end;  // the sequence's last segment, in the sweep's order
    float *to = nullptr;
    if (!OUT) {
        to = P.local + item_state;
        if (tid == 0 && zpart == 0) P.total[(size_t)it.slot * P.a.HV + hv] = linear_parts(lost ? (double)__int_as_float(0x7fc00000) : all);
    } else if (ends && !skip && p.end) {
        to = p.end + ((size_t)it.state * P.a.HV + hv) * ((size_t)P.a.K * P.a.V);
    }
    if (to) {
        // backwards the state's gradient passes the first token's decay too
        const float pass = OUT && p.reverse && it.seq_end > it.seq_begin ? exp2_wide(linear_log2(P.a.g[it.seq_begin * P.a.g_stride + hv])) : 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int y = y_of(i), z = z0 + col + j;
                if (y < p.DY && z < p.DZ) to[y * p.sy + z * p.sz] = S[i][j] * f * pass;
            }
    }
    if (OUT && p.chunk_states && !p.chunk_dot)
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) p.chunk_states[kept + (2 * i + j) * NT] = S[i][j] * f;
}

template <int NY>
cudaError_t launch(const LinearLaunch &P, const LinearSweep &p, bool outputs, cudaStream_t stream)
{
    const dim3 grid((unsigned)(outputs ? P.items : P.cut_items), (unsigned)P.a.HV, (unsigned)((p.DZ + kLinearZ - 1) / kLinearZ));
    if (outputs) linear_recurrent_kernel<NY, true><<<grid, Geometry<NY>::kThreads, 0, stream>>>(P, p);
    else linear_recurrent_kernel<NY, false><<<grid, Geometry<NY>::kThreads, 0, stream>>>(P, p);
    return cudaGetLastError();
}

cudaError_t launch_y(const LinearLaunch &P, const LinearSweep &p, bool outputs, cudaStream_t stream)
{
    if (p.DY <= 16) return launch<16>(P, p, outputs, stream);
    if (p.DY <= 32) return launch<32>(P, p, outputs, stream);
    if (p.DY <= 64) return launch<64>(P, p, outputs, stream);
    return launch<128>(P, p, outputs, stream);
}

}  // namespace

int launch_linear_recurrent(const LinearLaunch &P, const LinearSweep &p, bool outputs, cudaStream_t stream)
{
    return launch_y(P, p, outputs, stream) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace gdn
