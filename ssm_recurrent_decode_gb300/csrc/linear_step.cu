// linear_step.cu -- the single-token step of linear attention (gdn_linear_attention_step).
//
// The layout of step_kernel.cu without the delta rule: a state row of K values is read by K / 4 lanes, a CTA of eight
// warps takes 8 R rows per pass and lane group, and 1 to 8 CTAs share a (row, value head) tile. One pass over the state: with e = exp(g)
//     out = scale (e S q + v (k . q))     S <- e S + v k^T
// so the row dots use the values as they are read. Memory-bound: the state is read and written once. With rotary
// positions a CTA computes the head's cosines and sines once, in shared memory, while its state loads are under way.
#include <cmath>

#include "gdn_chain.cuh"
#include "gdn_linear.h"
#include "gdn_tile.cuh"
#include "rotary.cuh"

namespace gdn {

namespace {

struct LinearStepLaunch {
    gdn_linear_step_args a;
    const int32_t *idx;
    int32_t pad;
    float scale, magnitude;
    int wide;             // q and k may be read four elements at a time
};

// four channels of a q or k head, and the other members of their pairs
struct Head4 {
    float v[4], other[4];
};
template <typename Tin> __device__ __forceinline__ Head4 load_head(const gdn_linear_step_args &a, const Tin *x, int col, bool wide)
{
    Head4 h;
    if (wide) {
        const float4 x4 = load4(x + col);
        h.v[0] = x4.x, h.v[1] = x4.y, h.v[2] = x4.z, h.v[3] = x4.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h.v[i] = to_f32(x[col + i]);
    }
    const int half = a.rotary_dim / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = col + i;
        const int other = a.interleaved ? c ^ 1 : c >= half ? c - half : c + half;
        h.other[i] = c < a.rotary_dim ? to_f32(x[other]) : 0.f;
    }
    return h;
}
// turned by the row's position
__device__ __forceinline__ float4 turn_head(const gdn_linear_step_args &a, const Head4 &h, int col, const float (*cs)[2])
{
    float v[4];
    const int half = a.rotary_dim / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = col + i;
        v[i] = h.v[i];
        if (c >= a.rotary_dim) continue;
        const int pair = a.interleaved ? c >> 1 : c < half ? c : c - half;
        const bool second = a.interleaved ? c & 1 : c >= half;
        v[i] = fmaf(second ? h.other[i] : -h.other[i], cs[pair][1], v[i] * cs[pair][0]);
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

template <int K, typename Tin, typename TS, int R>
__global__ void __launch_bounds__(kThreads, 4) linear_step_kernel(const __grid_constant__ LinearStepLaunch P, int splits)
{
    using TL = Tile<K, R>;
    using TR = Tile<K, R / 2>;               // reduces R row dots
    const gdn_linear_step_args &a = P.a;
    const int HV = a.HV, V = a.V;
    const int tile = blockIdx.x / splits, blk = blockIdx.x - tile * splits;
    const int b = tile / HV, hv = tile - b * HV, h = hv / (HV / a.H);
    const size_t out_base = ((size_t)b * HV + hv) * V;
    const int first_row = blk * TL::ROWS_PASS, row_step = splits * TL::ROWS_PASS;
    __shared__ float cs[K / 2][2];
    ordinary_launch_start();
    // (asked for before the state: their chain of loads is the longer one)
    int position = 0;
    uint64_t turns = 0;
    if ((int)threadIdx.x < a.rotary_dim / 2) {
        position = a.positions[b];
        turns = rotary_turns(a.frequencies[threadIdx.x]);
    }

    int slot = b;
    if (P.idx) {
        slot = P.idx[b];
        const bool pad = slot == P.pad;
        if (pad || slot < 0 || slot >= a.num_slots) {   // uniform over the CTA
            if (!pad && blk == 0 && threadIdx.x == 0) raise_flag(a.err_flags, GDN_DEVERR_BAD_INDEX);
            for (int r = threadIdx.x; r < V; r += kThreads)
                if ((r / TL::ROWS_PASS) % splits == blk) store_out(a.out, a.out_dtype, out_base + r, 0.f);
            return;
        }
    }
    if (!GDN_IN(a.err_flags, ((long long)slot * HV + hv + 1) * V * K - 1, (long long)a.num_slots * HV * V * K)) return;
    TS *S = static_cast<TS *>(a.state) + ((size_t)slot * HV + hv) * (size_t)V * K;
    TL t;
    t.init();
    t.load(S, V, first_row);
    const Tin *qp = static_cast<const Tin *>(a.q) + b * a.q_stride + h * a.q_head_stride;
    const Tin *kp = static_cast<const Tin *>(a.k) + b * a.k_stride + h * a.k_head_stride;
    const Tin *vp = static_cast<const Tin *>(a.v) + b * a.v_stride + hv * a.v_head_stride;
    const Head4 qh = load_head<Tin>(a, qp, t.col, P.wide), kh = load_head<Tin>(a, kp, t.col, P.wide);
    const float e = expf(a.g[b * a.g_stride + hv]);
    if (a.rotary_dim > 0) {
        if ((int)threadIdx.x < a.rotary_dim / 2) {
            float c, s;
            rotary_cos_sin(position, turns, c, s);
            cs[threadIdx.x][0] = c * P.magnitude;
            cs[threadIdx.x][1] = s * P.magnitude;
        }
        __syncthreads();
    }
    const float4 q4 = scale4(turn_head(a, qh, t.col, cs), P.scale), k4 = turn_head(a, kh, t.col, cs);
    const float kq = group_sum<TL::LPR>(dot4(k4, q4));

    for (int row0 = first_row; row0 < V; row0 += row_step) {
        if (row0 != first_row) t.load(S, V, row0);
        float vv[R], x[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = t.row(row0, i);
            vv[i] = r < V ? to_f32(vp[r]) : 0.f;
            x[i] = dot4(t.s[i], q4);
        }
        TR tr;
        tr.init();
        tr.reduce_scatter(x);
        // lane `sub` of a row group holds the dots of rows (sub / DUP) M ..
#pragma unroll
        for (int m = 0; m < TR::M; ++m) {
            const int r = t.row(row0, (t.sub / TR::DUP) * TR::M + m);
            if (t.sub % TR::DUP == 0 && r < V) store_out(a.out, a.out_dtype, out_base + r, fmaf(e, x[m], to_f32(vp[r]) * kq));
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = t.row(row0, i);
            if (r < V) st_stream(S + (size_t)r * K + t.col, axpby4(e, t.s[i], vv[i], k4));
        }
    }
}

template <int K, typename Tin, typename TS, int R> int launch_rows(const LinearStepLaunch &p, cudaStream_t stream)
{
    const int splits = (p.a.V + Tile<K, R>::ROWS_PASS - 1) / Tile<K, R>::ROWS_PASS;
    const unsigned grid = (unsigned)p.a.B * (unsigned)p.a.HV * (unsigned)splits;
    return launch_ordinary(linear_step_kernel<K, Tin, TS, R>, dim3(grid), dim3(kThreads), 0, stream, p, splits) == cudaSuccess
               ? GDN_OK : GDN_ERR_LAUNCH;
}

template <int K, typename Tin, typename TS> int launch_k(const LinearStepLaunch &p, cudaStream_t stream)
{
    // enough CTAs for four per SM, with as many rows each as that leaves
    const int64_t tiles = (int64_t)p.a.B * p.a.HV, target = 4 * 152;
    const auto ctas = [&](int rows) { return tiles * ((p.a.V + rows - 1) / rows); };
    if (ctas(Tile<K, 8>::ROWS_PASS) >= target) return launch_rows<K, Tin, TS, 8>(p, stream);
    if (ctas(Tile<K, 4>::ROWS_PASS) >= target) return launch_rows<K, Tin, TS, 4>(p, stream);
    return launch_rows<K, Tin, TS, 2>(p, stream);
}

template <typename Tin, typename TS> int launch_t(const LinearStepLaunch &p, cudaStream_t stream)
{
    switch (p.a.K) {
    case 16: return launch_k<16, Tin, TS>(p, stream);
    case 32: return launch_k<32, Tin, TS>(p, stream);
    case 64: return launch_k<64, Tin, TS>(p, stream);
    default: return launch_k<128, Tin, TS>(p, stream);
    }
}

}  // namespace

}  // namespace gdn

extern "C" int gdn_linear_attention_step(const gdn_linear_step_args *args, const int32_t *cache_indices, int32_t pad_slot_id,
                                         gdn_stream_t stream)
{
    if (!args) return GDN_ERR_NULL;
    const gdn_linear_step_args &a = *args;
    const auto aligned = [](const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const auto dtype_ok = [](int d) { return d == GDN_F32 || d == GDN_BF16; };
    if (a.B < 0 || a.H < 1 || a.HV < 1 || a.HV % a.H || a.num_slots < 1) return GDN_ERR_SHAPE;
    if ((a.K != 16 && a.K != 32 && a.K != 64 && a.K != 128) || a.V < 1 || a.V > 1024) return GDN_ERR_SHAPE;
    if ((int64_t)a.B * a.HV * ((a.V + 15) / 16) > INT32_MAX) return GDN_ERR_SHAPE;
    if (!dtype_ok(a.in_dtype) || !dtype_ok(a.out_dtype) || !dtype_ok(a.state_dtype)) return GDN_ERR_DTYPE;
    if (a.rotary_dim < 0 || a.rotary_dim > a.K || a.rotary_dim % 2) return GDN_ERR_SHAPE;
    if (!cache_indices && a.num_slots < a.B) return GDN_ERR_SHAPE;
    if (a.B == 0) return GDN_OK;
    if (!a.q || !a.k || !a.v || !a.g || !a.state || !a.out || (a.rotary_dim && (!a.positions || !a.frequencies))) return GDN_ERR_NULL;
    for (int64_t s : {a.q_stride, a.q_head_stride, a.k_stride, a.k_head_stride, a.v_stride, a.v_head_stride, a.g_stride})
        if (s < 0) return GDN_ERR_SHAPE;
    const size_t es = a.in_dtype == GDN_BF16 ? 2 : 4;
    if (!aligned(a.q, es) || !aligned(a.k, es) || !aligned(a.v, es) || !aligned(a.g, 4) || !aligned(a.state, 16) ||
        !aligned(a.out, a.out_dtype == GDN_BF16 ? 2 : 4) || !aligned(cache_indices, 4) || !aligned(a.positions, 4) ||
        !aligned(a.frequencies, 8))
        return GDN_ERR_ALIGN;
    gdn::LinearStepLaunch p = {};
    p.a = a;
    p.idx = cache_indices;
    p.pad = pad_slot_id;
    p.scale = a.scale != 0.f ? a.scale : 1.0f / std::sqrt((float)a.K);
    p.magnitude = a.magnitude != 0.f ? a.magnitude : 1.f;
    p.wide = aligned(a.q, 4 * es) && aligned(a.k, 4 * es) && a.q_stride % 4 == 0 && a.k_stride % 4 == 0 && a.q_head_stride % 4 == 0 &&
             a.k_head_stride % 4 == 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    using gdn::bf16;
    if (a.state_dtype == GDN_BF16) return es == 2 ? gdn::launch_t<bf16, bf16>(p, s) : gdn::launch_t<float, bf16>(p, s);
    return es == 2 ? gdn::launch_t<bf16, float>(p, s) : gdn::launch_t<float, float>(p, s);
}
