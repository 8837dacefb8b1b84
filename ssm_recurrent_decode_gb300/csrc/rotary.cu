// rotary.cu -- rotary positions of q and k (gdn_rotary).
//
// A thread owns a vector of pairs (16 bytes of each channel range where pointers, strides and sizes allow, else single
// pairs) of one token and walks over heads, so that a pair's cosine and sine are computed once for all its heads. Memory-bound:
// each element is read and written once. The channels behind rotary_dim are copied by threads of their own, unless
// the call works in place.
#include "gdn_chain.cuh"
#include "gdn_common.cuh"
#include "gdn_rotary.h"
#include "rotary.cuh"

namespace gdn {

namespace {

struct RotaryLaunch {
    gdn_rotary_args a;
    float magnitude;
    int pairs;            // threads of a token and head group that turn; behind them those that copy
    int threads;          // both
    int heads;            // heads per thread
    int groups;           // head groups (of q and k together) per token
};

template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Vec { T v[VEC]; };

// VEC elements a vector; halves: a pair's members lie in two vectors, interleaved: side by side in one
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryLaunch R)
{
    using W = Vec<T, VEC>;
    constexpr int NP = INTER ? (VEC + 1) / 2 : VEC;                // pairs a thread turns
    const gdn_rotary_args &a = R.a;
    ordinary_launch_start();
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t tg = u / R.threads;
    const int j = (int)(u - tg * R.threads);
    const int64_t t = tg / R.groups;
    const int group = (int)(tg - t * R.groups);
    if (t >= a.T) return;
    const bool turn = j < R.pairs;
    // first channel of this thread's vector, and of its pairs' other members
    const int half = a.rotary_dim / 2;
    const int c0 = turn ? (INTER ? (VEC == 1 ? 2 * j : VEC * j) : VEC * j) : a.rotary_dim + VEC * (j - R.pairs);
    const int c1 = INTER ? c0 + 1 : c0 + half;                      // (interleaved: only where VEC is 1)
    float cs[NP], sn[NP];
    if (turn) {
        const int pos = a.positions[t];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            rotary_cos_sin(pos, rotary_turns(a.frequencies[(INTER ? c0 / 2 : c0) + i]), cs[i], sn[i]);
            cs[i] *= R.magnitude;
            sn[i] *= a.inverse ? -R.magnitude : R.magnitude;
        }
    }
    const int last = min(a.H + a.HK, (group + 1) * R.heads);
    // four heads' vectors are asked for before any is written (an output may be its input's memory, so the compiler keeps
    // the order: 16384 tokens x 48 heads of 128 in bf16 100 us one at a time, SUBST four)
    constexpr int NH = 4;
    constexpr bool kTwo = !(INTER && VEC > 1);
    for (int head0 = group * R.heads; head0 < last; head0 += NH) {
        W x[NH], y[kTwo ? NH : 1];
        T *out[NH];
#pragma unroll
        for (int k = 0; k < NH; ++k) {
            const int head = min(head0 + k, last - 1);
            const bool isq = head < a.H;
            const T *in = isq ? static_cast<const T *>(a.q) + t * a.q_stride + (int64_t)head * a.q_head_stride
                              : static_cast<const T *>(a.k) + t * a.k_stride + (int64_t)(head - a.H) * a.k_head_stride;
            out[k] = isq ? static_cast<T *>(a.q_out) + t * a.q_out_stride + (int64_t)head * a.q_out_head_stride
                         : static_cast<T *>(a.k_out) + t * a.k_out_stride + (int64_t)(head - a.H) * a.k_out_head_stride;
            x[k] = *reinterpret_cast<const W *>(in + c0);
            if (kTwo && turn) y[kTwo ? k : 0] = *reinterpret_cast<const W *>(in + c1);
        }
#pragma unroll
        for (int k = 0; k < NH; ++k) {
            if (head0 + k >= last) break;
            if (turn) {
                if constexpr (!kTwo) {
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const float p = to_f32(x[k].v[2 * i]), q = to_f32(x[k].v[2 * i + 1]);
                        x[k].v[2 * i] = from_f32<T>(p * cs[i] - q * sn[i]);
                        x[k].v[2 * i + 1] = from_f32<T>(q * cs[i] + p * sn[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const float p = to_f32(x[k].v[i]), q = to_f32(y[k].v[i]);
                        x[k].v[i] = from_f32<T>(p * cs[i] - q * sn[i]);
                        y[k].v[i] = from_f32<T>(q * cs[i] + p * sn[i]);
                    }
                    *reinterpret_cast<W *>(out[k] + c1) = y[k];
                }
            }
            *reinterpret_cast<W *>(out[k] + c0) = x[k];
        }
    }
}

template <typename T, int VEC, bool INTER> int launch(RotaryLaunch &R, cudaStream_t stream)
{
    const gdn_rotary_args &a = R.a;
    const bool in_place = a.q == a.q_out && (a.HK == 0 || a.k == a.k_out);
    R.pairs = INTER ? (VEC == 1 ? a.rotary_dim / 2 : a.rotary_dim / VEC) : a.rotary_dim / 2 / VEC;
    R.threads = R.pairs + (in_place ? 0 : (a.D - a.rotary_dim) / VEC);
    // Heads per thread: as many as leave every SM a full complement of threads, so that few threads repeat a pair's
    // cosine and sine.
    const int heads = a.H + a.HK;
    R.heads = 1;
    while (R.heads < 16 && R.heads < heads && (int64_t)a.T * R.threads * ((heads + 2 * R.heads - 1) / (2 * R.heads)) >= 152 * 2048) R.heads *= 2;
    R.groups = (heads + R.heads - 1) / R.heads;
    const int64_t n = (int64_t)a.T * R.groups * R.threads;
    const int64_t grid = (n + 255) / 256;
    if (grid > INT32_MAX) return GDN_ERR_SHAPE;
    return launch_ordinary(rotary_kernel<T, VEC, INTER>, dim3((unsigned)grid), dim3(256), 0, stream, R) == cudaSuccess ? GDN_OK
                                                                                                                    : GDN_ERR_LAUNCH;
}

template <typename T> int launch_t(RotaryLaunch &R, bool vec, cudaStream_t stream)
{
    constexpr int N = 16 / sizeof(T);
    if (R.a.interleaved) return vec ? launch<T, N, true>(R, stream) : launch<T, 1, true>(R, stream);
    return vec ? launch<T, N, false>(R, stream) : launch<T, 1, false>(R, stream);
}

}  // namespace

}  // namespace gdn

extern "C" int gdn_rotary(const gdn_rotary_args *args, gdn_stream_t stream)
{
    if (!args) return GDN_ERR_NULL;
    const gdn_rotary_args &a = *args;
    if (a.T < 0 || a.H < 1 || a.HK < 0 || (int64_t)a.H + a.HK > 65535 || a.D < 2 || a.D > 1024) return GDN_ERR_SHAPE;
    if (a.rotary_dim < 2 || a.rotary_dim > a.D || a.rotary_dim % 2) return GDN_ERR_SHAPE;
    if (a.dtype != GDN_F32 && a.dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (a.T == 0) return GDN_OK;
    if (!a.positions || !a.frequencies || !a.q || !a.q_out || (a.HK && (!a.k || !a.k_out))) return GDN_ERR_NULL;
    const int es = a.dtype == GDN_BF16 ? 2 : 4;
    const auto aligned = [](const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    if (!aligned(a.positions, 4) || !aligned(a.frequencies, 8)) return GDN_ERR_ALIGN;
    bool vec = a.D * es % 16 == 0 && a.rotary_dim * es % (a.interleaved ? 16 : 32) == 0;
    const auto tensor = [&](const void *p, int64_t stride, int64_t head, bool output, int heads) {
        if (!aligned(p, es)) return GDN_ERR_ALIGN;
        if (stride < 0 || head < 0) return GDN_ERR_SHAPE;
        // rows and heads of an output may not overlap
        if (output) {
            const bool rows = a.T == 1 || stride >= (heads > 1 ? (heads - 1) * head : 0) + a.D, in_row = heads == 1 || head >= a.D;
            const bool planes = heads == 1 || head >= (a.T - 1) * stride + a.D, in_plane = a.T == 1 || stride >= a.D;
            if (!(rows && in_row) && !(planes && in_plane)) return GDN_ERR_SHAPE;
        }
        if (!aligned(p, 16) || (a.T > 1 && stride * es % 16) || (heads > 1 && head * es % 16)) vec = false;
        return GDN_OK;
    };
    int rc = tensor(a.q, a.q_stride, a.q_head_stride, false, a.H);
    if (rc == GDN_OK) rc = tensor(a.q_out, a.q_out_stride, a.q_out_head_stride, true, a.H);
    if (rc == GDN_OK && a.HK) rc = tensor(a.k, a.k_stride, a.k_head_stride, false, a.HK);
    if (rc == GDN_OK && a.HK) rc = tensor(a.k_out, a.k_out_stride, a.k_out_head_stride, true, a.HK);
    if (rc != GDN_OK) return rc;
    // in place is the same rows; another layout over the same memory would be read after it was written
    if (a.q == a.q_out && (a.q_stride != a.q_out_stride || a.q_head_stride != a.q_out_head_stride)) return GDN_ERR_ARG;
    if (a.HK && a.k == a.k_out && (a.k_stride != a.k_out_stride || a.k_head_stride != a.k_out_head_stride)) return GDN_ERR_ARG;
    gdn::RotaryLaunch R = {};
    R.a = a;
    R.magnitude = a.magnitude != 0.f ? a.magnitude : 1.f;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return es == 2 ? gdn::launch_t<gdn::bf16>(R, vec, s) : gdn::launch_t<float>(R, vec, s);
}
