// rotary.cu -- rotary positions of q and k (gdn_rotary).
//
// A CTA takes a few tokens: their cosines and sines go to shared memory, once for all heads, then its threads walk over the
// tokens' heads in the order of memory, a vector of pairs each (16 bytes of each channel range where pointers, strides and sizes
// allow, else two elements, else one). Memory-bound: each element is read and written once. The channels behind rotary_dim are
// copied, unless the call works in place.
#include "gdn_chain.cuh"
#include "gdn_common.cuh"
#include "gdn_rotary.h"
#include "rotary.cuh"

namespace gdn {

namespace {

// One vector a thread at a time and six CTAs an SM (16384 tokens x 48 heads of 128 in bf16, 403 MB: 70 us, 0.85 of the copy rate;
// two vectors and four CTAs 81, four and two 115; a thread that kept its pairs' angles in registers and walked over the heads,
// whose warps touch rows 4 KB apart, 100 to 115).
constexpr int kThreads = 256, kResident = 6;

struct RotaryLaunch {
    gdn_rotary_args a;
    float magnitude;
    int pairs;            // vectors of a head that turn; behind them those that are copied
    int units;            // both
    int tokens;           // tokens per CTA
    int parts;            // CTAs (blockIdx.y) that share the tokens' vectors
};

template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Vec { T v[VEC]; };

// VEC elements a vector; halves: a pair's members lie in two vectors, interleaved: side by side in one (unless VEC is 1)
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads, kResident) rotary_kernel(const __grid_constant__ RotaryLaunch R)
{
    using W = Vec<T, VEC>;
    constexpr bool kTwo = !(INTER && VEC > 1);                     // two vectors
    constexpr int NP = kTwo ? VEC : VEC / 2;                       // pairs
    extern __shared__ float2 turned[];                             // [tokens, rotary_dim / 2] cosine, sine
    const gdn_rotary_args &a = R.a;
    ordinary_launch_start();
    const int half = a.rotary_dim / 2, heads = a.H + a.HK;
    const int64_t t0 = (int64_t)blockIdx.x * R.tokens;
    const int tokens = (int)min((int64_t)R.tokens, a.T - t0);
    // this thread's next vector, and the step to the one behind it
    const int first = blockIdx.y * kThreads + threadIdx.x, step = R.parts * kThreads;
    int u = first % R.units, head = first / R.units % heads, tk = first / R.units / heads;
    const int du = step % R.units, dh = step / R.units % heads, dt = step / R.units / heads;
    W x, y;
    T *out;
    int c0, at;                                                    // first channel; its place in `turned`, or -1: copied
    const auto load = [&]() {
        out = nullptr;
        if (tk >= tokens) return;
        const int64_t t = t0 + tk;
        const bool turn = u < R.pairs, isq = head < a.H;
        const int h = isq ? head : head - a.H;
        c0 = turn ? (INTER && VEC == 1 ? 2 * u : VEC * u) : a.rotary_dim + VEC * (u - R.pairs);
        at = turn ? tk * half + NP * u : -1;
        const T *in = isq ? static_cast<const T *>(a.q) + t * a.q_stride + h * a.q_head_stride
                          : static_cast<const T *>(a.k) + t * a.k_stride + h * a.k_head_stride;
        out = isq ? static_cast<T *>(a.q_out) + t * a.q_out_stride + h * a.q_out_head_stride
                  : static_cast<T *>(a.k_out) + t * a.k_out_stride + h * a.k_out_head_stride;
        if (!GDN_IN(nullptr, t, a.T) || !GDN_IN(nullptr, c0 + VEC - 1, a.D) || (turn && !GDN_IN(nullptr, at + NP - 1, R.tokens * half)) ||
            (turn && kTwo && !GDN_IN(nullptr, c0 + (INTER ? 1 : half) + VEC - 1, a.rotary_dim))) {
            out = nullptr;
            return;
        }
        x = *reinterpret_cast<const W *>(in + c0);
        if (kTwo && turn) y = *reinterpret_cast<const W *>(in + c0 + (INTER ? 1 : half));
        u += du;
        head += dh;
        tk += dt;
        if (u >= R.units) u -= R.units, ++head;
        if (head >= heads) head -= heads, ++tk;
    };
    load();                                                        // on its way while the angles are taken
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int k = i / half;
        float c, s;
        rotary_cos_sin(a.positions[t0 + k], rotary_turns(a.frequencies[i - k * half]), c, s);
        turned[i] = make_float2(c * R.magnitude, a.inverse ? -R.magnitude * s : R.magnitude * s);
    }
    __syncthreads();
    while (out) {
        if (at >= 0) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                T &p = kTwo ? x.v[j] : x.v[kTwo ? 0 : 2 * j], &q = kTwo ? y.v[j] : x.v[kTwo ? 0 : 2 * j + 1];
                const float2 cs = turned[at + j];
                const float f = to_f32(p), h = to_f32(q);
                p = from_f32<T>(f * cs.x - h * cs.y);
                q = from_f32<T>(h * cs.x + f * cs.y);
            }
            if (kTwo) *reinterpret_cast<W *>(out + c0 + (INTER ? 1 : half)) = y;
        }
        *reinterpret_cast<W *>(out + c0) = x;
        load();
    }
}

template <typename T, int VEC, bool INTER> int launch(RotaryLaunch &R, cudaStream_t stream)
{
    const gdn_rotary_args &a = R.a;
    const bool in_place = a.q == a.q_out && (a.HK == 0 || a.k == a.k_out);
    R.pairs = INTER && VEC > 1 ? a.rotary_dim / VEC : a.rotary_dim / 2 / VEC;
    R.units = R.pairs + (in_place ? 0 : (a.D - a.rotary_dim) / VEC);
    // Tokens of a CTA: up to four, as long as two rounds of CTAs remain (16384 tokens of 48 bf16 heads: 70 us at four, 72 at two,
    // 72 at eight; 4999 of 24 fp32 heads: 19.7 at two, 20.7 at four, 21.1 at one); few tokens are shared by CTAs, a vector a thread.
    constexpr int kCtas = kResident * 152, kTokens = 4;
    const int tokens = a.T / (2 * kCtas);
    R.tokens = tokens < 1 ? 1 : tokens > kTokens ? kTokens : tokens;
    const int64_t grid = ((int64_t)a.T + R.tokens - 1) / R.tokens;
    const int64_t vectors = (int64_t)R.tokens * (a.H + a.HK) * R.units;
    const int64_t parts = grid >= kCtas ? 1 : (vectors + kThreads - 1) / kThreads;
    R.parts = (int)(parts < 65535 ? parts : 65535);
    return launch_ordinary(rotary_kernel<T, VEC, INTER>, dim3((unsigned)grid, (unsigned)R.parts), dim3(kThreads),
                           (size_t)R.tokens * (a.rotary_dim / 2) * sizeof(float2), stream, R) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_LAUNCH;
}

template <typename T, bool INTER> int launch_vec(RotaryLaunch &R, int bytes, cudaStream_t stream)
{
    constexpr int N = 16 / sizeof(T);
    if (bytes >= 16) return launch<T, N, INTER>(R, stream);
    return bytes >= 2 * (int)sizeof(T) ? launch<T, 2, INTER>(R, stream) : launch<T, 1, INTER>(R, stream);
}

template <typename T> int launch_t(RotaryLaunch &R, int bytes, cudaStream_t stream)
{
    return R.a.interleaved ? launch_vec<T, true>(R, bytes, stream) : launch_vec<T, false>(R, bytes, stream);
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
    // bytes of a vector: 16, two elements or one
    int vec = 16;
    const auto limit = [&](int64_t bytes) {
        if (bytes % vec) vec = bytes % (2 * es) ? es : 2 * es;
    };
    limit((int64_t)a.D * es);
    limit((int64_t)a.rotary_dim * es / (a.interleaved ? 1 : 2));
    const auto tensor = [&](const void *p, int64_t stride, int64_t head, bool output, int heads) {
        if (!aligned(p, es)) return GDN_ERR_ALIGN;
        if (stride < 0 || head < 0) return GDN_ERR_SHAPE;
        // rows and heads of an output may not overlap
        if (output) {
            const bool rows = a.T == 1 || stride >= (heads > 1 ? (heads - 1) * head : 0) + a.D, in_row = heads == 1 || head >= a.D;
            const bool planes = heads == 1 || head >= (a.T - 1) * stride + a.D, in_plane = a.T == 1 || stride >= a.D;
            if (!(rows && in_row) && !(planes && in_plane)) return GDN_ERR_SHAPE;
        }
        limit((int64_t)(reinterpret_cast<uintptr_t>(p) % 16));
        if (a.T > 1) limit(stride * es);
        if (heads > 1) limit(head * es);
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
