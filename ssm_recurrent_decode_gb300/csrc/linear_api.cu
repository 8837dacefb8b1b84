// linear_api.cu -- host checks, workspace layout and dispatch of linear attention.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "linear_launch.h"

namespace gdn {

namespace {

constexpr int kSms = 152;              // GB300
constexpr size_t kWsAlign = 256;

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool overlap(const void *p, const void *q, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + bytes && b < a + bytes;
}

bool sizes_ok(const gdn_linear_args &a, bool uniform)
{
    return a.T >= 0 && a.S >= 1 && (int64_t)a.S + a.T / 16 <= INT32_MAX && a.H >= 1 && a.HV >= 1 && a.HV <= 65535 && a.HV % a.H == 0 && a.V >= 1 && a.V <= 128 &&
           (a.K == 16 || a.K == 32 || a.K == 64 || a.K == 128) && (!uniform || a.T % a.S == 0);
}

// what the backward pass keeps besides the states between segments
struct BackwardSpace {
    float *part;                       // [T, HV, K] dq, then dk of every value head
    float *qdq, *kdk;                  // [T, HV]
    float *dg_part;
    float *chunk_states, *chunk_dot;   // see LinearSweep
};

// Copies of inputs whose rows TMA cannot take, for value sizes that are not a multiple of eight (other rows that are not
// aligned to 16 bytes, which dense tensors and views of them have not, are read by plain loads instead).
struct PackedSpace {
    void *q, *k, *v, *d_o;
};

struct Carver {
    unsigned char *base;
    size_t used = 0;
    float *take(size_t count)
    {
        float *p = base ? reinterpret_cast<float *>(base + used) : nullptr;
        used += (count * sizeof(float) + kWsAlign - 1) / kWsAlign * kWsAlign;
        return p;
    }
};

int z_parts(int dz) { return (dz + kLinearZ - 1) / kLinearZ; }

void set_segments(LinearLaunch &P, bool uniform, int64_t seg)
{
    const int64_t longest = uniform ? P.Ls : P.a.T;
    if (seg >= longest) seg = longest > 0 ? longest : 1;
    P.seg = (int)seg;
    P.carried = longest > seg;
    P.items = (int)(uniform ? (int64_t)P.a.S * (P.Ls > 0 ? (P.Ls + seg - 1) / seg : 1) : P.a.S + P.a.T / seg);
    // (a sequence that is cut has more than seg rows, and at most twice as many segments as whole ones)
    P.cut_items = uniform || P.a.S <= kLinearSorted ? P.items : (int)std::min<int64_t>(P.items, 2 * (P.a.T / seg));
}

// Rows of a segment of equal sequences: as many segments as make the shortest run of rounds of CTAs, in units of a chunk's time.
// 1 x 32768 x 32 heads: nine segments (288 CTAs, two rounds of 29 chunks) 436 us, ten (320 CTAs, three rounds) 513 (both measured
// with outputs of one term; nine take 454 now).
int64_t uniform_segment(const gdn_linear_args &a, int64_t length, bool backward)
{
    const int64_t chunks = (length + kLinearChunk - 1) / kLinearChunk, tiles = (int64_t)a.S * a.HV;
    double best = 0.0;
    int64_t seg = length;
    for (int64_t n = 1; n <= 8 * kSms && (n == 1 || 2 * n <= chunks); ++n) {
        const int64_t per = (chunks + n - 1) / n;
        if (n > 1 && (n - 1) * per >= chunks) continue;          // as good as fewer
        // a CTA starts and ends in the time of a chunk; the pass for the segments' states takes 0.55 to 0.65 of one with
        // outputs, two of them beside the three of the gradients a quarter; a state of the carry 4 K V floats of traffic at 5 TB/s
        double cost = (double)((tiles * n + kSms - 1) / kSms) * (per + 1);
        if (n > 1) cost = cost * (backward ? 1.27 : 1.65) + 0.7e-6 * (double)(tiles * n) * a.K * a.V + 0.1 * n;
        if (n == 1 || cost < best) best = cost, seg = n == 1 ? length : per * kLinearChunk;
    }
    return seg;
}

// Splits the sequences into segments, by the call's sizes alone.
void plan(LinearLaunch &P, bool uniform, bool backward)
{
    const gdn_linear_args &a = P.a;
    P.Ls = uniform ? a.T / a.S : 0;
    P.tc = a.in_dtype == GDN_BF16;
    const int64_t longest = uniform ? P.Ls : a.T;
    if (P.tc) {
        // One CTA an SM, whole chunks. A cut sequence's keys and values are read twice, and its states between the segments go
        // through memory.
        int64_t seg = longest;
        if (uniform || a.S == 1) seg = uniform_segment(a, longest, backward);
        else {
            // The lengths are on the device; the longest sequences start first. No segment is longer than what an SM has to do in
            // all: its share of the tokens and, where that order is kept, of the sequences' starts and last chunks (a chunk and
            // a half each). 24 sequences of 8000 tokens, 32 heads: 136 us, 147 by the
            // share of the tokens alone.
            seg = ((int64_t)a.T + (a.S <= kLinearSorted ? 3 * kLinearChunk / 2 * (int64_t)a.S : 0)) * a.HV / kSms / kLinearChunk * kLinearChunk;
            if (seg < 2 * kLinearChunk) seg = 2 * kLinearChunk;
        }
        set_segments(P, uniform, seg);
        return;
    }
    const int64_t ctas = (int64_t)a.HV * z_parts(backward ? (a.K < a.V ? a.K : a.V) : a.V);
    int64_t seg = ((int64_t)a.T * ctas + 4 * kSms - 1) / (4 * kSms);
    seg = (seg + 15) / 16 * 16;
    if (seg < 48) seg = 48;
    if (backward && seg > 128) seg = 128;                // dg's sums run no longer than a segment
    set_segments(P, uniform, seg);
}

size_t carve(LinearLaunch &P, BackwardSpace *B, PackedSpace &packed, unsigned char *base)
{
    Carver w{base};
    const gdn_linear_args &a = P.a;
    packed = PackedSpace{};
    if (P.tc && a.V % 8) {
        const size_t qk = (size_t)a.T * a.H * a.K / 2, v = (size_t)a.T * a.HV * ((a.V + 7) / 8 * 4);      // in words
        packed.q = w.take(qk);
        packed.k = w.take(qk);
        packed.v = w.take(v);
        if (B) packed.d_o = w.take(v);
    }
    if (P.carried) {
        P.local = w.take((size_t)P.cut_items * a.HV * a.K * a.V);
        P.total = reinterpret_cast<float2 *>(w.take((size_t)P.cut_items * a.HV * 2));
    }
    if (B) {
        const size_t th = (size_t)a.T * a.HV;
        B->part = w.take(th * a.K);
        B->qdq = w.take(th);
        B->kdk = w.take(th);
        if (P.tc) {
            const size_t chunks = ((size_t)a.T / kLinearChunk + a.S) * a.HV;
            B->chunk_states = w.take(chunks * kLinearChunk * (a.K <= 64 ? 64 : 128));
            B->chunk_dot = w.take(chunks * 8);
            B->dg_part = w.take(chunks * 8);
        } else {
            const size_t parts = (size_t)P.items * a.HV * z_parts(a.K);
            B->chunk_states = w.take(parts * kLinearZ * (a.V <= 16 ? 16 : a.V <= 32 ? 32 : a.V <= 64 ? 64 : 128));
            B->chunk_dot = w.take(parts);
            B->dg_part = w.take(linear_dg_part_floats(P.items, a.HV));
        }
    }
    return w.used;
}

int check_rows(const void *p, int64_t stride, int64_t head, size_t es)
{
    if (stride < 0 || head < 0) return GDN_ERR_SHAPE;
    return aligned(p, es) ? GDN_OK : GDN_ERR_ALIGN;
}

// rows [T, heads, n] of an output: no two of them on the same memory
int check_output(const void *p, int64_t stride, int64_t head, int T, int heads, int n, size_t es)
{
    const int rc = check_rows(p, stride, head, es);
    if (rc != GDN_OK) return rc;
    const bool by_token = (T <= 1 || stride >= (heads > 1 ? (heads - 1) * head : 0) + n) && (heads == 1 || head >= n);
    const bool by_head = (heads == 1 || head >= (int64_t)(T - 1) * stride + n) && (T <= 1 || stride >= n);
    return by_token || by_head ? GDN_OK : GDN_ERR_SHAPE;
}

int check(const gdn_linear_args &a, bool states)
{
    if (!sizes_ok(a, !a.cu_seqlens)) return GDN_ERR_SHAPE;
    if (a.in_dtype != GDN_F32 && a.in_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (states && (a.num_states < 1 || (!a.state_indices && a.num_states < a.S))) return GDN_ERR_SHAPE;
    if (a.T > 0 && (!a.q || !a.k || !a.v || !a.g)) return GDN_ERR_NULL;
    const size_t es = a.in_dtype == GDN_BF16 ? 2 : 4;
    for (int rc : {check_rows(a.q, a.q_stride, a.q_head_stride, es), check_rows(a.k, a.k_stride, a.k_head_stride, es),
                   check_rows(a.v, a.v_stride, a.v_head_stride, es), check_rows(a.g, a.g_stride, 0, 4)})
        if (rc != GDN_OK) return rc;
    if (!aligned(a.cu_seqlens, 4) || !aligned(a.state_indices, 4) || !aligned(a.initial_state, 16) || !aligned(a.final_state, 16))
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

int check_workspace(const gdn_linear_args &a, size_t need)
{
    if (need == 0) return GDN_OK;
    if (!a.workspace) return GDN_ERR_NULL;
    if (a.workspace_bytes < need) return GDN_ERR_SHAPE;
    return aligned(a.workspace, 16) ? GDN_OK : GDN_ERR_ALIGN;
}

// the sweep (x, y, z) = (q, k, v); the others exchange roles
LinearSweep forward_sweep(const LinearLaunch &P)
{
    const gdn_linear_args &a = P.a;
    LinearSweep p = {};
    const int G = a.HV / a.H;
    p.x = a.q, p.x_stride = a.q_stride, p.x_head = a.q_head_stride, p.x_group = G;
    p.y = a.k, p.y_stride = a.k_stride, p.y_head = a.k_head_stride, p.y_group = G;
    p.z = a.v, p.z_stride = a.v_stride, p.z_head = a.v_head_stride, p.z_group = 1;
    p.DY = a.K, p.DZ = a.V;
    p.x_scale = P.scale, p.z_scale = 1.f;
    p.sy = 1, p.sz = a.K;
    return p;
}

int run(const LinearLaunch &P, const LinearSweep &p, cudaStream_t stream) 
{
    return P.tc ? launch_linear_chunk(P, p, true, stream) : launch_linear_recurrent(P, p, true, stream);
}

// An input's rows, copied where they need it.
int pack(const LinearLaunch &P, const void *&p, int64_t &stride, int64_t &head, int heads, int n, void *to, cudaStream_t stream)
{
    if (!to || P.a.T == 0 || (n % 8 == 0 && aligned(p, 16) && stride % 8 == 0 && (head % 8 == 0 || heads == 1))) return GDN_OK;
    const int rc = launch_linear_pack(p, stride, head, P.a.T, heads, n, to, stream);
    p = to;
    head = (n + 7) / 8 * 8;
    stride = heads * head;
    return rc;
}

int pack_inputs(LinearLaunch &P, const PackedSpace &packed, cudaStream_t stream)
{
    gdn_linear_args &a = P.a;
    int rc = pack(P, a.q, a.q_stride, a.q_head_stride, a.H, a.K, packed.q, stream);
    if (rc == GDN_OK) rc = pack(P, a.k, a.k_stride, a.k_head_stride, a.H, a.K, packed.k, stream);
    if (rc == GDN_OK) rc = pack(P, a.v, a.v_stride, a.v_head_stride, a.HV, a.V, packed.v, stream);
    return rc;
}

struct Rows {
    const void *p;
    int64_t stride, head;
};

// A sweep whose outputs are summed over the value heads that share a q/k head: dq or dk, and each value head's product
// with q or k.
struct Heads {
    Rows out, with;
    float *part, *dot;
};

bool direct(const LinearLaunch &P) { return P.tc && P.a.HV == P.a.H; }        // one value head a head: nothing to sum

void set_heads(const LinearLaunch &P, LinearSweep &p, const Heads &h)
{
    const gdn_linear_args &a = P.a;
    if (P.tc && h.dot)
        p.dot = h.dot, p.dot_with = h.with.p, p.dot_stride = h.with.stride, p.dot_head = h.with.head, p.dot_group = a.HV / a.H;
    if (direct(P)) p.out = const_cast<void *>(h.out.p), p.out_stride = h.out.stride, p.out_head = h.out.head, p.out_f32 = 0;
    else p.out = h.part, p.out_stride = (int64_t)a.HV * a.K, p.out_head = a.K, p.out_f32 = 1;
}

int fold_heads(const LinearLaunch &P, const Heads &h, cudaStream_t stream)
{
    if (direct(P) || (P.tc && !h.out.p)) return GDN_OK;
    return launch_linear_fold(P, {h.part, const_cast<void *>(h.out.p), h.out.stride, h.out.head, h.with.p, h.with.stride, h.with.head,
                                  P.tc ? nullptr : h.dot}, stream);
}

// the states between the segments
int run_states(const LinearLaunch &P, const LinearSweep &p, cudaStream_t stream)
{
    if (!P.carried) return GDN_OK;
    const int rc = P.tc ? launch_linear_chunk(P, p, false, stream) : launch_linear_recurrent(P, p, false, stream);
    return rc != GDN_OK ? rc : launch_linear_carry(P, p, stream);
}

LinearLaunch make(const gdn_linear_args &a, bool backward, bool states)
{
    LinearLaunch P;
    std::memset(&P, 0, sizeof(P));
    P.a = a;
    P.scale = a.scale != 0.f ? a.scale : 1.0f / std::sqrt((float)a.K);
    P.states = states;
    plan(P, !a.cu_seqlens, backward);
    return P;
}

}  // namespace

}  // namespace gdn

extern "C" {

size_t gdn_linear_workspace_bytes(int32_t T, int32_t S, int32_t H, int32_t HV, int32_t K, int32_t V, int32_t in_dtype,
                                  int32_t uniform, int32_t backward)
{
    gdn::LinearLaunch P;
    std::memset(&P, 0, sizeof(P));
    P.a.T = T, P.a.S = S, P.a.H = H, P.a.HV = HV, P.a.K = K, P.a.V = V, P.a.in_dtype = in_dtype;
    if (!gdn::sizes_ok(P.a, uniform != 0)) return 0;
    gdn::plan(P, uniform != 0, backward != 0);
    gdn::BackwardSpace B;
    gdn::PackedSpace packed;
    return gdn::carve(P, backward ? &B : nullptr, packed, nullptr);
}

int gdn_linear_attention(const gdn_linear_args *args, gdn_stream_t stream)
{
    if (!args) return GDN_ERR_NULL;
    const gdn_linear_args &a = *args;
    const bool states = a.initial_state || a.final_state;
    int rc = gdn::check(a, states);
    if (rc != GDN_OK) return rc;
    if (a.out_dtype != GDN_F32 && a.out_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (a.T > 0 && !a.o) return GDN_ERR_NULL;
    rc = gdn::check_output(a.o, a.o_stride, a.o_head_stride, a.T, a.HV, a.V, a.out_dtype == GDN_BF16 ? 2 : 4);
    if (rc != GDN_OK || (a.T == 0 && !a.final_state)) return rc;
    gdn::LinearLaunch P = gdn::make(a, false, states);
    gdn::PackedSpace packed;
    rc = gdn::check_workspace(a, gdn::carve(P, nullptr, packed, nullptr));
    if (rc != GDN_OK) return rc;
    gdn::carve(P, nullptr, packed, static_cast<unsigned char *>(a.workspace));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    rc = gdn::pack_inputs(P, packed, s);
    if (rc != GDN_OK) return rc;
    gdn::LinearSweep p = gdn::forward_sweep(P);
    p.start = a.initial_state;
    p.end = a.final_state;
    p.out = a.o, p.out_stride = a.o_stride, p.out_head = a.o_head_stride, p.out_f32 = a.out_dtype == GDN_F32;
    rc = gdn::run_states(P, p, s);
    return rc != GDN_OK ? rc : gdn::run(P, p, s);
}

int gdn_linear_attention_backward(const gdn_linear_grad_args *args, gdn_stream_t stream)
{
    if (!args) return GDN_ERR_NULL;
    const gdn_linear_grad_args &given = *args;
    const bool states = given.s.initial_state || given.d_final_state || given.d_initial_state;
    gdn_linear_args in = given.s;
    in.final_state = nullptr;
    int rc = gdn::check(in, states);
    if (rc != GDN_OK) return rc;
    if (in.T > 0 && !given.d_o) return GDN_ERR_NULL;
    const size_t es = in.in_dtype == GDN_BF16 ? 2 : 4, pool = states ? (size_t)in.num_states * in.HV * in.K * in.V * 4 : 0;
    for (int r : {gdn::check_rows(given.d_o, given.do_stride, given.do_head_stride, es),
                  given.dq ? gdn::check_output(given.dq, given.dq_stride, given.dq_head_stride, in.T, in.H, in.K, es) : (int)GDN_OK,
                  given.dk ? gdn::check_output(given.dk, given.dk_stride, given.dk_head_stride, in.T, in.H, in.K, es) : (int)GDN_OK,
                  given.dv ? gdn::check_output(given.dv, given.dv_stride, given.dv_head_stride, in.T, in.HV, in.V, es) : (int)GDN_OK,
                  given.dg && in.g_stride ? gdn::check_output(given.dg, given.dg_stride, in.HV, in.T, 1, in.HV, 4) : (int)GDN_OK})
        if (r != GDN_OK) return r;
    if (!gdn::aligned(given.dg, 4) || !gdn::aligned(given.d_final_state, 16) || !gdn::aligned(given.d_initial_state, 16)) return GDN_ERR_ALIGN;
    if (gdn::overlap(given.d_initial_state, given.d_final_state, pool) || gdn::overlap(given.d_initial_state, in.initial_state, pool)) return GDN_ERR_ARG;
    gdn::LinearLaunch P = gdn::make(in, true, states);
    gdn::BackwardSpace B;
    gdn::PackedSpace packed;
    rc = gdn::check_workspace(in, gdn::carve(P, &B, packed, nullptr));
    if (rc != GDN_OK) return rc;
    gdn::carve(P, &B, packed, static_cast<unsigned char *>(in.workspace));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    gdn_linear_grad_args q = *args;
    rc = gdn::pack_inputs(P, packed, s);
    if (rc == GDN_OK) rc = gdn::pack(P, q.d_o, q.do_stride, q.do_head_stride, in.HV, in.V, packed.d_o, s);
    if (rc != GDN_OK) return rc;
    const gdn_linear_args &a = P.a;
    const int G = a.HV / a.H;

    // forward: dq from the states
    if (q.dq || q.dg) {
        gdn::LinearSweep p = gdn::forward_sweep(P);
        p.start = a.initial_state;
        rc = gdn::run_states(P, p, s);
        if (rc != GDN_OK) return rc;
        p.x = q.d_o, p.x_stride = q.do_stride, p.x_head = q.do_head_stride, p.x_group = 1;
        p.y = a.v, p.y_stride = a.v_stride, p.y_head = a.v_head_stride, p.y_group = 1;
        p.z = a.k, p.z_stride = a.k_stride, p.z_head = a.k_head_stride, p.z_group = G;
        p.DY = a.V, p.DZ = a.K, p.sy = a.K, p.sz = 1;
        if (q.dg) p.chunk_states = B.chunk_states;
        const gdn::Heads h = {{q.dq, q.dq_stride, q.dq_head_stride}, {a.q, a.q_stride, a.q_head_stride}, B.part, q.dg ? B.qdq : nullptr};
        gdn::set_heads(P, p, h);
        rc = gdn::run(P, p, s);
        if (rc == GDN_OK) rc = gdn::fold_heads(P, h, s);
        if (rc != GDN_OK) return rc;
    }
    // backward: dv and dk from the states' gradients
    if (q.dk || q.dv || q.dg || q.d_initial_state) {
        gdn::LinearSweep p = gdn::forward_sweep(P);
        p.reverse = 1;
        p.start = q.d_final_state;
        p.x = a.k, p.x_stride = a.k_stride, p.x_head = a.k_head_stride;
        p.y = a.q, p.y_stride = a.q_stride, p.y_head = a.q_head_stride;
        p.z = q.d_o, p.z_stride = q.do_stride, p.z_head = q.do_head_stride;
        p.x_scale = 1.f, p.z_scale = P.scale;
        rc = gdn::run_states(P, p, s);
        if (rc != GDN_OK) return rc;
        // dk's sweep, then dv's, which starts where dk's leaves SMs empty (all gradients of 8 x 2048
        // tokens, 32 heads: 793 us, 807 one behind the other; of ten ragged sequences 255 and 275)
        const bool do_dk = q.dk || q.dg, do_dv = q.dv || q.d_initial_state, both = P.tc && do_dk && do_dv;
        const gdn::Heads h = {{q.dk, q.dk_stride, q.dk_head_stride}, {a.k, a.k_stride, a.k_head_stride}, B.part, q.dg ? B.kdk : nullptr};
        if (do_dk) {
            gdn::LinearSweep dk = p;
            dk.x = a.v, dk.x_stride = a.v_stride, dk.x_head = a.v_head_stride, dk.x_group = 1;
            dk.y = q.d_o, dk.y_stride = q.do_stride, dk.y_head = q.do_head_stride, dk.y_group = 1;
            dk.z = a.q, dk.z_stride = a.q_stride, dk.z_head = a.q_head_stride, dk.z_group = G;
            dk.DY = a.V, dk.DZ = a.K, dk.sy = a.K, dk.sz = 1;
            if (q.dg) dk.chunk_states = B.chunk_states, dk.chunk_dot = B.chunk_dot;
            dk.before_next = both;
            gdn::set_heads(P, dk, h);
            rc = gdn::run(P, dk, s);
            if (rc != GDN_OK) return rc;
        }
        if (do_dv) {
            p.end = q.d_initial_state;
            p.out = q.dv, p.out_stride = q.dv_stride, p.out_head = q.dv_head_stride, p.out_f32 = a.in_dtype == GDN_F32;
            p.early = both;
            rc = gdn::run(P, p, s);
            if (rc != GDN_OK) return rc;
        }
        if (do_dk) rc = gdn::fold_heads(P, h, s);
        if (rc != GDN_OK) return rc;
    }
    if (!q.dg) return GDN_OK;
    if (P.tc) return gdn::launch_linear_dg_chunks(P, B.qdq, B.kdk, B.chunk_dot, q.dg, q.dg_stride, B.dg_part, s);
    return gdn::launch_linear_dg(P, B.qdq, B.kdk, B.chunk_dot, gdn::z_parts(a.K), q.dg, q.dg_stride, B.dg_part, s);
}

}  // extern "C"
