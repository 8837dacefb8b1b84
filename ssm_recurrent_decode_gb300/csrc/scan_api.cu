// scan_api.cu -- host checks, workspace layout and dispatch of the selective scan.
#include <cstring>

#include "scan_launch.h"

namespace gdn {

namespace {
constexpr int kMaxState = 128;
constexpr int kSms = 152;             // GB300
constexpr size_t kWsAlign = 256;

size_t round_up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }
bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }
bool overlap(const void *p, const void *q, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + bytes && b < a + bytes;
}
bool sizes_ok(int T, int S, int D, int N, bool uniform)
{
    return T >= 0 && S >= 1 && D >= 1 && N >= 1 && N <= kMaxState && (!uniform || T % S == 0);
}

// Takes consecutive pieces of a workspace (only counts when base is null).
struct Carver {
    unsigned char *base;
    size_t used = 0;
    template <typename T> T *take(size_t count)
    {
        T *p = base ? reinterpret_cast<T *>(base + used) : nullptr;
        used += round_up(count * sizeof(T));
        return p;
    }
};

// Lays out the workspace of a call whose sizes, C, G, nct and W are set; returns its bytes.
size_t carve(ScanLaunch &P, bool uniform, bool backward, unsigned char *base)
{
    Carver w{base};
    const size_t dn = (size_t)P.a.D * P.a.N;
    // one sequence per chunk, or all rows in one chunk: no state crosses a chunk border; in a cluster it
    // crosses through shared memory
    const bool carried = P.G > 1 && !P.cluster && !(uniform && P.C == P.L);
    if (carried) {
        P.info = w.take<int4>(P.G);
        P.sumdt = w.take<float>((size_t)P.G * P.a.D);
        P.hin = w.take<float>(P.G * dn);
        if (!backward) P.init = w.take<float>(P.G * dn);
    }
    if (backward) {
        if (carried) {
            P.sumdt_head = w.take<float>((size_t)P.G * P.a.D);
            P.ein = w.take<float>(P.G * dn);
        }
        P.part_bc = w.take<float>((size_t)P.nct * P.a.T * 2 * P.a.N);
        P.part_a = w.take<float>(P.W * dn);
        P.part_d = w.take<float>((size_t)P.W * P.a.D);
    }
    return w.used;
}

// Splits a call whose sizes are set (by the sizes alone, so that the workspace can be sized before the
// call): channels per thread, rows per chunk, workers.
void plan(ScanLaunch &P, bool uniform, bool backward)
{
    const int64_t T = P.a.T;
    P.L = uniform ? P.a.T / P.a.S : 0;
    const auto tiles = [&](int cpt) { return (P.a.D + scan_channels(P.a.N, cpt) - 1) / scan_channels(P.a.N, cpt); };
    P.cpt = 4;
    P.nct = tiles(4);
    if (backward) {
        // (two channels a thread for N <= 8, whose tiles of four would leave room for one CTA per SM)
        if (scan_lanes(P.a.N) == 2) {
            P.cpt = 2;
            P.nct = tiles(2);
        }
        // Chunks of 64 rows (what the states kept per CTA allow), shorter ones where those would leave SMs
        // without work.
        const int64_t C = (T * P.nct + kScanBackCtas * kSms - 1) / (kScanBackCtas * kSms);
        P.C = (int)(C >= kScanBackChunk ? kScanBackChunk : C <= 16 ? 16 : (C + 7) / 8 * 8);
    } else {
        const int64_t kSlots = (int64_t)scan_ctas(scan_lanes(P.a.N)) * kSms;     // resident CTAs, by registers
        // Chunks of equal length that fill those slots once, and no shorter than the 32 rows below which a
        // chunk's own costs (its rates, states and launch) outweigh its rows.
        int64_t C = (T * P.nct + kSlots - 1) / kSlots;
        C = (C + 15) / 16 * 16;
        P.C = (int)(C < 32 ? 32 : C);
        if (C < 32 && T * tiles(2) <= 32 * kSlots) {
            P.cpt = 2;                           // too few rows for that: more threads for each
            P.nct = tiles(2);
        }
        if (T > 32 && T <= 8 * 32 && !(uniform && P.L <= 32)) {
            // a few chunks: a cluster of at most eight CTAs per channel tile, in one launch. Against three launches
            // (D = 1536, N = 16, bf16): 64 rows 9.7 and 14.2 us, 128 rows 12.8 and 14.8, 256 rows 15.9 and 17.5. A
            // cluster's CTA has up to 196 registers a thread, so many channel tiles take several rounds and lose:
            // 128 rows, D = 4096, N = 16: 28.7 and 19.3; 256 rows, D = 1536, N = 128: 57 and 39, in fp32 65 and 39.
            P.C = T <= 8 * 16 ? 16 : 32;
            P.cluster = 1;
        } else if (uniform && P.L > 0 && P.L <= 4 * P.C) {
            // About as long as the chunks would be: one pass over whole sequences. Against the same rows in chunks
            // (by cu_seqlens; bf16): 60 x 128, D = 64, N = 16: 17.0 and 37.3 us; 8 x 128, D = 1536: 22.8 and 31.2;
            // 16 x 512: 108 and 116; 64 x 256: 136 and 184; N = 128, 4 x 256: 68 and 108, 4 x 1024: 256 and 398.
            P.C = P.L;
        }
    }
    P.G = T > 0 ? (int)((T + P.C - 1) / P.C) : 1;   // without rows: one chunk of empty sequences
    P.W = 1;
    if (backward) {
        // two CTAs per SM (what their registers allow), each walking over chunks
        const int64_t fit = (int64_t)kScanBackCtas * kSms / P.nct, want = fit > 0 ? fit : 1;
        P.W = (int)(want < P.G ? want : P.G);
    }
}

int check(const mamba_scan_args &a, bool backward, bool states)
{
    const bool uniform = !a.cu_seqlens;
    if (!sizes_ok(a.T, a.S, a.D, a.N, uniform)) return GDN_ERR_SHAPE;
    if (a.in_dtype != GDN_F32 && a.in_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (!backward && a.out_dtype != GDN_F32 && a.out_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (states && a.num_states < 1) return GDN_ERR_SHAPE;
    if (states && !a.state_indices && a.num_states < a.S) return GDN_ERR_SHAPE;
    if (a.T > 0 && (!a.x || !a.dt || !a.A || !a.Bm || !a.Cm || (!backward && !a.y))) return GDN_ERR_NULL;
    if (a.x_stride < a.D || a.dt_stride < a.D || (a.z && a.z_stride < a.D) || a.B_stride < a.N || a.C_stride < a.N ||
        (!backward && a.y_stride < a.D))
        return GDN_ERR_SHAPE;
    const size_t es = a.in_dtype == GDN_BF16 ? 2 : 4;
    if (!aligned(a.x, es) || !aligned(a.dt, es) || !aligned(a.z, es) || !aligned(a.Bm, es) || !aligned(a.Cm, es) ||
        !aligned(a.A, 4) || !aligned(a.Dskip, 4) || !aligned(a.cu_seqlens, 4) || !aligned(a.state_indices, 4) ||
        !aligned(a.h0, 4) || !aligned(a.h_last, 4) || !aligned(a.y, a.out_dtype == GDN_BF16 ? 2 : 4))
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

int row_mode(const void *p, int64_t stride, size_t es)
{
    const auto on = [&](int64_t bytes) { return aligned(p, (size_t)bytes) && stride * (int64_t)es % bytes == 0; };
    return on(16) ? kRows16 : on(4) ? kRows4 : kRowsAny;
}

void set_inputs(ScanLaunch &P)
{
    const mamba_scan_args &a = P.a;
    const size_t es = a.in_dtype == GDN_BF16 ? 2 : 4;
    P.mode_x = row_mode(a.x, a.x_stride, es);
    P.mode_dt = row_mode(a.dt, a.dt_stride, es);
    P.mode_z = row_mode(a.z, a.z_stride, es);
    P.mode_b = row_mode(a.Bm, a.B_stride, es);
    P.mode_c = row_mode(a.Cm, a.C_stride, es);
    if (a.N % 4 == 0 && aligned(a.A, 16) && aligned(a.h0, 16) && aligned(a.h_last, 16)) P.vec |= kVecState;
}

int check_workspace(const mamba_scan_args &a, size_t need)
{
    if (need == 0) return GDN_OK;
    if (!a.workspace) return GDN_ERR_NULL;
    if (a.workspace_bytes < need) return GDN_ERR_SHAPE;
    return aligned(a.workspace, 16) ? GDN_OK : GDN_ERR_ALIGN;
}
}  // namespace

}  // namespace gdn

extern "C" {

size_t mamba_scan_workspace_bytes(int32_t T, int32_t S, int32_t D, int32_t N, int32_t uniform, int32_t backward)
{
    if (!gdn::sizes_ok(T, S, D, N, uniform != 0)) return 0;
    gdn::ScanLaunch P;
    std::memset(&P, 0, sizeof(P));
    P.a.T = T;
    P.a.S = S;
    P.a.D = D;
    P.a.N = N;
    gdn::plan(P, uniform != 0, backward != 0);
    return gdn::carve(P, uniform != 0, backward != 0, nullptr);
}

int mamba_selective_scan(const mamba_scan_args *args, gdn_stream_t stream)
{
    if (!args) return GDN_ERR_NULL;
    const int rc = gdn::check(*args, false, args->h0 || args->h_last);
    if (rc != GDN_OK || (args->T == 0 && !args->h_last)) return rc;
    gdn::ScanLaunch P;
    std::memset(&P, 0, sizeof(P));
    P.a = *args;
    const bool uniform = !args->cu_seqlens;
    gdn::plan(P, uniform, false);
    const size_t need = gdn::carve(P, uniform, false, nullptr);
    const int wrc = gdn::check_workspace(*args, need);
    if (wrc != GDN_OK) return wrc;
    gdn::carve(P, uniform, false, static_cast<unsigned char *>(args->workspace));
    gdn::set_inputs(P);
    P.has_states = args->h0 || args->h_last;
    const size_t os = args->out_dtype == GDN_BF16 ? 2 : 4;
    if (gdn::aligned(args->y, P.cpt * os) && args->y_stride % P.cpt == 0) P.vec |= gdn::kVecY;
    return gdn::launch_scan_forward(P, reinterpret_cast<cudaStream_t>(stream));
}

int mamba_selective_scan_backward(const mamba_scan_grad_args *args, gdn_stream_t stream)
{
    if (!args) return GDN_ERR_NULL;
    const mamba_scan_grad_args &q = *args;
    const bool states = q.s.h0 || q.dh_last || q.dh0;
    const int rc = gdn::check(q.s, true, states);
    if (rc != GDN_OK) return rc;
    if ((q.dz && !q.s.z) || (q.dDskip && !q.s.Dskip)) return GDN_ERR_ARG;
    if (q.s.T > 0 && !q.dy) return GDN_ERR_NULL;
    const int64_t D = q.s.D, N = q.s.N;
    // a sequence's first chunk may be done before its last one has read dh_last
    if (gdn::overlap(q.dh0, q.dh_last, (size_t)q.s.num_states * D * N * sizeof(float))) return GDN_ERR_ARG;
    if (q.dy_stride < D || (q.dx && q.dx_stride < D) || (q.ddt && q.ddt_stride < D) || (q.dz && q.dz_stride < D) ||
        (q.dBm && q.dB_stride < N) || (q.dCm && q.dC_stride < N))
        return GDN_ERR_SHAPE;
    const size_t es = q.s.in_dtype == GDN_BF16 ? 2 : 4;
    for (const void *p : {q.dy, (const void *)q.dx, (const void *)q.ddt, (const void *)q.dz, (const void *)q.dBm, (const void *)q.dCm})
        if (!gdn::aligned(p, es)) return GDN_ERR_ALIGN;
    for (const void *p : {(const void *)q.dh_last, (const void *)q.dA, (const void *)q.dDskip, (const void *)q.dh0})
        if (!gdn::aligned(p, 4)) return GDN_ERR_ALIGN;
    gdn::ScanLaunch P;
    std::memset(&P, 0, sizeof(P));
    P.a = q.s;
    P.g = q;
    const bool uniform = !q.s.cu_seqlens;
    gdn::plan(P, uniform, true);
    const size_t need = gdn::carve(P, uniform, true, nullptr);
    const int wrc = gdn::check_workspace(q.s, need);
    if (wrc != GDN_OK) return wrc;
    gdn::carve(P, uniform, true, static_cast<unsigned char *>(q.s.workspace));
    P.a.h_last = nullptr;
    gdn::set_inputs(P);
    if (!gdn::aligned(q.dh_last, 16) || !gdn::aligned(q.dh0, 16)) P.vec &= ~gdn::kVecState;
    P.has_states = states;
    P.mode_dy = gdn::row_mode(q.dy, q.dy_stride, es);
    const auto out_bit = [&](const void *p, int64_t stride, int bit) {
        if (p && gdn::aligned(p, 4 * es) && stride % 4 == 0) P.vec |= bit;
    };
    out_bit(q.dx, q.dx_stride, gdn::kVecDx);
    out_bit(q.ddt, q.ddt_stride, gdn::kVecDdt);
    out_bit(q.dz, q.dz_stride, gdn::kVecDz);
    return gdn::launch_scan_backward(P, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
