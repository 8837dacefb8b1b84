// scan_forward.cu -- the Mamba-1 selective scan over whole sequences (mamba_selective_scan).
//
// Source: "Triton decode kernel + MBU analysis", "Kernel design" (the per-token arithmetic) and
// "Prefill path" (a scan over the prompt).
#include "scan_common.cuh"

namespace gdn {

// Shared memory, in bytes.
template <typename Tin, class Sh> struct ScanSmem {
    static constexpr int RX = kScanTile * Sh::CB * (int)sizeof(Tin);     // a staged x, dt or z tile
    static constexpr int RB = kScanTile * Sh::NP * (int)sizeof(Tin);     // a staged B or C tile
    static constexpr int STAGE = 3 * RX + 2 * RB;
    static constexpr int HALF = 8;                                       // rows between two stores of outputs
    static constexpr int PARTS = Sh::NL <= 4 ? Sh::NL : 1;               // sums over n still to be joined
    static constexpr int Y = kScanWarps * HALF * PARTS * Sh::YP * 4;
    static constexpr int MAIN = 2 * STAGE + Y;
    static constexpr int SUMMARY = 2 * STAGE;
};

// One CTA: rows g C .. of channel tile ct. SUM: the summary pass (end state from zero and sum of dt
// of the sequence that goes on behind the chunk); else the outputs. Tiles of 16 rows are staged one
// ahead by asynchronous copies; a warp's channels are its own, so only the staging needs barriers.
template <typename Tin, int NL, int CPT, bool SUM>
__global__ void __launch_bounds__(kScanThreads, scan_ctas(NL)) scan_forward_kernel(const __grid_constant__ ScanLaunch P)
{
    using Sh = ScanShape<NL, CPT>;
    using Sm = ScanSmem<Tin, Sh>;
    constexpr int CB = Sh::CB, NP = Sh::NP, PP = Sh::P, CLN = Sh::CLN;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[kScanWarps];
    ordinary_launch_start();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, cl = lane / NL;
    const int ct = (int)(blockIdx.x % (unsigned)P.nct), g = (int)(blockIdx.x / (unsigned)P.nct);
    const int D = P.a.D, N = P.a.N;
    const int c0 = ct * CB, ncols = min(CB, D - c0);
    const int n0 = 4 * nl, wc = warp * Sh::CW + cl * CPT, d0 = c0 + wc;      // this thread's first entry and channel
    const int64_t dn = (int64_t)D * N;
    const bool vst = (P.vec & kVecState) != 0;
    const int row0 = (int)min((int64_t)g * P.C, (int64_t)P.a.T), row1 = (int)min((int64_t)(g + 1) * P.C, (int64_t)P.a.T);

    ScanIter load, use;
    if (SUM) {
        // only the rows of the sequence that goes on behind the chunk
        const int s = find_seq(P, row1 - 1, scratch, tid);
        const bool goes_on = s >= 0 && s < P.a.S && seq_bound(P, s + 1) > row1;
        const int first = goes_on ? max(seq_bound(P, s), row0) : row1;
        if (tid == 0 && ct == 0)
            P.info[g] = make_int4(goes_on ? s : -1, goes_on && seq_bound(P, s) >= row0, 0, 0);
        if (!goes_on) return;
        load.init(first, row1, s);
    } else {
        load.init(row0, row1, find_seq(P, row0, scratch, tid));
        // empty sequences pass their state on (each handled by one chunk's CTAs)
        if (P.a.h_last && P.a.h_last != P.a.h0 && (P.a.cu_seqlens || P.L == 0)) {
            for (int s = g; s < P.a.S; s += P.G) {
                if (seq_bound(P, s) != seq_bound(P, s + 1)) continue;
                const int64_t slot = P.a.state_indices ? (int64_t)P.a.state_indices[s] : s;
                if (slot < 0 || slot >= P.a.num_states) {
                    if (tid == 0) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
                    continue;
                }
                for (int i = tid; i < ncols * N; i += kScanThreads)
                    P.a.h_last[slot * dn + (int64_t)c0 * N + i] = P.a.h0 ? P.a.h0[slot * dn + (int64_t)c0 * N + i] : 0.f;
            }
        }
    }
    use = load;

    auto stage_tile = [&](const ScanTile &t, int b) {
        Tin *xs = reinterpret_cast<Tin *>(smem + b * Sm::STAGE);
        Tin *ds = xs + kScanTile * CB, *zs = ds + kScanTile * CB;
        Tin *Bs = zs + kScanTile * CB, *Cs = Bs + kScanTile * NP;
        const auto rows = [&](const void *base, int64_t stride, int col, int width, int mode) {
            return TileSource<Tin>{static_cast<const Tin *>(base), stride, t.t0, P.a.T, col, width, mode};
        };
        stage_rows<Tin, CB>(xs, rows(P.a.x, P.a.x_stride, c0, D, P.mode_x), t.n, tid);
        stage_rows<Tin, CB>(ds, rows(P.a.dt, P.a.dt_stride, c0, D, P.mode_dt), t.n, tid);
        stage_rows<Tin, NP>(Bs, rows(P.a.Bm, P.a.B_stride, 0, N, P.mode_b), t.n, tid);
        if (!SUM) {
            if (P.a.z) stage_rows<Tin, CB>(zs, rows(P.a.z, P.a.z_stride, c0, D, P.mode_z), t.n, tid);
            stage_rows<Tin, NP>(Cs, rows(P.a.Cm, P.a.C_stride, 0, N, P.mode_c), t.n, tid);
        }
    };
    ScanTile tl, nxt;
    if (load.next(P, nxt)) stage_tile(nxt, 0);
    cp_async_commit();

    f2 A2[4][PP], h[4][PP], dts[PP];
    zero_entries(A2);
    zero_entries(h);
    if (row0 < row1) load_rates(P.a.A, d0, D, n0, N, vst, A2);
#pragma unroll
    for (int p = 0; p < PP; ++p) dts[p] = 0ull;
    // a lane finishes CPT channels of every row it is given: the same ones in every tile
    const int oc = warp * Sh::CW + lane % CLN * CPT, orow = lane / CLN;
    const bool whole = (P.vec & kVecY) && oc + CPT <= ncols;
    f2 skip[PP];
#pragma unroll
    for (int p = 0; p < PP; ++p) {
        const int c = oc + 2 * p;
        skip[p] = pack2(!SUM && P.a.Dskip && c < ncols ? P.a.Dskip[c0 + c] : 0.f,
                        !SUM && P.a.Dskip && c + 1 < ncols ? P.a.Dskip[c0 + c + 1] : 0.f);
    }
    float *ys = reinterpret_cast<float *>(smem + 2 * Sm::STAGE) + warp * Sm::HALF * Sm::PARTS * Sh::YP;

    int b = 0;
    while (use.next(P, tl)) {
        cp_async_wait<0>();
        __syncthreads();             // the tile is here, and the buffers of the one before are free
        if (load.next(P, nxt)) stage_tile(nxt, b ^ 1);
        cp_async_commit();

        const Tin *xs = reinterpret_cast<const Tin *>(smem + b * Sm::STAGE);
        const Tin *ds = xs + kScanTile * CB, *zs = ds + kScanTile * CB;
        const Tin *Bs = zs + kScanTile * CB, *Cs = Bs + kScanTile * NP;
        if (tl.fresh) {
            const float *from = nullptr;
            if (!SUM && tl.seq >= 0)
                // (a sequence that goes on behind the chunk: in place, a later chunk's CTA may already have
                // written its row of h_last, so its initial state comes from the carry pass's copy)
                from = !tl.starts ? (P.hin ? P.hin + g * dn : nullptr)
                       : !P.a.h0  ? nullptr
                       : P.hin && g < P.G - 1 && P.info[g].x == tl.seq ? P.init + g * dn : P.a.h0 + tl.slot * dn;
            zero_entries(h);
            if (from) load_entries(from, d0, D, n0, N, vst, h);
        }

        f2 dt_tile[PP] = {};
        // rows behind the tile's last are zeros: dt = 0 leaves h as it is
#pragma unroll 1
        for (int t8 = 0; t8 < kScanTile; t8 += Sm::HALF) {
#pragma unroll
            for (int t4 = t8; t4 < t8 + Sm::HALF; t4 += 4) {       // eight rows' work to schedule among (401 -> 379 us)
                float acc[4 * CPT];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = t4 + k;
                    f2 dt[PP], u[PP], B[4], C[4], y[PP];
                    load_pairs(ds + t * CB + wc, dt);
                    load_pairs(xs + t * CB + wc, u);
                    load_twice(Bs + t * NP + n0, B);
                    if (!SUM) load_twice(Cs + t * NP + n0, C);
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        u[p] = mul2(dt[p], u[p]);
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            h[n][p] = fma2(decay2(dt[p], A2[n][p]), h[n][p], mul2(u[p], B[n]));
                            if (!SUM) y[p] = n == 0 ? mul2(C[n], h[n][p]) : fma2(C[n], h[n][p], y[p]);
                        }
                        if (SUM) dt_tile[p] = add2(dt_tile[p], dt[p]);
                        else if (NL > 4) {
                            const float2 v = unpack2(y[p]);
                            acc[k * CPT + 2 * p] = v.x;
                            acc[k * CPT + 2 * p + 1] = v.y;
                        }
                    }
                    // up to four lanes' sums are joined where the row is finished, more of them here by shuffles
                    if (!SUM && NL <= 4) store_pairs(ys + ((t - t8) * NL + nl) * Sh::YP + cl * CPT, y);
                }
                if (!SUM && NL > 4) {
                    constexpr int M = 4 * CPT, KEEP = M >= NL ? M / NL : 1, REP = M >= NL ? 1 : NL / M;
                    group_reduce<M, NL>(acc, nl);
                    if (nl % REP == 0) {
#pragma unroll
                        for (int i = 0; i < KEEP; ++i) {
                            const int v = nl / REP * KEEP + i;
                            ys[(t4 - t8 + v / CPT) * Sh::YP + cl * CPT + v % CPT] = acc[i];
                        }
                    }
                }
            }
            if (SUM) continue;
            __syncwarp();
            // skip, gate and output of these rows
#pragma unroll
            for (int r0 = 0; r0 < Sm::HALF; r0 += NL) {
                const int r = r0 + orow, t = t8 + r;
                if ((NL > Sm::HALF && r >= Sm::HALF) || t >= tl.n || oc >= ncols) continue;
                f2 y[PP], x2[PP], z2[PP];
                load_pairs(ys + r * Sm::PARTS * Sh::YP + lane % CLN * CPT, y);
#pragma unroll
                for (int q = 1; q < Sm::PARTS; ++q) {
                    f2 more[PP];
                    load_pairs(ys + (r * Sm::PARTS + q) * Sh::YP + lane % CLN * CPT, more);
#pragma unroll
                    for (int p = 0; p < PP; ++p) y[p] = add2(y[p], more[p]);
                }
                load_pairs(xs + t * CB + oc, x2);
                if (P.a.z) load_pairs(zs + t * CB + oc, z2);
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    y[p] = fma2(skip[p], x2[p], y[p]);
                    if (P.a.z) {
                        const float2 z = unpack2(z2[p]);
                        y[p] = mul2(y[p], mul2(z2[p], pack2(fast_sigmoid(z.x), fast_sigmoid(z.y))));
                    }
                    if (tl.seq < 0) y[p] = 0ull;
                }
                if (!GDN_IN(P.a.err_flags, (int64_t)tl.t0 + t, P.a.T)) continue;
                const int64_t o = (int64_t)(tl.t0 + t) * P.a.y_stride + c0 + oc;
                if (P.a.out_dtype == GDN_BF16)
                    store_row(static_cast<bf16 *>(P.a.y) + o, y, ncols - oc, whole);
                else
                    store_row(static_cast<float *>(P.a.y) + o, y, ncols - oc, whole);
            }
            __syncwarp();
        }
        if (SUM) {
#pragma unroll
            for (int p = 0; p < PP; ++p) dts[p] = add2(dts[p], dt_tile[p]);
        } else if (tl.ends && P.a.h_last && GDN_IN(P.a.err_flags, tl.slot, P.a.num_states)) {
            store_entries(P.a.h_last + tl.slot * dn, d0, D, n0, N, vst, h);
        }
        b ^= 1;
    }
    if (SUM && GDN_IN(P.a.err_flags, g, P.G)) {
        store_entries(P.hin + g * dn, d0, D, n0, N, vst, h);
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            const float2 v = unpack2(dts[p]);
            if (nl == 0 && d0 + 2 * p < D) P.sumdt[(int64_t)g * D + d0 + 2 * p] = v.x;
            if (nl == 0 && d0 + 2 * p + 1 < D) P.sumdt[(int64_t)g * D + d0 + 2 * p + 1] = v.y;
        }
    }
}

template <typename Tin, int NL, int CPT, bool SUM>
static cudaError_t launch_one(const ScanLaunch &P, int chunks, cudaStream_t stream)
{
    constexpr int bytes = SUM ? ScanSmem<Tin, ScanShape<NL, CPT>>::SUMMARY : ScanSmem<Tin, ScanShape<NL, CPT>>::MAIN;
    auto kern = scan_forward_kernel<Tin, NL, CPT, SUM>;
    if (bytes > 40 * 1024) {      // the kernels have a little static shared memory too
        const cudaError_t rc = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (rc != cudaSuccess) return rc;
    }
    return launch_ordinary(kern, dim3((unsigned)((int64_t)chunks * P.nct)), dim3(kScanThreads), bytes, stream, P);
}

template <typename Tin, int NL, int CPT> static int launch_shape(const ScanLaunch &P, cudaStream_t stream)
{
    if (P.hin) {
        if (launch_one<Tin, NL, CPT, true>(P, P.G - 1, stream) != cudaSuccess) return GDN_ERR_LAUNCH;
        if (launch_scan_carry(P, false, stream) != cudaSuccess) return GDN_ERR_LAUNCH;
    }
    return launch_one<Tin, NL, CPT, false>(P, P.G, stream) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

template <typename Tin, int NL> static int launch_lanes(const ScanLaunch &P, cudaStream_t stream)
{
    return P.cpt == 2 ? launch_shape<Tin, NL, 2>(P, stream) : launch_shape<Tin, NL, 4>(P, stream);
}

template <typename Tin> static int launch_typed(const ScanLaunch &P, cudaStream_t stream)
{
    switch (scan_lanes(P.a.N)) {
    case 2: return launch_lanes<Tin, 2>(P, stream);
    case 4: return launch_lanes<Tin, 4>(P, stream);
    case 8: return launch_lanes<Tin, 8>(P, stream);
    case 16: return launch_lanes<Tin, 16>(P, stream);
    default: return launch_lanes<Tin, 32>(P, stream);
    }
}

int launch_scan_forward(const ScanLaunch &P, cudaStream_t stream)
{
    return P.a.in_dtype == GDN_BF16 ? launch_typed<bf16>(P, stream) : launch_typed<float>(P, stream);
}

}  // namespace gdn
