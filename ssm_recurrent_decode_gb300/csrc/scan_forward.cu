// scan_forward.cu -- the Mamba-1 selective scan over whole sequences (mamba_selective_scan).
//
// Source: "Triton decode kernel + MBU analysis", "Kernel design" (the per-token arithmetic) and
// "Prefill path" (a scan over the prompt).
#include "scan_common.cuh"

namespace gdn {

// Shared memory of the scan kernels, in bytes.
template <typename Tin, class Sh> struct ScanSmem {
    static constexpr int RX = kScanTile * Sh::CB * (int)sizeof(Tin);     // a staged x, dt or z tile
    static constexpr int RB = kScanTile * Sh::NP * (int)sizeof(Tin);     // a staged B or C tile
    static constexpr int STAGE = 3 * RX + 2 * RB;
    static constexpr int Q = kScanTile * Sh::CB * 16;                    // {dt, dt, dt x, dt x}
    static constexpr int WIDE = sizeof(Tin) == 4 ? 0 : kScanTile * Sh::NP * 4;
    static constexpr int Y = kScanTile * Sh::YP * 4;
    static constexpr int MAIN = 2 * STAGE + Q + 2 * WIDE + Y;
};

// One CTA: rows g C .. of channel tile ct. SUM: the summary pass (end state from zero and sum of dt
// of the sequence that goes on behind the chunk); else the outputs.
template <typename Tin, int NL, int CPT, bool SUM>
__global__ void __launch_bounds__(kScanThreads) scan_forward_kernel(const __grid_constant__ ScanLaunch P)
{
    using Sh = ScanShape<NL, CPT>;
    using Sm = ScanSmem<Tin, Sh>;
    constexpr int CB = Sh::CB, NP = Sh::NP;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[kScanWarps];
    ordinary_launch_start();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, cl = lane / NL;
    const int ct = (int)(blockIdx.x % (unsigned)P.nct), g = (int)(blockIdx.x / (unsigned)P.nct);
    const int D = P.a.D, N = P.a.N;
    const int c0 = ct * CB, ncols = min(CB, D - c0);
    const int n0 = 4 * nl, wc = warp * Sh::CW + cl;          // this thread's channels: wc + c CLN
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

    f2 A2[CPT][2], h[CPT][2];
    float dts[CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        A2[c][0] = A2[c][1] = h[c][0] = h[c][1] = 0ull;
        if (row0 < row1) load_rates(P.a.A, c0 + wc + c * Sh::CLN, D, n0, N, vst, A2[c]);
        dts[c] = 0.f;
    }

    float4 *q = reinterpret_cast<float4 *>(smem + 2 * Sm::STAGE);
    float *wideB = reinterpret_cast<float *>(smem + 2 * Sm::STAGE + Sm::Q), *wideC = wideB + Sm::WIDE / 4;
    float *ys = reinterpret_cast<float *>(smem + 2 * Sm::STAGE + Sm::Q + 2 * Sm::WIDE);

    auto stage_tile = [&](const ScanTile &t, int b) {
        Tin *xs = reinterpret_cast<Tin *>(smem + b * Sm::STAGE);
        Tin *ds = xs + kScanTile * CB, *zs = ds + kScanTile * CB;
        Tin *Bs = zs + kScanTile * CB, *Cs = Bs + kScanTile * NP;
        const int64_t r = t.t0;
        stage_rows<Tin, CB>(xs, static_cast<const Tin *>(P.a.x) + r * P.a.x_stride + c0, P.a.x_stride, t.n, ncols, P.vec & kVecX, tid);
        stage_rows<Tin, CB>(ds, static_cast<const Tin *>(P.a.dt) + r * P.a.dt_stride + c0, P.a.dt_stride, t.n, ncols, P.vec & kVecDt, tid);
        stage_rows<Tin, NP>(Bs, static_cast<const Tin *>(P.a.Bm) + r * P.a.B_stride, P.a.B_stride, t.n, N, P.vec & kVecB, tid);
        if (!SUM) {
            if (P.a.z)
                stage_rows<Tin, CB>(zs, static_cast<const Tin *>(P.a.z) + r * P.a.z_stride + c0, P.a.z_stride, t.n, ncols, P.vec & kVecZ, tid);
            stage_rows<Tin, NP>(Cs, static_cast<const Tin *>(P.a.Cm) + r * P.a.C_stride, P.a.C_stride, t.n, N, P.vec & kVecC, tid);
        }
    };

    ScanTile tl, nxt;
    if (load.next(P, nxt)) stage_tile(nxt, 0);
    cp_async_commit();
    int b = 0;
    while (use.next(P, tl)) {
        cp_async_wait<0>();
        __syncthreads();             // the tile is here, and the buffers of the one before are free
        if (load.next(P, nxt)) stage_tile(nxt, b ^ 1);
        cp_async_commit();

        const Tin *xs = reinterpret_cast<const Tin *>(smem + b * Sm::STAGE);
        const Tin *ds = xs + kScanTile * CB, *zs = ds + kScanTile * CB;
        const Tin *Bs = zs + kScanTile * CB, *Cs = Bs + kScanTile * NP;
#pragma unroll
        for (int i = tid * 4; i < kScanTile * CB; i += kScanThreads * 4) {
            const float4 x4 = load4(xs + i), d4 = load4(ds + i);
            const float u0 = d4.x * x4.x, u1 = d4.y * x4.y, u2 = d4.z * x4.z, u3 = d4.w * x4.w;
            q[i] = make_float4(d4.x, d4.x, u0, u0);
            q[i + 1] = make_float4(d4.y, d4.y, u1, u1);
            q[i + 2] = make_float4(d4.z, d4.z, u2, u2);
            q[i + 3] = make_float4(d4.w, d4.w, u3, u3);
        }
        const float *Bf = as_f32(Bs, wideB, kScanTile * NP, tid);
        const float *Cf = SUM ? nullptr : as_f32(Cs, wideC, kScanTile * NP, tid);
        __syncthreads();

        if (tl.fresh) {
            const float *from = nullptr;
            if (!SUM && tl.seq >= 0)
                // (a sequence that goes on behind the chunk: in place, a later chunk's CTA may already have
                // written its row of h_last, so its initial state comes from the carry pass's copy)
                from = !tl.starts ? (P.hin ? P.hin + g * dn : nullptr)
                       : !P.a.h0  ? nullptr
                       : P.hin && g < P.G - 1 && P.info[g].x == tl.seq ? P.init + g * dn : P.a.h0 + tl.slot * dn;
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                h[c][0] = h[c][1] = 0ull;
                if (from) load_entries(from, c0 + wc + c * Sh::CLN, D, n0, N, vst, h[c]);
            }
        }

        float dt_tile[CPT];
#pragma unroll
        for (int c = 0; c < CPT; ++c) dt_tile[c] = 0.f;
        // rows behind the tile's last are zeros: dt = 0 leaves h as it is
#pragma unroll 1
        for (int t4 = 0; t4 < kScanTile; t4 += 4) {
            float acc[4 * CPT];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = t4 + k;
                const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(Bf + t * NP + n0);
                ulonglong2 C = make_ulonglong2(0, 0);
                if (!SUM) C = *reinterpret_cast<const ulonglong2 *>(Cf + t * NP + n0);
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(q + t * CB + wc + c * Sh::CLN);
                    h[c][0] = fma2(decay2(du.x, A2[c][0]), h[c][0], mul2(du.y, B.x));
                    h[c][1] = fma2(decay2(du.x, A2[c][1]), h[c][1], mul2(du.y, B.y));
                    if (SUM) {
                        dt_tile[c] += unpack2(du.x).x;
                    } else {
                        const float2 s = unpack2(fma2(C.y, h[c][1], mul2(C.x, h[c][0])));
                        acc[k * CPT + c] = s.x + s.y;
                    }
                }
            }
            if (!SUM) {
                constexpr int M = 4 * CPT;
                group_reduce<M, NL>(acc, nl);
                if (M >= NL) {
#pragma unroll
                    for (int i = 0; i < (M >= NL ? M / NL : 1); ++i) {
                        const int v = nl * (M / NL) + i;
                        ys[(t4 + v / CPT) * Sh::YP + wc + (v % CPT) * Sh::CLN] = acc[i];
                    }
                } else {
                    constexpr int R = M >= NL ? 1 : NL / M;
                    const int v = nl / R;
                    if (nl % R == 0) ys[(t4 + v / CPT) * Sh::YP + wc + (v % CPT) * Sh::CLN] = acc[0];
                }
            }
        }
        if (SUM) {
#pragma unroll
            for (int c = 0; c < CPT; ++c) dts[c] += dt_tile[c];
        } else {
            if (tl.ends && P.a.h_last) {
#pragma unroll
                for (int c = 0; c < CPT; ++c)
                    store_entries(P.a.h_last + tl.slot * dn, c0 + wc + c * Sh::CLN, D, n0, N, vst, h[c]);
            }
            __syncthreads();
            // skip, gate and output of the tile's rows
            for (int i = tid * 4; i < tl.n * CB; i += kScanThreads * 4) {
                const int r = i / CB, c = i % CB;
                if (c >= ncols) continue;
                float4 y = *reinterpret_cast<const float4 *>(ys + r * Sh::YP + c);
                if (P.a.Dskip) {
                    const float4 x4 = load4(xs + i);
                    const float *dp = P.a.Dskip + c0 + c;
                    y.x = fmaf(dp[0], x4.x, y.x);
                    if (c + 1 < ncols) y.y = fmaf(dp[1], x4.y, y.y);
                    if (c + 2 < ncols) y.z = fmaf(dp[2], x4.z, y.z);
                    if (c + 3 < ncols) y.w = fmaf(dp[3], x4.w, y.w);
                }
                if (P.a.z) {
                    const float4 z4 = load4(zs + i);
                    y.x *= z4.x * fast_sigmoid(z4.x);
                    y.y *= z4.y * fast_sigmoid(z4.y);
                    y.z *= z4.z * fast_sigmoid(z4.z);
                    y.w *= z4.w * fast_sigmoid(z4.w);
                }
                if (tl.seq < 0) y = make_float4(0.f, 0.f, 0.f, 0.f);
                const int64_t o = (int64_t)(tl.t0 + r) * P.a.y_stride + c0 + c;
                if (P.a.out_dtype == GDN_BF16)
                    store_row4(static_cast<bf16 *>(P.a.y) + o, y, ncols - c, P.vec & kVecY);
                else
                    store_row4(static_cast<float *>(P.a.y) + o, y, ncols - c, P.vec & kVecY);
            }
        }
        b ^= 1;
    }
    if (SUM) {
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const int d = c0 + wc + c * Sh::CLN;
            store_entries(P.hin + g * dn, d, D, n0, N, vst, h[c]);
            if (nl == 0 && d < D) P.sumdt[(int64_t)g * D + d] = dts[c];
        }
    }
}

template <typename Tin, int NL, int CPT, bool SUM>
static cudaError_t launch_one(const ScanLaunch &P, int chunks, cudaStream_t stream)
{
    constexpr int bytes = ScanSmem<Tin, ScanShape<NL, CPT>>::MAIN;
    auto kern = scan_forward_kernel<Tin, NL, CPT, SUM>;
    if (bytes > 48 * 1024) {
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

template <typename Tin> static int launch_typed(const ScanLaunch &P, cudaStream_t stream)
{
    switch (scan_shape(P.a.N).NL) {
    case 2: return launch_shape<Tin, 2, 2>(P, stream);
    case 4: return launch_shape<Tin, 4, 2>(P, stream);
    case 8: return launch_shape<Tin, 8, 2>(P, stream);
    case 16: return launch_shape<Tin, 16, 4>(P, stream);
    default: return launch_shape<Tin, 32, 4>(P, stream);
    }
}

int launch_scan_forward(const ScanLaunch &P, cudaStream_t stream)
{
    return P.a.in_dtype == GDN_BF16 ? launch_typed<bf16>(P, stream) : launch_typed<float>(P, stream);
}

}  // namespace gdn
