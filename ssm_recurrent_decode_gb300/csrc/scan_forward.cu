// scan_forward.cu -- the Mamba-1 selective scan over whole sequences (mamba_selective_scan).
//
// Source: "Triton decode kernel + MBU analysis", "Kernel design" (the per-token arithmetic) and
// "Prefill path" (a scan over the prompt).
#include "gdn_cluster.cuh"
#include "scan_common.cuh"

namespace gdn {

// Shared memory, in bytes.
template <typename Tin, class Sh> struct ScanSmem {
    static constexpr int RX = kScanTile * Sh::CB * (int)sizeof(Tin);     // a staged x, dt or z tile
    static constexpr int RB = kScanTile * Sh::NP * (int)sizeof(Tin);     // a staged B or C tile
    static constexpr int STAGE = 3 * RX + 2 * RB;
    static constexpr int HALF = 8;                                       // rows between two stores of outputs
    static constexpr int PARTS = Sh::NL <= 4 ? Sh::NL : 1;               // sums over n still to be joined
    static constexpr int JOIN = Sh::NL > 4 ? HALF * 32 * Sh::CPT * 4 : 0;   // a warp's sums before eight lanes' are joined
    static constexpr int Y = kScanWarps * (HALF * PARTS * Sh::YP * 4 + JOIN);
    static constexpr int MAIN = 2 * STAGE + Y;
    static constexpr int SUMMARY = 2 * STAGE;
};

// A thread's place: its CTA's chunk and channel tile, its lanes, its first state entry and channel.
template <class Sh> struct ScanPlace {
    int tid, lane, warp, nl, cl, ct, g, c0, ncols, n0, wc, d0, row0, row1;
    __device__ __forceinline__ ScanPlace(const ScanLaunch &P, int g_, int ct_)
    {
        tid = threadIdx.x;
        lane = tid & 31;
        warp = tid >> 5;
        nl = lane % Sh::NL;
        cl = lane / Sh::NL;
        g = g_;
        ct = ct_;
        c0 = ct * Sh::CB;
        ncols = min(Sh::CB, P.a.D - c0);
        n0 = 4 * nl;
        wc = warp * Sh::CW + cl * Sh::CPT;
        d0 = c0 + wc;
        row0 = (int)min((int64_t)g * P.C, (int64_t)P.a.T);
        row1 = (int)min((int64_t)(g + 1) * P.C, (int64_t)P.a.T);
    }
};

// What a summary is taken of: the rows from `first` on of the sequence that goes on behind the chunk.
struct ScanTail {
    int seq, first;
    bool goes_on, begins;       // begins: in this chunk
};
template <class Sh> __device__ __forceinline__ ScanTail scan_tail(const ScanLaunch &P, const ScanPlace<Sh> &at, int *scratch)
{
    ScanTail t;
    t.seq = find_seq(P, at.row1 - 1, scratch, at.tid);
    t.goes_on = t.seq >= 0 && t.seq < P.a.S && seq_bound(P, t.seq + 1) > at.row1;
    t.begins = t.goes_on && seq_bound(P, t.seq) >= at.row0;
    t.first = t.goes_on ? max(seq_bound(P, t.seq), at.row0) : at.row1;
    return t;
}

// Walks the rows of `load` tile by tile. SUM: only the states (h ends as the last row's) and the sum of dt; else
// the outputs too. start(tile, h) sets h where a sequence begins or the chunk does. Tiles of 16 rows are
// staged one ahead by asynchronous copies; a warp's channels are its own, so only the staging needs barriers.
template <typename Tin, class Sh, bool SUM, typename Start>
__device__ __forceinline__ void scan_pass(const ScanLaunch &P, unsigned char *smem, const ScanPlace<Sh> &at, ScanIter load,
                                          const f2 (&A2)[4][Sh::P], f2 (&h)[4][Sh::P], f2 (&dts)[Sh::P], Start start)
{
    using Sm = ScanSmem<Tin, Sh>;
    constexpr int NL = Sh::NL, CPT = Sh::CPT, CB = Sh::CB, NP = Sh::NP, PP = Sh::P, CLN = Sh::CLN;
    const int tid = at.tid, lane = at.lane, warp = at.warp, nl = at.nl, cl = at.cl, c0 = at.c0, ncols = at.ncols, n0 = at.n0,
              wc = at.wc, D = P.a.D, N = P.a.N;
    const int64_t dn = (int64_t)D * N;
    const bool vst = (P.vec & kVecState) != 0;
    ScanIter use = load;

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
    float *before = reinterpret_cast<float *>(smem + 2 * Sm::STAGE) + kScanWarps * Sm::HALF * Sm::PARTS * Sh::YP + warp * (Sm::JOIN / 4);

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
            zero_entries(h);
            if (tl.seq >= 0) start(tl, h);
        }

        f2 dt_tile[PP] = {};
        // rows behind the tile's last are zeros: dt = 0 leaves h as it is
#pragma unroll 1
        for (int t8 = 0; t8 < kScanTile; t8 += Sm::HALF) {
#pragma unroll
            for (int t4 = t8; t4 < t8 + Sm::HALF; t4 += 4) {       // eight rows' work to schedule among (401 -> 379 us)
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
                    }
                    // up to four lanes' sums are joined where the row is finished, more of them eight by eight below
                    if (!SUM && NL <= 4) store_pairs(ys + ((t - t8) * NL + nl) * Sh::YP + cl * CPT, y);
                    if (!SUM && NL > 4) store_pairs(before + ((t - t8) * 32 + lane) * CPT, y);
                }
            }
            if (!SUM && NL > 4) {
                // the eight rows' 256 sums, eight to a lane (each lane begins at another, for the banks): those of one
                // row and channel lane lie in NL / 8 lanes
                __syncwarp();
                f2 y[PP];
                load_pairs(before + (lane * 8 + (lane & 7)) * CPT, y);
#pragma unroll
                for (int i = 1; i < 8; ++i) {
                    f2 more[PP];
                    load_pairs(before + (lane * 8 + ((lane + i) & 7)) * CPT, more);
#pragma unroll
                    for (int p = 0; p < PP; ++p) y[p] = add2(y[p], more[p]);
                }
#pragma unroll
                for (int off = 1; off < NL / 8; off <<= 1)
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        const float2 v = unpack2(y[p]);
                        y[p] = add2(y[p], pack2(__shfl_xor_sync(kScanFull, v.x, off), __shfl_xor_sync(kScanFull, v.y, off)));
                    }
                constexpr int SHARE = NL >= 8 ? NL / 8 : 1;
                if (lane % SHARE == 0) store_pairs(ys + lane / 4 * Sh::YP + lane % 4 * 8 / NL * CPT, y);
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
                    if (P.a.z) y[p] = mul2(y[p], mul2(z2[p], sigmoid2(z2[p])));
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
            store_entries(P.a.h_last + tl.slot * dn, at.d0, D, n0, N, vst, h);
        }
        b ^= 1;
    }
}

// An empty sequence passes its state on: each is handled by one chunk's CTAs.
template <class Sh> __device__ __forceinline__ void pass_empty_on(const ScanLaunch &P, const ScanPlace<Sh> &at)
{
    if (!P.a.h_last || P.a.h_last == P.a.h0 || (!P.a.cu_seqlens && P.L != 0)) return;
    const int64_t dn = (int64_t)P.a.D * P.a.N;
    for (int s = at.g; s < P.a.S; s += P.G) {
        if (seq_bound(P, s) != seq_bound(P, s + 1)) continue;
        const int64_t slot = P.a.state_indices ? (int64_t)P.a.state_indices[s] : s;
        if (slot < 0 || slot >= P.a.num_states) {
            if (at.tid == 0) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
            continue;
        }
        for (int i = at.tid; i < at.ncols * P.a.N; i += kScanThreads) {
            const int64_t o = slot * dn + (int64_t)at.c0 * P.a.N + i;
            P.a.h_last[o] = P.a.h0 ? P.a.h0[o] : 0.f;
        }
    }
}

// One CTA: the rows of chunk g, channel tile ct. SUM: the summary pass (end state from zero and sum of dt
// of the sequence that goes on behind the chunk); else the outputs.
template <typename Tin, int NL, int CPT, bool SUM>
__global__ void __launch_bounds__(kScanThreads, scan_ctas(NL)) scan_forward_kernel(const __grid_constant__ ScanLaunch P)
{
    using Sh = ScanShape<NL, CPT>;
    constexpr int PP = Sh::P;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[kScanWarps];
    ordinary_launch_start();

    const ScanPlace<Sh> at(P, (int)(blockIdx.x / (unsigned)P.nct), (int)(blockIdx.x % (unsigned)P.nct));
    const int D = P.a.D, N = P.a.N, g = at.g;
    const int64_t dn = (int64_t)D * N;
    const bool vst = (P.vec & kVecState) != 0;
    ScanIter rows;
    if (SUM) {
        const ScanTail t = scan_tail(P, at, scratch);
        if (at.tid == 0 && at.ct == 0) P.info[g] = make_int4(t.goes_on ? t.seq : -1, t.begins, 0, 0);
        if (!t.goes_on) return;
        rows.init(t.first, at.row1, t.seq);
    } else {
        rows.init(at.row0, at.row1, find_seq(P, at.row0, scratch, at.tid));
        pass_empty_on(P, at);
    }
    f2 A2[4][PP], h[4][PP], dts[PP];
    zero_entries(A2);
    if (at.row0 < at.row1) load_rates(P.a.A, at.d0, D, at.n0, N, vst, A2);
    zero_entries(h);
    scan_pass<Tin, Sh, SUM>(P, smem, at, rows, A2, h, dts, [&](const ScanTile &tl, f2 (&v)[4][PP]) {
        if (SUM) return;             // from zero
        // (a sequence that goes on behind the chunk: in place, a later chunk's CTA may already have
        // written its row of h_last, so its initial state comes from the carry pass's copy)
        const float *from = !tl.starts ? (P.hin ? P.hin + g * dn : nullptr)
                            : !P.a.h0  ? nullptr
                            : P.hin && g < P.G - 1 && P.info[g].x == tl.seq ? P.init + g * dn : P.a.h0 + tl.slot * dn;
        if (from) load_entries(from, at.d0, D, at.n0, N, vst, v);
    });
    if (SUM && GDN_IN(P.a.err_flags, g, P.G)) {
        store_entries(P.hin + g * dn, at.d0, D, at.n0, N, vst, h);
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            const float2 v = unpack2(dts[p]);
            const int d = at.d0 + 2 * p;
            if (at.nl == 0 && d < D) P.sumdt[(int64_t)g * D + d] = v.x;
            if (at.nl == 0 && d + 1 < D) P.sumdt[(int64_t)g * D + d + 1] = v.y;
        }
    }
}

// A short call in one launch: its up to eight chunks are the CTAs of a thread-block cluster (per channel
// tile). Each takes its summary, reads those before it from the other CTAs' shared memory, folds them into
// the state it starts from, and takes its outputs. (One prompt of 128 tokens, D = 1536, N = 16: 11.9 us; in
// one pass without chunks 17.0, in three launches 20.)
template <typename Tin, int NL, int CPT>
__global__ void __launch_bounds__(kScanThreads) scan_cluster_kernel(const __grid_constant__ ScanLaunch P)
{
    using Sh = ScanShape<NL, CPT>;
    constexpr int PP = Sh::P;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[kScanWarps];
    __shared__ int2 info[8];                         // per rank: goes on, begins there
    // a thread's entries n = 0 .. 3 of each channel: the initial state of the sequence that goes on, its end
    // state from zero, and its channels' sums of dt
    __shared__ float4 first_state[2 * PP][kScanThreads], end_state[2 * PP][kScanThreads], sum_dt[kScanThreads];
    ordinary_launch_start();

    // the cluster's CTAs are consecutive: rank g of channel tile ct
    const ScanPlace<Sh> at(P, (int)(blockIdx.x % (unsigned)P.G), (int)(blockIdx.x / (unsigned)P.G));
    const int D = P.a.D, N = P.a.N, tid = at.tid;
    const int64_t dn = (int64_t)D * N;
    const bool vst = (P.vec & kVecState) != 0;
    f2 A2[4][PP], h[4][PP], dts[PP];
    load_rates(P.a.A, at.d0, D, at.n0, N, vst, A2);

    const auto put = [&](float4 (&to)[2 * PP][kScanThreads], const f2 (&v)[4][PP]) {
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            const float2 a = unpack2(v[0][p]), b = unpack2(v[1][p]), c = unpack2(v[2][p]), d = unpack2(v[3][p]);
            to[2 * p][tid] = make_float4(a.x, b.x, c.x, d.x);
            to[2 * p + 1][tid] = make_float4(a.y, b.y, c.y, d.y);
        }
    };
    const auto get = [&](const float4 (&from)[2 * PP][kScanThreads], f2 (&v)[4][PP]) {
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            const float4 x = from[2 * p][tid], y = from[2 * p + 1][tid];
            v[0][p] = pack2(x.x, y.x);
            v[1][p] = pack2(x.y, y.y);
            v[2][p] = pack2(x.z, y.z);
            v[3][p] = pack2(x.w, y.w);
        }
    };
    const ScanTail tail = scan_tail(P, at, scratch);
    const bool goes_on = tail.goes_on && at.g + 1 < P.G;
    cluster_sync_all();              // the others' shared memory exists
    ScanIter rows;
    if (goes_on) {
        rows.init(tail.first, at.row1, tail.seq);
        zero_entries(h);
        scan_pass<Tin, Sh, true>(P, smem, at, rows, A2, h, dts, [](const ScanTile &, f2 (&)[4][PP]) {});
        put(end_state, h);
        const float2 s0 = unpack2(dts[0]), s1 = unpack2(dts[PP - 1]);
        sum_dt[tid] = make_float4(s0.x, s0.y, s1.x, s1.y);
        // read before any CTA of the cluster writes a final state: h_last may be h0
        f2 v[4][PP];
        zero_entries(v);
        if (tail.begins && P.a.h0) {
            const int64_t slot = P.a.state_indices ? (int64_t)P.a.state_indices[tail.seq] : tail.seq;
            if (slot >= 0 && slot < P.a.num_states) load_entries(P.a.h0 + slot * dn, at.d0, D, at.n0, N, vst, v);
        }
        put(first_state, v);
    }
    // everyone's flags to everyone, so that none has to be fetched below
    if (tid < P.G) cluster_st_s32x2(cluster_map(smem_u32(&info[at.g]), tid), goes_on, tail.begins);
    cluster_sync_all();

    // the state this chunk starts from: the summaries of the chunks before it, from the one on in which
    // its first row's sequence begins
    f2 carry[4][PP];
    zero_entries(carry);
    int from = at.g;
    while (from > 0 && info[from - 1].x && (from == at.g || !info[from].y)) --from;
    struct Summary {
        float4 end[2 * PP], dt;
    };
    const auto fetch = [&](int r) {
        Summary q;
        q.dt = cluster_ld_f32x4(cluster_map(smem_u32(&sum_dt[tid]), r));
#pragma unroll
        for (int c = 0; c < 2 * PP; ++c) q.end[c] = cluster_ld_f32x4(cluster_map(smem_u32(&end_state[c][tid]), r));
        return q;
    };
    if (from < at.g) {
        if (info[from].y) {
#pragma unroll
            for (int c = 0; c < 2 * PP; c += 2) {
                const float4 x = cluster_ld_f32x4(cluster_map(smem_u32(&first_state[c][tid]), from)),
                             y = cluster_ld_f32x4(cluster_map(smem_u32(&first_state[c + 1][tid]), from));
                carry[0][c / 2] = pack2(x.x, y.x);
                carry[1][c / 2] = pack2(x.y, y.y);
                carry[2][c / 2] = pack2(x.z, y.z);
                carry[3][c / 2] = pack2(x.w, y.w);
            }
        }
        // a remote load takes most of a microsecond: as many ranks' as the registers hold are under way together
        constexpr int BATCH = PP == 1 ? 7 : 4;
        for (int r0 = from; r0 < at.g; r0 += BATCH) {
            Summary q[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (r0 + i < at.g) q[i] = fetch(r0 + i);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (r0 + i >= at.g) break;
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    const f2 dt = p == 0 ? pack2(q[i].dt.x, q[i].dt.y) : pack2(q[i].dt.z, q[i].dt.w);
                    const float4 ex = q[i].end[2 * p], ey = q[i].end[2 * p + 1];
                    const float lx[4] = {ex.x, ex.y, ex.z, ex.w}, ly[4] = {ey.x, ey.y, ey.z, ey.w};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float2 c = unpack2(carry[n][p]), a = unpack2(decay2(dt, A2[n][p]));
                        // no product with the decay where nothing is carried: 0 x inf is not 0
                        carry[n][p] = pack2(c.x == 0.f ? lx[n] : fmaf(a.x, c.x, lx[n]), c.y == 0.f ? ly[n] : fmaf(a.y, c.y, ly[n]));
                    }
                }
            }
        }
    }
    cluster_sync_all();              // every CTA has read what it needs of the others

    rows.init(at.row0, at.row1, find_seq(P, at.row0, scratch, tid));
    pass_empty_on(P, at);
    zero_entries(h);
    scan_pass<Tin, Sh, false>(P, smem, at, rows, A2, h, dts, [&](const ScanTile &tl, f2 (&v)[4][PP]) {
        if (!tl.starts) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int p = 0; p < PP; ++p) v[n][p] = carry[n][p];
        } else if (goes_on && tl.seq == tail.seq) {
            get(first_state, v);
        } else if (P.a.h0) {
            load_entries(P.a.h0 + tl.slot * dn, at.d0, D, at.n0, N, vst, v);
        }
    });
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

template <typename Tin, int NL, int CPT> static cudaError_t launch_cluster(const ScanLaunch &P, cudaStream_t stream)
{
    constexpr int bytes = ScanSmem<Tin, ScanShape<NL, CPT>>::MAIN;
    auto kern = scan_cluster_kernel<Tin, NL, CPT>;
    const cudaError_t rc = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (rc != cudaSuccess) return rc;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    set_programmatic(attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)P.G;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(P.G * P.nct));
    cfg.blockDim = dim3(kScanThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, P);
}

template <typename Tin, int NL, int CPT> static int launch_shape(const ScanLaunch &P, cudaStream_t stream)
{
    if (P.cluster) return launch_cluster<Tin, NL, CPT>(P, stream) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
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
