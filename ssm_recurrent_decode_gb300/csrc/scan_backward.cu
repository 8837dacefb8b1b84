// scan_backward.cu -- gradients of the Mamba-1 selective scan (mamba_selective_scan_backward).
//
// Per state entry, with g = dy silu(z), u = dt x, a = exp(dt A) and e the gradient that arrives from
// the next token:
//     dh = C g + e,   e' = a dh,   w = e' h_{t-1}      (e' goes on to the token before; w = dL/d(dt A))
//     dC += g h,  dB += u dh  (sums over channels)     du = sum_n B dh,  ddt = x du + sum_n A w
//     dA += dt w  (sum over tokens)                    dx = dt du + D g
// Launches: (1) per chunk the end state from zero and what its rows send to the row before it (one
// pass, one exp per entry: the products of the decays from the chunk's first row give both); (2) the
// carries over the chunks; (3) the gradients; (4) sums of the per-CTA parts of dB, dC, dA, dD.
#include "scan_common.cuh"

namespace gdn {

constexpr int kBackTile = 8;        // token rows per tile: their states and decays fit a thread's registers
constexpr int kBackTiles = kScanBackChunk / kBackTile;

template <typename Tin, class Sh> struct BackSmem {
    static constexpr int R = kBackTile;
    static constexpr int RX = R * Sh::CB * (int)sizeof(Tin);              // a staged x, dt, z or dy tile
    static constexpr int RB = R * Sh::NP * (int)sizeof(Tin);              // a staged B or C tile
    static constexpr int STAGE = 4 * RX + 2 * RB;
    static constexpr int SUMS = kScanWarps * R * Sh::YP * 4;              // a value per row and channel
    // Sums over the state's lanes: up to four lanes' are joined through shared memory where the rows are finished,
    // four rows at a time (bf16: the room is there beside two CTAs' stages), others by shuffles (8 x 2048 rows,
    // N = 16, bf16: 760 us joined, 778 by shuffles).
    static constexpr bool JOINED = Sh::NL <= 4 && sizeof(Tin) == 2;
    static constexpr int LANES = JOINED ? Sh::NL : 1, HALF = JOINED ? 4 : R;       // HALF rows are finished at a time
    static constexpr int JOIN = kScanWarps * HALF * LANES * Sh::YP * 4;
    static constexpr int JOIN_Y = JOINED ? JOIN : SUMS;       // the shuffled sums of C h are taken with the states, all rows'
    static constexpr int PART = kScanWarps * R * 2 * Sh::NP * 4;          // dB and dC per warp
    static constexpr int STATES = (kBackTiles - 2) * 4 * kScanThreads * 8 * Sh::P;   // not before the first and the last tile
    static constexpr int SUMMARY = 2 * STAGE + SUMS;
    static constexpr int MAIN = 2 * STAGE + SUMS + JOIN_Y + 2 * JOIN + PART + STATES;
};

// the sum of LANES vectors of pairs, one row pitch apart
template <int LANES, int PITCH, int P> __device__ __forceinline__ void join_lanes(const float *from, f2 (&v)[P])
{
    load_pairs(from, v);
#pragma unroll
    for (int q = 1; q < LANES; ++q) {
        f2 more[P];
        load_pairs(from + q * PITCH, more);
#pragma unroll
        for (int p = 0; p < P; ++p) v[p] = add2(v[p], more[p]);
    }
}

// Staging that the summary and the gradient kernel share, and g = dy silu(z) of a tile.
template <typename Tin, class Sh> struct BackTile {
    using Sm = BackSmem<Tin, Sh>;
    static constexpr int CB = Sh::CB, NP = Sh::NP, R = kBackTile;
    const ScanLaunch &P;
    unsigned char *smem;
    int tid, c0, ncols;

    __device__ __forceinline__ BackTile(const ScanLaunch &P_, unsigned char *s, int tid_, int c0_)
        : P(P_), smem(s), tid(tid_), c0(c0_), ncols(min(CB, P_.a.D - c0_))
    {
    }
    __device__ __forceinline__ Tin *raw(int b, int k) const      // k: 0 x, 1 dt, 2 z, 3 dy
    {
        return reinterpret_cast<Tin *>(smem + b * Sm::STAGE + k * Sm::RX);
    }
    __device__ __forceinline__ Tin *raw_bc(int b, int k) const   // k: 0 B, 1 C
    {
        return reinterpret_cast<Tin *>(smem + b * Sm::STAGE + 4 * Sm::RX + k * Sm::RB);
    }
    // rows t0 .. t0 + n - 1 into buffer b (LAST: as the tile's last rows); grads: also what only the gradients need
    template <bool LAST> __device__ __forceinline__ void stage(int b, int t0, int n, bool grads)
    {
        const auto rows = [&](const void *base, int64_t stride, int col, int width, int mode) {
            return TileSource<Tin>{static_cast<const Tin *>(base), stride, t0, P.a.T, col, width, mode};
        };
        stage_rows<Tin, CB, R, LAST>(raw(b, 0), rows(P.a.x, P.a.x_stride, c0, P.a.D, P.mode_x), n, tid);
        stage_rows<Tin, CB, R, LAST>(raw(b, 1), rows(P.a.dt, P.a.dt_stride, c0, P.a.D, P.mode_dt), n, tid);
        stage_rows<Tin, NP, R, LAST>(raw_bc(b, 0), rows(P.a.Bm, P.a.B_stride, 0, P.a.N, P.mode_b), n, tid);
        if (grads) {
            if (P.a.z) stage_rows<Tin, CB, R, LAST>(raw(b, 2), rows(P.a.z, P.a.z_stride, c0, P.a.D, P.mode_z), n, tid);
            stage_rows<Tin, CB, R, LAST>(raw(b, 3), rows(P.g.dy, P.g.dy_stride, c0, P.a.D, P.mode_dy), n, tid);
            stage_rows<Tin, NP, R, LAST>(raw_bc(b, 1), rows(P.a.Cm, P.a.C_stride, 0, P.a.N, P.mode_c), n, tid);
        }
    }
    // g of this warp's channels into gs [R][YP]; the warp alone reads it
    __device__ __forceinline__ void gate(int b, float *gs, int lane, int warp)
    {
        constexpr int CLN = Sh::CLN, NL = Sh::NL, PP = Sh::P;
        const int c = lane % CLN * Sh::CPT;
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += NL) {
            const int r = r0 + lane / CLN;
            if (NL > R && r >= R) break;
            f2 g[PP], z[PP];
            load_pairs(raw(b, 3) + r * CB + warp * Sh::CW + c, g);
            if (P.a.z) {
                load_pairs(raw(b, 2) + r * CB + warp * Sh::CW + c, z);
#pragma unroll
                for (int p = 0; p < PP; ++p) g[p] = mul2(g[p], mul2(z[p], sigmoid2(z[p])));
            }
            store_pairs(gs + r * Sh::YP + c, g);
        }
    }
};

// (1) The summaries of chunk g: for the sequence that goes on behind the chunk its end state from
// zero, for the sequence that began before it what its rows send back. Usually one and the same.
template <typename Tin, int NL, int CPT>
__global__ void __launch_bounds__(kScanThreads, 4) scan_back_summary_kernel(const __grid_constant__ ScanLaunch P)
{
    using Sh = ScanShape<NL, CPT>;
    using Sm = BackSmem<Tin, Sh>;
    constexpr int R = kBackTile, NP = Sh::NP, CB = Sh::CB, PP = Sh::P;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[kScanWarps];
    ordinary_launch_start();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, cl = lane / NL;
    const int ct = (int)(blockIdx.x % (unsigned)P.nct), g = (int)(blockIdx.x / (unsigned)P.nct);
    const int D = P.a.D, N = P.a.N, c0 = ct * CB;
    const int n0 = 4 * nl, wc = warp * Sh::CW + cl * CPT, d0 = c0 + wc;
    const int64_t dn = (int64_t)D * N;
    const bool vst = (P.vec & kVecState) != 0;
    const int row0 = g * P.C, row1 = (int)min((int64_t)P.a.T, (int64_t)row0 + P.C);

    const int sh = find_seq(P, row0, scratch, tid), st = find_seq(P, row1 - 1, scratch, tid);
    const bool before = sh >= 0 && sh < P.a.S && seq_bound(P, sh) < row0;
    const bool behind = st >= 0 && st < P.a.S && seq_bound(P, st + 1) > row1;
    const int head_end = before ? min(seq_bound(P, sh + 1), row1) : row0;
    const int tail_begin = behind ? max(seq_bound(P, st), row0) : row1;
    if (tid == 0 && ct == 0)
        P.info[g] = make_int4(behind ? st : -1, behind && seq_bound(P, st) >= row0, before ? sh : -1,
                              before && seq_bound(P, sh + 1) <= row1);

    BackTile<Tin, Sh> T(P, smem, tid, c0);
    float *gs = reinterpret_cast<float *>(smem + 2 * Sm::STAGE) + warp * R * Sh::YP;
    // rows row0 .. head_end - 1 (head) and tail_begin .. row1 - 1 (tail); tiles do not cross either border
    auto clip = [&](int pos) {
        int end = min(row1, pos + R);
        if (pos < head_end) end = min(end, head_end);
        if (pos < tail_begin) end = min(end, tail_begin);
        return end - pos;
    };
    auto first_at = [&](int pos) { return pos >= head_end && pos < tail_begin ? tail_begin : pos; };   // skips what is neither
    int pos = first_at(row0), b = 0;
    if (pos < row1) T.template stage<false>(0, pos, clip(pos), true);
    cp_async_commit();

    f2 A2[4][PP], h[4][PP], prod[4][PP], e[4][PP], dt_head[PP] = {}, dt_tail[PP] = {};
    load_rates(P.a.A, d0, D, n0, N, vst, A2);
    zero_entries(h);
    zero_entries(e);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int p = 0; p < PP; ++p) prod[n][p] = pack2(1.f, 1.f);

    while (pos < row1) {
        const bool head = pos < head_end, tail = pos >= tail_begin;
        const int next = first_at(pos + clip(pos));
        cp_async_wait<0>();
        __syncthreads();
        if (next < row1) T.template stage<false>(b ^ 1, next, clip(next), true);
        cp_async_commit();
        T.gate(b, gs, lane, warp);
        __syncwarp();
        const Tin *xs = T.raw(b, 0), *ds = T.raw(b, 1), *Bs = T.raw_bc(b, 0), *Cs = T.raw_bc(b, 1);
        f2 dts[PP] = {};
#pragma unroll
        for (int t = 0; t < R; ++t) {
            f2 dt[PP], u[PP], gv[PP], B[4], C[4];
            load_pairs(ds + t * CB + wc, dt);
            load_pairs(xs + t * CB + wc, u);
            load_pairs(gs + t * Sh::YP + cl * CPT, gv);
            load_twice(Bs + t * NP + n0, B);
            load_twice(Cs + t * NP + n0, C);
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                dts[p] = add2(dts[p], dt[p]);
                u[p] = mul2(u[p], dt[p]);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const f2 a = decay2(dt[p], A2[n][p]);
                    h[n][p] = fma2(a, h[n][p], mul2(u[p], B[n]));
                    prod[n][p] = mul2(prod[n][p], a);
                    e[n][p] = fma2(prod[n][p], mul2(C[n], gv[p]), e[n][p]);
                }
            }
        }
        if (!tail) zero_entries(h);          // the sequence that goes on behind the chunk has not begun
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            if (head) dt_head[p] = add2(dt_head[p], dts[p]);
            if (tail) dt_tail[p] = add2(dt_tail[p], dts[p]);
        }
        if (head && next >= head_end && before) store_entries(P.ein + g * dn, d0, D, n0, N, vst, e);
        __syncwarp();
        pos = next;
        b ^= 1;
    }
    if (behind) store_entries(P.hin + g * dn, d0, D, n0, N, vst, h);
#pragma unroll
    for (int p = 0; p < PP; ++p) {
        const float2 ht = unpack2(dt_head[p]), tt = unpack2(dt_tail[p]);
        const int d = d0 + 2 * p;
        const int64_t o = (int64_t)g * D + d;
        if (nl == 0 && d < D) {
            P.sumdt[o] = tt.x;
            P.sumdt_head[o] = ht.x;
        }
        if (nl == 0 && d + 1 < D) {
            P.sumdt[o + 1] = tt.y;
            P.sumdt_head[o + 1] = ht.y;
        }
    }
}

// (3) The gradients. A CTA owns a channel tile and walks the chunks w, w + W, ..., so that dA and dD
// stay in registers. In a chunk it takes each sequence's rows forward once, keeping the state before
// every tile in shared memory, then tile by tile backwards: the tile's states again, now kept in
// registers, and the recurrence of dh through them (the decays a third time: one instruction pair
// each, where keeping them would take another 128 registers).
template <typename Tin, int NL, int CPT>
__global__ void __launch_bounds__(kScanThreads, kScanBackCtas) scan_back_kernel(const __grid_constant__ ScanLaunch P)
{
    using Sh = ScanShape<NL, CPT>;
    using Sm = BackSmem<Tin, Sh>;
    constexpr int R = kBackTile, NP = Sh::NP, CB = Sh::CB, CLN = Sh::CLN, YP = Sh::YP, PP = Sh::P;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[kScanWarps];
    ordinary_launch_start();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, cl = lane / NL;
    const int ct = (int)(blockIdx.x % (unsigned)P.nct), w = (int)(blockIdx.x / (unsigned)P.nct);
    const int D = P.a.D, N = P.a.N, c0 = ct * CB;
    const int n0 = 4 * nl, wc = warp * Sh::CW + cl * CPT, d0 = c0 + wc;
    const int64_t dn = (int64_t)D * N;
    const bool vst = (P.vec & kVecState) != 0;

    BackTile<Tin, Sh> T(P, smem, tid, c0);
    // per warp: g [R][YP], and of HALF rows the sums over n of C h, B dh and A w
    float *gs = reinterpret_cast<float *>(smem + 2 * Sm::STAGE) + warp * R * YP;
    float *sum_y = reinterpret_cast<float *>(smem + 2 * Sm::STAGE + Sm::SUMS) + warp * (Sm::JOIN_Y / 4 / kScanWarps);
    float *sum_u = reinterpret_cast<float *>(smem + 2 * Sm::STAGE + Sm::SUMS + Sm::JOIN_Y) + warp * (Sm::JOIN / 4 / kScanWarps),
          *sum_w = sum_u + Sm::JOIN / 4;
    float *part = reinterpret_cast<float *>(smem + 2 * Sm::STAGE + Sm::SUMS + Sm::JOIN_Y + 2 * Sm::JOIN);
    float *states = reinterpret_cast<float *>(smem + Sm::MAIN - Sm::STATES);

    f2 A2[4][PP], dA[4][PP];
    zero_entries(A2);
    zero_entries(dA);
    if (P.a.T > 0) load_rates(P.a.A, d0, D, n0, N, vst, A2);
    // a lane finishes CPT channels of every row it is given: the same ones in every tile
    const int oc = warp * Sh::CW + lane % CLN * CPT, orow = lane / CLN;
    f2 skip[PP], dD[PP] = {};
#pragma unroll
    for (int p = 0; p < PP; ++p) {
        const int c = oc + 2 * p;
        skip[p] = pack2(P.a.Dskip && c < T.ncols ? P.a.Dskip[c0 + c] : 0.f, P.a.Dskip && c + 1 < T.ncols ? P.a.Dskip[c0 + c + 1] : 0.f);
    }

    // a gradient of the final state goes straight through an empty sequence
    if (P.g.dh0 && (P.a.cu_seqlens || P.L == 0)) {
        for (int s = w; s < P.a.S; s += P.W) {
            if (seq_bound(P, s) != seq_bound(P, s + 1)) continue;
            const int64_t slot = P.a.state_indices ? (int64_t)P.a.state_indices[s] : s;
            if (slot < 0 || slot >= P.a.num_states) {
                if (tid == 0) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
                continue;
            }
            for (int i = tid; i < T.ncols * N; i += kScanThreads) {
                const int64_t o = slot * dn + (int64_t)c0 * N + i;
                P.g.dh0[o] = P.g.dh_last ? P.g.dh_last[o] : 0.f;
            }
        }
    }

    for (int g = w; g < P.G; g += P.W) {
        const int row0 = (int)min((int64_t)g * P.C, (int64_t)P.a.T), row1 = (int)min((int64_t)(g + 1) * P.C, (int64_t)P.a.T);
        if (row0 >= row1) break;
        int end = row1;
        int s = find_seq(P, row1 - 1, scratch, tid);
        while (end > row0) {
            // the rows ra .. rb - 1 of one sequence (or of none)
            bool live = s >= 0 && s < P.a.S;
            const int first = live ? seq_bound(P, s) : s < 0 ? row0 : min(seq_bound(P, P.a.S), end - 1);
            const int ra = max(row0, min(first, end - 1));
            const bool starts = live && ra == first, ends = live && seq_bound(P, s + 1) <= row1;
            int64_t slot = 0;
            if (live) {
                slot = P.a.state_indices ? (int64_t)P.a.state_indices[s] : s;
                if (P.has_states && (slot < 0 || slot >= P.a.num_states)) live = false;
            }
            if (!live && tid == 0) raise_flag(P.a.err_flags, GDN_DEVERR_BAD_INDEX);
            const int rb = end, nt = (rb - ra + R - 1) / R;
            end = ra;
            s = s >= P.a.S ? P.a.S - 1 : s - 1;
            while (s >= 0 && seq_bound(P, s) >= end) --s;

            // jobs 0 .. nt - 2: tiles 0 .. nt - 2 forward; jobs nt - 1 .. 2 nt - 2: tiles nt - 1 .. 0 backward
            auto tile_of = [&](int j) { return j < nt - 1 ? j : 2 * nt - 2 - j; };
            // A tile of fewer than R rows has them at its end, behind rows of zeros. Such a row passes h and e on and adds
            // (e h) 0 to dA: before the first row that is no number only where that row's own share of dA is none.
            // Behind the last row it would also be where the state there, which dA does not see, is infinite or NaN.
            auto stage_job = [&](int j, int buf) {
                const int t0 = ra + tile_of(j) * R;
                T.template stage<true>(buf, t0, live ? min(R, rb - t0) : 0, j >= nt - 1);      // of no sequence: zeros
            };
            const int first_job = live ? 0 : nt - 1;
            __syncthreads();                 // the buffers of the rows before are free
            stage_job(first_job, 0);
            cp_async_commit();

            f2 h[4][PP], e[4][PP];
            zero_entries(h);
            zero_entries(e);
            const float *hf = nullptr;      // where the rows' first state is
            if (live) {
                hf = starts ? (P.a.h0 ? P.a.h0 + slot * dn : nullptr) : P.hin ? P.hin + g * dn : nullptr;
                const float *ef = ends ? (P.g.dh_last ? P.g.dh_last + slot * dn : nullptr) : P.ein ? P.ein + g * dn : nullptr;
                if (hf) load_entries(hf, d0, D, n0, N, vst, h);
                if (ef) load_entries(ef, d0, D, n0, N, vst, e);
            }

            int b = 0;
            for (int j = first_job; j < 2 * nt - 1; ++j, b ^= 1) {
                const bool back = j >= nt - 1;
                const int tile = tile_of(j), t0 = ra + tile * R, n = min(R, rb - t0), lead = R - n;
                cp_async_wait<0>();
                __syncthreads();
                if (j + 1 < 2 * nt - 1) stage_job(j + 1, b ^ 1);
                cp_async_commit();
                const Tin *xs = T.raw(b, 0), *ds = T.raw(b, 1), *zs = T.raw(b, 2), *dys = T.raw(b, 3);
                const Tin *Bs = T.raw_bc(b, 0), *Cs = T.raw_bc(b, 1);

                if (!back) {
                    if (tile > 0) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) store_pairs(states + (((tile - 1) * 4 + q) * kScanThreads + tid) * CPT, h[q]);
                    }
#pragma unroll 2
                    for (int t = 0; t < R; ++t) {
                        f2 dt[PP], u[PP], B[4];
                        load_pairs(ds + t * CB + wc, dt);
                        load_pairs(xs + t * CB + wc, u);
                        load_twice(Bs + t * NP + n0, B);
#pragma unroll
                        for (int p = 0; p < PP; ++p) {
                            u[p] = mul2(u[p], dt[p]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) h[k][p] = fma2(decay2(dt[p], A2[k][p]), h[k][p], mul2(u[p], B[k]));
                        }
                    }
                    continue;
                }

                T.gate(b, gs, lane, warp);
                // the tile's states, hp[t] before row t
                f2 hp[R + 1][4][PP];
                if (tile == nt - 1 || !live) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
#pragma unroll
                        for (int p = 0; p < PP; ++p) hp[0][q][p] = h[q][p];
                    }
                } else if (tile == 0) {
                    zero_entries(hp[0]);
                    if (hf) load_entries(hf, d0, D, n0, N, vst, hp[0]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        load_pairs(states + (((tile - 1) * 4 + q) * kScanThreads + tid) * CPT, hp[0][q]);
                    }
                }
#pragma unroll
                for (int t4 = 0; t4 < R; t4 += 4) {
                    float acc[4 * CPT];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int t = t4 + k;
                        f2 dt[PP], u[PP], B[4], C[4], y[PP];
                        load_pairs(ds + t * CB + wc, dt);
                        load_pairs(xs + t * CB + wc, u);
                        load_twice(Bs + t * NP + n0, B);
                        if (!Sm::JOINED) load_twice(Cs + t * NP + n0, C);
#pragma unroll
                        for (int p = 0; p < PP; ++p) {
                            u[p] = mul2(u[p], dt[p]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                hp[t + 1][q][p] = fma2(decay2(dt[p], A2[q][p]), hp[t][q][p], mul2(u[p], B[q]));
                                if (!Sm::JOINED) y[p] = q == 0 ? mul2(C[q], hp[t + 1][q][p]) : fma2(C[q], hp[t + 1][q][p], y[p]);
                            }
                            if (!Sm::JOINED) {
                                const float2 v = unpack2(y[p]);
                                acc[k * CPT + 2 * p] = v.x;
                                acc[k * CPT + 2 * p + 1] = v.y;
                            }
                        }
                    }
                    if (!Sm::JOINED && P.g.dz) {
                        constexpr int M = 4 * CPT, KEEP = M >= NL ? M / NL : 1, REP = M >= NL ? 1 : NL / M;
                        group_reduce<M, NL>(acc, nl);
                        if (nl % REP == 0) {
#pragma unroll
                            for (int i = 0; i < KEEP; ++i) {
                                const int v = nl / REP * KEEP + i;
                                sum_y[(t4 + v / CPT) * YP + cl * CPT + v % CPT] = acc[i];
                            }
                        }
                    }
                }
                __syncwarp();
                // backwards, HALF rows at a time
#pragma unroll
                for (int half = R - Sm::HALF; half >= 0; half -= Sm::HALF) {
#pragma unroll
                for (int t = half + Sm::HALF - 1; t >= half; --t) {
                    f2 dt[PP], u[PP], gv[PP], B[4], C[4], db[4], dc[4], us[PP], ws[PP], ys[PP];
                    load_pairs(ds + t * CB + wc, dt);
                    load_pairs(xs + t * CB + wc, u);
                    load_pairs(gs + t * YP + cl * CPT, gv);
                    load_twice(Bs + t * NP + n0, B);
                    load_twice(Cs + t * NP + n0, C);
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        u[p] = mul2(u[p], dt[p]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const f2 dh = fma2(C[q], gv[p], e[q][p]);
                            dc[q] = p == 0 ? mul2(gv[p], hp[t + 1][q][p]) : fma2(gv[p], hp[t + 1][q][p], dc[q]);
                            db[q] = p == 0 ? mul2(u[p], dh) : fma2(u[p], dh, db[q]);
                            us[p] = q == 0 ? mul2(B[q], dh) : fma2(B[q], dh, us[p]);
                            if (Sm::JOINED) ys[p] = q == 0 ? mul2(C[q], hp[t + 1][q][p]) : fma2(C[q], hp[t + 1][q][p], ys[p]);
                            e[q][p] = mul2(decay2(dt[p], A2[q][p]), dh);
                            const f2 wv = mul2(e[q][p], hp[t][q][p]);
                            ws[p] = q == 0 ? mul2(wv, A2[q][p]) : fma2(wv, A2[q][p], ws[p]);
                            dA[q][p] = fma2(wv, dt[p], dA[q][p]);
                        }
                    }
                    if (Sm::JOINED) {
                        const int o = ((t - half) * NL + nl) * YP + cl * CPT;
                        store_pairs(sum_y + o, ys);
                        store_pairs(sum_u + o, us);
                        store_pairs(sum_w + o, ws);
                    } else {
                        constexpr int M = 2 * CPT, KEEP = M >= NL ? M / NL : 1, REP = M >= NL ? 1 : NL / M;
                        float v[M];
#pragma unroll
                        for (int p = 0; p < PP; ++p) {
                            const float2 uv = unpack2(us[p]), wv = unpack2(ws[p]);
                            v[2 * p] = uv.x;
                            v[2 * p + 1] = uv.y;
                            v[CPT + 2 * p] = wv.x;
                            v[CPT + 2 * p + 1] = wv.y;
                        }
                        group_reduce<M, NL>(v, nl);
                        if (nl % REP == 0) {
#pragma unroll
                            for (int i = 0; i < KEEP; ++i) {
                                const int k = nl / REP * KEEP + i;      // the first half: sums of B dh, the second: of A w
                                (k < CPT ? sum_u : sum_w)[(t - half) * YP + cl * CPT + k % CPT] = v[i];
                            }
                        }
                    }
                    {
                        float v[8];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 x2 = unpack2(db[q]), y2 = unpack2(dc[q]);
                            v[q] = x2.x + x2.y;
                            v[4 + q] = y2.x + y2.y;
                        }
                        constexpr int KEEP = 8 >= CLN ? 8 / CLN : 1, REP = 8 >= CLN ? 1 : CLN / 8;
                        group_reduce<8, CLN>(v, cl, NL);
                        if (cl % REP == 0) {
#pragma unroll
                            for (int i = 0; i < KEEP; ++i) {
                                const int k = cl / REP * KEEP + i;      // 0 .. 3: dB, 4 .. 7: dC
                                part[((warp * R + t) * 2 + k / 4) * NP + n0 + k % 4] = v[i];
                            }
                        }
                    }
                }
                __syncwarp();
                // this warp's per-channel gradients of these rows
#pragma unroll
                for (int r0 = 0; r0 < Sm::HALF; r0 += NL) {
                    const int r = half + r0 + orow;
                    if ((NL > Sm::HALF && orow >= Sm::HALF) || r < lead || oc >= T.ncols) continue;
                    const int sc = (r - half) * Sm::LANES * YP + lane % CLN * CPT;
                    f2 x2[PP], d2[PP], y2[PP], z2[PP], g2[PP], u2[PP], w2[PP], s2[PP], gx[PP], gt[PP], gz[PP];
                    load_pairs(xs + r * CB + oc, x2);
                    load_pairs(ds + r * CB + oc, d2);
                    load_pairs(gs + r * YP + lane % CLN * CPT, g2);
                    join_lanes<Sm::LANES, YP>(sum_u + sc, u2);
                    join_lanes<Sm::LANES, YP>(sum_w + sc, w2);
                    if (P.g.dz) {
                        load_pairs(dys + r * CB + oc, y2);
                        load_pairs(zs + r * CB + oc, z2);
                        join_lanes<Sm::LANES, YP>(sum_y + (Sm::JOINED ? sc : r * YP + lane % CLN * CPT), s2);
                    }
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        gx[p] = fma2(u2[p], d2[p], mul2(skip[p], g2[p]));
                        gt[p] = fma2(u2[p], x2[p], mul2(pack2(kLn2, kLn2), w2[p]));      // A2 = A log2(e)
                        dD[p] = fma2(g2[p], x2[p], dD[p]);
                        if (P.g.dz) {
                            // silu'(z) = s (1 + z (1 - s)) at s = sigmoid(z)
                            const f2 sg = sigmoid2(z2[p]), one = pack2(1.f, 1.f);
                            const f2 slope = mul2(sg, fma2(z2[p], fma2(sg, pack2(-1.f, -1.f), one), one));
                            gz[p] = mul2(mul2(y2[p], fma2(skip[p], x2[p], s2[p])), slope);
                        }
                    }
                    const int64_t row = t0 + r - lead;
                    if (!GDN_IN(P.a.err_flags, row, P.a.T)) continue;
                    const int left = T.ncols - oc, col = c0 + oc;
                    if (P.g.dx) store_row(static_cast<Tin *>(P.g.dx) + row * P.g.dx_stride + col, gx, left, (P.vec & kVecDx) && left >= CPT);
                    if (P.g.ddt) store_row(static_cast<Tin *>(P.g.ddt) + row * P.g.ddt_stride + col, gt, left, (P.vec & kVecDdt) && left >= CPT);
                    if (P.g.dz) store_row(static_cast<Tin *>(P.g.dz) + row * P.g.dz_stride + col, gz, left, (P.vec & kVecDz) && left >= CPT);
                }
                __syncwarp();
                }
                __syncthreads();
                // this channel tile's share of dB and dC: the warps' sums in order
                for (int i = tid; i < n * 2 * NP; i += kScanThreads) {
                    const int r = i / (2 * NP), k = i / NP % 2, nn = i % NP;
                    if (nn >= N) continue;
                    float v = 0.f;
#pragma unroll
                    for (int q = 0; q < kScanWarps; ++q) v += part[((q * R + lead + r) * 2 + k) * NP + nn];
                    const int64_t o = ((int64_t)ct * P.a.T + t0 + r) * 2 * N + k * N + nn;
                    if (GDN_IN(P.a.err_flags, o, (int64_t)P.nct * P.a.T * 2 * N)) P.part_bc[o] = v;
                }
            }
            if (starts && live && P.g.dh0 && GDN_IN(P.a.err_flags, slot, P.a.num_states)) store_entries(P.g.dh0 + slot * dn, d0, D, n0, N, vst, e);
        }
    }

    store_entries(P.part_a + w * dn, d0, D, n0, N, vst, dA);
    // dD: the lanes that share channels
#pragma unroll
    for (int p = 0; p < PP; ++p) {
        float2 v = unpack2(dD[p]);
#pragma unroll
        for (int off = CLN; off < 32; off <<= 1) {
            v.x += __shfl_xor_sync(kScanFull, v.x, off);
            v.y += __shfl_xor_sync(kScanFull, v.y, off);
        }
        const int c = oc + 2 * p;
        if (orow == 0 && c < T.ncols) P.part_d[(int64_t)w * D + c0 + c] = v.x;
        if (orow == 0 && c + 1 < T.ncols) P.part_d[(int64_t)w * D + c0 + c + 1] = v.y;
    }
}

// (4) The parts' sums, in the order of channel tiles (dB, dC) or workers (dA, dD).
template <typename Tin> __global__ void __launch_bounds__(256) scan_back_sum_kernel(const __grid_constant__ ScanLaunch P)
{
    ordinary_launch_start();
    const int64_t N = P.a.N, rows = (int64_t)P.a.T * 2 * N, dn = (int64_t)P.a.D * N;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < rows) {
        float v = 0.f;
#pragma unroll 8
        for (int k = 0; k < P.nct; ++k) v += P.part_bc[k * rows + i];
        const int64_t t = i / (2 * N), n = i % (2 * N);
        if (n < N) {
            if (P.g.dBm) static_cast<Tin *>(P.g.dBm)[t * P.g.dB_stride + n] = from_f32<Tin>(v);
        } else if (P.g.dCm) {
            static_cast<Tin *>(P.g.dCm)[t * P.g.dC_stride + n - N] = from_f32<Tin>(v);
        }
    } else if (i < rows + dn) {
        const int64_t j = i - rows;
        float v = 0.f;
#pragma unroll 8
        for (int k = 0; k < P.W; ++k) v += P.part_a[k * dn + j];
        if (P.g.dA) P.g.dA[j] = v;
    } else if (i < rows + dn + P.a.D) {
        const int64_t j = i - rows - dn;
        float v = 0.f;
#pragma unroll 8
        for (int k = 0; k < P.W; ++k) v += P.part_d[(int64_t)k * P.a.D + j];
        if (P.g.dDskip) P.g.dDskip[j] = v;
    }
}

template <typename Kern> static cudaError_t launch_sized(Kern kern, int64_t ctas, int bytes, const ScanLaunch &P, cudaStream_t stream)
{
    if (bytes > 40 * 1024) {      // the kernels have a little static shared memory too
        const cudaError_t rc = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (rc != cudaSuccess) return rc;
    }
    return launch_ordinary(kern, dim3((unsigned)ctas), dim3(kScanThreads), bytes, stream, P);
}

template <typename Tin, int NL, int CPT> static int launch_shape(const ScanLaunch &P, cudaStream_t stream)
{
    using Sm = BackSmem<Tin, ScanShape<NL, CPT>>;
    if (P.hin) {
        if (launch_sized(scan_back_summary_kernel<Tin, NL, CPT>, (int64_t)P.G * P.nct, Sm::SUMMARY, P, stream) != cudaSuccess)
            return GDN_ERR_LAUNCH;
        if (launch_scan_carry(P, true, stream) != cudaSuccess) return GDN_ERR_LAUNCH;
    }
    if (launch_sized(scan_back_kernel<Tin, NL, CPT>, (int64_t)P.W * P.nct, Sm::MAIN, P, stream) != cudaSuccess) return GDN_ERR_LAUNCH;
    const int64_t outs = (int64_t)P.a.T * 2 * P.a.N + (int64_t)P.a.D * P.a.N + P.a.D;
    return launch_ordinary(scan_back_sum_kernel<Tin>, dim3((unsigned)((outs + 255) / 256)), dim3(256), 0, stream, P) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_LAUNCH;
}

template <typename Tin> static int launch_typed(const ScanLaunch &P, cudaStream_t stream)
{
    switch (scan_lanes(P.a.N)) {
    case 2: return launch_shape<Tin, 2, 2>(P, stream);
    case 4: return launch_shape<Tin, 4, 4>(P, stream);
    case 8: return launch_shape<Tin, 8, 4>(P, stream);
    case 16: return launch_shape<Tin, 16, 4>(P, stream);
    default: return launch_shape<Tin, 32, 4>(P, stream);
    }
}

int launch_scan_backward(const ScanLaunch &P, cudaStream_t stream)
{
    return P.a.in_dtype == GDN_BF16 ? launch_typed<bf16>(P, stream) : launch_typed<float>(P, stream);
}

}  // namespace gdn
