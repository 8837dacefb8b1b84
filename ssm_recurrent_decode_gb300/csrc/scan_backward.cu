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
    static constexpr int Q = R * Sh::CB * 16;                             // {dt, dt, u, u}
    static constexpr int GG = R * Sh::CB * 8;                             // {g, g}
    static constexpr int WIDE = sizeof(Tin) == 4 ? 0 : R * Sh::NP * 4;
    static constexpr int SUMS = R * Sh::YP * 4;                           // per-channel sums of one kind
    static constexpr int PART = kScanWarps * R * 2 * Sh::NP * 4;          // dB and dC per warp
    static constexpr int STATES = kBackTiles * Sh::CPT * kScanThreads * 16;
    static constexpr int SUMMARY = 2 * STAGE + Q + GG + 2 * WIDE;
    static constexpr int MAIN = 2 * STAGE + Q + GG + 2 * WIDE + 3 * SUMS + PART + STATES;
};

// Staging, conversion and addressing that the summary and the gradient kernel share.
template <typename Tin, class Sh> struct BackTile {
    using Sm = BackSmem<Tin, Sh>;
    static constexpr int CB = Sh::CB, NP = Sh::NP, R = kBackTile;
    const ScanLaunch &P;
    unsigned char *smem;
    int tid, c0, ncols;
    float4 *q;
    f2 *gg;
    float *wideB, *wideC;
    const float *Bf, *Cf;

    __device__ __forceinline__ BackTile(const ScanLaunch &P_, unsigned char *s, int tid_, int c0_)
        : P(P_), smem(s), tid(tid_), c0(c0_), ncols(min(CB, P_.a.D - c0_))
    {
        q = reinterpret_cast<float4 *>(smem + 2 * Sm::STAGE);
        gg = reinterpret_cast<f2 *>(smem + 2 * Sm::STAGE + Sm::Q);
        wideB = reinterpret_cast<float *>(smem + 2 * Sm::STAGE + Sm::Q + Sm::GG);
        wideC = wideB + Sm::WIDE / 4;
    }
    __device__ __forceinline__ Tin *raw(int b, int k) const      // k: 0 x, 1 dt, 2 z, 3 dy
    {
        return reinterpret_cast<Tin *>(smem + b * Sm::STAGE + k * Sm::RX);
    }
    __device__ __forceinline__ Tin *raw_bc(int b, int k) const   // k: 0 B, 1 C
    {
        return reinterpret_cast<Tin *>(smem + b * Sm::STAGE + 4 * Sm::RX + k * Sm::RB);
    }
    __device__ __forceinline__ void rows(Tin *dst, const void *src, int64_t stride, int64_t t0, int n, int bit)
    {
        stage_rows<Tin, CB, R>(dst, static_cast<const Tin *>(src) + t0 * stride + c0, stride, n, ncols, P.vec & bit, tid);
    }
    // rows t0 .. t0 + n - 1 into buffer b; grads: also what only the gradients need
    __device__ __forceinline__ void stage(int b, int t0, int n, bool grads)
    {
        rows(raw(b, 0), P.a.x, P.a.x_stride, t0, n, kVecX);
        rows(raw(b, 1), P.a.dt, P.a.dt_stride, t0, n, kVecDt);
        stage_rows<Tin, NP, R>(raw_bc(b, 0), static_cast<const Tin *>(P.a.Bm) + (int64_t)t0 * P.a.B_stride, P.a.B_stride, n,
                               P.a.N, P.vec & kVecB, tid);
        if (grads) {
            if (P.a.z) rows(raw(b, 2), P.a.z, P.a.z_stride, t0, n, kVecZ);
            rows(raw(b, 3), P.g.dy, P.g.dy_stride, t0, n, kVecDy);
            stage_rows<Tin, NP, R>(raw_bc(b, 1), static_cast<const Tin *>(P.a.Cm) + (int64_t)t0 * P.a.C_stride, P.a.C_stride,
                                   n, P.a.N, P.vec & kVecC, tid);
        }
    }
    __device__ __forceinline__ void widen(int b, bool grads)
    {
        const Tin *xs = raw(b, 0), *ds = raw(b, 1), *zs = raw(b, 2), *dys = raw(b, 3);
        for (int i = tid * 4; i < R * CB; i += kScanThreads * 4) {
            const float4 x4 = load4(xs + i), d4 = load4(ds + i);
            const float u0 = d4.x * x4.x, u1 = d4.y * x4.y, u2 = d4.z * x4.z, u3 = d4.w * x4.w;
            q[i] = make_float4(d4.x, d4.x, u0, u0);
            q[i + 1] = make_float4(d4.y, d4.y, u1, u1);
            q[i + 2] = make_float4(d4.z, d4.z, u2, u2);
            q[i + 3] = make_float4(d4.w, d4.w, u3, u3);
            if (grads) {
                float4 g = load4(dys + i);
                if (P.a.z) {
                    const float4 z4 = load4(zs + i);
                    g.x *= z4.x * fast_sigmoid(z4.x);
                    g.y *= z4.y * fast_sigmoid(z4.y);
                    g.z *= z4.z * fast_sigmoid(z4.z);
                    g.w *= z4.w * fast_sigmoid(z4.w);
                }
                *reinterpret_cast<float4 *>(gg + i) = make_float4(g.x, g.x, g.y, g.y);
                *reinterpret_cast<float4 *>(gg + i + 2) = make_float4(g.z, g.z, g.w, g.w);
            }
        }
        Bf = as_f32(raw_bc(b, 0), wideB, R * NP, tid);
        if (grads) Cf = as_f32(raw_bc(b, 1), wideC, R * NP, tid);
    }
};

// (1) The summaries of chunk g: for the sequence that goes on behind the chunk its end state from
// zero, for the sequence that began before it what its rows send back. Usually one and the same.
template <typename Tin, int NL>
__global__ void __launch_bounds__(kScanThreads) scan_back_summary_kernel(const __grid_constant__ ScanLaunch P)
{
    using Sh = ScanShape<NL, 2>;
    constexpr int CPT = 2, R = kBackTile, NP = Sh::NP, CB = Sh::CB;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[kScanWarps];
    ordinary_launch_start();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, cl = lane / NL;
    const int ct = (int)(blockIdx.x % (unsigned)P.nct), g = (int)(blockIdx.x / (unsigned)P.nct);
    const int D = P.a.D, N = P.a.N, c0 = ct * CB;
    const int n0 = 4 * nl, wc = warp * Sh::CW + cl;
    const int64_t dn = (int64_t)D * N;
    const bool vst = (P.vec & kVecState) != 0;
    const int row0 = g * P.C, row1 = min(P.a.T, row0 + P.C);

    const int sh = find_seq(P, row0, scratch, tid), st = find_seq(P, row1 - 1, scratch, tid);
    const bool before = sh >= 0 && sh < P.a.S && seq_bound(P, sh) < row0;
    const bool behind = st >= 0 && st < P.a.S && seq_bound(P, st + 1) > row1;
    const int head_end = before ? min(seq_bound(P, sh + 1), row1) : row0;
    const int tail_begin = behind ? max(seq_bound(P, st), row0) : row1;
    if (tid == 0 && ct == 0)
        P.info[g] = make_int4(behind ? st : -1, behind && seq_bound(P, st) >= row0, before ? sh : -1,
                              before && seq_bound(P, sh + 1) <= row1);

    f2 A2[CPT][2], h[CPT][2], prod[CPT][2], e[CPT][2];
    float dt_head[CPT], dt_tail[CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        load_rates(P.a.A, c0 + wc + c * Sh::CLN, D, n0, N, vst, A2[c]);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            h[c][p] = e[c][p] = 0ull;
            prod[c][p] = pack2(1.f, 1.f);
        }
        dt_head[c] = dt_tail[c] = 0.f;
    }

    BackTile<Tin, Sh> T(P, smem, tid, c0);
    // rows row0 .. head_end - 1 (head) and tail_begin .. row1 - 1 (tail); tiles do not cross either border
    auto clip = [&](int pos) {
        int end = min(row1, pos + R);
        if (pos < head_end) end = min(end, head_end);
        if (pos < tail_begin) end = min(end, tail_begin);
        return end - pos;
    };
    auto first_at = [&](int pos) { return pos >= head_end && pos < tail_begin ? tail_begin : pos; };   // skips what is neither
    int pos = first_at(row0), b = 0;
    if (pos < row1) T.stage(0, pos, clip(pos), true);
    cp_async_commit();
    while (pos < row1) {
        const bool head = pos < head_end, tail = pos >= tail_begin;
        const int next = first_at(pos + clip(pos));
        cp_async_wait<0>();
        __syncthreads();
        if (next < row1) T.stage(b ^ 1, next, clip(next), true);
        cp_async_commit();
        T.widen(b, true);
        __syncthreads();
        float dts[CPT] = {};
#pragma unroll
        for (int t = 0; t < R; ++t) {
            const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(T.Bf + t * NP + n0);
            const ulonglong2 C = *reinterpret_cast<const ulonglong2 *>(T.Cf + t * NP + n0);
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                const int ch = t * CB + wc + c * Sh::CLN;
                const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(T.q + ch);
                const f2 g2 = T.gg[ch];
                const f2 a0 = decay2(du.x, A2[c][0]), a1 = decay2(du.x, A2[c][1]);
                dts[c] += unpack2(du.x).x;
                if (tail) {
                    h[c][0] = fma2(a0, h[c][0], mul2(du.y, B.x));
                    h[c][1] = fma2(a1, h[c][1], mul2(du.y, B.y));
                }
                if (head) {
                    prod[c][0] = mul2(prod[c][0], a0);
                    prod[c][1] = mul2(prod[c][1], a1);
                    e[c][0] = fma2(prod[c][0], mul2(C.x, g2), e[c][0]);
                    e[c][1] = fma2(prod[c][1], mul2(C.y, g2), e[c][1]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            if (head) dt_head[c] += dts[c];
            if (tail) dt_tail[c] += dts[c];
        }
        pos = next;
        b ^= 1;
    }
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int d = c0 + wc + c * Sh::CLN;
        if (behind) store_entries(P.hin + g * dn, d, D, n0, N, vst, h[c]);
        if (before) store_entries(P.ein + g * dn, d, D, n0, N, vst, e[c]);
        if (nl == 0 && d < D) {
            P.sumdt[(int64_t)g * D + d] = dt_tail[c];
            P.sumdt_head[(int64_t)g * D + d] = dt_head[c];
        }
    }
}

// (3) The gradients. A CTA owns a channel tile and walks the chunks w, w + W, ..., so that dA and dD
// stay in registers. In a chunk it takes each sequence's rows forward once, keeping the state before
// every tile in shared memory, then tile by tile backwards: the tile's states and decays again, now
// kept in registers, and the recurrence of dh through them.
template <typename Tin, int NL>
__global__ void __launch_bounds__(kScanThreads) scan_back_kernel(const __grid_constant__ ScanLaunch P)
{
    using Sh = ScanShape<NL, 2>;
    using Sm = BackSmem<Tin, Sh>;
    constexpr int CPT = 2, R = kBackTile, NP = Sh::NP, CB = Sh::CB, CLN = Sh::CLN, YP = Sh::YP;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[kScanWarps];
    ordinary_launch_start();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, cl = lane / NL;
    const int ct = (int)(blockIdx.x % (unsigned)P.nct), w = (int)(blockIdx.x / (unsigned)P.nct);
    const int D = P.a.D, N = P.a.N, c0 = ct * CB;
    const int n0 = 4 * nl, wc = warp * Sh::CW + cl;
    const int64_t dn = (int64_t)D * N;
    const bool vst = (P.vec & kVecState) != 0;

    BackTile<Tin, Sh> T(P, smem, tid, c0);
    float *sum_y = reinterpret_cast<float *>(smem + 2 * Sm::STAGE + Sm::Q + Sm::GG + 2 * Sm::WIDE);
    float *sum_u = sum_y + R * YP, *sum_w = sum_u + R * YP, *part = sum_w + R * YP;
    ulonglong2 *states = reinterpret_cast<ulonglong2 *>(smem + Sm::MAIN - Sm::STATES);

    f2 A2[CPT][2], dA[CPT][2];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        A2[c][0] = A2[c][1] = dA[c][0] = dA[c][1] = 0ull;
        if (P.a.T > 0) load_rates(P.a.A, c0 + wc + c * CLN, D, n0, N, vst, A2[c]);
    }
    float4 dD = make_float4(0.f, 0.f, 0.f, 0.f);
    const int ec = tid * 4 % CB;            // the four channels this thread finishes in every tile

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
            // the rows ra .. end - 1 of one sequence (or of none)
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

            f2 h[CPT][2], e[CPT][2];
            {
                const float *hf = starts ? (P.a.h0 && live ? P.a.h0 + slot * dn : nullptr) : P.hin ? P.hin + g * dn : nullptr;
                const float *ef = ends ? (P.g.dh_last && live ? P.g.dh_last + slot * dn : nullptr) : P.ein ? P.ein + g * dn : nullptr;
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    h[c][0] = h[c][1] = e[c][0] = e[c][1] = 0ull;
                    if (live && hf) load_entries(hf, c0 + wc + c * CLN, D, n0, N, vst, h[c]);
                    if (live && ef) load_entries(ef, c0 + wc + c * CLN, D, n0, N, vst, e[c]);
                }
            }

            // jobs 0 .. nt - 2: tiles 0 .. nt - 2 forward; jobs nt - 1 .. 2 nt - 2: tiles nt - 1 .. 0 backward
            auto tile_of = [&](int j) { return j < nt - 1 ? j : 2 * nt - 2 - j; };
            auto stage_job = [&](int j, int buf) {
                const int t0 = ra + tile_of(j) * R;
                T.stage(buf, t0, live ? min(R, rb - t0) : 0, j >= nt - 1);      // of no sequence: zeros
            };
            const int first_job = live ? 0 : nt - 1;
            __syncthreads();                 // the buffers of the rows before are free
            stage_job(first_job, 0);
            cp_async_commit();
            int b = 0;
            for (int j = first_job; j < 2 * nt - 1; ++j, b ^= 1) {
                const bool back = j >= nt - 1;
                const int tile = tile_of(j), t0 = ra + tile * R, n = min(R, rb - t0);
                cp_async_wait<0>();
                __syncthreads();
                if (j + 1 < 2 * nt - 1) stage_job(j + 1, b ^ 1);
                cp_async_commit();
                T.widen(b, back);
                __syncthreads();

                if (!back || tile == nt - 1) {
#pragma unroll
                    for (int c = 0; c < CPT; ++c)
                        states[(tile * CPT + c) * kScanThreads + tid] = make_ulonglong2(h[c][0], h[c][1]);
                }
                if (!back) {
#pragma unroll
                    for (int t = 0; t < R; ++t) {
                        const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(T.Bf + t * NP + n0);
#pragma unroll
                        for (int c = 0; c < CPT; ++c) {
                            const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(T.q + t * CB + wc + c * CLN);
                            h[c][0] = fma2(decay2(du.x, A2[c][0]), h[c][0], mul2(du.y, B.x));
                            h[c][1] = fma2(decay2(du.x, A2[c][1]), h[c][1], mul2(du.y, B.y));
                        }
                    }
                    continue;
                }

                // the tile's states (before each row) and decays
                f2 hp[R + 1][CPT][2], a[R][CPT][2];
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const ulonglong2 v = states[(tile * CPT + c) * kScanThreads + tid];
                    hp[0][c][0] = v.x;
                    hp[0][c][1] = v.y;
                }
#pragma unroll
                for (int t4 = 0; t4 < R; t4 += 4) {
                    float acc[4 * CPT];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int t = t4 + k;
                        const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(T.Bf + t * NP + n0);
                        const ulonglong2 C = *reinterpret_cast<const ulonglong2 *>(T.Cf + t * NP + n0);
#pragma unroll
                        for (int c = 0; c < CPT; ++c) {
                            const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(T.q + t * CB + wc + c * CLN);
                            a[t][c][0] = decay2(du.x, A2[c][0]);
                            a[t][c][1] = decay2(du.x, A2[c][1]);
                            hp[t + 1][c][0] = fma2(a[t][c][0], hp[t][c][0], mul2(du.y, B.x));
                            hp[t + 1][c][1] = fma2(a[t][c][1], hp[t][c][1], mul2(du.y, B.y));
                            const float2 y = unpack2(fma2(C.y, hp[t + 1][c][1], mul2(C.x, hp[t + 1][c][0])));
                            acc[k * CPT + c] = y.x + y.y;
                        }
                    }
                    if (P.g.dz) {
                        constexpr int M = 4 * CPT;
                        group_reduce<M, NL>(acc, nl);
                        constexpr int KEEP = M >= NL ? M / NL : 1, REP = M >= NL ? 1 : NL / M;
                        if (nl % REP == 0) {
#pragma unroll
                            for (int i = 0; i < KEEP; ++i) {
                                const int v = nl / REP * KEEP + i;
                                sum_y[(t4 + v / CPT) * YP + wc + (v % CPT) * CLN] = acc[i];
                            }
                        }
                    }
                }
                // backwards
#pragma unroll
                for (int t = R - 1; t >= 0; --t) {
                    const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(T.Bf + t * NP + n0);
                    const ulonglong2 C = *reinterpret_cast<const ulonglong2 *>(T.Cf + t * NP + n0);
                    f2 db[2], dc[2];
                    float uw[2 * CPT];
#pragma unroll
                    for (int c = 0; c < CPT; ++c) {
                        const int ch = t * CB + wc + c * CLN;
                        const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(T.q + ch);
                        const f2 g2 = T.gg[ch];
                        f2 us, ws;
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const f2 Bp = p ? B.y : B.x, Cp = p ? C.y : C.x;
                            const f2 dh = fma2(Cp, g2, e[c][p]);
                            dc[p] = c == 0 ? mul2(g2, hp[t + 1][c][p]) : fma2(g2, hp[t + 1][c][p], dc[p]);
                            db[p] = c == 0 ? mul2(du.y, dh) : fma2(du.y, dh, db[p]);
                            us = p == 0 ? mul2(Bp, dh) : fma2(Bp, dh, us);
                            e[c][p] = mul2(a[t][c][p], dh);
                            const f2 wv = mul2(e[c][p], hp[t][c][p]);
                            ws = p == 0 ? mul2(wv, A2[c][p]) : fma2(wv, A2[c][p], ws);
                            dA[c][p] = fma2(wv, du.x, dA[c][p]);
                        }
                        const float2 u = unpack2(us), wsum = unpack2(ws);
                        uw[c] = u.x + u.y;
                        uw[CPT + c] = wsum.x + wsum.y;
                    }
                    {
                        constexpr int M = 2 * CPT;
                        group_reduce<M, NL>(uw, nl);
                        constexpr int KEEP = M >= NL ? M / NL : 1, REP = M >= NL ? 1 : NL / M;
                        if (nl % REP == 0) {
#pragma unroll
                            for (int i = 0; i < KEEP; ++i) {
                                const int v = nl / REP * KEEP + i;
                                (v < CPT ? sum_u : sum_w)[t * YP + wc + (v % CPT) * CLN] = uw[i];
                            }
                        }
                    }
                    {
                        const float2 b0 = unpack2(db[0]), b1 = unpack2(db[1]), k0 = unpack2(dc[0]), k1 = unpack2(dc[1]);
                        float bc[8] = {b0.x, b0.y, b1.x, b1.y, k0.x, k0.y, k1.x, k1.y};
                        group_reduce<8, CLN>(bc, cl, NL);
                        constexpr int KEEP = 8 >= CLN ? 8 / CLN : 1, REP = 8 >= CLN ? 1 : CLN / 8;
                        if (cl % REP == 0) {
#pragma unroll
                            for (int i = 0; i < KEEP; ++i) {
                                const int v = cl / REP * KEEP + i;      // 0 .. 3: dB, 4 .. 7: dC
                                part[((warp * R + t) * 2 + v / 4) * NP + n0 + v % 4] = bc[i];
                            }
                        }
                    }
                }
                __syncthreads();

                // per-channel gradients of the tile's rows
                for (int i = tid * 4; i < n * CB; i += kScanThreads * 4) {
                    const int r = i / CB;
                    if (ec >= T.ncols) break;
                    const float4 x4 = load4(T.raw(b, 0) + i), d4 = load4(T.raw(b, 1) + i), dy4 = load4(T.raw(b, 3) + i);
                    const float4 u4 = *reinterpret_cast<const float4 *>(sum_u + r * YP + ec);
                    const float4 w4 = *reinterpret_cast<const float4 *>(sum_w + r * YP + ec);
                    const float xv[4] = {x4.x, x4.y, x4.z, x4.w}, dv[4] = {d4.x, d4.y, d4.z, d4.w},
                                yv[4] = {dy4.x, dy4.y, dy4.z, dy4.w}, uv[4] = {u4.x, u4.y, u4.z, u4.w},
                                wv[4] = {w4.x, w4.y, w4.z, w4.w};
                    float zv[4] = {}, pre[4] = {}, dskip[4] = {}, gx[4], gt[4], gz[4] = {}, gd[4];
                    if (P.a.z) {
                        const float4 z4 = load4(T.raw(b, 2) + i);
                        zv[0] = z4.x; zv[1] = z4.y; zv[2] = z4.z; zv[3] = z4.w;
                        if (P.g.dz) {
                            const float4 s4 = *reinterpret_cast<const float4 *>(sum_y + r * YP + ec);
                            pre[0] = s4.x; pre[1] = s4.y; pre[2] = s4.z; pre[3] = s4.w;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (P.a.Dskip && ec + k < T.ncols) dskip[k] = P.a.Dskip[c0 + ec + k];
                        float gk = yv[k];
                        if (P.a.z) {
                            const float sg = fast_sigmoid(zv[k]);
                            gk = yv[k] * (zv[k] * sg);
                            gz[k] = yv[k] * fmaf(dskip[k], xv[k], pre[k]) * (sg * fmaf(zv[k], 1.f - sg, 1.f));
                        }
                        gx[k] = fmaf(uv[k], dv[k], dskip[k] * gk);
                        gt[k] = fmaf(uv[k], xv[k], kLn2 * wv[k]);      // A2 = A log2(e)
                        gd[k] = gk * xv[k];
                        if (!live) gx[k] = gt[k] = gz[k] = gd[k] = 0.f;
                    }
                    dD.x += gd[0]; dD.y += gd[1]; dD.z += gd[2]; dD.w += gd[3];
                    const int64_t row = t0 + r;
                    const int left = T.ncols - ec, col = c0 + ec;
                    if (P.g.dx)
                        store_row4(static_cast<Tin *>(P.g.dx) + row * P.g.dx_stride + col, make_float4(gx[0], gx[1], gx[2], gx[3]), left, P.vec & kVecDx);
                    if (P.g.ddt)
                        store_row4(static_cast<Tin *>(P.g.ddt) + row * P.g.ddt_stride + col, make_float4(gt[0], gt[1], gt[2], gt[3]), left, P.vec & kVecDdt);
                    if (P.g.dz)
                        store_row4(static_cast<Tin *>(P.g.dz) + row * P.g.dz_stride + col, make_float4(gz[0], gz[1], gz[2], gz[3]), left, P.vec & kVecDz);
                }
                // this channel tile's share of dB and dC: the warps' sums in order
                for (int i = tid; i < n * 2 * NP; i += kScanThreads) {
                    const int r = i / (2 * NP), k = i / NP % 2, nn = i % NP;
                    if (nn >= N) continue;
                    float v = 0.f;
#pragma unroll
                    for (int q = 0; q < kScanWarps; ++q) v += part[((q * R + r) * 2 + k) * NP + nn];
                    P.part_bc[((int64_t)ct * P.a.T + t0 + r) * 2 * N + k * N + nn] = live ? v : 0.f;
                }
            }
            if (starts && live && P.g.dh0) {
#pragma unroll
                for (int c = 0; c < CPT; ++c) store_entries(P.g.dh0 + slot * dn, c0 + wc + c * CLN, D, n0, N, vst, e[c]);
            }
        }
    }

#pragma unroll
    for (int c = 0; c < CPT; ++c) store_entries(P.part_a + w * dn, c0 + wc + c * CLN, D, n0, N, vst, dA[c]);
    // dD: the threads that share four channels
    __syncthreads();
    reinterpret_cast<float4 *>(smem)[tid] = dD;
    __syncthreads();
    if (tid * 4 < CB) {
        float v[4] = {};
        for (int k = tid; k < kScanThreads; k += CB / 4) {
            const float4 o = reinterpret_cast<const float4 *>(smem)[k];
            v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
        }
        for (int k = 0; k < 4; ++k)
            if (ec + k < T.ncols) P.part_d[(int64_t)w * D + c0 + ec + k] = v[k];
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
    if (bytes > 48 * 1024) {
        const cudaError_t rc = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (rc != cudaSuccess) return rc;
    }
    return launch_ordinary(kern, dim3((unsigned)ctas), dim3(kScanThreads), bytes, stream, P);
}

template <typename Tin, int NL> static int launch_shape(const ScanLaunch &P, cudaStream_t stream)
{
    using Sm = BackSmem<Tin, ScanShape<NL, 2>>;
    if (P.hin) {
        if (launch_sized(scan_back_summary_kernel<Tin, NL>, (int64_t)P.G * P.nct, Sm::SUMMARY, P, stream) != cudaSuccess)
            return GDN_ERR_LAUNCH;
        if (launch_scan_carry(P, true, stream) != cudaSuccess) return GDN_ERR_LAUNCH;
    }
    if (launch_sized(scan_back_kernel<Tin, NL>, (int64_t)P.W * P.nct, Sm::MAIN, P, stream) != cudaSuccess) return GDN_ERR_LAUNCH;
    const int64_t outs = (int64_t)P.a.T * 2 * P.a.N + (int64_t)P.a.D * P.a.N + P.a.D;
    return launch_ordinary(scan_back_sum_kernel<Tin>, dim3((unsigned)((outs + 255) / 256)), dim3(256), 0, stream, P) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_LAUNCH;
}

template <typename Tin> static int launch_typed(const ScanLaunch &P, cudaStream_t stream)
{
    switch (scan_shape_backward(P.a.N).NL) {
    case 2: return launch_shape<Tin, 2>(P, stream);
    case 4: return launch_shape<Tin, 4>(P, stream);
    case 8: return launch_shape<Tin, 8>(P, stream);
    case 16: return launch_shape<Tin, 16>(P, stream);
    default: return launch_shape<Tin, 32>(P, stream);
    }
}

int launch_scan_backward(const ScanLaunch &P, cudaStream_t stream)
{
    return P.a.in_dtype == GDN_BF16 ? launch_typed<bf16>(P, stream) : launch_typed<float>(P, stream);
}

}  // namespace gdn
