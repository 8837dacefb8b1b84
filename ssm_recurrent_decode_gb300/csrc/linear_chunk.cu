// linear_chunk.cu -- linear attention in bf16 on the tensor cores (tcgen05), 128 tokens at a time.
//
// For a chunk of rows r, s = 0 .. 127 in the sweep's order, with G the running sum of the log decays inside it and
// State the state before it (roles x, y, z as in linear_launch.h):
//     out_r = sum_{s <= r} (x_r . y_s) e^{G_r - G_s} z_s + e^{G_r} State^T x_r
//     State <- e^{G_last} State + sum_s e^{G_last - G_s} y_s z_s^T
// Four products a chunk, each with fp32 sums in tensor memory:
//     scores  [r, s] = x y^T                      both operands as loaded
//     inter   [r, z] = x State                    State from registers through shared memory, as two bf16 terms
//     out     [r, z] = inter e^{G_r} + P z        P = scores times decays, two bf16 terms, in tensor memory over the scores
//     update  [y, z] = Y^T z                      Y = y e^{G_last - G_s}, three bf16 terms, in tensor memory, 64 tokens at a time
// The terms are what keeps fp32: x, y and z are bf16 and exact, the state itself stays in fp32 registers (a lane of
// tensor memory is a row y of it, the columns z are shared by two warpgroups), a product's sum is added to it in fp32
// once a chunk. Two terms keep 16 bits of what leads to a token's bf16 output; the update's three keep all 24.
//
// One CTA owns a segment of a sequence and a value head. Warps 0-3: P, inter's decays and the outputs (a thread a row
// r); warps 4-7 and 8-11: Y and the state; 12: issues the MMAs; 13: decays, and z's non-finite values; 14, 15:
// copies x, y and z (cp.async of 16 bytes, whose zero fill ends a sequence inside a tile) into a ring of 32 KB tiles.
//
// A product with a zero of P would carry a later token's NaN to earlier ones; warp 13 looks z's tile over (one
// multiply-add a pair), and in the rare tile that has a non-finite value sets it to zero, notes the column's first
// such row, and the outputs and the state get their NaN from there.
//
// Every wait is bounded; a wait that gives up raises GDN_DEVERR_TIMEOUT and ends the CTA, its MMAs and copies done.
#include <mutex>

#include "gdn_chain.cuh"
#include "linear_common.cuh"
#include "tc_ops.cuh"

namespace gdn {

namespace {

constexpr int kRows = 128;                            // tokens per chunk
constexpr uint32_t kBlock = 16384;                    // 128 rows of 64 columns
constexpr uint32_t kTile = 2 * kBlock;
constexpr int kThreadsChunk = 512;
constexpr int kLoaders = 64;
constexpr long long kWaitLimit = 1LL << 31;           // SM clock cycles, about one second

// columns of tensor memory
constexpr uint32_t kScores = 0, kOut = 128, kUpdate = 256, kY = 384;

template <int NS> struct Smem {
    static constexpr int kSlots = NS == 3 ? 4 : 5;    // NS: bf16 terms of the state
    static constexpr uint32_t kStates = kSlots * kTile;
    static constexpr uint32_t kDecays = kStates + NS * kTile;         // float2 [2][128]: G = x + y in powers of two
    static constexpr uint32_t kBad = kDecays + 2 * kRows * 8;         // uint8 [2][128]: first non-finite row of a column of z
    static constexpr uint32_t kBars = kBad + 2 * kRows;
    static constexpr uint32_t kBytes = kBars + 512;
    static_assert(kBytes <= 232448, "more than an SM's shared memory");
};

struct Bars {
    uint64_t full[5], empty[5];
    uint64_t decays[2], decays_free[2], z_ok[2];
    uint64_t scores, p_ready, inter, out, out_read, y_ready, y_free, update, state_ready, done;
    LinearItem item;
    uint32_t tmem;
    int abort_flag, zero, bad[2];
    float sums[8];
};
static_assert(sizeof(Bars) <= 512, "");

// Copies one tile: rows of a tensor in the sweep's order, zeros behind n rows and behind dim columns up to 64 * blocks.
template <int BLOCKS>
__device__ __forceinline__ void load_tile(uint32_t dst, const bf16 *src, int64_t stride, int64_t first, int dir, int n, int dim,
                                          bool wide, int tid)
{
    constexpr int CH = 8 * BLOCKS;                    // 16-byte chunks of a row
#pragma unroll 8
    for (int i = 0; i < kRows * CH / kLoaders; ++i) {
        const int e = tid + i * kLoaders, r = e / CH, c = e % CH;
        const uint32_t to = dst + (c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        const bool row = r < n;
        const bf16 *from = src + (first + (int64_t)dir * (row ? r : 0)) * stride;
        if (wide) {
            const bool in = row && c * 8 < dim;
            cp_async16(to, in ? from + c * 8 : from, in);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = c * 8 + 2 * j;
                const uint32_t lo = row && k < dim ? reinterpret_cast<const uint16_t *>(from)[k] : 0;
                const uint32_t hi = row && k + 1 < dim ? reinterpret_cast<const uint16_t *>(from)[k + 1] : 0;
                w[j] = lo | hi << 16;
            }
            st_shared16(to, w[0], w[1], w[2], w[3]);
        }
    }
}

// two values as N bf16 terms each: word i holds term i of both
template <int N> __device__ __forceinline__ void split(float a, float b, uint32_t (&w)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w[i] = pack_bf16(a, b);
        if (i + 1 < N) {
            a -= low_bf16(w[i]);
            b -= high_bf16(w[i]);
        }
    }
}

// YB, ZB: blocks of 64 columns of x and y, of z. OUT: outputs (else the state a segment ends with from zero).
template <int YB, int ZB, int NS, bool OUT>
__global__ void __launch_bounds__(kThreadsChunk, 1)
    linear_chunk_kernel(const __grid_constant__ LinearLaunch P, const __grid_constant__ LinearSweep p, const int wide)
{
    using M = Smem<NS>;
    constexpr int kSlots = M::kSlots;
    constexpr int YP = 64 * YB, ZP = 64 * ZB;
    constexpr int TILES = OUT ? 3 : 2;                // x, y, z (x only with outputs)
    constexpr int YI = OUT ? 1 : 0, ZI = OUT ? 2 : 1;
    extern __shared__ __align__(1024) unsigned char sm[];
    Bars &B = *reinterpret_cast<Bars *>(sm + M::kBars);
    const uint32_t sbase = smem_u32(sm);
    float2(*decays)[kRows] = reinterpret_cast<float2(*)[kRows]>(sm + M::kDecays);
    uint8_t(*first_bad)[kRows] = reinterpret_cast<uint8_t(*)[kRows]>(sm + M::kBad);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = blockIdx.y;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&B.full[i], kLoaders), mbar_init(&B.empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&B.decays[i], 32), mbar_init(&B.decays_free[i], OUT ? 384 : 256), mbar_init(&B.z_ok[i], 32);
        mbar_init(&B.scores, 1), mbar_init(&B.inter, 1), mbar_init(&B.out, 1), mbar_init(&B.y_free, 1), mbar_init(&B.update, 1);
        mbar_init(&B.p_ready, 128), mbar_init(&B.out_read, 128), mbar_init(&B.y_ready, 256), mbar_init(&B.state_ready, 256);
        mbar_init(&B.done, 1);
        B.abort_flag = B.zero = B.bad[0] = B.bad[1] = 0;
        fence_barrier_init();
    }
    if (warp == 13) {
        const LinearItem it = linear_item(P, blockIdx.x, OUT && hv == 0);
        if (lane == 0) B.item = it;
    }
    __syncthreads();
    const LinearItem it = B.item;
    if (it.seq < 0 || (sbase & 1023u)) return;
    const bool whole = it.seq_end - it.seq_begin <= P.seg;
    if (!OUT && (whole || it.state < 0)) return;
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&B.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tcl_fence_before();
    __syncthreads();
    tcl_fence_after();
    const uint32_t tmem = B.tmem;
    const int n = it.n, chunks = (n + kRows - 1) / kRows;
    const int64_t first = p.reverse ? it.begin + n - 1 : it.begin;
    const int dir = p.reverse ? -1 : 1;
    const bool skip = it.state < 0;
    const long long limit = P.wait_limit > 0 ? P.wait_limit : kWaitLimit;
    volatile int *abort_flag = &B.abort_flag;
    bool ok = true;
    const auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok && !mbar_wait_warp(bar, parity & 1u, abort_flag, limit)) {
            ok = false;
            *abort_flag = 1;
            if (lane == 0) raise_flag(P.a.err_flags, GDN_DEVERR_TIMEOUT);
        }
        return ok;
    };
    const size_t state_at = ((size_t)(skip ? 0 : it.state) * P.a.HV + hv) * ((size_t)P.a.K * P.a.V);
    const size_t item_at = ((size_t)blockIdx.x * P.a.HV + hv) * ((size_t)P.a.K * P.a.V);

    if (warp >= 14) {
        // ---------------------------------------------------------------- copies
        const int t = tid - 14 * 32;
        const bf16 *src[3] = {static_cast<const bf16 *>(OUT ? p.x : p.y) + (int64_t)(hv / (OUT ? p.x_group : p.y_group)) * (OUT ? p.x_head : p.y_head),
                              static_cast<const bf16 *>(OUT ? p.y : p.z) + (int64_t)(hv / (OUT ? p.y_group : p.z_group)) * (OUT ? p.y_head : p.z_head),
                              static_cast<const bf16 *>(p.z) + (int64_t)(hv / p.z_group) * p.z_head};
        const int64_t stride[3] = {OUT ? p.x_stride : p.y_stride, OUT ? p.y_stride : p.z_stride, p.z_stride};
        int filled = 0;
        for (int i = 0; i < chunks && ok; ++i) {
            const int64_t at = first + (int64_t)dir * i * kRows;
            const int rows = min(kRows, n - i * kRows);
#pragma unroll
            for (int k = 0; k < TILES; ++k) {
                const int m = i * TILES + k, slot = m % kSlots;
                if (m >= kSlots && !wait(&B.empty[slot], m / kSlots - 1)) break;
                const uint32_t dst = sbase + slot * kTile;
                if (k == ZI) load_tile<ZB>(dst, src[k], stride[k], at, dir, rows, p.DZ, wide & 4, t);
                else load_tile<YB>(dst, src[k], stride[k], at, dir, rows, p.DY, wide & (OUT && k == 0 ? 1 : 2), t);
                cp_async_commit();
                if (m > 0) {                          // the tile before has landed: hand it on
                    cp_async_wait<1>();
                    fence_proxy_async();
                    mbar_arrive(&B.full[(m - 1) % kSlots]);
                }
                filled = m + 1;
            }
        }
        cp_async_wait<0>();
        if (ok && filled) {
            fence_proxy_async();
            mbar_arrive(&B.full[(filled - 1) % kSlots]);
        }
    } else if (warp == 13) {
        // ---------------------------------------------------------------- decays; z's non-finite values
        double all = 0.0;
        for (int i = 0; i < chunks; ++i) {
            const int b = i & 1;
            if (i >= 2 && !wait(&B.decays_free[b], (i >> 1) - 1)) break;
            double s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = i * kRows + lane * 4 + j;
                const double d = r < n ? linear_decay(P, hv, (int)first + dir * r, it.seq_end, p.reverse) : 0.0;
                s[j] = j ? s[j - 1] + d : d;
            }
            double sum = s[3];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(kAll, sum, o);
                if (lane >= o) sum += v;
            }
            const double before = lane ? __shfl_up_sync(kAll, sum, 1) : (__shfl_up_sync(kAll, sum, 1), 0.0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // 1/256 steps and the rest: differences of the first are exact, of the second small
                const double G = before + s[j], hi = rint(G * 256.0) * (1.0 / 256.0);
                decays[b][lane * 4 + j] = make_float2((float)hi, (float)(G - hi));
            }
            all += __shfl_sync(kAll, sum, 31);
            mbar_arrive(&B.decays[b]);
            const int m = i * TILES + ZI, slot = m % kSlots;
            if (!wait(&B.full[slot], m / kSlots)) break;
            const uint4 *z = reinterpret_cast<const uint4 *>(sm + slot * kTile);
            __nv_bfloat162 acc = __float2bfloat162_rn(0.f);
            const __nv_bfloat162 none = acc;
#pragma unroll 8
            for (int e = lane; e < ZB * (int)kBlock / 16; e += 32) {
                const uint4 v = z[e];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) acc = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]), none, acc);
            }
            const bool bad = __any_sync(kAll, __hisnan(acc.x) || __hisnan(acc.y));
            if (bad) {
                uint16_t *e = reinterpret_cast<uint16_t *>(sm + slot * kTile);
                for (int c = lane; c < ZP; c += 32) {
                    int from = 255;
                    for (int r = 0; r < kRows; ++r) {
                        uint16_t &v = e[(c >> 6) * (kBlock / 2) + r * 64 + ((((c & 63) >> 3) ^ (r & 7)) << 3) + (c & 7)];
                        if ((v & 0x7F80) == 0x7F80) {
                            if (from == 255) from = r;
                            v = 0;
                        }
                    }
                    first_bad[b][c] = (uint8_t)from;
                }
                fence_proxy_async();
            }
            if (lane == 0) B.bad[b] = bad;
            __syncwarp();
            mbar_arrive(&B.z_ok[b]);
        }
        if (!OUT && lane == 0) P.total[(size_t)blockIdx.x * P.a.HV + hv] = (float)all;
    } else if (warp == 12) {
        // ---------------------------------------------------------------- MMAs
        constexpr uint32_t id_scores = tc_idesc(128, 128, false), id_z = tc_idesc(128, ZP, true);
        for (int i = 0; i < chunks; ++i) {
            const int mx = i * TILES, my = mx + YI, mz = mx + ZI;
            const uint32_t tx = sbase + (mx % kSlots) * kTile, ty = sbase + (my % kSlots) * kTile, tz = sbase + (mz % kSlots) * kTile;
            if constexpr (OUT) {
                if (!wait(&B.full[mx % kSlots], mx / kSlots) || !wait(&B.full[my % kSlots], my / kSlots)) break;
                tcl_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < YP / 16; ++k) {
                        const uint32_t o = (k >> 2) * kBlock + (k & 3) * 32;
                        tcl_mma_ss(tmem + kScores, tc_desc(tx + o, 16), tc_desc(ty + o, 16), id_scores, k > 0);
                    }
                    tcl_commit(&B.scores);
                }
                __syncwarp();
                if (!wait(&B.state_ready, i) || (i > 0 && !wait(&B.out_read, i - 1))) break;
                tcl_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int t = 0; t < NS; ++t)
#pragma unroll
                        for (int k = 0; k < YP / 16; ++k) {
                            const uint32_t a = tx + (k >> 2) * kBlock + (k & 3) * 32, s = sbase + M::kStates + t * kTile + k * 2048;
                            tcl_mma_ss(tmem + kOut, tc_desc(a, 16), tc_desc(s, YP * 128), id_z, t + k > 0);
                        }
                    tcl_commit(&B.inter);
                }
                __syncwarp();
            }
            if (!wait(&B.z_ok[i & 1], i >> 1)) break;
            bool go = true;
            for (int h = 0; h < 2 && go; ++h) {
                go = wait(&B.y_ready, 2 * i + h);
                if (!go) break;
                tcl_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int t = 0; t < 3; ++t)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t a = tmem + kY + (k >> 1) * 48 + t * 16 + (k & 1) * 8;
                            tcl_mma_ts(tmem + kUpdate, a, tc_desc(tz + (4 * h + k) * 2048, kBlock), id_z, h + t + k > 0);
                        }
                    tcl_commit(&B.y_free);
                    if (h == 1) {
                        tcl_commit(&B.update);
                        if (OUT) tcl_commit(&B.empty[mx % kSlots]);
                        tcl_commit(&B.empty[my % kSlots]);
                        if (!OUT) tcl_commit(&B.empty[mz % kSlots]);
                    }
                }
                __syncwarp();
            }
            if (!go) break;
            if constexpr (OUT) {
                if (!wait(&B.p_ready, i)) break;
                tcl_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t a = tmem + kScores + (k >> 1) * 32 + t * 16 + (k & 1) * 8;
                            tcl_mma_ts(tmem + kOut, a, tc_desc(tz + k * 2048, kBlock), id_z, true);
                        }
                    tcl_commit(&B.out);
                    tcl_commit(&B.empty[mz % kSlots]);
                }
                __syncwarp();
            }
        }
        // every MMA has completed before the tensor memory is freed
        if (lane == 0) {
            tcl_commit(&B.done);
            mbar_wait(&B.done, 0u, &B.zero, kWaitLimit);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- Y and the state
        const int half = warp >= 8, y = tid & 127;    // this thread's row of the state; columns half * ZP / 2 ..
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        constexpr int ZC = ZP / 2;
        const bool active = (warp & 3) * 32 < YP;     // (YP = 64: lanes 64 .. 127 of Y are zero)
        const float z_inv = 1.f / p.z_scale;
        float S[ZC];
        {
            const float *from = nullptr;
            if (OUT && !skip) {
                if (!whole) from = P.local + item_at;
                else if (p.start) from = p.start + state_at;
            }
#pragma unroll
            for (int c = 0; c < ZC; ++c) {
                const int z = half * ZC + c;
                S[c] = from && y < p.DY && z < p.DZ ? from[y * p.sy + z * p.sz] * z_inv : 0.f;
            }
        }
        if (!active) {
            uint32_t zero[16] = {};
            for (int k = 0; k < 3; ++k) tcl_st16(tmem + lanes + kY + half * 48 + k * 16, zero);
            tcl_wait_st();
        }
        const auto put_state = [&]() {
            if (!active) return;
#pragma unroll
            for (int c = 0; c < ZC; c += 8) {
                uint32_t w[4][NS];
#pragma unroll
                for (int j = 0; j < 4; ++j) split<NS>(S[c + 2 * j], S[c + 2 * j + 1], w[j]);
                const int z = half * ZC + c;
                const uint32_t to = sbase + M::kStates + (z >> 6) * (YP * 128) + y * 128 + ((((z & 63) >> 3) ^ (y & 7)) << 4);
#pragma unroll
                for (int t = 0; t < NS; ++t) st_shared16(to + t * kTile, w[0][t], w[1][t], w[2][t], w[3][t]);
            }
        };
        if (OUT) {
            put_state();
            fence_proxy_async();
            tcl_fence_before();
            mbar_arrive(&B.state_ready);
        }
        for (int i = 0; i < chunks; ++i) {
            const int b = i & 1, m = i * TILES + YI, slot = m % kSlots;
            if (!wait(&B.decays[b], i >> 1) || !wait(&B.full[slot], m / kSlots)) break;
            const float2 end = decays[b][kRows - 1];
            bool go = true;
            for (int h = 0; h < 2; ++h) {
                const int s0 = 64 * h + 32 * half;
                const float2 d = decays[b][s0 + lane];
                const float weight = ex2(end.x - d.x) * ex2(end.y - d.y);
                if (2 * i + h > 0 && !wait(&B.y_free, 2 * i + h - 1)) {
                    go = false;
                    break;
                }
                tcl_fence_after();
                if (active) {
                    const uint16_t *ty = reinterpret_cast<const uint16_t *>(sm + slot * kTile + (y >> 6) * kBlock);
                    uint32_t w[3][16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int s = s0 + 2 * j + e;
                            const uint32_t raw = ty[s * 64 + ((((y & 63) >> 3) ^ (s & 7)) << 3) + (y & 7)];
                            v[e] = __uint_as_float(raw << 16) * __shfl_sync(kAll, weight, 2 * j + e);
                        }
                        uint32_t t[3];
                        split<3>(v[0], v[1], t);
                        w[0][j] = t[0], w[1][j] = t[1], w[2][j] = t[2];
                    }
#pragma unroll
                    for (int k = 0; k < 3; ++k) tcl_st16(tmem + lanes + kY + half * 48 + k * 16, w[k]);
                    tcl_wait_st();
                }
                tcl_fence_before();
                mbar_arrive(&B.y_ready);
            }
            if (!go || !wait(&B.update, i)) break;
            tcl_fence_after();
            const float decay = ex2(end.x) * ex2(end.y);
            const bool bad = *(volatile int *)&B.bad[b];
            if (active) {
#pragma unroll
                for (int c = 0; c < ZC; c += 32) {
                    float u[32];
                    tcl_ld32(tmem + lanes + kUpdate + half * ZC + c, u);
#pragma unroll
                    for (int j = 0; j < 32; ++j) S[c + j] = fmaf(S[c + j], decay, u[j]);
                    if (bad)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (first_bad[b][half * ZC + c + j] < kRows) S[c + j] = __int_as_float(0x7fc00000);
                }
            }
            tcl_fence_before();
            mbar_arrive(&B.decays_free[b]);
            if (OUT && i + 1 < chunks) {
                if (!wait(&B.inter, i)) break;        // the product with the state before has read it
                put_state();
                fence_proxy_async();
                mbar_arrive(&B.state_ready);
            }
        }
        const bool ends = p.reverse ? it.index == 0 : it.begin + n == it.seq_end;
        float *to = nullptr;
        if (!OUT) to = P.local + item_at;
        else if (ends && !skip && p.end) to = p.end + state_at;
        if (ok && to) {
            const float pass = OUT && p.reverse && it.seq_end > it.seq_begin ? exp2_wide(linear_log2(P.a.g[it.seq_begin * P.a.g_stride + hv])) : 1.f;
            const float f = pass * p.z_scale;
#pragma unroll
            for (int c = 0; c < ZC; ++c) {
                const int z = half * ZC + c;
                if (y < p.DY && z < p.DZ) to[y * p.sy + z * p.sz] = S[c] * f;
            }
        }
        if (OUT && p.with_end && ends) {
            float d = 0.f;
            if (!skip) {
                const float *w = p.with_end + state_at;
#pragma unroll
                for (int c = 0; c < ZC; ++c) {
                    const int z = half * ZC + c;
                    if (y < p.DY && z < p.DZ) d = fmaf(S[c] * p.z_scale, w[y * p.sy + z * p.sz], d);
                }
            }
            d = group_sum<32>(d);
            if (lane == 0) B.sums[warp - 4] = d;
        }
    } else if constexpr (OUT) {
        // ---------------------------------------------------------------- P, inter's decays, outputs
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        const int r = tid;
        const float f = p.x_scale * p.z_scale;
        for (int i = 0; i < chunks; ++i) {
            const int b = i & 1;
            if (!wait(&B.decays[b], i >> 1)) break;
            const float2 G = decays[b][r];
            if (!wait(&B.scores, i)) break;
            tcl_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t w[32] = {};
                if (c <= warp) {
                    float v[32];
                    tcl_ld32(tmem + lanes + kScores + c * 32, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int s = c * 32 + 2 * j;
                        const float4 d = *reinterpret_cast<const float4 *>(&decays[b][s]);
                        const float p0 = s <= r ? v[2 * j] * ex2((G.x - d.x) + (G.y - d.y)) : 0.f;
                        const float p1 = s + 1 <= r ? v[2 * j + 1] * ex2((G.x - d.z) + (G.y - d.w)) : 0.f;
                        uint32_t t[2];
                        split<2>(p0, p1, t);
                        w[j] = t[0], w[16 + j] = t[1];
                    }
                }
                tcl_st32(tmem + lanes + kScores + c * 32, w);
            }
            const float er = ex2(G.x) * ex2(G.y);
            if (!wait(&B.inter, i)) break;
            tcl_fence_after();
#pragma unroll 1
            for (int c = 0; c < ZP; c += 32) {
                float v[32];
                tcl_ld32(tmem + lanes + kOut + c, v);
                uint32_t w[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j] * er);
                tcl_st32(tmem + lanes + kOut + c, w);
            }
            tcl_wait_st();
            tcl_fence_before();
            mbar_arrive(&B.p_ready);
            if (!wait(&B.out, i)) break;
            tcl_fence_after();
            const bool bad = *(volatile int *)&B.bad[b];
            const bool mine = i * kRows + r < n;
            const int64_t t = first + (int64_t)dir * (i * kRows + r);
            const bf16 *with = p.dot && mine ? static_cast<const bf16 *>(p.dot_with) + t * p.dot_stride + (int64_t)(hv / p.dot_group) * p.dot_head : nullptr;
            float dot = 0.f;
#pragma unroll 1
            for (int c = 0; c < ZP; c += 32) {
                float v[32];
                tcl_ld32(tmem + lanes + kOut + c, v);
                if (c + 32 >= ZP) {
                    tcl_fence_before();
                    mbar_arrive(&B.out_read);
                }
                if (mine) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = skip ? 0.f : v[j] * f;
                    if (bad)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (first_bad[b][c + j] <= r && !skip) v[j] = __int_as_float(0x7fc00000);
                    const int left = p.DZ - c;            // columns there are
                    if (with) {
                        if ((wide & 8) && left >= 32) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) {
                                const uint4 q = *reinterpret_cast<const uint4 *>(with + c + j);
                                const uint32_t e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) dot = fmaf(v[j + 2 * k], low_bf16(e[k]), fmaf(v[j + 2 * k + 1], high_bf16(e[k]), dot));
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j < left) dot = fmaf(v[j], to_f32(with[c + j]), dot);
                        }
                    }
                    if (p.out) {
                        const int64_t to = t * p.out_stride + (int64_t)hv * p.out_head + c;
                        if (p.out_f32) {
                            float *o = static_cast<float *>(p.out) + to;
                            if ((wide & 16) && left >= 32) {
#pragma unroll
                                for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4 *>(o + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (j < left) o[j] = v[j];
                            }
                        } else {
                            bf16 *o = static_cast<bf16 *>(p.out) + to;
                            if ((wide & 16) && left >= 32) {
#pragma unroll
                                for (int j = 0; j < 32; j += 8)
                                    *reinterpret_cast<uint4 *>(o + j) = make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]),
                                                                                   pack_bf16(v[j + 4], v[j + 5]), pack_bf16(v[j + 6], v[j + 7]));
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (j < left) o[j] = __float2bfloat16_rn(v[j]);
                            }
                        }
                    }
                }
                __syncwarp();
            }
            mbar_arrive(&B.decays_free[b]);
            if (with) p.dot[t * P.a.HV + hv] = dot;
        }
    }
    tcl_fence_before();
    __syncthreads();
    if (OUT && p.with_end && tid == 0 && (p.reverse ? it.index == 0 : it.begin + n == it.seq_end)) {
        float s = 0.f;
        for (int w = 0; w < 8; ++w) s += B.sums[w];
        p.end_dot[(size_t)it.seq * P.a.HV + hv] = s;
    }
    if (warp == 12) {
        tcl_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

constexpr int kMaxDevices = 64;

template <int YB, int ZB, int NS, bool OUT>
int launch(const LinearLaunch &P, const LinearSweep &p, int wide, cudaStream_t stream)
{
    const auto kernel = linear_chunk_kernel<YB, ZB, NS, OUT>;
    static std::mutex lock;
    static bool raised[kMaxDevices] = {};             // the shared-memory limit, a function attribute of each device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GDN_ERR_LAUNCH;
    {
        std::lock_guard<std::mutex> g(lock);
        if (!raised[dev]) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<NS>::kBytes) != cudaSuccess) return GDN_ERR_LAUNCH;
            raised[dev] = true;
        }
    }
    kernel<<<dim3((unsigned)P.items, (unsigned)P.a.HV), kThreadsChunk, Smem<NS>::kBytes, stream>>>(P, p, wide);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

template <int YB, int ZB> int launch_size(const LinearLaunch &P, const LinearSweep &p, bool outputs, int wide, cudaStream_t stream)
{
    if (!outputs) return launch<YB, ZB, 2, false>(P, p, wide, stream);
    // what dg is summed from keeps the state whole
    return p.dot ? launch<YB, ZB, 3, true>(P, p, wide, stream) : launch<YB, ZB, 2, true>(P, p, wide, stream);
}

}  // namespace

int launch_linear_chunk(const LinearLaunch &P, const LinearSweep &p, bool outputs, cudaStream_t stream)
{
    const auto wide_rows = [](const void *q, int64_t stride, int64_t head, int n, int es) {
        return q && reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride * es % 16 == 0 && head * es % 16 == 0 && n * es % 16 == 0;
    };
    int wide = 0;
    if (wide_rows(p.x, p.x_stride, p.x_head, p.DY, 2)) wide |= 1;
    if (wide_rows(p.y, p.y_stride, p.y_head, p.DY, 2)) wide |= 2;
    if (wide_rows(p.z, p.z_stride, p.z_head, p.DZ, 2)) wide |= 4;
    if (wide_rows(p.dot_with, p.dot_stride, p.dot_head, p.DZ, 2)) wide |= 8;
    if (wide_rows(p.out, p.out_stride, p.out_head, 8, p.out_f32 ? 4 : 2)) wide |= 16;
    if (p.DY <= 64) return p.DZ <= 64 ? launch_size<1, 1>(P, p, outputs, wide, stream) : launch_size<1, 2>(P, p, outputs, wide, stream);
    return p.DZ <= 64 ? launch_size<2, 1>(P, p, outputs, wide, stream) : launch_size<2, 2>(P, p, outputs, wide, stream);
}

}  // namespace gdn
