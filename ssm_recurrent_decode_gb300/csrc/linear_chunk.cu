// linear_chunk.cu -- linear attention in bf16 on the tensor cores (tcgen05), 128 tokens at a time.
//
// For a chunk of rows r, s = 0 .. 127 in the sweep's order, with G the running sum of the log decays inside it and
// State the state before it (roles x, y, z as in linear_launch.h):
//     out_r = sum_{s <= r} (x_r . y_s) e^{G_r - G_s} z_s + e^{G_r} State^T x_r
//     State <- e^{G_last} State + sum_s e^{G_last - G_s} y_s z_s^T
// Four products a chunk, each with fp32 sums in tensor memory:
//     scores  [r, s] = x y^T                      both operands as loaded
//     inter   [r, z] = x State                    State from registers through shared memory, as two or three bf16 terms
//     out     [r, z] = inter e^{G_r} + P z        P = scores times decays, two bf16 terms, in tensor memory over the scores
//     update  [y, z] = Y^T z                      Y = y e^{G_last - G_s}, three bf16 terms, in tensor memory, 32 tokens at a time
// The terms are what keeps fp32: x, y and z are bf16 and exact, the state itself stays in fp32 registers (a lane of tensor
// memory is a row y of it, the columns z are shared by two warpgroups), a product's sum is added to it in fp32 once a chunk. The
// update's three terms keep 24 bits of the state; how many the outputs need is said at launch_size.
//
// One CTA owns a segment of a sequence and a value head. Its 24 warps are groups of four, which take turns on a chunk so that
// each one's latencies are covered by the others' work:
//   0, 1   two quarters of Y each, P between them, blocks of 32 columns in turn
//   2      inter's decays and the outputs (a thread a row r)
//   3, 4   the state, half its columns each
//   5      a warp each: MMAs of scores, inter and out; MMAs of the update; the decays, and z's non-finite values; copies of x, y
//          and z by TMA into a ring of 32 KB tiles (by plain loads what is not aligned to 16 bytes)
// What a chunk takes (5.5 us with two terms of the state, 10 with three and dg, 3.1 without outputs) is set by no one unit: the
// tensor pipe is active 24 to 40% of the time, 31 to 47% of the issue slots are used (8 x 2048 and 1 x 16384 tokens of 16 heads). A
// chunk's stages follow one another, and the seven tiles and 512 columns of tensor memory hold the operands of two chunks. The steps
// there, for 1 x 32768 tokens of 32 heads (both passes): 16 warps in step 1073 us; tiles by TMA, decays as factors of rows and of
// columns, one term for bf16 outputs 747; groups of warps with registers of their own (24 ragged prompts 316 -> 260) and outputs
// stored from registers as whole sectors 666; the update's weights apart from the other decays 597; states loaded as whole rows,
// decays in integers 513; whole rounds of CTAs 436; a token's heads side by side 423; two terms for bf16 outputs, as their cancelling
// sums need, 454.
// A tile may end in another sequence's rows: their y's weigh nothing, their scores are not looked at, their outputs are not
// written.
//
// A product with a zero of P would carry a later token's NaN to earlier ones; z's tile is looked over (one multiply-add a
// pair), and in the rare tile that has a non-finite value the outputs' product takes it as zero, the column's first such
// row is noted, and the outputs get their NaN from there.
//
// Every wait is bounded; a wait that gives up raises GDN_DEVERR_TIMEOUT and ends the CTA once its MMAs and copies are done. The outputs
// of its segment and head are NaN then, what other kernels read of it too.
#include <atomic>
#include <cstring>
#include <mutex>

#include "gdn_chain.cuh"
#include "linear_common.cuh"
#include "tc_ops.cuh"
#include "tma_map.h"

namespace gdn {

namespace {

constexpr int kRows = 128;                            // tokens per chunk
// The tensor cores cut off what a sum's step has below its largest term's last bit, towards zero. Measured on zero-mean inputs, in the
// states after a chunk: what 32 tokens bring is low by 0.4 to 1.2e-7 from their own steps and by 1.5e-7 more for every 32 tokens
// behind them whose share is not lost beside theirs (uncorrected: 1.1e-7 after 32 tokens, 3.4e-7 after 128, 2.2e-7
// under decays of 0.01 a token, 0.6e-7 of 0.5). Over many chunks that would add up, and where a difference of such sums counts (dg) it
// shows; so the update's weights carry it back, 32 tokens at a time in the sweep's order (states are then off by -0.9 to 1.3e-7
// on average, 0.7 to 2.0e-7 in norm, forwards and backwards, over decays of 0 to 2 a token; with one constant for all 128 it was -1.9e-7 for
// long memories and 3.2e-7 for short ones, and rows in one order for both sweeps would be low by 6.6e-7 backwards under 0.03).
// Outputs are low by 1.2 to 2.4e-7. (In the weights' exponents it costs nothing; as a factor of its own 3% of 1 x 32768 tokens.)
constexpr float kCutOwn = 0.9e-7f, kCutLater = 1.5e-7f, kCutOut = 2e-7f;
constexpr uint32_t kBlock = 16384;                    // 128 rows of 64 columns
constexpr uint32_t kTile = 2 * kBlock;
constexpr int kThreadsChunk = 768;
constexpr int kLoaders = 32;
// Registers a thread: 80 at launch; the groups that hold the state take more of them, the others give some up
// (2 x 128 + 4 x 56 = 6 x 80 for each of 128 threads). All four warps of a group execute the same of the two.
constexpr int kStateRegisters = 128, kOtherRegisters = 56;
static_assert(2 * kStateRegisters + 4 * kOtherRegisters <= 6 * 80, "more registers than the CTA has");
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegisters)); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegisters)); }
constexpr uint32_t kWaitLimit = 1u << 30;              // SM clock cycles, about half a second
// The limit of the waits that can give up (0: kWaitLimit); set only by the test hook below. The waits for copies and MMAs in
// flight always use kWaitLimit.
std::atomic<uint32_t> g_wait_limit{0};

// columns of tensor memory
constexpr uint32_t kScores = 0, kOut = 128, kUpdate = 256, kY = 384;
// Y: 48 columns for 32 tokens (16 tokens: three terms of eight columns); two buffers behind the others, two more where there are
// no outputs
__host__ __device__ constexpr uint32_t y_column(bool outputs, int buffer) { return outputs || buffer < 2 ? kY + 48 * buffer : 48 * (buffer - 2); }

constexpr int kMostSlots = 7;

// what the decays' warp says of a chunk's rows; G: sum of the log decays up to and with the row in the sweep's order, as a
// power of two, hi + lo with hi in steps of 1/256 (differences of hi are exact, lo is small)
struct Decays {
    float nhi[kRows], nlo[kRows];                     // -hi, -lo
    float col[kRows];                                 // e^{(G at the end of the row's 32) - G}
    float weight[2][kRows];                           // e^{(G at the chunk's end) - G}; 0 for rows behind the sequence. Two, since
                                                      // the state's warps come to a chunk last
};

struct ChunkMaps {
    CUtensorMap x, y, z;
};

struct Bars {
    uint64_t full[kMostSlots], empty[kMostSlots];     // tiles
    uint64_t weights[2], weight_free[2], rows, rows_free;              // Decays: its weights; the rest of it
    uint64_t z_raw[3], z_ok[2], bad_read;             // z's tile may be used for the update; for the outputs; first_bad was read
    uint64_t y_ready[4], y_free[4];                   // quarters of Y: written; used
    uint64_t scores, p_ready, inter, out, out_read, update[2], update_read, state_ready, done[2];
    float end_hi[2], end_lo[2];                       // G at the chunk's end
    uint32_t tmem;
    uint8_t abort_flag, bad[2];
};

// Seven tiles of shared memory: NS for the state's bf16 terms (0: no outputs), the others for x, y and z; and what the
// 227 KB leave besides.
template <int NS> struct Smem {
    static constexpr int kSlots = 7 - NS;
    static constexpr uint32_t kStates = kSlots * kTile;
    static constexpr uint32_t kDecays = 7 * kTile;
    static constexpr uint32_t kBad = kDecays + sizeof(Decays);        // uint8 [128]: first non-finite row of a column of z
    static constexpr uint32_t kBars = kBad + kRows;
    static constexpr uint32_t kBytes = kBars + sizeof(Bars);
    static_assert(kSlots <= kMostSlots && kBytes <= 232448 && sizeof(LinearItem) <= 64 && 64 + sizeof(LinearScan) <= sizeof(Decays), "more than an SM's shared memory");
};

// A tile by plain loads, for rows that TMA cannot copy (not 16-byte aligned): zeros behind n rows and dim columns.
// (2048 tokens of 8 heads of 128 x 128: 182 us, 35 by TMA; with 4-byte loads, 16 on their way a lane, 131 where rows are aligned
// to that, 342 where not, and ten ragged sequences' gradients, which never come here, 232 against 224 by its registers.)
template <int BLOCKS>
__device__ __forceinline__ void load_tile(uint32_t dst, const bf16 *src, int64_t stride, int n, int dim, int tid)
{
    constexpr int CH = 8 * BLOCKS;                    // 16-byte chunks of a row
#pragma unroll 2
    for (int e = tid; e < kRows * CH; e += kLoaders) {
        const int r = e / CH, c = e % CH;
        const uint32_t to = dst + (c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        const uint16_t *from = reinterpret_cast<const uint16_t *>(src + (int64_t)(r < n ? r : 0) * stride);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = c * 8 + 2 * j;
            const uint32_t lo = r < n && k < dim ? from[k] : 0, hi = r < n && k + 1 < dim ? from[k + 1] : 0;
            w[j] = lo | hi << 16;
        }
        st_shared16(to, w[0], w[1], w[2], w[3]);
    }
}

// Waits for a barrier's phase, every lane of a warp with one answer; false once the CTA gives up. A try suspends the warp
// for up to a millisecond (`suspend` ns), so that warps that wait leave the scheduler to those that work.
__device__ __forceinline__ bool try_phase(uint64_t *bar, uint32_t parity, uint32_t suspend)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(smem_u32(bar)), "r"(parity), "r"(suspend)
                 : "memory");
    return done != 0;
}
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, Bars *B, uint32_t limit)
{
    const uint32_t t0 = clock();
    bool done;
    do {
        done = try_phase(bar, parity & 1u, min(limit, 1000000u));
    } while (!done && !*(volatile uint8_t *)&B->abort_flag && (uint32_t)clock() - t0 < limit);
    done = __all_sync(kAll, done);
    if (!done) *(volatile uint8_t *)&B->abort_flag = 1;
    return done;
}
// Waits for what is in flight, whether or not the CTA has given up.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity)
{
    for (const uint32_t t0 = clock(); !try_phase(bar, parity & 1u, 1000000u) && (uint32_t)clock() - t0 < kWaitLimit;);
}

// 32 tokens of Y, from row s0 of y's tile, into the buffer at taddr: lane y of tensor memory takes column y.
__device__ __forceinline__ void make_y(const unsigned char *tile, int y, int s0, int rows, const float *weight, uint32_t taddr)
{
    const uint16_t *ty = reinterpret_cast<const uint16_t *>(tile + (y >> 6) * kBlock) + (y & 7);
    const int yc = (y & 63) >> 3;
#pragma unroll 1
    for (int k = 0; k < 2; ++k, s0 += 16) {           // 16 tokens: one step of the product
        // (step by step for all of them, so that the steps' latencies overlap)
        uint32_t raw[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) raw[j] = ty[(s0 + j) * 64 + ((yc ^ (j & 7)) << 3)];
#pragma unroll
        for (int j = 0; j < 16; ++j) raw[j] <<= 16;
        if (rows < s0 + 16) {                         // rows behind belong to no one or another sequence
#pragma unroll
            for (int j = 0; j < 16; ++j) raw[j] = s0 + j < rows ? raw[j] : 0;
        }
        f2 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = mul2(pair(raw[2 * j], raw[2 * j + 1]), *reinterpret_cast<const f2 *>(&weight[s0 + 2 * j]));
#pragma unroll
        for (int t = 0; t < 3; ++t) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = pack_bf16(v[j]);
            tcl_st8(taddr + k * 24 + t * 8, w);
            if (t < 2)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = fma2(pair(w[j] << 16, w[j] & 0xFFFF0000u), pair(-1.f, -1.f), v[j]);
        }
    }
    tcl_wait_st();
}

// YB, ZB: blocks of 64 columns of x and y, of z. NS: bf16 terms of the state; 0: no outputs, only the state a segment ends
// with from zero.
template <int YB, int ZB, int NS>
__global__ void __launch_bounds__(kThreadsChunk, 1)
    linear_chunk_kernel(const __grid_constant__ LinearLaunch P, const __grid_constant__ LinearSweep p,
                        const __grid_constant__ ChunkMaps maps, const int wide)
{
    using M = Smem<NS>;
    constexpr bool OUT = NS > 0;
    constexpr int kSlots = M::kSlots;
    constexpr int YP = 64 * YB, ZP = 64 * ZB;
    constexpr int NP = 2;                             // terms of P
    constexpr int TILES = OUT ? 3 : 2;                // x, y, z (x only with outputs)
    constexpr int YI = OUT ? 1 : 0, ZI = OUT ? 2 : 1;
    extern __shared__ __align__(1024) unsigned char sm[];
    Bars &B = *reinterpret_cast<Bars *>(sm + M::kBars);
    const uint32_t sbase = smem_u32(sm);
    Decays &decays = *reinterpret_cast<Decays *>(sm + M::kDecays);
    uint8_t *first_bad = sm + M::kBad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = blockIdx.x % P.a.HV;               // (a token's heads lie side by side in memory)

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&B.full[i], kLoaders), mbar_init(&B.empty[i], 2);
        for (int i = 0; i < 2; ++i) mbar_init(&B.weights[i], 32), mbar_init(&B.weight_free[i], 512);
        mbar_init(&B.rows, 32), mbar_init(&B.rows_free, 384), mbar_init(&B.bad_read, 128);
        for (int i = 0; i < 2; ++i) mbar_init(&B.z_ok[i], 32), mbar_init(&B.done[i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&B.y_ready[i], 128), mbar_init(&B.y_free[i], 1);
        for (int i = 0; i < 3; ++i) mbar_init(&B.z_raw[i], 32);
        mbar_init(&B.scores, 1), mbar_init(&B.inter, 1), mbar_init(&B.out, 1), mbar_init(&B.update[0], 1), mbar_init(&B.update[1], 1);
        mbar_init(&B.p_ready, 384), mbar_init(&B.out_read, 128), mbar_init(&B.state_ready, 256), mbar_init(&B.update_read, 256);
        B.abort_flag = B.bad[0] = B.bad[1] = 0;
        fence_barrier_init();
    }
    LinearItem *found = reinterpret_cast<LinearItem *>(sm + M::kDecays);       // (the decays come later)
    const int turn = warp == 22 ? linear_turn(P, blockIdx.x / P.a.HV) : blockIdx.x / P.a.HV;
    linear_find<kThreadsChunk>(P, turn, !OUT, OUT && hv == 0, 22, *reinterpret_cast<LinearScan *>(sm + M::kDecays + 64), found);
    const LinearItem it = *found;
    if (OUT && p.before_next && tid == 0) grid_launch_dependents();
    // (a CTA of a launch that may have started early ends behind the launch before it, on every path)
    const auto leave = [&]() {
        if (OUT && p.early && tid == 0) grid_dependency_wait();
    };
    if (it.seq < 0) return leave();
    // (the tiles' swizzle needs the 1024 bytes that the declaration asks for)
    if (!linear_in(P, it) || !GDN_IN(P.a.err_flags, sbase & 1023u, 1)) return leave();
    const bool whole = it.seq_end - it.seq_begin <= P.seg;
    if (!OUT && (whole || it.state < 0)) return;
    const int n = it.n, chunks = (n + kRows - 1) / kRows;
    const auto fill = [&](float v, int first, int warps) {         // the segment's outputs, a warp a row
        for (int r = first; p.out && r < n; r += warps)
            for (int c = lane; c < p.DZ; c += 32) {
                const int64_t at = (int64_t)(it.begin + r) * p.out_stride + (int64_t)hv * p.out_head + c;
                if (p.out_f32) static_cast<float *>(p.out)[at] = v;
                else static_cast<bf16 *>(p.out)[at] = __float2bfloat16_rn(v);
            }
    };
    if (it.state < 0) {                               // a bad state index: zeros
        fill(0.f, warp, kThreadsChunk / 32);
        return leave();
    }
    if (warp == 20) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&B.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tcl_fence_before();
    __syncthreads();
    tcl_fence_after();
    const uint32_t tmem = B.tmem;
    if (YB == 1 && warp < 4 && warp >= 2) {           // lanes 64 .. 127 of Y are zero
        const uint32_t zero[16] = {};
        for (int b = 0; b < (OUT ? 2 : 4); ++b)
            for (int k = 0; k < 48; k += 16) tcl_st16(tmem + ((uint32_t)(32 * warp) << 16) + y_column(OUT, b) + k, zero);
        tcl_wait_st();
    }
    if (YB == 1) {
        tcl_fence_before();
        __syncthreads();
        tcl_fence_after();
    }
    bool ok = true;
    const auto wait = [&](uint64_t *bar, uint32_t parity) { return ok = ok && wait_phase(bar, parity, &B, P.wait_limit); };
    const size_t state_at = ((size_t)it.state * P.a.HV + hv) * ((size_t)P.a.K * P.a.V);
    const size_t item_at = ((size_t)it.slot * P.a.HV + hv) * ((size_t)P.a.K * P.a.V);

    if (warp >= 20) {
        give_registers();
        if (warp == 23) {
            // ---------------------------------------------------------------- copies
            const int hx = OUT ? hv / p.x_group : 0, hy = hv / p.y_group, hz = hv / p.z_group;
            int issued = 0;
            for (int i = 0; i < chunks && ok; ++i) {
                const int at = it.begin + kRows * (p.reverse ? chunks - 1 - i : i);
#pragma unroll 1
                for (int k = 0; k < TILES; ++k) {
                    const int m = i * TILES + k, slot = m % kSlots;
                    const int which = k + 3 - TILES;      // 0: x, 1: y, 2: z
                    const bool tma = wide >> which & 1;
                    if (m >= kSlots && !wait(&B.empty[slot], m / kSlots - 1)) break;
                    const uint32_t dst = sbase + slot * kTile;
                    if (tma) {
                        if (lane == 0) {
                            const CUtensorMap *map = which == 0 ? &maps.x : which == 1 ? &maps.y : &maps.z;
                            const int head = which == 0 ? hx : which == 1 ? hy : hz, blocks = which == 2 ? ZB : YB;
                            mbar_arrive_expect_tx(&B.full[slot], blocks * kBlock);
                            mbar_arrive_n(&B.full[slot], kLoaders - 1);
                            for (int c = 0; c < blocks; ++c) tma_rows(dst + c * kBlock, map, 64 * c, head, at, &B.full[slot]);
                        }
                        __syncwarp();
                    } else {
                        const int rows = min(kRows, it.begin + n - at);
                        if (which == 2)
                            load_tile<ZB>(dst, static_cast<const bf16 *>(p.z) + hz * p.z_head + at * p.z_stride, p.z_stride, rows, p.DZ, lane);
                        else if (which == 1)
                            load_tile<YB>(dst, static_cast<const bf16 *>(p.y) + hy * p.y_head + at * p.y_stride, p.y_stride, rows, p.DY, lane);
                        else
                            load_tile<YB>(dst, static_cast<const bf16 *>(p.x) + hx * p.x_head + at * p.x_stride, p.x_stride, rows, p.DY, lane);
                        fence_proxy_async();
                        mbar_arrive(&B.full[slot]);
                    }
                    issued = m + 1;
                }
            }
            // Copies in flight land before the CTA ends (whether this warp gave up or another one will: nobody else may look
            // for the last tiles then).
            for (int m = max(0, issued - kSlots); m < issued; ++m)
                if (wide >> (m % TILES + 3 - TILES) & 1) drain(&B.full[m % kSlots], m / kSlots);
        } else if (warp == 22) {
            // ---------------------------------------------------------------- decays; z's non-finite values
            // Sums as 64-bit integers in steps of 2^-40 (fp64 runs at two operations a clock and SM, and this warp is on every
            // chunk's path); lane l takes the rows 4 l .. 4 l + 3 in the sweep's order, the next chunk's already loaded.
            double all = 0.0;
            const float cut = 1.44269504f * (kCutOwn + kCutLater * (3 - (lane >> 3)));   // (a lane's four rows lie in the same 32)
            float g[4];
            const auto fetch = [&](int i) {
                const int c = p.reverse ? chunks - 1 - i : i, at = it.begin + c * kRows, rows = min(kRows, n - c * kRows);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = p.reverse ? kRows - 1 - lane * 4 - j : lane * 4 + j, t = at + r + (p.reverse ? 1 : 0);
                    g[j] = r < rows && t < it.seq_end ? P.a.g[t * P.a.g_stride + hv] : 0.f;
                }
            };
            if (chunks > 0) fetch(0);
            for (int i = 0; i < chunks; ++i) {
                const int rows = min(kRows, n - kRows * (p.reverse ? chunks - 1 - i : i));
                long long s[4];
                bool nan[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const long long d = linear_fixed(g[j], nan[j]);
                    if (j) nan[j] |= nan[j - 1];
                    s[j] = j ? s[j - 1] + d : d;
                }
                if (i + 1 < chunks) fetch(i + 1);
                long long sum = s[3];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long v = __shfl_up_sync(kAll, sum, o);
                    if (lane >= o) sum += v;
                }
                const bool nan_before = (__ballot_sync(kAll, nan[3]) & ((1u << lane) - 1)) != 0;
                const long long before = sum - s[3];
                float hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    linear_parts(before + s[j], hi[j], lo[j]);
                    if (nan_before || nan[j]) lo[j] = __int_as_float(0x7fc00000);
                }
                const float hi32 = __shfl_sync(kAll, hi[3], lane | 7), lo32 = __shfl_sync(kAll, lo[3], lane | 7);
                const float hi_end = __shfl_sync(kAll, hi[3], 31), lo_end = __shfl_sync(kAll, lo[3], 31);
                if (!OUT) all += (double)hi_end + (double)lo_end;
                if (i >= 2 && !wait(&B.weight_free[i & 1], (i >> 1) - 1)) break;
                if (lane == 0) B.end_hi[i & 1] = hi_end, B.end_lo[i & 1] = lo_end;    // (the state's warps take its factor: this one's steps are on every chunk's path)
                float lo_cut = lo_end + cut;                  // what the weights carry back is a factor too
                if (rows < kRows && !p.reverse) lo_cut += 1.44269504f * kCutLater * (((rows - 1) >> 5) - 3);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = p.reverse ? kRows - 1 - lane * 4 - j : lane * 4 + j;
                    const float w = r < rows ? ex2(hi_end - hi[j]) * ex2(lo_cut - lo[j]) : 0.f;
                    decays.weight[i & 1][r] = w;
                }
                mbar_arrive(&B.weights[i & 1]);
                if (OUT) {
                    if (i > 0 && !wait(&B.rows_free, i - 1)) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = p.reverse ? kRows - 1 - lane * 4 - j : lane * 4 + j;
                        decays.nhi[r] = -hi[j];
                        decays.nlo[r] = -lo[j];
                        decays.col[r] = ex2(hi32 - hi[j]) * ex2(lo32 - lo[j]);
                    }
                    mbar_arrive(&B.rows);
                }
                const int b = i & 1;
                const int m = i * TILES + ZI, slot = m % kSlots;
                if (!wait(&B.full[slot], m / kSlots)) break;
                uint4 *z = reinterpret_cast<uint4 *>(sm + slot * kTile);
                const __nv_bfloat162 none = __float2bfloat162_rn(0.f);
                __nv_bfloat162 acc[4] = {none, none, none, none};
                const auto look = [&](const uint4 (&v)[4]) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[j] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]), none, acc[j]);
                    }
                };
                {
                    uint4 v[2][4];
                    const uint4 *from = z + lane;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[0][k] = from[32 * k];
#pragma unroll 1
                    for (int e = 0; e < ZB * (int)kBlock / 16 / 32; e += 8, from += 256) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[1][k] = from[128 + 32 * k];
                        look(v[0]);
                        if (e + 8 < ZB * (int)kBlock / 16 / 32)
#pragma unroll
                            for (int k = 0; k < 4; ++k) v[0][k] = from[256 + 32 * k];
                        look(v[1]);
                    }
                }
                acc[0] = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
                const bool bad = __any_sync(kAll, __hisnan(acc[0].x) || __hisnan(acc[0].y));
                if (bad && rows < kRows) {
                    // rows behind the sequence (or before it, none) are another's: zero
                    for (int e = lane; e < ZB * kRows * 8; e += 32)
                        if ((e >> 3) % kRows >= rows) z[e] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async();
                }
                // (a phase is waited for only when the one before it is known to be complete: parities repeat)
                if (OUT && bad && i >= 2 && !wait(&B.update[b], (i >> 1) - 1)) break;
                __syncwarp();
                mbar_arrive(&B.z_raw[i % 3]);
                if (!OUT) continue;
                if (i >= 1 && !wait(&B.bad_read, i - 1)) break;
                if (bad) {
                    // the update has its NaN; the outputs' product takes zeros, and the column's first row is noted
                    if (!wait(&B.update[i & 1], i >> 1)) break;
                    uint16_t *e = reinterpret_cast<uint16_t *>(z);
                    for (int k = lane; k < ZP; k += 32) {
                        int from = 255;
                        for (int j = 0; j < rows; ++j) {
                            const int r = p.reverse ? rows - 1 - j : j;
                            uint16_t &v = e[(k >> 6) * (kBlock / 2) + r * 64 + ((((k & 63) >> 3) ^ (r & 7)) << 3) + (k & 7)];
                            if ((v & 0x7F80) == 0x7F80) {
                                if (from == 255) from = r;
                                v = 0;
                            }
                        }
                        first_bad[k] = (uint8_t)from;
                    }
                    fence_proxy_async();
                }
                if (lane == 0) B.bad[b] = bad;
                __syncwarp();
                mbar_arrive(&B.z_ok[b]);
            }
            if (!OUT && lane == 0) P.total[(size_t)it.slot * P.a.HV + hv] = linear_parts(all);
        } else if (warp == 20) {
            // ---------------------------------------------------------------- MMAs: scores, inter, out
            constexpr uint32_t id_scores = tc_idesc(128, 128, false), id_z = tc_idesc(128, ZP, true);
            const uint64_t state = tc_desc(sbase + M::kStates, YP * 128);
            for (int i = 0; OUT && i < chunks; ++i) {
                const int mx = i * TILES, my = mx + YI, mz = mx + ZI;
                const uint64_t tx = tc_desc(sbase + (mx % kSlots) * kTile, 16), ty = tc_desc(sbase + (my % kSlots) * kTile, 16);
                const uint64_t tz = tc_desc(sbase + (mz % kSlots) * kTile, kBlock);
                // (descriptors step in units of 16 bytes; two arrivals free a tile: of two products, or one with a plain one)
                if (!wait(&B.full[mx % kSlots], mx / kSlots) || !wait(&B.full[my % kSlots], my / kSlots)) break;
                tcl_fence_after();
                if (lane == 0) {
#pragma unroll 1
                    for (int k = 0; k < YP / 16; ++k) {
                        const uint32_t o = ((k >> 2) * kBlock + (k & 3) * 32) >> 4;
                        tcl_mma_ss(tmem + kScores, tx + o, ty + o, id_scores, k > 0);
                    }
                    tcl_commit(&B.scores);
                    tcl_commit(&B.empty[my % kSlots]);
                }
                __syncwarp();
                if (!wait(&B.state_ready, i) || (i > 0 && !wait(&B.out_read, i - 1))) break;
                tcl_fence_after();
                if (lane == 0) {
#pragma unroll 1
                    for (int t = NS - 1; t >= 0; --t)         // the small terms first: sums are cut off, not rounded
#pragma unroll 1
                        for (int k = 0; k < YP / 16; ++k)
                            tcl_mma_ss(tmem + kOut, tx + (((k >> 2) * kBlock + (k & 3) * 32) >> 4), state + ((t * kTile + k * 2048) >> 4), id_z,
                                       t < NS - 1 || k > 0);
                    tcl_commit(&B.inter);
                    mbar_arrive(&B.empty[mx % kSlots]);
                    tcl_commit(&B.empty[mx % kSlots]);
                }
                __syncwarp();
                if (!wait(&B.z_ok[i & 1], i >> 1) || !wait(&B.p_ready, i)) break;
                tcl_fence_after();
                if (lane == 0) {
#pragma unroll 1
                    for (int t = NP - 1; t >= 0; --t)
#pragma unroll 1
                        for (int k = 0; k < 8; ++k)
                            tcl_mma_ts(tmem + kOut, tmem + kScores + k * 16 + t * 8, tz + (k * 2048 >> 4), id_z, true);
                    tcl_commit(&B.out);
                    tcl_commit(&B.empty[mz % kSlots]);
                }
                __syncwarp();
            }
            // every MMA has completed before the tensor memory is freed
            if (lane == 0) {
                tcl_commit(&B.done[0]);
                drain(&B.done[0], 0);
            }
            __syncwarp();
        } else if (warp == 21) {
            // ---------------------------------------------------------------- MMAs: update
            constexpr uint32_t id_z = tc_idesc(128, ZP, true);
            for (int i = 0; i < chunks; ++i) {
                const int my = i * TILES + YI, mz = i * TILES + ZI;
                const uint64_t tz = tc_desc(sbase + (mz % kSlots) * kTile, kBlock);
                if (!wait(&B.z_raw[i % 3], i / 3) || (i > 0 && !wait(&B.update_read, i - 1))) break;
                bool go = true;
#pragma unroll 1
                for (int u = 0; u < 4 && go; ++u) {       // 32 tokens each, in the sweep's order
                    go = wait(&B.y_ready[u], i);
                    if (!go) break;
                    tcl_fence_after();
                    if (lane == 0) {
                        const uint32_t y = tmem + y_column(OUT, OUT ? u & 1 : u);
                        const uint64_t z = tz + (p.reverse ? 3 - u : u) * (4096 >> 4);
#pragma unroll
                        for (int t = 2; t >= 0; --t)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                tcl_mma_ts(tmem + kUpdate, y + k * 24 + t * 8, z + (k * 2048 >> 4), id_z, u > 0 || t < 2 || k > 0);
                        tcl_commit(&B.y_free[u]);
                        if (u == 3) {
                            tcl_commit(&B.update[i & 1]);
                            tcl_commit(&B.empty[my % kSlots]);
                            tcl_commit(&B.empty[mz % kSlots]);
                            if (!OUT) {
                                mbar_arrive(&B.empty[my % kSlots]);
                                mbar_arrive(&B.empty[mz % kSlots]);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (!go) break;
            }
            if (lane == 0) {
                tcl_commit(&B.done[1]);
                drain(&B.done[1], 0);
            }
            __syncwarp();
        }
    } else if (warp >= 12) {
        take_registers();
        // ---------------------------------------------------------------- the state
        const int half = warp >= 16, y = tid & 127;    // this thread's row of the state; columns half * ZP / 2 ..
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        constexpr int ZC = ZP / 2;
        const bool active = (warp & 3) * 32 < YP;     // (YP = 64: lanes 64 .. 127 of Y are zero)
        const float z_inv = 1.f / p.z_scale;
        const int sy = (int)p.sy, sz = (int)p.sz;
        f2 S[ZC / 2];
        {
            const float *from = nullptr;
            if (OUT) {
                if (!whole) from = P.local + item_at;
                else if (p.start) from = p.start + state_at;
            }
            const int left = from && y < p.DY ? p.DZ - half * ZC : 0;             // columns there are to load
            from += y * sy + half * ZC * sz;
            float v[ZC];
            if (left >= ZC && sz == 1) {
#pragma unroll
                for (int c = 0; c < ZC; c += 4) *reinterpret_cast<float4 *>(&v[c]) = *reinterpret_cast<const float4 *>(from + c);
            } else if (left >= ZC) {
#pragma unroll
                for (int c = 0; c < ZC; ++c, from += sz) v[c] = *from;
            } else {
#pragma unroll
                for (int c = 0; c < ZC; ++c) v[c] = c < left ? from[c * sz] : 0.f;
            }
#pragma unroll
            for (int c = 0; c < ZC / 2; ++c) S[c] = pair(v[2 * c] * z_inv, v[2 * c + 1] * z_inv);
        }
        const auto put_state = [&]() {
            if (!active) return;
#pragma unroll
            for (int c = 0; c < ZC; c += 8) {
                uint32_t w[4][NS > 0 ? NS : 1];
#pragma unroll
                for (int j = 0; j < 4; ++j) split(S[c / 2 + j], w[j]);
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
            const int c0 = p.reverse ? chunks - 1 - i : i, at = it.begin + c0 * kRows;
            const size_t chunk = ((size_t)(at / kRows + it.seq) * P.a.HV + hv) * (128 * ZP) + (tid - 384);
            const bool mine = NS != 3 || GDN_IN(P.a.err_flags, at / kRows + it.seq, P.a.T / kRows + P.a.S);
            if (!wait(&B.weights[i & 1], i >> 1)) break;
            if (NS == 3 && p.chunk_dot) {
                // the product of this state's gradient, as it reaches the chunk's last row, and the state behind that row
                float d = 0.f;
                const int next = at + min(kRows, n - c0 * kRows);
                if (active && mine) {
#pragma unroll
                    for (int c = 0; c < ZC / 2; ++c) {
                        const float2 v = unpair(S[c]);
                        d = fmaf(v.x, p.chunk_states[chunk + 512 * c], fmaf(v.y, p.chunk_states[chunk + 512 * c + 256], d));
                    }
                    d *= exp2_wide(linear_decay(P, hv, next - 1, it.seq_end, 1)) * p.z_scale;
                }
                d = group_sum<32>(d);
                if (lane == 0 && mine) p.chunk_dot[((size_t)(at / kRows + it.seq) * P.a.HV + hv) * 8 + warp - 12] = d;
            }
            const float end_hi = B.end_hi[i & 1], end_lo = B.end_lo[i & 1];
            mbar_arrive(&B.weight_free[i & 1]);
            const float decay = linear_decay_factor(end_hi, end_lo);
            if (!wait(&B.update[i & 1], i >> 1)) break;
            tcl_fence_after();
            if (active) {
                const f2 decay2 = pair(decay, decay);
                const uint32_t from = tmem + lanes + kUpdate + half * ZC;
                uint32_t u[2][16];
                tcl_ld16_start(from, u[0]);
#pragma unroll
                for (int c = 0; c < ZC; c += 16) {
                    uint32_t(&v)[16] = u[(c >> 4) & 1];
                    tcl_ld16_wait(v);
                    if (c + 16 < ZC) tcl_ld16_start(from + c + 16, u[((c >> 4) & 1) ^ 1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) S[c / 2 + j] = fma2(S[c / 2 + j], decay2, pair(v[2 * j], v[2 * j + 1]));
                }
                if (NS == 3 && p.chunk_states && !p.chunk_dot && mine)
#pragma unroll
                    for (int c = 0; c < ZC / 2; ++c) {
                        const float2 v = unpair(S[c]);
                        p.chunk_states[chunk + 512 * c] = v.x;
                        p.chunk_states[chunk + 512 * c + 256] = v.y;
                    }
            }
            tcl_fence_before();
            mbar_arrive(&B.update_read);
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
        else if (ends && p.end) to = p.end + state_at;
        if (ok && to) {
            const float pass = OUT && p.reverse && it.seq_end > it.seq_begin ? exp2_wide(linear_log2(P.a.g[it.seq_begin * P.a.g_stride + hv])) : 1.f;
            const float f = pass * p.z_scale;
            const int left = y < p.DY ? p.DZ - half * ZC : 0;
            to += y * sy + half * ZC * sz;
            if (left >= ZC && sz == 1) {
#pragma unroll
                for (int c = 0; c < ZC / 2; c += 2) {
                    const float2 v = unpair(S[c]), w = unpair(S[c + 1]);
                    *reinterpret_cast<float4 *>(to + 2 * c) = make_float4(v.x * f, v.y * f, w.x * f, w.y * f);
                }
            } else if (left >= ZC) {
#pragma unroll
                for (int c = 0; c < ZC / 2; ++c, to += 2 * sz) {
                    const float2 v = unpair(S[c]);
                    to[0] = v.x * f;
                    to[sz] = v.y * f;
                }
            } else {
#pragma unroll
                for (int c = 0; c < ZC / 2; ++c) {
                    const float2 v = unpair(S[c]);
                    if (2 * c < left) to[2 * c * sz] = v.x * f;
                    if (2 * c + 1 < left) to[(2 * c + 1) * sz] = v.y * f;
                }
            }
        }
    } else if (warp < 8) {
        give_registers();
        // ---------------------------------------------------------------- two quarters of Y; P
        const int group = warp >> 2, quad = warp & 3, r = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        for (int i = 0; i < chunks; ++i) {
            const int m = i * TILES + YI, slot = m % kSlots;
            const int rows = min(kRows, n - kRows * (p.reverse ? chunks - 1 - i : i));
            if (!wait(&B.weights[i & 1], i >> 1) || !wait(&B.full[slot], m / kSlots)) break;
            bool go = true;
#pragma unroll 1
            for (int k = 0; k < 2 && go; ++k) {
                // quarters group and 2 + group, in the sweep's order; with outputs both in the same buffer
                const int u = 2 * k + group;
                go = OUT ? k ? wait(&B.y_free[group], i) : i == 0 || wait(&B.y_free[2 + group], i - 1) : i == 0 || wait(&B.y_free[u], i - 1);
                if (!go) break;
                tcl_fence_after();
                if (32 * quad < YP) make_y(sm + slot * kTile, r, 32 * (p.reverse ? 3 - u : u), rows, decays.weight[i & 1], tmem + lanes + y_column(OUT, OUT ? group : u));
                tcl_fence_before();
                mbar_arrive(&B.y_ready[u]);
                if (!OUT || k == 1) continue;
                // P, while the first half is being used
                go = wait(&B.rows, i) && wait(&B.scores, i);
                if (!go) break;
                const float hi = -decays.nhi[r], lo = -decays.nlo[r];
                tcl_fence_after();
                // Blocks of 32 columns s, every other one, over which P's terms are laid (16 columns: eight of the first term,
                // eight of the second). In the row's own 32 the decay is taken for each element, and the columns it does not
                // see (s > r; backwards s < r and rows behind the sequence) are zero; the columns of other 32s have theirs as
                // a factor of the column times one of the row.
                const int from = p.reverse ? r : 0, to = p.reverse ? rows : r + 1;
#pragma unroll 1
                for (int c = group; c < 4; c += 2) {
                    const bool none = p.reverse ? c < quad : c > quad;
                    const bool each = c == quad || (p.reverse && rows < c * 32 + 32);
                    float f = 0.f;
                    if (!none && !each) {
                        const int end = p.reverse ? c * 32 : c * 32 + 31;
                        f = ex2(hi + decays.nhi[end]) * ex2(lo + decays.nlo[end]);
                    }
                    const uint32_t at = tmem + lanes + kScores + c * 32;
                    if (none) {
                        const uint32_t zero[16] = {};
                        tcl_st16(at, zero);
                        tcl_st16(at + 16, zero);
                        continue;
                    }
                    const auto convert = [&](int h, const uint32_t (&v)[16]) {
                        const int s0 = c * 32 + h * 16;
                        f2 q[8];
                        if (each) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int s = s0 + 2 * j;
                                const f2 d = add2(add2(pair(hi, hi), *reinterpret_cast<const f2 *>(&decays.nhi[s])),
                                                  add2(pair(lo, lo), *reinterpret_cast<const f2 *>(&decays.nlo[s])));
                                const float2 e = unpair(d);
                                const float p0 = __uint_as_float(v[2 * j]) * ex2(e.x), p1 = __uint_as_float(v[2 * j + 1]) * ex2(e.y);
                                q[j] = pair(s >= from && s < to ? p0 : 0.f, s + 1 >= from && s + 1 < to ? p1 : 0.f);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) q[j] = mul2(*reinterpret_cast<const f2 *>(&decays.col[s0 + 2 * j]), pair(f, f));
#pragma unroll
                            for (int j = 0; j < 8; ++j) q[j] = mul2(pair(v[2 * j], v[2 * j + 1]), q[j]);
                        }
#pragma unroll
                        for (int k = 0; k < NP; ++k) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[j] = pack_bf16(q[j]);
                            tcl_st8(at + h * 16 + k * 8, w);
                            if (k + 1 < NP)
#pragma unroll
                                for (int j = 0; j < 8; ++j) q[j] = fma2(pair(w[j] << 16, w[j] & 0xFFFF0000u), pair(-1.f, -1.f), q[j]);
                        }
                    };
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[16];
                        tcl_ld16(at + h * 16, v);
                        convert(h, v);
                    }
                }
                mbar_arrive(&B.rows_free);
                tcl_wait_st();
                tcl_fence_before();
                mbar_arrive(&B.p_ready);
            }
            if (!go) break;
            mbar_arrive(&B.weight_free[i & 1]);
        }
    } else {
        give_registers();
        if constexpr (OUT) {
        // ---------------------------------------------------------------- inter's decays, outputs
        const int quad = warp & 3, r = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const float f = p.x_scale * p.z_scale * (1.f + kCutOut);
        for (int i = 0; i < chunks; ++i) {
            {
                if (!wait(&B.rows, i)) break;
                const float er = ex2(-decays.nhi[r]) * ex2(-decays.nlo[r]);
                mbar_arrive(&B.rows_free);
                if (!wait(&B.inter, i)) break;
                tcl_fence_after();
                const f2 er2 = pair(er, er);
                const uint32_t at = tmem + lanes + kOut;
#pragma unroll 1
                for (int c = 0; c < ZP; c += 16) {
                    uint32_t u[16];
                    tcl_ld16(at + c, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 q = unpair(mul2(pair(u[2 * j], u[2 * j + 1]), er2));
                        u[2 * j] = __float_as_uint(q.x), u[2 * j + 1] = __float_as_uint(q.y);
                    }
                    tcl_st16(at + c, u);
                }
                tcl_wait_st();
                tcl_fence_before();
                mbar_arrive(&B.p_ready);
            }
            if (!wait(&B.out, i)) break;
            tcl_fence_after();
            const int b = i & 1, c0 = p.reverse ? chunks - 1 - i : i, rows = min(kRows, n - c0 * kRows);
            const bool bad = *(volatile uint8_t *)&B.bad[b];
            const int64_t t = it.begin + c0 * kRows + r;
            const bool mine = r < rows && linear_in(P, (int)t, hv, P.a.HV);
            const bf16 *with = NS == 3 && p.dot && mine ? static_cast<const bf16 *>(p.dot_with) + t * p.dot_stride + (int64_t)(hv / p.dot_group) * p.dot_head : nullptr;
            float dot = 0.f;
            if (bad) {
                // columns whose z is not finite from a row on: NaN from there
#pragma unroll 1
                for (int c = 0; c < ZP; ++c) {
                    const int fb = first_bad[c];
                    if (fb == 255) continue;          // the same in every lane
                    uint32_t v;
                    const uint32_t at = tmem + lanes + kOut + c;
                    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(v) : "r"(at) : "memory");
                    if (p.reverse ? r <= fb : r >= fb) v = 0x7fc00000u;
                    __syncwarp();
                    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(at), "r"(v) : "memory");
                }
            }
            const auto take = [&](int c, const uint32_t (&u)[16]) {
                f2 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = mul2(pair(u[2 * j], u[2 * j + 1]), pair(f, f));
                if (!mine) return;
                const int left = p.DZ - c;            // columns there are
                if (NS == 3 && with) {
                    float d = 0.f;
                    if ((wide & 8) && left >= 16) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(with + c + 8 * j);
                            const uint32_t e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 o = unpair(v[4 * j + k]);
                                d = fmaf(o.x, low_bf16(e[k]), fmaf(o.y, high_bf16(e[k]), d));
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 o = unpair(v[j]);
                            if (2 * j < left) d = fmaf(o.x, to_f32(with[c + 2 * j]), d);
                            if (2 * j + 1 < left) d = fmaf(o.y, to_f32(with[c + 2 * j + 1]), d);
                        }
                    }
                    dot += d;
                }
                if (!p.out) return;
                const int64_t to = t * p.out_stride + (int64_t)hv * p.out_head + c;
                if ((wide & 16) && left >= 16) {
                    // whole sectors of 32 bytes
                    uint32_t w[16];
                    if (p.out_f32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 e = unpair(v[j]);
                            w[2 * j] = __float_as_uint(e.x), w[2 * j + 1] = __float_as_uint(e.y);
                        }
                        st_global32(static_cast<float *>(p.out) + to, w);
                        st_global32(static_cast<float *>(p.out) + to + 8, w + 8);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = pack_bf16(v[j]);
                        st_global32(static_cast<bf16 *>(p.out) + to, w);
                    }
                    return;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 e = unpair(v[j]);
                    if (p.out_f32) {
                        if (2 * j < left) static_cast<float *>(p.out)[to + 2 * j] = e.x;
                        if (2 * j + 1 < left) static_cast<float *>(p.out)[to + 2 * j + 1] = e.y;
                    } else {
                        if (2 * j < left) static_cast<bf16 *>(p.out)[to + 2 * j] = __float2bfloat16_rn(e.x);
                        if (2 * j + 1 < left) static_cast<bf16 *>(p.out)[to + 2 * j + 1] = __float2bfloat16_rn(e.y);
                    }
                }
            };
            {
                const uint32_t at = tmem + lanes + kOut;
#pragma unroll 1
                for (int c = 0; c < ZP; c += 16) {
                    uint32_t u[16];
                    tcl_ld16(at + c, u);
                    if (c + 16 >= ZP) {
                        tcl_fence_before();
                        mbar_arrive(&B.out_read);
                    }
                    take(c, u);
                    __syncwarp();
                }
            }
            if (NS == 3 && with) p.dot[t * P.a.HV + hv] = dot;
            mbar_arrive(&B.bad_read);
        }
        }
    }
    tcl_fence_before();
    __syncthreads();
    if (B.abort_flag && warp >= 12 && warp < 20) {    // (warps with registers to spare)
        const float none = __int_as_float(0x7fc00000);
        if (tid == 384) raise_flag(P.a.err_flags, GDN_DEVERR_TIMEOUT);
        if (!OUT) {
            if (tid == 384) P.total[(size_t)it.slot * P.a.HV + hv] = make_float2(none, none);          // and with it the states of the segments behind
        } else {
            fill(none, warp - 12, 8);
            if (NS == 3 && p.dot)
                for (int r = tid - 384; r < n; r += 256) p.dot[(size_t)(it.begin + r) * P.a.HV + hv] = none;
            if (p.end && (p.reverse ? it.index == 0 : it.begin + n == it.seq_end))
                for (int e = tid - 384; e < P.a.K * P.a.V; e += 256) p.end[state_at + e] = none;
        }
    }
    if (warp == 20) {
        tcl_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    leave();
}

constexpr int kMaxDevices = 64;

template <int YB, int ZB, int NS>
int launch(const LinearLaunch &P, const LinearSweep &p, const ChunkMaps &maps, int wide, cudaStream_t stream)
{
    const auto kernel = linear_chunk_kernel<YB, ZB, NS>;
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
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const int64_t ctas = (int64_t)(NS > 0 ? P.items : P.cut_items) * P.a.HV;
    if (ctas > INT32_MAX) return GDN_ERR_SHAPE;
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreadsChunk);
    cfg.dynamicSmemBytes = Smem<NS>::kBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (p.early) set_programmatic(attr[cfg.numAttrs++]);
    return cudaLaunchKernelEx(&cfg, kernel, P, p, maps, wide) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

template <int YB, int ZB> int launch_size(const LinearLaunch &P, const LinearSweep &p, bool outputs, const ChunkMaps &maps, int wide, cudaStream_t stream)
{
    if (!outputs) return launch<YB, ZB, 0>(P, p, maps, wide, stream);
    // Terms of the state and of P: two of each, whose remainder is at most 2^-16 of a term of the outputs' sums. One would do where
    // the sums' terms do not cancel (zero-mean inputs: 0.0023 of the norm off, 0.0017 with two as by rounding the exact result to bf16),
    // but keys or values with a common mean leave outputs far below their terms: 1024 tokens of mean 1 and spread 0.1, q
    // orthogonal to the mean: 0.38 off with one term, 0.0017 with two. (32768 tokens of 32 heads: 455 us, 423 with one; 24 ragged
    // prompts 148 and 136; gradients of 8 x 2048 816 and 790.) What dg is summed from keeps the state whole, as three.
    return p.dot ? launch<YB, ZB, 3>(P, p, maps, wide, stream) : launch<YB, ZB, 2>(P, p, maps, wide, stream);
}

}  // namespace

int launch_linear_chunk(const LinearLaunch &launch, const LinearSweep &p, bool outputs, cudaStream_t stream)
{
    LinearLaunch P = launch;
    const uint32_t limit = g_wait_limit.load(std::memory_order_relaxed);
    P.wait_limit = limit ? limit : kWaitLimit;
    const auto wide_rows = [](const void *q, int64_t stride, int64_t head, int n, int es) {
        return q && reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride * es % 16 == 0 && head * es % 16 == 0 && n * es % 16 == 0;
    };
    int wide = 0;
    ChunkMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    const int HV = P.a.HV;
    if (outputs && encode_head_rows(&maps.x, p.x, P.a.T, HV / p.x_group, p.DY, p.x_stride, p.x_head, kRows)) wide |= 1;
    if (encode_head_rows(&maps.y, p.y, P.a.T, HV / p.y_group, p.DY, p.y_stride, p.y_head, kRows)) wide |= 2;
    if (encode_head_rows(&maps.z, p.z, P.a.T, HV / p.z_group, p.DZ, p.z_stride, p.z_head, kRows)) wide |= 4;
    if (wide_rows(p.dot_with, p.dot_stride, p.dot_head, p.DZ, 2)) wide |= 8;
    if (reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.out_stride * (p.out_f32 ? 4 : 2) % 32 == 0 && p.out_head * (p.out_f32 ? 4 : 2) % 32 == 0) wide |= 16;
    if (p.DY <= 64) return p.DZ <= 64 ? launch_size<1, 1>(P, p, outputs, maps, wide, stream) : launch_size<1, 2>(P, p, outputs, maps, wide, stream);
    return p.DZ <= 64 ? launch_size<2, 1>(P, p, outputs, maps, wide, stream) : launch_size<2, 2>(P, p, outputs, maps, wide, stream);
}

}  // namespace gdn

extern "C" int64_t gdn_linear_set_wait_limit(int64_t cycles)
{
    return gdn::g_wait_limit.exchange(cycles <= 0 ? 0u : cycles < gdn::kWaitLimit ? (uint32_t)cycles : gdn::kWaitLimit);
}
