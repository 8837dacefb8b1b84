// scan_carry.cu -- the selective scan's pass over the chunks: from each chunk's end state counted
// from zero to the state that the next chunk starts from, and backwards the same for e.
#include "scan_common.cuh"

namespace gdn {

constexpr int kCarryThreads = 64;      // small CTAs: the loads in flight are spread over the SMs
constexpr int kCarryU = 16;            // chunks whose loads are in flight while as many are worked on

// One thread per state entry walks the chunks in order (blockIdx.y = 0) or backwards (1). The traffic is 12
// bytes per entry and chunk, the loads do not depend on the carry; what counted was instructions: 73 per
// entry and chunk with every chunk's borders looked at by every thread (57 us for 256 chunks of 24576 entries
// in both directions), some 15 where a batch of chunks has none (30 us).
__global__ void __launch_bounds__(kCarryThreads) scan_carry_kernel(const __grid_constant__ ScanLaunch P)
{
    ordinary_launch_start();
    const int lane = threadIdx.x & 31;
    const int64_t dn = (int64_t)P.a.D * P.a.N;
    const int64_t at = (int64_t)blockIdx.x * kCarryThreads + threadIdx.x;
    const bool live = at < dn;
    const int64_t i = live ? at : dn - 1;
    const bool back = blockIdx.y != 0;
    const int d = (int)(i / P.a.N);
    const float A2 = finite_rate(P.a.A[i] * kLog2e);
    const float *boundary = back ? P.g.dh_last : P.a.h0;
    // position k of this direction is chunk k, or G - 1 - k
    const int64_t vstep = back ? -dn : dn, sstep = back ? -(int64_t)P.a.D : P.a.D;
    float *val = (back ? P.ein + (P.G - 1) * dn : P.hin) + i;
    const float *sums = (back ? P.sumdt_head + (int64_t)(P.G - 1) * P.a.D : P.sumdt) + d;
    const int last = P.G - 1;             // nothing goes on behind the last position

    float loc[kCarryU], sum[kCarryU], loc2[kCarryU], sum2[kCarryU];
    int4 info = make_int4(-1, 0, -1, 0), info2;          // of position k0 + lane
    const auto fetch = [&](int k0, float (&lo)[kCarryU], float (&su)[kCarryU], int4 &in) {
        const int mine = min(k0 + (lane & (kCarryU - 1)), last);
        in = P.info[back ? P.G - 1 - mine : mine];
        const float *v = val + k0 * vstep, *s = sums + k0 * sstep;
#pragma unroll
        for (int k = 0; k < kCarryU; ++k) {
            lo[k] = k0 + k < last ? *v : 0.f;
            su[k] = k0 + k < last ? *s : 0.f;
            v += vstep;
            s += sstep;
        }
    };
    float carry = 0.f;
    fetch(0, loc, sum, info);
    for (int k0 = 0; k0 < P.G; k0 += kCarryU) {
        const bool more = k0 + kCarryU < P.G;
        if (more) fetch(k0 + kCarryU, loc2, sum2, info2);
        // (the last position's own record is not looked at: forward, no summary wrote it)
        const bool inner = k0 + (lane & (kCarryU - 1)) < last;
        const int seq = !inner ? -1 : back ? info.z : info.x, edge = back ? info.w : info.y;
        const bool plain = k0 + kCarryU <= last && __all_sync(kScanFull, seq >= 0 && !edge);
        float *v = val + k0 * vstep;
        if (plain) {
            // no product with the decay where nothing is carried: 0 x inf is not 0
#pragma unroll
            for (int k = 0; k < kCarryU; ++k) {
                if (live) *v = carry;
                v += vstep;
                carry = carry == 0.f ? loc[k] : fmaf(ex2_approx(fmaf(A2, sum[k], kDecayBias)), carry, loc[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kCarryU; ++k) {
                const int sq = __shfl_sync(kScanFull, seq, k), ed = __shfl_sync(kScanFull, edge, k);
                if (k0 + k >= P.G) break;
                if (live) *v = carry;
                v += vstep;
                if (sq >= 0 && ed) {      // the sequence begins (backwards: ends) in this chunk
                    carry = 0.f;
                    const int64_t slot = P.a.state_indices ? (int64_t)P.a.state_indices[sq] : sq;
                    if (boundary && slot >= 0 && slot < P.a.num_states) carry = boundary[slot * dn + i];
                    if (!back && P.init && live) P.init[(int64_t)(k0 + k) * dn + i] = carry;
                }
                const float next = carry == 0.f ? loc[k] : fmaf(ex2_approx(fmaf(A2, sum[k], kDecayBias)), carry, loc[k]);
                carry = sq >= 0 ? next : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < kCarryU; ++k) {
            loc[k] = loc2[k];
            sum[k] = sum2[k];
        }
        info = info2;
    }
}

cudaError_t launch_scan_carry(const ScanLaunch &P, bool both, cudaStream_t stream)
{
    const int64_t dn = (int64_t)P.a.D * P.a.N;
    return launch_ordinary(scan_carry_kernel, dim3((unsigned)((dn + kCarryThreads - 1) / kCarryThreads), both ? 2 : 1),
                           dim3(kCarryThreads), 0, stream, P);
}

}  // namespace gdn
