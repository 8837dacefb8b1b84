// scan_carry.cu -- the selective scan's pass over the chunks: from each chunk's end state counted
// from zero to the state that the next chunk starts from, and backwards the same for e.
#include "scan_common.cuh"

namespace gdn {

constexpr int kCarryThreads = 64;      // small CTAs: the loads in flight are spread over the SMs

// One thread per state entry walks the chunks in order (blockIdx.y = 0) or backwards (1). The loads of a
// chunk do not depend on the carry: those of the next U chunks are in flight while U chunks are worked
// on. The traffic is 12 bytes per entry and chunk.
__global__ void __launch_bounds__(kCarryThreads) scan_carry_kernel(const __grid_constant__ ScanLaunch P)
{
    ordinary_launch_start();
    const int64_t dn = (int64_t)P.a.D * P.a.N;
    const int64_t i = (int64_t)blockIdx.x * kCarryThreads + threadIdx.x;
    if (i >= dn) return;
    const bool back = blockIdx.y != 0;
    const int d = (int)(i / P.a.N);
    const float A = finite_rate(P.a.A[i]);
    float *val = back ? P.ein : P.hin;
    const float *sums = back ? P.sumdt_head : P.sumdt;
    const float *boundary = back ? P.g.dh_last : P.a.h0;
    float carry = 0.f;
    constexpr int U = 8;
    // chunk of position k in this direction; nothing goes on behind the last (before the first)
    const auto chunk = [&](int k) { return back ? P.G - 1 - k : k; };
    float loc[U], sum[U];
    int seq[U], edge[U];
    const auto fetch = [&](int k0, float (&lo)[U], float (&su)[U], int (&sq)[U], int (&ed)[U]) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool on = k0 + k < P.G - 1;
            const int g = chunk(on ? k0 + k : 0);
            const int4 info = P.info[g];
            lo[k] = on ? val[g * dn + i] : 0.f;
            su[k] = on ? sums[(int64_t)g * P.a.D + d] : 0.f;
            sq[k] = on ? (back ? info.z : info.x) : -1;
            ed[k] = back ? info.w : info.y;
        }
    };
    fetch(0, loc, sum, seq, edge);
    for (int k0 = 0; k0 < P.G; k0 += U) {
        float loc2[U], sum2[U], decay[U];
        int seq2[U], edge2[U];
        if (k0 + U < P.G) fetch(k0 + U, loc2, sum2, seq2, edge2);      // while this batch is worked on
#pragma unroll
        for (int k = 0; k < U; ++k) decay[k] = expf(A * sum[k]);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (k0 + k >= P.G) break;
            const int g = chunk(k0 + k);
            val[g * dn + i] = carry;
            if (seq[k] >= 0 && edge[k]) {           // the sequence begins (backwards: ends) in this chunk
                carry = 0.f;
                if (boundary) {
                    const int64_t slot = P.a.state_indices ? (int64_t)P.a.state_indices[seq[k]] : seq[k];
                    if (slot >= 0 && slot < P.a.num_states) carry = boundary[slot * dn + i];
                }
                if (!back && P.init) P.init[g * dn + i] = carry;
            }
            // where nothing goes on there is no carry, and where it is zero no product: 0 x inf is not 0
            const float next = carry == 0.f ? loc[k] : fmaf(decay[k], carry, loc[k]);
            carry = seq[k] >= 0 ? next : 0.f;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            loc[k] = loc2[k];
            sum[k] = sum2[k];
            seq[k] = seq2[k];
            edge[k] = edge2[k];
        }
    }
}

cudaError_t launch_scan_carry(const ScanLaunch &P, bool both, cudaStream_t stream)
{
    const int64_t dn = (int64_t)P.a.D * P.a.N;
    return launch_ordinary(scan_carry_kernel, dim3((unsigned)((dn + kCarryThreads - 1) / kCarryThreads), both ? 2 : 1),
                           dim3(kCarryThreads), 0, stream, P);
}

}  // namespace gdn
