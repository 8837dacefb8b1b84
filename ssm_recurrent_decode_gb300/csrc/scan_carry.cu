// scan_carry.cu -- the selective scan's pass over the chunks: from each chunk's end state counted
// from zero to the state that the next chunk starts from, and backwards the same for e.
#include "scan_common.cuh"

namespace gdn {

constexpr int kCarryThreads = 64;      // small CTAs: the loads in flight are spread over the SMs

// One thread per state entry walks the chunks in order (blockIdx.y = 0) or backwards (1). Two loads
// per chunk do not depend on the carry, so U chunks' values are in flight at a time; the traffic is
// 12 bytes per entry and chunk.
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
    constexpr int U = 16;
    for (int k0 = 0; k0 < P.G; k0 += U) {
        float loc[U], sum[U];
        int seq[U], edge[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool on = k0 + k < P.G - 1;       // nothing goes on behind the last chunk (before the first)
            const int g = back ? P.G - 1 - (k0 + k) : k0 + k;
            const int4 info = on ? P.info[g] : make_int4(-1, 0, -1, 0);
            seq[k] = back ? info.z : info.x;
            edge[k] = back ? info.w : info.y;
            loc[k] = seq[k] >= 0 ? val[g * dn + i] : 0.f;
            sum[k] = seq[k] >= 0 ? sums[(int64_t)g * P.a.D + d] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (k0 + k >= P.G) break;
            const int g = back ? P.G - 1 - (k0 + k) : k0 + k;
            val[g * dn + i] = carry;
            if (seq[k] < 0) {
                carry = 0.f;
                continue;
            }
            if (edge[k]) {                          // the sequence begins (backwards: ends) in this chunk
                carry = 0.f;
                if (boundary) {
                    const int64_t slot = P.a.state_indices ? (int64_t)P.a.state_indices[seq[k]] : seq[k];
                    if (slot >= 0 && slot < P.a.num_states) carry = boundary[slot * dn + i];
                }
                if (!back && P.init) P.init[g * dn + i] = carry;
            }
            // no product with the decay where nothing is carried: 0 x inf is not 0
            carry = carry == 0.f ? loc[k] : fmaf(expf(A * sum[k]), carry, loc[k]);
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
