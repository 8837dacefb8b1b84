// scan_launch.h -- launch parameters of the selective scan (internal to libgdn_decode.so).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mamba_scan.h"

namespace gdn {

// how the rows of an input tensor may be copied
enum { kRowsAny = 0, kRows4 = 1, kRows16 = 2 };
// whole-vector access to outputs and states (bits of ScanLaunch::vec)
enum { kVecY = 1, kVecState = 2, kVecDx = 4, kVecDdt = 8, kVecDz = 16 };

struct ScanLaunch {
    mamba_scan_args a;
    int L;              // rows per sequence without cu_seqlens
    int C, G;           // rows per chunk, chunks
    int cpt;            // channels per thread
    int nct;            // channel tiles
    int cluster;        // a short forward call: its G chunks are a thread-block cluster, in one launch
    int vec;
    int mode_x, mode_dt, mode_z, mode_b, mode_c, mode_dy;
    int has_states;     // state indices are checked
    // workspace
    int4 *info;         // [G] x: sequence that goes on behind the chunk (-1: none), y: it begins inside,
                        //         z: sequence that began before the chunk (-1: none), w: it ends inside
    float *sumdt;       // [G, D] sum of dt over the rows of info.x's sequence
    float *hin;         // [G, D, N] the state that chunk ends with from zero; then the state it starts from
    float *init;        // [G, D, N] initial state of info.x's sequence, when it begins in the chunk
    // backward only
    mamba_scan_grad_args g;
    float *sumdt_head;  // [G, D] sum of dt over the rows of info.z's sequence
    float *ein;         // [G, D, N] e that the chunk sends to the row before it, from zero; then e at its last row
    float *part_bc;     // [nct, T, 2 N] each channel tile's share of dBm and dCm
    float *part_a;      // [W, D, N] each worker's share of dA
    float *part_d;      // [W, D] each worker's share of dDskip
    int W;              // workers per channel tile
};

// lanes along the state for a state size, and the channels of a CTA of four warps
inline int scan_lanes(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }
inline int scan_channels(int N, int cpt) { return 4 * (32 / scan_lanes(N)) * cpt; }

constexpr int kScanBackChunk = 64;   // most token rows per chunk of the backward pass
constexpr int kScanBackCtas = 2;     // its resident CTAs per SM

// Resident CTAs per SM of the forward kernel by its registers, which chunks are counted out for. Shared memory
// allows as many for states above 16 and for 9 to 16 entries in bf16 at four channels a thread; fewer for 9 to 16 in fp32
// (73 KB a CTA: 3) and up to 8 (67 KB in bf16: 3; 116 KB in fp32: 1), whose chunks then take a second round or more:
// 32768 rows, D = 1536: N = 4, 8 and 16 in bf16 272, 258 and 379 us, in fp32 379, 380 and 401. Wide states (N above 32) ran faster with more registers a
// thread than with a fourth CTA (N = 128, 4 x 1024 rows, fp32: 245 against 323 us), narrow ones a little slower
// (N = 16, 32768 rows: 382 against 379; 24 ragged prompts of 8000: 131 against 123 to 129), and six CTAs of 80
// registers were slower for both.
constexpr int scan_ctas(int lanes) { return lanes >= 16 ? 3 : 4; }

// The carry pass over the chunks (forward; with both also the backward one, over e).
cudaError_t launch_scan_carry(const ScanLaunch &P, bool both, cudaStream_t stream);

int launch_scan_forward(const ScanLaunch &P, cudaStream_t stream);
int launch_scan_backward(const ScanLaunch &P, cudaStream_t stream);

}  // namespace gdn
