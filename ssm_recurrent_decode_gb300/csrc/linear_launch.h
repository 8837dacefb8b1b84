// linear_launch.h -- launch parameters of linear attention (internal to libgdn_decode.so).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gdn_linear.h"

namespace gdn {

// One sweep over the sequences with a state. All four products of the operation and its gradients have the form
//     State_t[y, z] = decay_t State_{t-1}[y, z] + y_t[y] z_t[z]        out_t[z] = sum_y State_t[y, z] x_t[y]
// with the roles (x, y, z) = (q, k, v) for o, (do, v, k) for dq, and, from the last token to the first with the
// decay of the token behind, (k, q, do) for dv and (v, do, q) for dk.
struct LinearSweep {
    const void *x, *y, *z;             // x may be null: no outputs
    int64_t x_stride, x_head, y_stride, y_head, z_stride, z_head;
    int x_group, y_group, z_group;     // value heads that share a head of x, y, z
    int DY, DZ;                        // sizes of x and y, of z
    float x_scale, z_scale;
    int reverse;
    void *out;                         // [T, HV (or heads), DZ]
    int64_t out_stride, out_head;
    int out_f32;                       // out is fp32, else bf16
    int64_t sy, sz;                    // strides of the state's memory [V, K] along y and z
    const float *start;                // [num_states, HV, V, K] states to start from, or null: zero
    float *end;                        // [num_states, HV, V, K] states to end with, or null
    // of the tensor-core kernel:
    float *dot;                        // [T, HV] or null: sum_z out_t[z] dot_with_t[z], before rounding
    const void *dot_with;
    int64_t dot_stride, dot_head;
    int dot_group;
    // for dg, per chunk (chunk c of sequence s: its first row / 128 + s; of the fp32 kernel per segment) and value head:
    float *chunk_states;               // the state behind it, in the kernel's own order
    float *chunk_dot;                  // given, chunk_states is read, and the parts of its product with the state the
                                       // sweep comes with are written (8, or one per part of z)
    // Two sweeps that need nothing of each other: the second one's CTAs take the SMs that the first one's last CTAs leave empty
    // (programmatic dependent launch), and end behind them.
    int before_next;                   // the launch behind this one may start early
    int early;                         // this one may
};

struct LinearLaunch {
    gdn_linear_args a;
    float scale;
    int Ls;             // rows per sequence without cu_seqlens
    int seg;            // rows per segment of a sequence
    int items;          // most segments (of all sequences) there can be; every sequence has at least one
    int cut_items;      // most segments of sequences that have several: the CTAs of the pass without outputs
    int carried;        // a sequence may have several segments
    int states;         // state indices are checked
    int tc;             // the tensor-core kernel
    // workspace
    float *local;       // [cut_items, HV, V, K] the state that a segment ends with from zero; then the one it starts with
    float2 *total;      // [cut_items, HV] log2 of the segment's decay, as two numbers
    uint32_t wait_limit;  // SM clock cycles of a wait that can give up
};

constexpr int kLinearSorted = 64;      // up to so many sequences, the longest start first, and a warp finds a segment; a block beyond
constexpr int kLinearZ = 64;           // columns of z per CTA of the fp32 kernel

// The sweep on the CUDA cores in fp32 (any size, stride); outputs: p.x given. Without: local and total.
int launch_linear_recurrent(const LinearLaunch &P, const LinearSweep &p, bool outputs, cudaStream_t stream);
// The same for bf16 inputs on the tensor cores.
int launch_linear_chunk(const LinearLaunch &P, const LinearSweep &p, bool outputs, cudaStream_t stream);
constexpr int kLinearChunk = 128;      // its tokens per chunk

// bf16 rows [T, heads, n] copied to dense rows of n rounded up to eight, zeros behind
int launch_linear_pack(const void *from, int64_t stride, int64_t head, int T, int heads, int n, void *to, cudaStream_t stream);

// Between the two: local from end states to start states.
int launch_linear_carry(const LinearLaunch &P, const LinearSweep &p, cudaStream_t stream);

// Sum over the value heads that share one: out[t, h] = sum part[t, h G ..], and dot[t, hv] = part[t, hv] . with[t, h]
struct LinearFold {
    const float *part;                 // [T, HV, K]
    void *out;                         // or null
    int64_t out_stride, out_head;
    const void *with;
    int64_t with_stride, with_head;
    float *dot;                        // [T, HV] or null
};
int launch_linear_fold(const LinearLaunch &P, const LinearFold &f, cudaStream_t stream);

// dg from the products per token and segment: dg_t = sum over the rows from t to the segment's end of (q.dq - k.dk), plus
// the segment's products (parts of them).
size_t linear_dg_part_floats(int items, int HV);
int launch_linear_dg(const LinearLaunch &P, const float *qdq, const float *kdk, const float *segment_dot, int parts, float *dg,
                     int64_t dg_stride, float *part, cudaStream_t stream);

// The same from products per token and chunk (chunk_dot), of the tensor-core kernel. `part`: 8 a chunk and head.
int launch_linear_dg_chunks(const LinearLaunch &P, const float *qdq, const float *kdk, const float *chunk_dot, float *dg,
                            int64_t dg_stride, float *part, cudaStream_t stream);

}  // namespace gdn
