/*
 * mamba_scan.h -- C ABI of the Mamba-1 selective scan over whole sequences and of its backward
 * pass in libgdn_decode.so; conventions as in gdn_decode.h (device pointers owned by the caller,
 * nothing allocated or synchronised, launches only on `stream`, host-side checks before any CUDA
 * call, negative gdn_status on error). The scan turns a prompt into the state that
 * mamba_selective_scan_decode (mamba_decode.h) continues from.
 *
 * The operation, for every sequence s with tokens t = first(s) .. last(s), channel d and state entry n:
 *     h_t[d,n] = exp(dt_t[d] A[d,n]) h_{t-1}[d,n] + dt_t[d] x_t[d] Bm_t[n],   h_{first-1} = h0[s]
 *     y_t[d]   = (sum_n Cm_t[n] h_t[d,n] + Dskip[d] x_t[d]) * silu(z_t[d])
 *     h_last[s] = h_{last(s)}
 * which is mamba_selective_scan_decode token by token: dt is used as given, arithmetic and states are
 * fp32. Its gradients, with g_t = dy_t silu(z_t) and e_t = exp(dt_{t+1} A) dh_{t+1} (e at the last
 * token: dh_last, or 0):
 *     dh_t = Cm_t g_t + e_t          w_t = dh_t exp(dt_t A) h_{t-1}     du_t[d] = sum_n dh_t[d,n] Bm_t[n]
 *     dx_t = dt_t du_t + Dskip g_t   ddt_t = x_t du_t + sum_n A w_t     dz_t = dy_t (y_t before the gate) silu'(z_t)
 *     dBm_t[n] = sum_d dh_t dt_t x_t   dCm_t[n] = sum_d g_t h_t   dA = sum_t dt_t w_t   dDskip = sum_t g_t x_t
 *     dh0[s] = exp(dt A) dh at first(s)
 * Source: the recurrence of "Triton decode kernel + MBU analysis", section "Kernel design"; the same
 * page's "Prefill path" names the scan over a prompt.
 *
 * Sequences are packed end to end: token rows 0 .. T-1. With cu_seqlens sequence s owns rows
 * cu_seqlens[s] .. cu_seqlens[s+1]-1 (it may be empty: its final state is then its initial one);
 * without, T rows are S sequences of T / S tokens each. Two sequences of a call may not name the same
 * state row (the result is then undefined).
 */
#ifndef MAMBA_SCAN_H
#define MAMBA_SCAN_H

#include <stddef.h>
#include <stdint.h>

#include "gdn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mamba_scan_args {
    int32_t T;                    /* token rows, >= 0 */
    int32_t S;                    /* sequences, >= 1; without cu_seqlens a divisor of T */
    int32_t D;                    /* channels */
    int32_t N;                    /* state entries per channel, 1 .. 128 */
    int32_t in_dtype;             /* gdn_dtype of x, dt, Bm, Cm, z (and of dy and the token gradients) */
    int32_t out_dtype;            /* gdn_dtype of y */
    const void *x;                /* [T, D], row stride x_stride */
    int64_t x_stride;
    const void *dt;               /* [T, D], row stride dt_stride */
    int64_t dt_stride;
    const float *A;               /* [D, N] dense */
    const void *Bm;               /* [T, N], row stride B_stride */
    int64_t B_stride;
    const void *Cm;               /* [T, N], row stride C_stride */
    int64_t C_stride;
    const float *Dskip;           /* [D] or NULL */
    const void *z;                /* [T, D], row stride z_stride, or NULL: no gate */
    int64_t z_stride;
    const int32_t *cu_seqlens;    /* [S + 1], from 0 to T without a decrease, or NULL */
    const int32_t *state_indices; /* [S]: row of each sequence in h0, h_last, dh_last and dh0, or NULL: row s */
    int32_t num_states;           /* rows of those buffers */
    const float *h0;              /* [num_states, D, N] or NULL: start from zero */
    float *h_last;                /* [num_states, D, N] or NULL; may be h0 itself (in place); where it
                                     overlaps h0 otherwise, no row written may be a row that another sequence
                                     reads. Rows that no sequence names are left as they are */
    void *y;                      /* [T, D] out_dtype, row stride y_stride */
    int64_t y_stride;
    void *workspace;              /* mamba_scan_workspace_bytes bytes, 16-byte aligned (NULL when that is 0) */
    size_t workspace_bytes;
    int32_t *err_flags;           /* optional device word: GDN_DEVERR_BAD_INDEX is ORed in for a state index
                                     outside [0, num_states) (that sequence's y is zeroed, its states and
                                     gradients are left out) and for rows that cu_seqlens gives to no sequence
                                     (their y and gradients are zeroed) */
} mamba_scan_args;

/* The gradients. s holds the forward call's inputs (s.y, s.h_last and s.out_dtype are not used, s.workspace
 * is this call's). Token gradients have in_dtype and rows of their own strides; a NULL gradient is not
 * written. dBm and dCm sum over channels, dA and dDskip over tokens, in a fixed order in fp32. */
typedef struct mamba_scan_grad_args {
    mamba_scan_args s;
    const void *dy;               /* [T, D] in_dtype, row stride dy_stride */
    int64_t dy_stride;
    const float *dh_last;         /* [num_states, D, N] or NULL: zero */
    void *dx;                     /* [T, D] */
    int64_t dx_stride;
    void *ddt;                    /* [T, D] */
    int64_t ddt_stride;
    void *dz;                     /* [T, D]; only with z */
    int64_t dz_stride;
    void *dBm;                    /* [T, N] */
    int64_t dB_stride;
    void *dCm;                    /* [T, N] */
    int64_t dC_stride;
    float *dA;                    /* [D, N] dense */
    float *dDskip;                /* [D]; only with Dskip */
    float *dh0;                   /* [num_states, D, N]; rows that no sequence names are left as they are;
                                     may not overlap dh_last. Without h0 too: the gradient at a start
                                     from zero */
} mamba_scan_grad_args;

/* Bytes of workspace that a call with these sizes needs; uniform: non-zero when cu_seqlens is NULL.
 * 0 for sizes that the calls refuse. The backward pass keeps every channel tile's share of dBm and dCm,
 * 8 T N bytes a tile of 128 channels (N up to 16), 64 (up to 32), 32 (up to 64) or 16, which for wide
 * states is many times the inputs: T = 16384 and D = 4096 take 1.6 GB at N = 64, 5.4 GB at N = 128. */
size_t mamba_scan_workspace_bytes(int32_t T, int32_t S, int32_t D, int32_t N, int32_t uniform, int32_t backward);

/*
 * mamba_selective_scan -- the scan. Returns GDN_OK, GDN_ERR_NULL (a missing pointer, or no workspace
 * where one is needed), GDN_ERR_SHAPE (negative sizes, N outside 1..128, T not a multiple of S without
 * cu_seqlens, a row stride below the row, a workspace that is too small), GDN_ERR_DTYPE, GDN_ERR_ALIGN
 * (a pointer not aligned to its element, or the workspace not to 16 bytes) or GDN_ERR_LAUNCH. Any row
 * stride is accepted; rows that are 16-byte aligned (pointer and stride) are copied faster. Other outputs
 * than h_last may not overlap the inputs, one another or the workspace (not checked).
 */
int mamba_selective_scan(const mamba_scan_args *args, gdn_stream_t stream);

/* mamba_selective_scan_backward -- its gradients; the same status codes, and GDN_ERR_ARG for dz without
 * z, dDskip without Dskip or dh0 over dh_last. Recomputes the states from the inputs: nothing of the
 * forward call has to be kept. */
int mamba_selective_scan_backward(const mamba_scan_grad_args *args, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_SCAN_H */
