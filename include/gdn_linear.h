/*
 * gdn_linear.h -- C ABI of linear attention with a decay for each head in libgdn_decode.so: whole
 * sequences (prompts), their backward pass, and the single-token step over a pool of states.
 * Conventions as in gdn_decode.h (device pointers owned by the caller, nothing allocated or
 * synchronised, launches only on `stream`, host-side checks before any CUDA call, negative
 * gdn_status on error).
 *
 * The operation, for value head hv with q/k head h = hv / (HV / H) and every token t of a sequence:
 *     S_t = exp(g_t) S_{t-1} + v_t k_t^T          (state [V, K], S_{first-1} = initial_state or 0)
 *     o_t = scale S_t q_t
 * g is one log decay per token and head, or one per head (g_stride 0). It is the step of gdn_decode.h
 * without the delta rule's subtraction (delta = v); "Optimization Log: Qwen3.5-27B Dense on B200",
 * Kernel 4, has that step. The gradients, with D_t the gradient of S_t:
 *     D_t  = scale do_t q_t^T + exp(g_{t+1}) D_{t+1}       (at the last token: + d_final_state)
 *     dq_t = scale S_t^T do_t     dk_t = D_t^T v_t     dv_t = D_t k_t     dg_t = exp(g_t) <D_t, S_{t-1}>
 *     d_initial_state = exp(g_first) D_first
 * with dq and dk summed over the value heads that share them, and dg over tokens where g is one per head.
 *
 * Arithmetic and states are fp32 whatever the inputs' type (states are stored in fp32, for the step also in
 * bf16). With bf16 inputs the sequences' products take what is not bf16 already as a sum of bf16 numbers: the
 * states carried from token to token keep 24 bits; where a token's output or gradient is summed, the state that it
 * meets and its scores times decays keep 16 bits, so that the sum is off by at most 2^-16 of the sum of its terms'
 * magnitudes beside what fp32 sums lose. Where dg is asked for, the states that dq and dk meet keep 24 bits: the last
 * bits of dq and dk may depend on it.
 *
 * A log decay below -200 counts as -200 (a factor of 0 in fp32). Log decays may be positive; no sum of consecutive
 * ones may then leave +-87 (fp32's powers of two). Infinite inputs count as NaN, and a NaN reaches outputs of its own
 * token and of later ones (gradients of k and v: of earlier ones; of g, which is summed over tokens: of any token of its
 * sequence), and no other sequence.
 *
 * Sequences are packed end to end: token rows 0 .. T-1. With cu_seqlens sequence s owns rows
 * cu_seqlens[s] .. cu_seqlens[s+1]-1 (it may be empty: its final state is then its initial one); without,
 * T rows are S sequences of T / S tokens each. Rows that cu_seqlens gives to no sequence may hold
 * anything and are not written. Two sequences of a call may not name the same state row (the result is then undefined).
 */
#ifndef GDN_LINEAR_H
#define GDN_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#include "gdn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdn_linear_args {
    int32_t T;                    /* token rows, >= 0 */
    int32_t S;                    /* sequences, >= 1; without cu_seqlens a divisor of T */
    int32_t H;                    /* q/k heads */
    int32_t HV;                   /* value heads, a multiple of H */
    int32_t K;                    /* key size: 16, 32, 64 or 128 */
    int32_t V;                    /* value size, 1 .. 128 */
    int32_t in_dtype;             /* gdn_dtype of q, k, v (and of do and the token gradients) */
    int32_t out_dtype;            /* gdn_dtype of o */
    const void *q;                /* q[t,h,:] at q + t q_stride + h q_head_stride; k, v and o alike */
    int64_t q_stride, q_head_stride;
    const void *k;
    int64_t k_stride, k_head_stride;
    const void *v;
    int64_t v_stride, v_head_stride;
    const float *g;               /* g[t,hv] at g + t g_stride + hv; g_stride 0: one per head */
    int64_t g_stride;
    float scale;                  /* 0 selects K^-1/2 */
    const int32_t *cu_seqlens;    /* [S + 1], from 0 without a decrease to at most T, or NULL */
    const int32_t *state_indices; /* [S]: row of each sequence in the state buffers, or NULL: row s */
    int32_t num_states;           /* rows of those buffers */
    const float *initial_state;   /* [num_states, HV, V, K] or NULL: start from zero */
    float *final_state;           /* [num_states, HV, V, K] or NULL; may be initial_state itself (in place).
                                     Rows that no sequence names are left as they are */
    void *o;                      /* [T, HV, V] out_dtype */
    int64_t o_stride, o_head_stride;
    void *workspace;              /* gdn_linear_workspace_bytes bytes, 16-byte aligned (NULL when that is 0);
                                     calls that may run at the same time need one each */
    size_t workspace_bytes;
    int32_t *err_flags;           /* optional device word: GDN_DEVERR_BAD_INDEX is ORed in for a state index
                                     outside [0, num_states) and for a sequence whose cu_seqlens leave 0 .. T or
                                     decrease (its rows are not written; of such a table, rows that two
                                     other sequences claim hold either one's outputs, dg is undefined, and
                                     sequences of more than T rows together may be left out whole); where the state index
                                     is bad, the sequence's outputs and gradients are zeroed and its states left
                                     out. GDN_DEVERR_TIMEOUT when a bounded wait gave up: the outputs,
                                     states and gradients that needed what it waited for are NaN */
} gdn_linear_args;

/* The gradients. s holds the forward call's inputs (s.o, s.final_state and s.out_dtype are not used,
 * s.workspace is this call's). Token gradients have in_dtype; a NULL gradient is not written. */
typedef struct gdn_linear_grad_args {
    gdn_linear_args s;
    const void *d_o;              /* [T, HV, V] */
    int64_t do_stride, do_head_stride;
    const float *d_final_state;   /* [num_states, HV, V, K] or NULL: zero */
    void *dq;                     /* [T, H, K] */
    int64_t dq_stride, dq_head_stride;
    void *dk;                     /* [T, H, K] */
    int64_t dk_stride, dk_head_stride;
    void *dv;                     /* [T, HV, V] */
    int64_t dv_stride, dv_head_stride;
    float *dg;                    /* like g: rows dg_stride apart, or [HV] when g_stride is 0 */
    int64_t dg_stride;
    float *d_initial_state;       /* [num_states, HV, V, K]; rows that no sequence names are left as they are;
                                     may not overlap d_final_state or initial_state. Also without
                                     initial_state: the gradient at a start from zero */
} gdn_linear_grad_args;

/* The single-token step: request row b on state slot cache_indices[b]. q and k may be turned by rotary
 * positions first (gdn_rotary.h): rotary_dim channels of each head, with positions[b]. */
typedef struct gdn_linear_step_args {
    int32_t B;                    /* request rows */
    int32_t H, HV;                /* q/k heads, value heads (a multiple of H) */
    int32_t K;                    /* 16, 32, 64 or 128 */
    int32_t V;                    /* 1 .. 1024 */
    int32_t num_slots;
    int32_t in_dtype;             /* gdn_dtype of q, k, v */
    int32_t out_dtype;            /* gdn_dtype of out */
    int32_t state_dtype;          /* gdn_dtype of state; bf16: computed in fp32, rounded to nearest even when
                                     stored; out comes from the unrounded state */
    const void *q;                /* q[b,h,:] at q + b q_stride + h q_head_stride; k and v alike */
    int64_t q_stride, q_head_stride;
    const void *k;
    int64_t k_stride, k_head_stride;
    const void *v;
    int64_t v_stride, v_head_stride;
    const float *g;               /* g[b,hv] at g + b g_stride + hv; g_stride 0: one per head */
    int64_t g_stride;
    float scale;                  /* 0 selects K^-1/2 */
    int32_t rotary_dim;           /* 0: q and k as given; else even, at most K */
    int32_t interleaved;          /* pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2) */
    const int32_t *positions;     /* [B] */
    const double *frequencies;    /* [rotary_dim / 2] radians a position */
    float magnitude;              /* factor of the turned channels; 0 selects 1 */
    void *state;                  /* [num_slots, HV, V, K], 16-byte aligned, in place */
    void *out;                    /* [B, HV, V] dense */
    int32_t *err_flags;
} gdn_linear_step_args;

/* Bytes of workspace that a call with these sizes needs; uniform: non-zero when cu_seqlens is NULL. 0 for
 * sizes that the calls refuse. It goes by how the sequences are cut: fewer tokens or sequences may need more. */
size_t gdn_linear_workspace_bytes(int32_t T, int32_t S, int32_t H, int32_t HV, int32_t K, int32_t V, int32_t in_dtype,
                                  int32_t uniform, int32_t backward);

/*
 * gdn_linear_attention -- outputs and final states. Returns GDN_OK, GDN_ERR_NULL (a missing pointer, or no
 * workspace where one is needed), GDN_ERR_SHAPE (sizes out of range, T not a multiple of S without cu_seqlens,
 * a stride that makes heads or rows of an output overlap, a workspace that is too small), GDN_ERR_DTYPE,
 * GDN_ERR_ALIGN (a pointer not aligned to its element, a state buffer or the workspace not to 16 bytes) or
 * GDN_ERR_LAUNCH. Any row and head strides are accepted; bf16 rows that are 16-byte aligned (pointers,
 * strides and head sizes) are read faster, and where V is not a multiple of 8 the workspace takes a copy of
 * the others. Outputs may not overlap inputs, one another or the workspace, but for final_state on
 * initial_state (not checked).
 */
int gdn_linear_attention(const gdn_linear_args *args, gdn_stream_t stream);

/* gdn_linear_attention_backward -- its gradients; the same status codes, and GDN_ERR_ARG for
 * d_initial_state over d_final_state or initial_state. Recomputes the states from the inputs: nothing of
 * the forward call has to be kept. Sums are taken in a fixed order. */
int gdn_linear_attention_backward(const gdn_linear_grad_args *args, gdn_stream_t stream);

/* gdn_linear_attention_step -- one token of each request row; cache_indices (int32 [B] on the device) may be
 * NULL: row b on slot b. A row whose index is pad_slot_id is skipped (state untouched, out zeroed), one whose
 * index is outside [0, num_slots) as well, and raises GDN_DEVERR_BAD_INDEX. Two rows may not name one slot. */
int gdn_linear_attention_step(const gdn_linear_step_args *args, const int32_t *cache_indices, int32_t pad_slot_id,
                              gdn_stream_t stream);

/*
 * gdn_linear_set_wait_limit -- test hook, not for production use: sets, for the whole process, the number of SM clock cycles
 * after which a wait of the bf16 sequences' kernel gives up; 0 restores the default (2^30 cycles, about half a second).
 * With a limit below a copy's latency a test can make the waits run out and check that the call returns normally, reports
 * GDN_DEVERR_TIMEOUT and leaves NaN. The waits that let copies and MMAs in flight finish keep the default limit.
 * Returns the previous setting. Launches nothing.
 */
int64_t gdn_linear_set_wait_limit(int64_t cycles);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LINEAR_H */
