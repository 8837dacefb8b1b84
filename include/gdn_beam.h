/*
 * gdn_beam.h -- C ABI of beam search over the decode's recurrent states in libgdn_decode.so;
 * conventions as in gdn_decode.h (device pointers owned by the caller, nothing allocated or
 * synchronised, launches only on `stream`, host-side checks before any CUDA call, negative gdn_status
 * on error). The source pages have no counterpart: a search step is what stands between two decode
 * steps of a model whose states live in a slot pool.
 *
 * One search step after the decode has given every beam's logits:
 *   gdn_beam_select   picks, per batch entry, the best K of beams x vocab continuations
 *   gdn_beam_reorder  gives each chosen continuation a slot that holds its parent's states
 */
#ifndef GDN_BEAM_H
#define GDN_BEAM_H

#include <stddef.h>
#include <stdint.h>

#include "gdn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_BEAM_MAX_BEAMS 32
#define GDN_BEAM_MAX_SELECT 64
#define GDN_BEAM_MAX_POOLS 128

typedef struct gdn_beam_select_args {
    int32_t batch;              /* batch entries, >= 0 */
    int32_t beams;              /* beams of each, 1 .. 32 */
    int32_t vocab;              /* tokens, >= 1 */
    int32_t K;                  /* continuations chosen for each batch entry, 1 .. 64 */
    int32_t logits_dtype;       /* gdn_dtype */
    int32_t num_rows;           /* rows of logits */
    const void *logits;         /* [num_rows, vocab], row stride row_stride (any, >= vocab) */
    int64_t row_stride;
    const int32_t *rows;        /* [batch, beams]: logits row of each beam (states that are decoded in slot
                                   order have their logits there), or NULL: row batch_entry * beams + beam */
    const float *scores;        /* [batch, beams]: cumulative log-probability; -inf (or NaN): no beam */
    const uint8_t *finished;    /* [batch, beams] or NULL: non-zero: the beam has ended; its one candidate is
                                   itself, with its score and eos_token, and its logits are not read */
    int32_t eos_token;          /* 0 .. vocab - 1 when finished or out_finished is given */
    float *out_scores;          /* [batch, K], best first; -inf where there is no candidate left */
    int32_t *out_parents;       /* [batch, K]: the beam continued; -1 where there is none */
    int32_t *out_tokens;        /* [batch, K]: the token; -1 where there is none */
    uint8_t *out_finished;      /* [batch, K] or NULL: 1 where the token is eos_token, else 0 */
    void *workspace;            /* gdn_beam_select_workspace_bytes bytes, 16-byte aligned */
    size_t workspace_bytes;
    int32_t *err_flags;         /* optional device word: GDN_DEVERR_BAD_INDEX for a row outside
                                   [0, num_rows) of a beam whose logits are read (one that lives and has
                                   not ended); that beam then has no candidates */
} gdn_beam_select_args;

/* Workspace bytes for these sizes; 0 for sizes that the call refuses. */
size_t gdn_beam_select_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t K);

/*
 * gdn_beam_select -- per batch entry the K best candidates (beam, token) by
 *     scores[beam] + logits[row, token] - log(sum_v exp(logits[row, v]))
 * in descending order; equal ones by the lower beam, within a beam by the larger logit, then the
 * lower token. A logit of -inf or NaN forbids its token; a row of such logits gives no candidate.
 * (+inf logits share their row's whole probability.) One pass over the logits in two launches; the
 * sums run in fp32 over short ranges and in fp64 over those, and scores are compared in fp64 and
 * rounded once. The result does not depend on timing.
 * The outputs may not overlap one another or the workspace, nor, with more than one batch entry, rows,
 * scores or finished, except that with K = beams an output may be one of those three itself (in place;
 * the type's size being the same).
 * Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_ALIGN, GDN_ERR_ARG (eos_token
 * outside the vocabulary where it is used, or an output over the workspace or an input as above) or
 * GDN_ERR_LAUNCH.
 */
int gdn_beam_select(const gdn_beam_select_args *args, gdn_stream_t stream);

/* One pool of states: slot s starts at base + s * slot_stride bytes and holds slot_bytes bytes. */
typedef struct gdn_beam_pool {
    void *base;
    int64_t slot_stride;        /* bytes, >= slot_bytes */
    int64_t slot_bytes;         /* bytes, >= 0 */
} gdn_beam_pool;

typedef struct gdn_beam_reorder_args {
    int32_t batch;              /* batch entries, >= 0 */
    int32_t beams;              /* beams of each, 1 .. 32 */
    int32_t num_slots;          /* slots of every pool */
    int32_t num_pools;          /* 0 .. 128 */
    const gdn_beam_pool *pools; /* HOST array of num_pools entries, read during the call */
    const int32_t *slots;       /* [batch, beams]: each beam's slot, all different */
    const int32_t *parents;     /* [batch, beams]: the beam that each new beam continues; outside
                                   [0, beams): the new beam continues none, and only gets a slot */
    int32_t *new_slots;         /* [batch, beams]: each new beam's slot; may not overlap slots or parents */
    int32_t *err_flags;         /* optional device word: GDN_DEVERR_BAD_INDEX for a copy from or to a
                                   slot outside [0, num_slots); the copy is skipped */
} gdn_beam_reorder_args;

/*
 * gdn_beam_reorder -- new_slots and the copies they need, in place in the pools. A parent's first
 * new beam (the lowest) takes over its slot and nothing is copied; each further one, and each new beam
 * without a parent, takes the slot of a beam that nobody continues, both in ascending order, and the
 * parent's states are copied there (not for a new beam without a parent). No slot is both read and
 * written. The next decode step reads its slots from new_slots (cache_indices of
 * gdn_decode_step_indexed). One launch for up to 2048 beams. A chained decode call may not directly
 * follow this one on the stream (it writes states: the first layer's call has to be an ordinary one).
 * Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_ALIGN, GDN_ERR_ARG (new_slots overlaps slots or
 * parents) or GDN_ERR_LAUNCH.
 */
int gdn_beam_reorder(const gdn_beam_reorder_args *args, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_BEAM_H */
