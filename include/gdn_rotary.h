/*
 * gdn_rotary.h -- C ABI of rotary positions in libgdn_decode.so; conventions as in gdn_decode.h. They turn
 * q and k before linear attention (gdn_linear.h), whose single-token step can also turn them itself.
 *
 * The operation: the first rotary_dim channels of every head are pairs (a_i, b_i), i < rotary_dim / 2, at
 * channels (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved. With the angle
 * phi = positions[t] frequencies[i]:
 *     a_i' = magnitude (a_i cos phi - b_i sin phi)     b_i' = magnitude (b_i cos phi + a_i sin phi)
 * The other channels are copied. inverse turns by -phi: with the same magnitude that is the transpose, so
 * the gradients of the inputs are the inverse call on the gradients of the outputs. Frequencies are fp64
 * radians a position, so any scaling for long contexts is a choice of that table; angles are taken
 * modulo a turn in 64-bit fixed point, whose error does not grow with the position, and rounded to fp32: within
 * 1e-7 radians of the exact product, at position 10^6 too, where an fp32 product would be off by 0.03.
 */
#ifndef GDN_ROTARY_H
#define GDN_ROTARY_H

#include <stdint.h>

#include "gdn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdn_rotary_args {
    int32_t T;                    /* token rows, >= 0 */
    int32_t H;                    /* heads of q, >= 1 */
    int32_t HK;                   /* heads of k; 0: no k */
    int32_t D;                    /* channels of a head, 2 .. 1024 */
    int32_t rotary_dim;           /* channels turned: even, 2 .. D */
    int32_t interleaved;
    int32_t inverse;
    int32_t dtype;                /* gdn_dtype of q, k and their outputs; arithmetic is fp32 */
    float magnitude;              /* 0 selects 1 */
    const int32_t *positions;     /* [T] */
    const double *frequencies;    /* [rotary_dim / 2], finite */
    const void *q;                /* q[t,h,:] at q + t q_stride + h q_head_stride */
    int64_t q_stride, q_head_stride;
    void *q_out;                  /* may be q itself with q's strides (in place) */
    int64_t q_out_stride, q_out_head_stride;
    const void *k;
    int64_t k_stride, k_head_stride;
    void *k_out;
    int64_t k_out_stride, k_out_head_stride;
} gdn_rotary_args;

/* gdn_rotary -- turns q and k. Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_ALIGN (a
 * pointer not aligned to its element) or GDN_ERR_LAUNCH. Outputs may not overlap the inputs but for in place, nor
 * one another (not checked). */
int gdn_rotary(const gdn_rotary_args *args, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ROTARY_H */
