/*
 * m3_rotary.h -- C ABI of the norm of queries and keys for each head with the
 * position rotation in the same pass (AMD MI355X / gfx950), and its gradients.
 *
 * For every row x (dim channels of one token and head of q or k):
 *     n = w x / sqrt(mean(x^2) + eps)        (norm; w = 1 without a weight)
 *     angle_i = sum_a position[a][token] * inv_freq[a][i],   i < rot / 2
 *     (n_u, n_v) -> (n_u cos - n_v sin, n_u sin + n_v cos)   for pair i
 * where pair i is the channels (2i, 2i + 1), or (i, i + rot / 2) with halves,
 * and channels from rot on are not turned.  Several axes (time, height, width)
 * are rows of inv_freq: an axis has its frequencies at the pairs it turns and
 * zeros elsewhere.  Arithmetic is fp32 with angles in fp64, taken modulo a
 * turn; every output is rounded once.  mean(x^2) + eps has to be a normal fp32
 * number: eps may be 0, but then a row of zeros gives NaN, and so does the
 * gradient of its weight.
 *
 * Rows and strides are those of m3_linear.h (m3_rows_t: channels contiguous,
 * 16-byte aligned rows), and ownership, streams and errors those of m3_ssm.h.
 * An output's rows may be its own input's rows (same pointer and strides);
 * outputs overlap nothing else (M3_ERR_INVALID_ARGUMENT where one starts at
 * another operand's address).
 */
#ifndef M3_ROTARY_H
#define M3_ROTARY_H

#include "m3_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Supported: dim a multiple of 8 from 8 to 256; rot a multiple of 8 from 8 to
 * dim; axes 1 to 4; tokens >= 0; q_heads >= 1, k_heads >= 0 (0: no keys, their
 * pointers are not read).  Other sizes are M3_ERR_UNSUPPORTED, and so are more
 * rows than one launch has threads for: tokens (ceil(q_heads / n) +
 * ceil(k_heads / n)) up to 2^26 - 5, with 256 / n the power of two that dim / 8
 * lanes fit in. */
typedef struct {
    int64_t tokens;
    int32_t q_heads, k_heads;
    int32_t dim, rot;
    int32_t axes;
    int32_t io_dtype;   /* m3_dtype_t of the rows                          */
    int32_t pos_int64;  /* positions are int64 (else int32)                */
    int32_t halves;     /* pairs (i, i + rot/2) instead of (2i, 2i + 1)    */
    int32_t norm;       /* RMS norm before the rotation                    */
    float eps;          /* inside the square root                          */
} m3_rotary_shape_t;

/* positions [axes][tokens], inv_freq [axes][rot / 2] fp32; q_weight and
 * k_weight [dim] fp32 or NULL (they need norm).  inv_freq and the weights start
 * at multiples of 16 bytes. */
m3_status_t m3_norm_rotate(const m3_rotary_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                           const void *positions, const float *inv_freq, const float *q_weight,
                           const float *k_weight, const m3_rows_t *q_out, const m3_rows_t *k_out,
                           hipStream_t stream);

/* Bytes of device workspace of the gradients (0: invalid or unsupported): one
 * partial sum of each weight's gradient per workgroup. */
size_t m3_norm_rotate_backward_workspace_bytes(const m3_rotary_shape_t *shape);

/* Gradients of sum(gq * q') + sum(gk * k') for the outputs q', k' of
 * m3_norm_rotate.  dq, dk: rows like q and k (dq may be gq's rows, dk gk's).
 * dq_weight, dk_weight: [dim] fp32, summed over tokens and heads in an order
 * that depends on the sizes only; given exactly where the weight is. */
m3_status_t m3_norm_rotate_backward(const m3_rotary_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                                    const void *positions, const float *inv_freq, const float *q_weight,
                                    const float *k_weight, const m3_rows_t *gq, const m3_rows_t *gk,
                                    const m3_rows_t *dq, const m3_rows_t *dk, float *dq_weight,
                                    float *dk_weight, void *workspace, size_t workspace_bytes,
                                    hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* M3_ROTARY_H */
