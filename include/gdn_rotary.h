/*
 * gdn_rotary.h -- C ABI of the rotary positions of the softmax-attention layers (B200, sm_100a).
 *
 * The hybrid model's softmax layers (include/gdn_attention.h) take queries and keys whose
 * positions are written into them as rotations: pair i of a head, (x1, x2), at position p becomes
 *     y1 = a (x1 cos t - x2 sin t),   y2 = a (x1 sin t + x2 cos t),   t = p f_i,
 * for the first rot_dim elements of the head; the others pass unchanged.  Pair i is
 * (x[2i], x[2i+1]) in the interleaved layout and (x[i], x[i + rot_dim/2]) in the half layout.
 * The rotation is linear, so its backward is its transpose: the rotation by -t, scaled by a.
 *
 * Frequencies.  f_i = base^(-2i/rot_dim), then by `scaling`:
 *   GDN_ROPE_NONE    f_i as it is
 *   GDN_ROPE_LINEAR  f_i / factor (positions interpolated)
 *   GDN_ROPE_NTK     base replaced by base * factor^(rot_dim / (rot_dim - 2)) (rot_dim >= 4)
 *   GDN_ROPE_RAMP    by parts: with r_i = original_len f_i / (2 pi), the turns that pair i makes over
 *                    the original context, and w = clamp((r_i - beta_slow) / (beta_fast - beta_slow),
 *                    0, 1): f_i (w + (1 - w) / factor); fast pairs keep f_i, slow ones are interpolated
 * A table stores each frequency as a fraction of a turn per position in 64-bit fixed point,
 * round(f_i / (2 pi) 2^64) mod 2^64.  The angle of position p is then p times that, modulo 2^64: whole
 * turns drop out exactly, and that angle is off by less than 2^-30 turns at every int32 position (a
 * table entry by less than 2^-62 turns): far positions lose nothing.  For the sine and cosine the angle,
 * less than half a turn, is rounded to fp32: another 2^-26 turns (9.4e-8 radians) at most.
 *
 * Layouts: rows of heads with the elements of a head contiguous; row and head strides in
 * ELEMENTS are the caller's (so q and k may be slices of one projection's output).
 *   q, q_out     [R, H, d]      k, k_out   [R, H_kv, d]      dtype = desc->dtype (bf16 or fp32)
 *   positions    [T] int32 (device), R a multiple of T: row r stands at positions[r % T] (the views of
 *                the noisy stream share their positions); any int32 value is valid
 *   turns        [rot_dim / 2] uint64 (device), as gdn_rotary_frequencies wrote them
 * q_out may be q (same strides: in place), else must not overlap an input or the other output; the same
 * for k.  Tensors whose extents overlap count as apart when they have one row stride and their rows
 * alternate (slices of one projection's output); any other overlap is refused.
 * Arithmetic is fp32, rounded once to the dtype.
 *
 * All calls validate on the host (no partial launch on error), then enqueue on `stream` and
 * return; nothing is allocated, nothing synchronises.  Errors: GDN_ERR_INVALID_ARG (sizes, strides,
 * NULL, overlaps), GDN_ERR_ALIGNMENT (positions not 4-byte, turns not 8-byte, or a tensor not aligned to its
 * element), GDN_ERR_UNSUPPORTED (head_dim > 256), GDN_ERR_CUDA (launch failure).  Tensors whose
 * bases and strides are 16-byte multiples, with rot_dim a multiple of 32 bytes and head_dim of
 * 16, move in 16-byte vectors; all others take a slower path, element by element.
 */
#ifndef GDN_ROTARY_H
#define GDN_ROTARY_H

#include "gdn_dual.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GDN_ROPE_NONE = 0, GDN_ROPE_LINEAR = 1, GDN_ROPE_NTK = 2, GDN_ROPE_RAMP = 3 } gdn_rotary_scaling;

/* Host only: the frequencies of a table into turns_host [rot_dim / 2].  rot_dim even, 0 .. 256
 * (0: nothing is rotated); base > 0 and finite; factor >= 1; GDN_ROPE_RAMP also needs
 * original_len > 0 and beta_fast > beta_slow >= 0 (ignored otherwise). */
gdn_status gdn_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor,
                                  double original_len, double beta_fast, double beta_slow,
                                  uint64_t *turns_host);

/* num_rows R >= 0; num_positions T >= 1 dividing R; num_heads H >= 0 and num_kv_heads H_kv >= 0, not
 * both 0 (with 0 heads the tensor may be NULL); head_dim d in [1, 256]; rot_dim even, 0 .. d;
 * interleaved 0 or 1; dtype a gdn_dtype; scale a, finite; strides in elements, >= 0 (an output's
 * rows and heads must not overlap one another); reserved 0. */
typedef struct {
    int32_t num_rows;
    int32_t num_positions;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t rot_dim;
    int32_t interleaved;
    int32_t dtype;
    float scale;
    int32_t reserved;
    int64_t q_row_stride, q_head_stride;
    int64_t k_row_stride, k_head_stride;
    int64_t q_out_row_stride, q_out_head_stride;
    int64_t k_out_row_stride, k_out_head_stride;
} gdn_rotary_desc;

/* q_out, k_out = the rotated q, k. */
gdn_status gdn_rotary_forward(const gdn_rotary_desc *desc, const uint64_t *turns, const int32_t *positions,
                              const void *q, const void *k, void *q_out, void *k_out, gdn_stream_t stream);

/* Given the gradients of q_out and k_out (in q, k), the gradients of q and k (in q_out, k_out). */
gdn_status gdn_rotary_backward(const gdn_rotary_desc *desc, const uint64_t *turns, const int32_t *positions,
                               const void *q, const void *k, void *q_out, void *k_out, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ROTARY_H */
