/*
 * exact_attention_51_gb300 -- C ABI of the rotary positions.
 *
 * Rotary positions turn the pairs of a query's or key's head by an angle that
 * grows with its position p, so that scores q . k depend on position
 * differences alone:
 *
 *     (y1, y2) = a * (x1 cos t - x2 sin t,  x2 cos t + x1 sin t),   t = p f_i
 *
 * for pair i of the first rot_dim elements of each head; elements from rot_dim
 * on are copied.  Pairs are (x_i, x_{i + rot_dim/2}) (half layout) or
 * (x_{2i}, x_{2i+1}) (interleaved).  f_i is the pair's frequency in radians a
 * position and a the attention factor (1 unless the scaling sets another).
 *
 * Frequencies are passed as phases: u_i = f_i / (2 pi) * 2^64 mod 2^64, the
 * fraction of a turn that a position adds, in units of 2^-64.  p * u_i mod
 * 2^64 is then the exact angle mod one turn: the reduction of the angle of a
 * far position is one integer product, at any int32 position, negative ones
 * among them.  What is left is the fraction's own error times the position: of
 * attn_rope_phases, which computes in fp64, 2^-52 of a turn (2^-35 at position
 * 2^17, 2^-21 at 2^31); of a table rounded to the unit 2^-65.  The angle is cut to
 * 2^-32 of a turn, cos and sin and the rotation are fp32 (the two within 2^-22), and the
 * result is rounded once to the tensor's type.
 *
 * Conventions (status codes, streams, ownership, thread safety) as in
 * include/attn_fwd.h.
 */
#ifndef EXACT_ATTENTION_51_GB300_ATTN_ROPE_H
#define EXACT_ATTENTION_51_GB300_ATTN_ROPE_H

#include <stddef.h>
#include <stdint.h>

#include "attn_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of attn_rope. */
enum attn_rope_dtype { ATTN_ROPE_BF16 = 0, ATTN_ROPE_F16 = 1, ATTN_ROPE_F32 = 2 };

/* Frequency scalings of attn_rope_phases, for rows longer than the trained
 * length L = original_positions by a factor s. */
enum attn_rope_scaling {
  ATTN_ROPE_NONE = 0,   /* f_i = base^(-2i / rot_dim) */
  ATTN_ROPE_LINEAR = 1, /* f_i / s */
  ATTN_ROPE_NTK = 2,    /* base replaced by base * s^(rot_dim / (rot_dim - 2)) */
  ATTN_ROPE_YARN = 3    /* g f_i + (1 - g) f_i / s, g = clamp((L f_i / 2 pi - beta_slow) /
                           (beta_fast - beta_slow), 0, 1); attention factor 0.1 ln s + 1 */
};

/*
 * Fills phases[0 .. rot_dim/2) (host memory) for these frequencies, and
 * *attention_factor (may be NULL) with the scaling's factor on cos and sin; in
 * fp64, each to 2^-52 of a turn.
 *
 *   rot_dim   even, 2..512.          base     finite, > 1.
 *   factor    s: finite, >= 1 (ignored by ATTN_ROPE_NONE).
 *   original_positions, beta_fast, beta_slow: ATTN_ROPE_YARN only; L >= 1,
 *             beta_fast > beta_slow, both finite.
 * ATTN_ROPE_NTK needs rot_dim > 2.  Host-only; anything else is
 * ATTN_ERR_INVALID_ARG and writes nothing.
 */
ATTN_API int attn_rope_phases(uint64_t* phases, float* attention_factor, int rot_dim, double base,
                              int scaling, double factor, int original_positions,
                              double beta_fast, double beta_slow);

/*
 * Rotates x [B, H, N, d] into y.
 *
 *   x, y       device pointers of `dtype`, elements of a head adjacent, other
 *              dims at the given strides (in elements: batch, head, position),
 *              so that [B, H, N, d], [B, N, H, d] and slices of a fused
 *              projection are all read in place.  x's strides are >= 0 (0
 *              broadcasts); y's must give every element a place of its own.
 *              y may be x with the same strides (in place); any other overlap
 *              of the two's extents is ATTN_ERR_ALIAS.
 *   d          even, 2..512.         rot_dim  even, 2..d.
 *   positions  device int32; row b, n is at position
 *              positions[b * position_stride_b + n] (position_stride_b 0: the
 *              same for the whole batch), or, where NULL, position0 + n (within int32).
 *   phases     device uint64 [rot_dim / 2], 8-byte aligned.
 *   attention_factor  finite.
 *
 * Pointers are aligned to their element; rows of whole 16-byte chunks
 * (base, strides and d) run the vector paths.
 * Enqueues one kernel.
 */
ATTN_API int attn_rope(const void* x, void* y, int dtype, int B, int H, int N, int d,
                       int64_t x_stride_b, int64_t x_stride_h, int64_t x_stride_n,
                       int64_t y_stride_b, int64_t y_stride_h, int64_t y_stride_n,
                       const int32_t* positions, int64_t position_stride_b, int position0,
                       const uint64_t* phases, int rot_dim, int interleaved,
                       float attention_factor, void* stream);

/*
 * Gradient of attn_rope: dx from dy, both [B, H, N, d].  The rotation is
 * linear in x, so this is its transpose, the turn by -t times the same factor;
 * arguments as attn_rope with dy for x and dx for y.  An x that was broadcast
 * (stride 0) takes the sum of its dx, which is the caller's.
 */
ATTN_API int attn_rope_bwd(const void* dy, void* dx, int dtype, int B, int H, int N, int d,
                           int64_t dy_stride_b, int64_t dy_stride_h, int64_t dy_stride_n,
                           int64_t dx_stride_b, int64_t dx_stride_h, int64_t dx_stride_n,
                           const int32_t* positions, int64_t position_stride_b, int position0,
                           const uint64_t* phases, int rot_dim, int interleaved,
                           float attention_factor, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTENTION_51_GB300_ATTN_ROPE_H */
