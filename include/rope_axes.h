/*
 * rope_axes.h -- C ABI of the rotary embedding by positions with several axes (time, height and
 * width of images and video beside text), alone and on the way into a paged cache (libattn.so).
 *
 * Semantics. A token has a position p_a on each of 1 .. 4 axes. Frequency j < D/2 belongs to one
 * axis a(j) and has the inverse frequency w_j, both by `layout` and the sections n_0, n_1, ..
 * (their sum is D/2, n_a the frequencies of axis a):
 *   ROPE_AXES_SECTIONS     the first n_0 frequencies of one ladder are axis 0's, the next n_1 axis
 *                          1's and so on; w_j = theta^(-2j/D)
 *   ROPE_AXES_INTERLEAVED  the same ladder, the axes in turn: with A axes, frequency j is axis
 *                          (j mod A)'s while j < A n_(j mod A), and else axis 0's. Every axis a > 0
 *                          must find its turns: A (n_a - 1) + a < D/2 where n_a > 0
 *   ROPE_AXES_SEPARATE     sections as in the first, each with a ladder of its own: the i-th
 *                          frequency of axis a is theta^(-i/n_a)
 * The rotation of element pairs (j, j + D/2) is that of rope_qk.h, value for value, with the angle
 * fp32(p_a(j) / pos_scale) * w_j: w_j rounded once to fp32, one fp32 product, cos and sin correctly
 * rounded, each output within 2 fp32 ulps before it is rounded once. Equal positions on all axes
 * give rope_qk's results bit for bit (sections, interleaved). A token with a negative position on
 * any axis is not rotated.
 *
 * Ownership, threading and errors are those of rope_qk.h.
 */
#ifndef ROPE_AXES_H
#define ROPE_AXES_H

#include <stdint.h>

#include "rope_qk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ROPE_AXES_MOST 4

typedef enum rope_axes_layout {
  ROPE_AXES_SECTIONS = 0,
  ROPE_AXES_INTERLEAVED = 1,
  ROPE_AXES_SEPARATE = 2
} rope_axes_layout;

/* Rotates queries and keys, into other tensors or in place.
 *  q, q_out   device [T][Hq][D], the heads of a token contiguous; q_out may be q (then with one
 *             token stride), else it must not overlap an input. Both NULL with Hq 0
 *  k, k_out   the same, [T][Hkv][D]
 *  T          0 .. 33554431 times 16, or times 4096 / D (rounded down) for D above 256: that many
 *             workgroups of so many tokens are a launch; Hq, Hkv 0 .. 4096, not both 0
 *  D          even, 2 .. 512; dtype any rope_dtype; any strides and alignment (0: heads * D; the
 *             widest access that they allow is used)
 *  position_ids   device int32: axis a of token t at a * ids_stride + t
 *  sections   host int32[axes], none negative
 *  direction  +1 forward, -1 the transposed rotation (gradients)
 *  theta, pos_scale  as in rope_qk_apply_ex */
int32_t rope_qk_apply_axes(const void* q, void* q_out, const void* k, void* k_out, int64_t T, int32_t Hq,
                           int32_t Hkv, int32_t D, int64_t q_stride, int64_t q_out_stride,
                           int64_t k_stride, int64_t k_out_stride, const int32_t* position_ids,
                           int64_t ids_stride, const int32_t* sections, int32_t axes, int32_t layout,
                           double theta, double pos_scale, int32_t dtype, int32_t direction,
                           void* stream);

/* Writes new keys and values into the cache rows that a slot map names, the keys rotated, and the
 * rotated queries to q_out (as kv_append, which finds the rows by a block table). One launch.
 *  q, q_out, k, v, k_cache, v_cache, strides and sizes as in kv_append of attn.h (T as above)
 *  slots      device int64[T]: token t goes to slot slots[t] % page_size of page slots[t] /
 *             page_size; a number outside 0 .. num_pages * page_size - 1 (-1) is no slot, and its
 *             token is not written. No two tokens may name one slot: it would hold parts of either
 *  position_ids, sections, axes, layout  as above. axes 1 with one section of D/2 is the ordinary
 *             rotation. A token with a negative position is written as it is */
int32_t kv_append_slots(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                        void* v_cache, int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride,
                        int64_t q_out_stride, int64_t k_stride, int64_t v_stride, int32_t num_pages,
                        int32_t page_size, int64_t page_stride, int64_t slot_stride,
                        int64_t head_stride, const int64_t* slots, const int32_t* position_ids,
                        int64_t ids_stride, const int32_t* sections, int32_t axes, int32_t layout,
                        double theta, double pos_scale, int32_t dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_AXES_H */
