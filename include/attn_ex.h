/*
 * attn_ex.h -- C ABI of the attention of attn.h (libattn.so) with what a model may put between
 * the scores and the softmax, and of masks that let a prefix be seen as a whole.
 *
 * Semantics. As in attn.h, with i and j positions in the sequence:
 *     s_ij = scale * sum_d q_id k_jd
 *     s_ij = cap * tanh(s_ij / cap)            where cap is not 0
 *     s_ij = s_ij - slopes[h] * |i - j|        where slopes are given, h the query head
 * and query i, of a sequence that holds m tokens, sees the keys of the positions j < m with
 *     j <= i  or  j < prefix                   where prefix lengths are given
 * so that the first `prefix` tokens of a sequence (an image, a question) see each other and the
 * others are causal. A query at a negative position sees no key, whatever the prefix. The
 * prefixes are part of a plan; cap and slopes are the same in a forward and its backward. lse
 * belongs to the scores as the softmax sees them. tanh is formed in fp32 within 2^-22 of its value
 * (for each fp32 argument on gfx950, where all were tried), distances are exact up to 2^24 and rounded
 * to 24 bits beyond; the backward has
 *     dS_ij = P_ij (dP_ij - D_i) (1 - tanh(..)^2)
 * and no gradient of slopes; D_i is formed as sum_j P_ij dP_ij, and for dq up to D = 64 dS enters the product
 * in two parts of the storage type (one past 65504 in f16 overflows as in attn.h). Scores that are
 * infinite are capped like others. Precision, layouts,
 * limits, ownership, threading and errors are those of attn.h. With cap 0 and without slopes the
 * calls are those of attn.h, and so are their results.
 */
#ifndef ATTN_EX_H
#define ATTN_EX_H

#include <stdint.h>

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* attn_plan with prefixes. The plan's size is attn_plan_ints, and any attn_fwd, attn_bwd or call
 * below takes it.
 *  prefix_lens  device int32[num_seqs] or NULL: every row of sequence s sees its first
 *               prefix_lens[s] keys (clamped to what the sequence holds) */
int32_t attn_plan_ex(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* seqused,
                     const int32_t* prefix_lens, int64_t T, int32_t Hq, int32_t Hkv, int32_t* plan,
                     int64_t plan_ints, void* stream);

/* attn_fwd with changed scores.
 *  cap     0 for none; else positive, cap log2 e below 1e30 and scale / cap within 1e-30 .. 1e30
 *  slopes  device float[Hq] or NULL, finite */
int32_t attn_fwd_ex(const void* q, const void* k, const void* v, void* out, float* lse, int64_t T,
                    int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride, int64_t k_stride,
                    int64_t v_stride, int64_t out_stride, const int32_t* plan, int32_t num_seqs,
                    double scale, double cap, const float* slopes, int32_t dtype, int32_t fill,
                    void* stream);

/* Floats of attn_bwd_ex's scratch, or -1: those of attn_bwd, and with slopes (biased not 0) 8 bytes
 * more for each row and query head. */
int64_t attn_bwd_ex_scratch_floats(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv, int32_t D,
                                   int32_t biased);

/* Its gradients, as attn_bwd. */
int32_t attn_bwd_ex(const void* dout, const void* q, const void* k, const void* v, const void* out,
                    const float* lse, float* scratch, void* dq, void* dk, void* dv, int64_t T,
                    int32_t Hq, int32_t Hkv, int32_t D, int64_t dout_stride, int64_t q_stride,
                    int64_t k_stride, int64_t v_stride, int64_t out_stride, int64_t dq_stride,
                    int64_t dk_stride, int64_t dv_stride, const int32_t* plan, int32_t num_seqs,
                    double scale, double cap, const float* slopes, int32_t dtype, int32_t fill,
                    void* stream);

/* paged_plan with prefixes (size: paged_plan_ints): every new token at a position sees the first
 * prefix_lens[s] of the keys that sequence s holds, those of this call among them. */
int32_t paged_plan_ex(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* kv_lens,
                      const int32_t* prefix_lens, int64_t T, int32_t Hq, int32_t Hkv, int32_t* plan,
                      int64_t plan_ints, void* stream);

/* attn_paged with changed scores; its workspace is paged_workspace_floats. */
int32_t attn_paged_ex(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                      float* workspace, int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride,
                      int64_t out_stride, int32_t num_pages, int32_t page_size, int64_t page_stride,
                      int64_t slot_stride, int64_t head_stride, const int32_t* block_table,
                      int32_t max_pages, int64_t table_stride, const int32_t* plan, int32_t num_seqs,
                      double scale, double cap, const float* slopes, int32_t dtype, int32_t fill,
                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_EX_H */
