/*
 * attn.h -- C ABI of the attention kernels for MI355X (gfx950): causal attention over
 * packed sequences, forward and backward, and attention over a paged key/value cache with
 * the append that fills it (libattn.so, which loads librope_qk.so beside it).
 *
 * The attention is what stands between the rotation of rope_qk.h and the output projection:
 * packed samples must not see each other ("Packing non contamine" on the Unsloth page cited
 * in rope_qk.h), so a token attends to the tokens of its own sequence up to itself.
 *
 * Semantics. Query head h reads key/value head h / (Hq / Hkv). Of a sequence that holds m
 * tokens, the n newest of them are queries (packed attention: n = m); query i sits at
 * position m - n + i and sees the keys of the positions 0 .. m - n + i:
 *     s_ij = scale * sum_d q_id k_jd,  lse_i = ln sum_j exp(s_ij),
 *     out_i = sum_j exp(s_ij - lse_i) v_j
 * A query that sees no key (a negative position) gets out = 0 and lse = -inf. Keys that a
 * query does not see have no influence on its outputs, whatever they hold
 * (infinities and NaN among it), and queries that do not see a key none on its gradients.
 * Products are formed on the matrix cores from the storage type into fp32; the softmax and
 * its sums are fp32; the weights (and dS, backward) are rounded to the storage type before the
 * second product, and outputs once at the end. In f16 a dS past 65504 overflows there. Scores
 * of any size, in any mixture, are weighed forward as their fp32 values differ, as long as fp32
 * holds s_ij log2 e; the backward forms the weights again from lse, with a relative error of
 * |lse| 2^-22. Results do not depend on the order of execution: no atomics on them.
 *
 * Layouts. Rows are [token][head][D], the heads of a token contiguous; every tensor has a
 * token stride in elements (0 = heads * D, else at least that: tokens do not overlap), so q, k
 * and v may be views of one fused projection. D is a multiple of 8, 8 .. 256 (backward: 8 ..
 * 128). Data pointers are 16-byte aligned and strides multiples of 8 elements, below 2^24.
 * dtype is ROPE_BF16 or ROPE_F16 (the append takes ROPE_F32 too). lse is float [T][Hq].
 * A launch has at most 8388607 workgroups: attention refuses (ROPE_EINVAL) what needs more,
 * T * Hq / 128 + (2 num_seqs + 3) Hkv of them.
 *
 * Ownership, threading and errors are those of rope_qk.h: the caller owns every buffer, the
 * library allocates nothing, keeps no state, never synchronizes, and only enqueues work on
 * `stream`; arguments are checked on the host before any HIP call (rope_status codes).
 * An output must not overlap an input or another output, except where stated.
 */
#ifndef ATTN_H
#define ATTN_H

#include <stdint.h>

#include "rope_qk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_ROW_TILE 128   /* packed query rows (token-major, the heads of a group minor) */
#define ATTN_KEY_TILE 128   /* keys of a work item of the dK/dV pass */
#define ATTN_PLAN_HEADER 16 /* int32 words before a plan's items */

/* ---- packed sequences -------------------------------------------------------------- */

/* int32 words of a plan for num_seqs sequences in T rows, or -1 for bad arguments. */
int64_t attn_plan_ints(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv);

/* Writes the plan of a packed batch: the list of work items, the longest first. One small
 * launch per batch, which serves every layer, forward and backward.
 *  cu_seqlens  device int32[num_seqs + 1]; sequence s is the rows cu_seqlens[s] ..
 *              cu_seqlens[s+1] - 1. Entries are read as clamped to [0, T] and to be
 *              non-decreasing (a smaller entry counts as the largest before it), so any
 *              contents are memory-safe.
 *  seqused     device int32[num_seqs] or NULL: sequence s holds its first seqused[s] rows
 *              only (padded layouts); the others belong to no sequence
 *  T           rows, 0 .. 2^31 - 1, with T * Hq / Hkv below 2^31
 *  Hq, Hkv     head counts, 1 .. 4096, Hq a multiple of Hkv
 *  plan        device int32[plan_ints], 16-byte aligned, written; plan_ints at least
 *              attn_plan_ints(T, num_seqs, Hq, Hkv) */
int32_t attn_plan(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* seqused, int64_t T,
                  int32_t Hq, int32_t Hkv, int32_t* plan, int64_t plan_ints, void* stream);

/* Causal attention of packed sequences.
 *  q, k, v     device [T][Hq][D], [T][Hkv][D], [T][Hkv][D], read
 *  out, lse    device [T][Hq][D] and float [T][Hq], written
 *  plan        written by attn_plan for the same T, num_seqs, Hq and Hkv. Where it was made
 *              for others, or by paged_plan, memory stays safe and nothing is written.
 *  scale       positive, and times log2 e within 1e-37 .. 3e38; usually D^-0.5
 *  fill        rows of no sequence: 0 leaves out and lse as they are, 1 writes out = 0 and
 *              lse = -inf */
int32_t attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int64_t T,
                 int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride, int64_t k_stride,
                 int64_t v_stride, int64_t out_stride, const int32_t* plan, int32_t num_seqs,
                 double scale, int32_t dtype, int32_t fill, void* stream);

/* Floats of attn_bwd's scratch, or -1 for bad arguments: 0.5 MB of partial sums for each of D
 * columns, twice that for D up to 64 (67 MB at D = 64 and 128), whatever T is, and 8 bytes a row
 * and query head. */
int64_t attn_bwd_scratch_floats(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv, int32_t D);

/* Its gradients, from dout and what attn_fwd read and wrote:
 *     dP_ij = dout_i . v_j,  D_i = dout_i . out_i,  dS_ij = P_ij (dP_ij - D_i),
 *     dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dout_i
 * with i over the queries of every head that reads key/value head j's head.
 *  scratch     device float[attn_bwd_scratch_floats(...)], 16-byte aligned: calls that may
 *              run at the same time need one each
 *  dq, dk, dv  device, written; token strides as the others'
 *  fill        as in attn_fwd: 1 writes zeros to the gradients of rows of no sequence
 * D is at most 128. */
int32_t attn_bwd(const void* dout, const void* q, const void* k, const void* v, const void* out,
                 const float* lse, float* scratch, void* dq, void* dk, void* dv, int64_t T,
                 int32_t Hq, int32_t Hkv, int32_t D, int64_t dout_stride, int64_t q_stride,
                 int64_t k_stride, int64_t v_stride, int64_t out_stride, int64_t dq_stride,
                 int64_t dk_stride, int64_t dv_stride, const int32_t* plan, int32_t num_seqs,
                 double scale, int32_t dtype, int32_t fill, void* stream);

/* ---- paged cache ------------------------------------------------------------------- *
 *
 * A cache is two tensors [num_pages][page_size][Hkv][D] (keys and values) of one layout:
 * page_stride, slot_stride and head_stride in elements, the D elements of a row contiguous,
 * so pages may hold their heads in either order or be parts of a larger allocation. Position
 * p of sequence s lies in page block_table[s * table_stride + p / page_size], slot p %
 * page_size. kv_lens[s] counts the tokens that sequence s holds, the new ones included; the
 * new tokens are rows cu_seqlens[s] .. cu_seqlens[s+1] - 1 of q, k and v, so token i of them
 * is at position kv_lens[s] - n + i. Entries of cu_seqlens count as clamped to [0, T], and are
 * non-decreasing (where they are not, memory stays safe, but append and plan may differ in whose
 * token it is). A page number outside 0 .. num_pages - 1 is no page. */

/* Writes the new tokens' keys and values into the cache, the keys rotated as rope_qk_fwd
 * rotates them at their position, and the new queries, rotated, to q_out. One launch.
 *  q, q_out    device [T][Hq][D]; both NULL (or Hq 0): keys and values only. q_out may be q.
 *              Rows at no position (of no sequence, or at a negative one) are copied as
 *              they are.
 *  k, v        device [T][Hkv][D], read; tokens at no position, behind the table's last
 *              page or on no page are not written to the cache
 *  T           0 .. 8388607 (a workgroup each); Hq 0 .. 4096, Hkv 1 .. 4096
 *  D           even, 2 .. 512; dtype any rope_dtype; any strides and alignment (the widest
 *              access that they allow is used)
 *  theta, pos_scale  as in rope_qk_apply_ex
 * Two tokens of one call must not share a cache row: it would hold parts of either, in no order. */
int32_t kv_append(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                  void* v_cache, int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride,
                  int64_t q_out_stride, int64_t k_stride, int64_t v_stride, int32_t num_pages,
                  int32_t page_size, int64_t page_stride, int64_t slot_stride, int64_t head_stride,
                  const int32_t* block_table, int32_t max_pages, int64_t table_stride,
                  const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* kv_lens, double theta,
                  double pos_scale, int32_t dtype, void* stream);

/* int32 words of a paged plan and floats of attn_paged's workspace, or -1. The workspace has room
 * for the splits of any batch of these sizes: about 2048 of them over all key/value heads, of 32
 * rows of D + 4 floats where T * Hq / Hkv is at most 32, else of 128 rows (D = 128, 8 heads: 35
 * and 139 MB). */
int64_t paged_plan_ints(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv);
int64_t paged_workspace_floats(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv, int32_t D);

/* Writes the plan of one step of a batch: which rows attend to which keys, and how the keys
 * are split over the chip. One small launch, which serves every layer of the step.
 * cu_seqlens and kv_lens as above, read now: later changes of kv_lens do not reach the
 * plan. Other arguments as in attn_plan. */
int32_t paged_plan(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* kv_lens, int64_t T,
                   int32_t Hq, int32_t Hkv, int32_t* plan, int64_t plan_ints, void* stream);

/* Attention of the new tokens over the cache, causal among themselves: one token of a
 * sequence (decode), a chunk of a prompt, or both in one batch.
 *  q, out, lse as in attn_fwd
 *  workspace   device float[paged_workspace_floats(...)], 16-byte aligned, scratch: calls
 *              that may run at the same time need one each
 *  plan        written by paged_plan for the same T, num_seqs, Hq and Hkv (as in attn_fwd)
 *  max_pages   entries of a sequence's row of block_table; keys behind them, and keys on no
 *              page, are seen by no query
 *  fill        as in attn_fwd
 * The cache is 16-byte aligned with strides that are multiples of 8 elements. */
int32_t attn_paged(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                   float* workspace, int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride,
                   int64_t out_stride, int32_t num_pages, int32_t page_size, int64_t page_stride,
                   int64_t slot_stride, int64_t head_stride, const int32_t* block_table,
                   int32_t max_pages, int64_t table_stride, const int32_t* plan, int32_t num_seqs,
                   double scale, int32_t dtype, int32_t fill, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H */
