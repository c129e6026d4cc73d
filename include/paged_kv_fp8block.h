/*
 * paged_kv_fp8block.h - C ABI of block-paged KV pools of 8-bit codes with a
 * scale for each block and kv head: the write that encodes rows and keeps the
 * scales, the attention that reads them, and the copy of scales that goes
 * with a copy-on-write.
 *
 * The pools of paged_kv.h's FP8 calls have one scale each, which the caller
 * must know before the first row arrives; here the scales follow the rows.
 *
 *   k_cache, v_cache    E4M3 codes [num_blocks, block_size, num_kv_heads, head_dim]
 *   k_scales, v_scales  float32 [num_blocks, num_kv_heads], zeros at first
 *   value of slot b * block_size + o, head h = code * scales[b][h]
 *
 * Scales that the write makes are powers of two in [2^-60, 2^60]: a block
 * whose scale grows has its earlier codes shifted in exponent, which loses
 * nothing but what falls among E4M3's subnormals, however often it happens.
 * The attention reads any scale; one outside [2^-60, 2^60] is taken as the
 * nearest end (a NaN as 2^-60).
 *
 * The codes have the type and layout of paged_kv.h's FP8 pools, so that no call
 * can tell the two apart.  Only the calls below, and paged_kv_copy_blocks together
 * with paged_kv_copy_block_scales, are for these pools.  Calls that take one scale
 * for a pool (all that end in _fp8 or _fp8kv, paged_attention_scores_fp8kv among
 * them) read or write other values here, and paged_kv_compact moves codes between
 * blocks whose scales differ: none of them reports it.  There is no scoring and no
 * eviction of these pools' tokens.
 *
 * Layouts, alignment, streams and errors are those of paged_kv.h.
 */
#ifndef PAGED_KV_FP8BLOCK_H_
#define PAGED_KV_FP8BLOCK_H_

#include "paged_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * paged_kv_write_fp8block - encode new K/V rows and scatter them into the
 * pools, growing the scales of the blocks they go to.
 *
 * For a block b that the call writes rows to, and each kv head h, K and V
 * apart, with top = the largest |x| of those rows:
 *   need = the least power of two in [2^-60, 2^60] with top <= 448 need
 *   old  = 0 if the call writes the block's first slot (the block begins
 *          anew: what else it holds is of an earlier sequence), else scales[b][h]
 *   scales[b][h] = new = max(old, need)
 *   code of x = E4M3(RNE(x / new)), saturated at +-448; NaN stays NaN
 * and, where the block goes on (old > 0 or 0 alike) and new > old, every code
 * of it that the call does not write becomes E4M3(RNE(value * old / new)).
 * Codes that the call does not write are otherwise left as they are.
 * A division by new is a product with its reciprocal in fp32.  For the powers of two
 * that this call makes that is the same; a scale that the caller put there (finite;
 * below 0 or a NaN it counts as 0) need not be one, and a code may then be its
 * neighbour where the quotient lies within 2^-22 of the border between two.
 * Rows are expected finite: an infinity saturates, and takes its scale to 2^60; a
 * NaN has no part in the scale.
 *
 *   k, v            device, [num_tokens, num_kv_heads, head_dim] of `dtype`
 *                   (PKV_DTYPE_BF16 or _F32), token strides in ELEMENTS (0: dense)
 *   slot_mapping    device int64 [num_tokens], as paged_kv_write (slots < 0 are
 *                   skipped, slots past the pool too, with
 *                   PKV_DEVERR_SLOT_OUT_OF_RANGE; two tokens with one slot: which
 *                   one lands is unspecified, and the scale covers that one)
 *   block_size      8, 16, 32 or 64; head_dim a multiple of 16, at most 1024
 *   workspace       device scratch of workspace_bytes >=
 *                   paged_kv_write_fp8block_workspace (may be NULL where that is
 *                   0), 16-byte aligned; overwritten; not shared by calls that may
 *                   run concurrently
 * Blocks that several tables name must not be written (copy-on-write belongs
 * to the cache manager).  num_tokens == 0 is a no-op.
 */
pkv_status paged_kv_write_fp8block(const void* k, const void* v, const int64_t* slot_mapping, void* k_cache,
                                   void* v_cache, float* k_scales, float* v_scales, int64_t num_tokens,
                                   int64_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                                   int64_t k_token_stride, int64_t v_token_stride, void* workspace,
                                   size_t workspace_bytes, pkv_dtype dtype, void* stream);

/* Bytes of workspace that paged_kv_write_fp8block wants (pure host arithmetic). */
size_t paged_kv_write_fp8block_workspace(int64_t num_tokens, int64_t num_blocks, int32_t block_size);

/*
 * paged_kv_copy_block_scales - the scales' part of a copy-on-write: for every
 * pair i and layer l, row copies[i][1] of layer l's k_scales and v_scales
 * becomes row copies[i][0].  The codes go through paged_kv_copy_blocks
 * (PKV_DTYPE_FP8_E4M3).
 *   k_scales, v_scales  device float32, num_layers arrays of [num_blocks,
 *                       num_kv_heads], layer l at element offset l *
 *                       layer_stride (0: dense)
 *   copies              HOST int32 [num_copies, 2], checked as
 *                       paged_kv_copy_blocks checks it
 */
pkv_status paged_kv_copy_block_scales(float* k_scales, float* v_scales, const int32_t* copies, int32_t num_copies,
                                      int32_t num_layers, int64_t layer_stride, int64_t num_blocks,
                                      int32_t num_kv_heads, void* stream);

/*
 * paged_attention_forward_fp8block - paged_attention_forward over such pools:
 * softmax(scale * q k^T) v with k and v the values above, q and out bf16,
 * head_dim 128.
 *
 *   window, num_sink  as paged_attention_window_forward; window 0: no window
 *                     (num_sink is ignored).  A window needs causal != 0.
 *   the rest          as paged_attention_forward (the same block sizes, groups,
 *                     query counts, workspace and errors)
 * Numerics: q is split into two E4M3 terms for each row's own power-of-two
 * scale (off by at most 2^-17 of the row's largest |q|, or by 2^-136 where that
 * is more; calls of many rows may leave out more of a row so small that none of
 * its logits moves by 2^-16; the tensor cores multiply codes by codes), logits
 * and sums are fp32; a weight times its V scale is split into E5M2 terms of 9
 * bits together in calls of few rows, and rounded to fp16 in calls of many (at
 * least 11 bits for those above 2^-21 of the row's largest).
 * q is expected finite, and a row's largest |q| times scale times a K scale it
 * meets below 2^110, so that logits stay in fp32.  A NaN makes its row NaN; a row
 * with an infinity, or past that bound, may be NaN or anything else.  Other rows are
 * as without it.
 */
pkv_status paged_attention_forward_fp8block(const void* q, const void* k_cache, const void* v_cache,
                                            const float* k_scales, const float* v_scales,
                                            const int32_t* block_tables, const int32_t* context_lens,
                                            const int32_t* query_start_loc, void* out, int32_t num_seqs,
                                            int64_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int64_t num_blocks, int32_t block_size,
                                            int32_t max_blocks_per_seq, int32_t max_query_len, float scale,
                                            int32_t causal, int32_t window, int32_t num_sink, void* workspace,
                                            size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_KV_FP8BLOCK_H_ */
