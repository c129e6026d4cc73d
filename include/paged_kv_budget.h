/*
 * paged_kv_budget.h - C ABI of the operators that keep a block-paged KV
 * cache (paged_kv.h) within a budget of tokens per sequence: the attention
 * weight each cached token has been paid, the choice of the tokens to keep,
 * and the compaction of their rows.
 *
 * A step that evicts, per layer:
 *   paged_attention_scores   adds the step's attention weights to the running
 *                            scores of the sequences' cached tokens;
 *   paged_kv_select          picks the positions a budget keeps;
 *   paged_kv_compact         moves their K/V rows and scores to the front;
 * and once for all layers the host block manager gives the blocks past the
 * budget back (pkv_bm_compact, paged_kv_blocks.h).
 *
 * Running scores: float32 [num_rows, num_kv_heads, max_len], contiguous, the
 * caller's.  scores[row][h][j] belongs to the token at cache position j (its
 * index in the sequence's block table) of the sequence that owns `row`.
 * score_rows (device int32 [num_seqs]) names each batch sequence's row, so a
 * sequence keeps its row while the batch around it changes; NULL means row s
 * for sequence s.  A row < 0 leaves that sequence out of the call; a row >=
 * num_rows does too and sets PKV_DEVERR_BAD_SEQUENCE.  Two sequences with the
 * same row in one call: which one's values land is unspecified.
 *
 * Each kv head keeps its own choice of tokens: after a compaction, cache
 * position j of different heads may hold different tokens.  The rows keep
 * their order, so a later step's tokens follow them and causal attention is
 * unchanged.  Cached keys carry the rotation of the position they were
 * written at (paged_kv_write_rope takes positions apart from the slots).
 *
 * Pools with a scale for each block (paged_kv_fp8block.h) are not for these calls,
 * which know no such scales and cannot tell such pools from FP8 pools of one scale:
 * scores of them would be of other keys, and rows moved between blocks would change
 * their values, unreported.
 *
 * Layouts, alignment, streams and errors are those of paged_kv.h.
 */
#ifndef PAGED_KV_BUDGET_H_
#define PAGED_KV_BUDGET_H_

#include "paged_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * paged_attention_scores - accumulate the attention weight paid to each
 * cached token.
 *
 * For sequence s with L = context_lens[s] tokens and n queries (query_start_loc),
 * each query i < n and q head h of kv head k's group, let
 *   w[i][h][j] = softmax over the visible keys j of scale * q[i][h] . K[j][k]
 * (visible: j <= L - n + i, or all j < L when causal == 0).  Then for j < L
 *   paid[k][j] = sum over i and the heads h of k's group of w[i][h][j]
 *   out[row][k][j] = paid[k][j] + decay * scores[row][k][j]   for j < L - n
 *   out[row][k][j] = paid[k][j]                               for j >= L - n
 * (the step's own tokens start at this step: their slots may hold the scores
 * of tokens long gone).  decay == 0 reads no old score.  Entries at j >= L are
 * left as they were.  n == 0 leaves the row as it was.
 * Everything is accumulated in fp32; sums are taken in a fixed order, so equal
 * calls give equal bits.
 *
 *   q, k_cache, block_tables, context_lens, query_start_loc, scale, causal,
 *   dtype       as paged_attention_forward (same shapes supported)
 *   max_query_len  0, or a promise that no sequence has more queries (it picks
 *               the kernels): one that does is invalid, below
 *   scores      device float32 [num_rows, num_kv_heads, max_len]: the old scores
 *   scores_out  where the new ones go: the same layout; may be `scores` itself,
 *               must not overlap it otherwise
 *   decay       finite, >= 0: 1 accumulates, 0 starts afresh
 *   workspace   device scratch of workspace_bytes >=
 *               paged_attention_scores_workspace_min, 256-byte aligned;
 *               overwritten; not shared by calls that may run concurrently
 * A sequence with L > max_len, L > max_blocks_per_seq * block_size, n > L, n >
 * max_query_len > 0 or a non-monotone query_start_loc (an entry below an
 * earlier one) sets PKV_DEVERR_BAD_SEQUENCE and leaves its row as it was.  An
 * out-of-pool block id is read as a block of zeros and sets
 * PKV_DEVERR_BLOCK_OUT_OF_RANGE, as in paged_attention_forward.
 * bf16 queries: a sequence has at most 65536 * floor(128 / group) queries (group: q
 * heads per kv head); a call whose num_tokens, max_context and max_query_len
 * would allow more returns PKV_ERR_UNSUPPORTED.
 */
pkv_status paged_attention_scores(const void* q, const void* k_cache, const int32_t* block_tables,
                                  const int32_t* context_lens, const int32_t* query_start_loc,
                                  const int32_t* score_rows, const float* scores, float* scores_out,
                                  int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int64_t num_blocks, int32_t block_size,
                                  int32_t max_blocks_per_seq, int32_t num_rows, int32_t max_len,
                                  int32_t max_query_len, float scale, int32_t causal, float decay, void* workspace,
                                  size_t workspace_bytes, pkv_dtype dtype, void* stream);

/*
 * paged_attention_scores_fp8kv - the same over an FP8 K pool (E4M3 codes read
 * as code * k_scale; q bf16; head_dim 128), as paged_attention_forward_fp8kv.
 * q is rounded to fp16: |q| must stay below 65504.
 */
pkv_status paged_attention_scores_fp8kv(const void* q, const void* k_cache, const int32_t* block_tables,
                                        const int32_t* context_lens, const int32_t* query_start_loc,
                                        const int32_t* score_rows, const float* scores, float* scores_out,
                                        int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
                                        int32_t block_size, int32_t max_blocks_per_seq, int32_t num_rows,
                                        int32_t max_len, int32_t max_query_len, float scale, int32_t causal,
                                        float decay, float k_scale, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * Bytes of workspace for a batch of this shape; max_context is the smaller of
 * max_len and max_blocks_per_seq * block_size.  Pure host arithmetic.  _size
 * is what the call makes use of, _min the least it accepts (sequences whose
 * logits do not fit are computed twice instead of stored).
 */
size_t paged_attention_scores_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads,
                                             int32_t num_kv_heads, int64_t max_context);
size_t paged_attention_scores_workspace_min(int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads,
                                            int32_t num_kv_heads, int64_t max_context);

/*
 * paged_kv_select - the positions a budget keeps of each (sequence, kv head).
 *
 * Of the L = context_lens[s] positions: all of them when L <= budget; else
 * exactly `budget`: the first num_sink, the last num_recent, and of those
 * between the ones with the highest scores[row][h][j], ties to the lowest
 * position (a NaN ranks below every number, -0 equals +0).
 *   kept   device int32 [num_seqs, num_kv_heads, budget]: the kept positions in
 *          ascending order, then -1
 * num_sink, num_recent >= 0, num_sink + num_recent <= budget, 1 <= budget.
 * A sequence left out (score row < 0) or with L < 0 or L > max_len (sets
 * PKV_DEVERR_BAD_SEQUENCE) gets -1 throughout.
 */
pkv_status paged_kv_select(const float* scores, const int32_t* score_rows, const int32_t* context_lens,
                           int32_t* kept, int32_t num_seqs, int32_t num_kv_heads, int32_t num_rows, int32_t max_len,
                           int32_t budget, int32_t num_sink, int32_t num_recent, void* stream);

/*
 * paged_kv_compact - move the kept tokens of each (sequence, kv head) to the
 * front of its cache, in K, V and the running scores: for r = 0, 1, ... while
 * kept[s][h][r] >= 0,
 *   position r of dst_block_tables[s]  =  position kept[s][h][r] of block_tables[s]
 *   scores[row][h][r]                  =  scores[row][h][kept[s][h][r]]
 * (bit-exact; sources are read as they were before the call).
 *   kept              device int32 [num_seqs, num_kv_heads, budget], ascending
 *                     positions, then -1 (paged_kv_select's output)
 *   dst_block_tables  device int32 [num_seqs, max_blocks_per_seq], or NULL: in
 *                     place.  Entry j of the first ceil(kept / block_size) is
 *                     either block_tables' entry j or a block that no sequence
 *                     of the call reads (pkv_bm_compact hands out such tables)
 *   scores            device float32 [num_rows, num_kv_heads, max_len] or NULL
 *   dtype             PKV_DTYPE_BF16, _F32 or _FP8_E4M3 (the pools' element, of
 *                     one scale for a pool); head_dim * element size a multiple
 *                     of 16
 * A block written in place must belong to this sequence alone (no other table
 * of the call or of a later step reads its old rows).  Positions not ascending
 * set PKV_DEVERR_BAD_SEQUENCE, and the rows of that head are unspecified.  A
 * source position past the table (or, for scores, past max_len) or in a block
 * outside the pool reads as zeros and sets PKV_DEVERR_BLOCK_OUT_OF_RANGE; a
 * destination block outside the pool is skipped and sets it too.
 */
pkv_status paged_kv_compact(void* k_cache, void* v_cache, const int32_t* block_tables,
                            const int32_t* dst_block_tables, const int32_t* kept, const int32_t* score_rows,
                            float* scores, int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim,
                            int64_t num_blocks, int32_t block_size, int32_t max_blocks_per_seq, int32_t budget,
                            int32_t num_rows, int32_t max_len, pkv_dtype dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_KV_BUDGET_H_ */
