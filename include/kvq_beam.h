/*
 * kvq_beam.h — beam search and parallel sampling over the paged caches (libkvq.so).
 *
 * The calls of one step that keeps several continuations ("beams") of each
 * request, in the order of use:
 *   beam_select          the best candidates of each request from the logits
 *   kv_blocks_fork       the block tables follow the parents: full blocks are
 *                        shared, a partly filled last one is given a copy
 *   kv_blocks_copy       those copies, in every layer's pools
 *   kv_blocks_resize_shared, and kv_slot_map and fp8_kv_append of kvq_spec.h
 *                        the new tokens
 *   fp8_group_attention  decode attention that reads the blocks a request's
 *                        beams share once (for up to 128 query rows a kv head)
 * and, now and then, kv_blocks_compact, after which the pool's end is unused.
 * Everything that changes from step to step is read on the device: no call
 * copies to the host or waits, so a step captures into a CUDA graph. The
 * conventions of kvq.h hold: the caller owns all memory, errors are found on the
 * host before anything is enqueued, device buffers start on 256-byte boundaries
 * (logits: on a boundary of their type).
 *
 * Sequences come in groups of `width`: sequence b belongs to request b / width,
 * and a request with fewer continuations leaves the others empty (length 0).
 * Several table entries may name one block. shares[block], device int32
 * [num_blocks], counts the references beyond the first: 0 for a free block and
 * for one that a single entry names, so that blocks which a resize grants need
 * no care. A holder outside the tables, such as a prefix cache, counts itself in
 * shares. kv_blocks_resize (kvq_spec.h) knows no shares: what it takes from a
 * sequence is free for everyone, so that on tables whose blocks may be shared
 * kv_blocks_resize_shared stands for it.
 */
#ifndef KVQ_BEAM_H_
#define KVQ_BEAM_H_

#include "kvq_spec.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KVQ_BEAM_MAX_WIDTH 64     /* sequences of a request                     */
#define KVQ_BEAM_MAX_OUT 128      /* candidates of a request                    */
#define KVQ_COPY_MAX_BUFFERS 160  /* buffers of one kv_blocks_copy              */

#define KVQ_LOGITS_FP16 0
#define KVQ_LOGITS_FP32 1
#define KVQ_LOGITS_BF16 2

/* ------------------------------------------------------------------------ */
/* Selection                                                                 */
/* ------------------------------------------------------------------------ */

/* The n_out best candidates (beam i, token t) of each request by
 *   score(i, t) = scores[i] + logits[i, t] - log(sum_u exp(logits[i, u])),
 * best first, those of one beam in the order of their logits, equal logits by the
 * lower t, equal scores of different beams by the lower i:
 *   logits      : device, row b at logits + b * row_stride elements, vocab
 *                 elements of the type that logits_type names; row_stride >=
 *                 vocab (rows need no alignment beyond their type's)
 *   scores      : device float32 [groups * width]; a value that is not finite
 *                 makes the beam a dead one, ended or not: all its candidates
 *                 score -inf
 *   finished    : device uint8 [groups * width] or NULL; a beam that has ended
 *                 (not 0) offers (end_token, scores[i]) alone, its other tokens
 *                 score -inf and its logits are not read
 *   end_token   : in [0, vocab) where finished is given
 *   out_scores  : device float32 [groups, n_out]
 *   out_parents : device int32 [groups, n_out], i, the beam within its request
 *   out_tokens  : device int32 [groups, n_out], t
 * A NaN logit counts as -inf and +inf as the largest float32; a token at -inf
 * scores -inf, and candidates at -inf fill up what finite ones leave, by the
 * lower i * vocab + t. Sums are float32 within a thread (at most 64 additions
 * one after the other, of 16 or 32 terms each), float64 or whole numbers beyond.
 * The logarithm of a sum is off by less than 2^-18, in rows of up to 160000
 * tokens by 2^-20 at most in what was tried (a constant tail: every term carries
 * the same rounding of its exponent); scores of two beams that are closer may
 * come in the other order than exact ones. Scores are compared in float64 and
 * rounded once. A row gives the same wherever it starts, and the same call the
 * same bits.
 * One launch. KVQ_ERR_UNSUPPORTED for width > KVQ_BEAM_MAX_WIDTH or n_out >
 * KVQ_BEAM_MAX_OUT, KVQ_ERR_ARG for n_out > vocab. */
KVQ_API kvq_status beam_select(const void* logits, int32_t logits_type, int64_t row_stride, const float* scores,
                               const uint8_t* finished, int32_t end_token, int32_t groups, int32_t width, int32_t vocab,
                               int32_t n_out, float* out_scores, int32_t* out_parents, int32_t* out_tokens, void* stream);

/* ------------------------------------------------------------------------ */
/* Blocks that several sequences share                                       */
/* ------------------------------------------------------------------------ */

/* Workspace of kv_blocks_fork (groups requests) and kv_blocks_compact (any
 * number) for pools of up to num_blocks blocks. Zero it once after allocating it:
 * the calls leave it as they need it, for pools of other sizes too. Calls that
 * overlap on the device must not share it. 0 for sizes the calls refuse. */
KVQ_API size_t kv_blocks_workspace_bytes(int32_t groups, int32_t num_blocks);

/* Every sequence becomes a copy of its parent, in place:
 *   block_table   : device int32 [batch, max_blocks], n_held: device int32
 *                   [batch], seq_lens: device int32 [batch], all updated
 *   parents       : device int32 [batch], the parent's place within the request,
 *                   0 .. width - 1 (its own: stays); any other value empties the
 *                   sequence and gives its blocks back
 *   shares        : device int32 [num_blocks], updated
 *   free_blocks, free_count : the stack of kv_blocks_resize, updated
 *   copy_src, copy_dst : device int32 [batch], copy_count: device int32 [1]:
 *                   blocks whose content has to be copied before the next append
 *                   (kv_blocks_copy); entries from copy_count on stay as they were
 *   granted       : device int32 [batch] or NULL; 0 where a sequence lacks a last
 *                   block of its own (see below), else 1
 *   shared_blocks : device int32 [batch / width] or NULL; the leading full blocks
 *                   that all sequences of the request with a length above 0 have
 *                   in common (0 without any)
 * With p the parent: seq_lens[b] = seq_lens[p], n_held[b] = ceil(seq_lens[p] /
 * block_tokens) (blocks held beyond that are not inherited: grow again after the
 * call), the held entries are p's, those behind become -1. A block that loses
 * its last reference is freed; freed blocks are pushed in descending order, the
 * lowest on top. Then every sequence whose last block is partly filled and has
 * other references gets a block of its own from the top of the stack, in the
 * order of b, and a (copy_src, copy_dst) pair, except that where only such
 * sequences of its request share that block the first of them keeps it. When the
 * stack runs out, the sequences left go on sharing (granted 0) and must not be
 * appended to.
 * A partly filled block is shared within a request only. Entries that name no
 * block of the pool are passed on and not counted.
 * The same inputs always give the same tables. KVQ_ERR_UNSUPPORTED for batch >
 * KVQ_SPEC_MAX_BATCH, width > KVQ_BEAM_MAX_WIDTH or batch * max_blocks >= 2^31;
 * KVQ_ERR_SHAPE for batch % width != 0. */
KVQ_API kvq_status kv_blocks_fork(int32_t* block_table, int32_t batch, int32_t max_blocks, int32_t* n_held,
                                  int32_t* seq_lens, const int32_t* parents, int32_t width, int32_t block_tokens,
                                  int32_t* shares, int32_t* free_blocks, int32_t* free_count, int32_t num_blocks,
                                  int32_t* copy_src, int32_t* copy_dst, int32_t* copy_count, int32_t* granted,
                                  int32_t* shared_blocks, void* ws, size_t ws_bytes, void* stream);

/* kv_blocks_resize (kvq_spec.h) for such tables: a sequence that would release a
 * block with other references (shares above 0, device int32 [num_blocks], read
 * alone) is refused like a target outside the table: granted 0, left as it was.
 * All else is as there. To shorten a sequence that shares blocks, lower
 * seq_lens and call kv_blocks_fork with every sequence its own parent: it keeps
 * the counts, frees what nobody holds any more, and copies a block that others
 * hold in full and the shorter one in part. */
KVQ_API kvq_status kv_blocks_resize_shared(int32_t* block_table, int32_t batch, int32_t max_blocks, int32_t* n_held,
                                           const int32_t* target_tokens, int32_t block_tokens, const int32_t* shares,
                                           int32_t* free_blocks, int32_t* free_count, int32_t num_blocks,
                                           int32_t* granted, void* stream);

/* One buffer of blocks: block i is the block_bytes bytes at base + i *
 * block_bytes (a multiple of 16). For an fp8_pool or nvfp4_pool: its memory, and
 * its bytes divided by num_blocks. */
typedef struct {
  void* base;
  int64_t block_bytes;
} kvq_block_buffer;

/* Copy block src[i] to block dst[i] for i < min(*count, n_pairs) in each of
 * n_buffers buffers (a host array, read before the call returns). Pairs that name
 * no block of [0, num_blocks) are skipped. No block may be the destination of two
 * pairs, or the source of one and the destination of another. count: device int32
 * [1], or NULL for n_pairs. One launch. */
KVQ_API kvq_status kv_blocks_copy(const kvq_block_buffer* buffers, int32_t n_buffers, int32_t num_blocks,
                                  const int32_t* src, const int32_t* dst, int32_t n_pairs, const int32_t* count,
                                  void* stream);

/* Empty the pool's blocks from keep_blocks on: the used ones among them (those
 * not on the stack), in ascending order, move to the free ones below, in
 * ascending order. Table entries (the first n_held[b] of each row) and shares
 * follow; the stack then holds the blocks below keep_blocks that are still free,
 * the lowest on top (entries behind the new count stay as they were).
 *   moved_to      : device int32 [num_blocks]: where each block is now (itself where
 *                   it stays), for holders outside the tables
 *   copy_src, copy_dst : device int32 [max_copies], copy_count: device int32 [1]
 *   done          : device int32 [1]: 1, or 0 where the free blocks below or
 *                   max_copies do not suffice: then nothing changes (copy_count
 *                   0, moved_to the identity)
 * To be followed by kv_blocks_copy in every pool. keep_blocks in [0, num_blocks].
 * (A pool that grows again gets its upper blocks back by pushing their numbers.) */
KVQ_API kvq_status kv_blocks_compact(int32_t* block_table, int32_t batch, int32_t max_blocks, const int32_t* n_held,
                                     int32_t keep_blocks, int32_t* shares, int32_t* free_blocks, int32_t* free_count,
                                     int32_t num_blocks, int32_t* moved_to, int32_t* copy_src, int32_t* copy_dst,
                                     int32_t max_copies, int32_t* copy_count, int32_t* done, void* ws, size_t ws_bytes,
                                     void* stream);

/* ------------------------------------------------------------------------ */
/* Attention                                                                 */
/* ------------------------------------------------------------------------ */

/* Workspace of fp8_group_attention: a status word at offset 0 (as
 * kv_decode_workspace_bytes) and the partial results that the call's kernels
 * hand over: at head_dim 128 some 34 to 38 MB, and 520 bytes for every query
 * head of every sequence, two or three times. Zero it once after allocating it
 * (the status word collects errors until it is cleared). One workspace serves one
 * stream: calls that overlap on the device (two captured graphs among them) must
 * not share it. 0 for shapes the call refuses. */
KVQ_API size_t fp8_group_workspace_bytes(int32_t batch, int32_t width, int32_t kv_heads, int32_t q_heads,
                                         int32_t head_dim);

/* Decode attention over the FP8 paged cache for sequences that share leading
 * blocks: as fp8_decode_attention (q in fp16),
 *   out[b, hq] = softmax(q[b, hq] . (k_scale K)^T * softmax_scale) (v_scale V)
 * over tokens 0 .. seq_lens[b] - 1 of sequence b, zeros where seq_lens[b] <= 0,
 * but the blocks that a group's sequences share are read (and converted) once for
 * all of the group's query rows of a kv head, width * (q_heads / kv_heads), up to
 * 128 of them, and once for every 128 beyond:
 *   q             : device fp16, row b at q + b * q_row_stride is [q_heads, D]
 *   block_table   : device int32 [batch, max_blocks]
 *   seq_lens      : device int32 [batch], the new tokens included
 *   shared_blocks : device int32 [batch / width]: the first shared_blocks[g] table
 *                   entries of all sequences of group g with a length above 0 are
 *                   the same, and each of those has at least 16 times as many
 *                   tokens (kv_blocks_fork writes such numbers; a smaller one, 0
 *                   included, only costs time)
 *   out           : device [batch, q_heads, D], fp32 if out_fp32, else fp16
 * Rows of a block behind a sequence's last token do not reach it, NaN bytes
 * included. softmax_scale <= 0 selects 1/sqrt(D). max_seq_len bounds seq_lens[b];
 * max_seq_len <= max_blocks * 16. Lengths, counts and table entries are clamped on
 * the device: a bad one gives wrong numbers, never an access outside the buffers.
 * The softmax weights go into the value product in two fp16 parts (2^-22
 * relative), but over shared blocks for fp16 output with width * (q_heads /
 * kv_heads) > 16 in one (2^-11 relative, as the output itself, so that an output
 * that is small beside the values it is made of may be off by several steps):
 * two would take such calls 1.2 to 1.7 times as long, as fp32 output, which has
 * them, does. Scores, sums and outputs accumulate in fp32. The same call gives
 * the same bits.
 * KVQ_ERR_UNSUPPORTED for batch > KVQ_SPEC_MAX_BATCH, width >
 * KVQ_BEAM_MAX_WIDTH, q_heads / kv_heads > KVQ_TREE_MAX_GQA or batch * q_heads >=
 * 2^31; KVQ_ERR_SHAPE for batch % width != 0. */
KVQ_API kvq_status fp8_group_attention(const uint16_t* q, int64_t q_row_stride, const fp8_pool* k, const fp8_pool* v,
                                       const int32_t* block_table, const int32_t* seq_lens,
                                       const int32_t* shared_blocks, int32_t batch, int32_t width, int32_t q_heads,
                                       int32_t max_blocks, int32_t max_seq_len, void* out, int32_t out_fp32,
                                       float softmax_scale, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_BEAM_H_ */
