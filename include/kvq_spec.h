/*
 * kvq_spec.h — speculative decoding over the paged FP8 cache (libkvq.so).
 *
 * The calls of one serving step that verifies several drafted tokens a
 * sequence, in the order of use:
 *   kv_blocks_resize   the block tables grow to what the step needs
 *   kv_slot_map        each new token's place in the pools
 *   fp8_kv_append      the new tokens' keys and values go to their places
 *   fp8_tree_attention the drafted tokens attend over the cache and, through
 *                      the tree's mask, to one another
 *   fp8_kv_accept      the accepted path moves to the end of the sequence
 *   kv_blocks_resize   the blocks that only rejected tokens held come back
 * Every input that changes from step to step (lengths, tables, trees) is read
 * on the device: no call copies to the host or waits, so a step captures into
 * a CUDA graph and replays with new lengths. kvq.h's conventions hold: the
 * caller owns all memory, errors are found on the host before anything is
 * enqueued, device buffers start on 256-byte boundaries, except that q, k_new
 * and v_new may start on any 16-byte boundary and have a row stride, so that
 * they can be slices of a fused projection's output.
 *
 * A slot is the place of one token in the pools: block * block_tokens + row.
 * A call without tokens, rows or requests is refused: a step that adds nothing
 * makes none.
 * Calls that work on one pool, table or workspace run on one stream, or are
 * ordered by the caller.
 */
#ifndef KVQ_SPEC_H_
#define KVQ_SPEC_H_

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KVQ_SPEC_MAX_BATCH 4096 /* requests of one call                       */
#define KVQ_TREE_MAX 256        /* nodes of one request's tree                */
#define KVQ_TREE_MAX_GQA 64     /* query heads per kv head in tree attention  */

/* ------------------------------------------------------------------------ */
/* Block tables and slot maps (any paged cache)                              */
/* ------------------------------------------------------------------------ */

/* Give every request the blocks that target_tokens[b] tokens need:
 *   block_table   : device int32 [batch, max_blocks]; entries [0, n_held[b])
 *                   are request b's blocks
 *   n_held        : device int32 [batch], updated
 *   target_tokens : device int32 [batch]
 *   free_blocks   : device int32 [num_blocks], a stack of the free blocks:
 *                   entries [0, *free_count), the last one on top
 *   free_count    : device int32 [1], updated
 *   granted       : device int32 [batch], 1 where the request got what it asked
 *                   for, 0 where it was left as it was; may be NULL
 * need_b = ceil(target_tokens[b] / block_tokens). A request with fewer is
 * shrunk first: table entries need_b .. n_held[b]-1 go back to the stack and
 * become -1. Requests with more then grow in the order of b, each granted while
 * the running sum of growth asked for (a refused request's counted too) is at
 * most the blocks then free; its new entries follow the held ones. A target
 * below 0 or above max_blocks * block_tokens is refused. Blocks are pushed so
 * that the first one released (lowest b, then lowest entry) ends on top: a
 * growth and the shrink that undoes it leave the stack as it was.
 * One launch; the same inputs always give the same tables. KVQ_ERR_UNSUPPORTED
 * for batch > KVQ_SPEC_MAX_BATCH or batch * max_blocks >= 2^31. */
KVQ_API kvq_status kv_blocks_resize(int32_t* block_table, int32_t batch, int32_t max_blocks, int32_t* n_held,
                                    const int32_t* target_tokens, int32_t block_tokens, int32_t* free_blocks,
                                    int32_t* free_count, int32_t num_blocks, int32_t* granted, void* stream);

/* The places of each request's new tokens (request b holds seq_lens[b] tokens
 * and adds new_lens[b], negative ones counted as 0), flattened over requests:
 *   offsets   : device int32 [batch + 1], the exclusive prefix sum of new_lens
 *               (at most n_rows: what does not fit n_rows rows is cut off)
 *   slots     : device int64 [n_rows]; row offsets[b] + i is position
 *               p = seq_lens[b] + i: block_table[b, p / block_tokens] *
 *               block_tokens + p % block_tokens, or -1 where p lies outside the
 *               table's row or 31 bits, or its entry outside [0, num_blocks)
 *   seq_ids   : device int32 [n_rows], b; may be NULL
 *   positions : device int32 [n_rows], p (-1 where it leaves 31 bits): the
 *               token's place in the cache. For the nodes of a tree that is
 *               not their depth, which a rotary embedding goes by. May be NULL
 * Rows behind the last request get -1 in all three, which the append skips: a
 * padded batch needs no other care. */
KVQ_API kvq_status kv_slot_map(const int32_t* block_table, int32_t batch, int32_t max_blocks, const int32_t* seq_lens,
                               const int32_t* new_lens, int32_t block_tokens, int32_t num_blocks, int32_t n_rows,
                               int32_t* offsets, int64_t* slots, int32_t* seq_ids, int32_t* positions, void* stream);

/* ------------------------------------------------------------------------ */
/* FP8 pools: append by slot, accept                                         */
/* ------------------------------------------------------------------------ */

/* Quantize new tokens into a key and a value pool (same shape, format and
 * scale granularity) with the scales the pools hold:
 *   k_new, v_new : device fp16, row i at k_new + i * k_row_stride elements is
 *                  [kv_heads, D]; strides are multiples of 8, at least
 *                  kv_heads * D
 *   slots        : device int64 [n_tokens]; tokens whose slot is outside
 *                  [0, num_blocks * 16) are skipped. No two tokens of a call
 *                  may share a slot.
 * byte = FP8(fl32(x / scale)), as fp8_kv_quantize with static_scale. Only the
 * named rows of a block are written. */
KVQ_API kvq_status fp8_kv_append(const fp8_pool* k, const fp8_pool* v, const uint16_t* k_new, int64_t k_row_stride,
                                 const uint16_t* v_new, int64_t v_row_stride, const int64_t* slots, int32_t n_tokens,
                                 void* stream);

/* Keep the accepted tokens of each request's tree: the pool rows at positions
 * seq_lens[b] + path[b, i] move to positions seq_lens[b] + i for i <
 * n_accepted[b], in both pools, and new_lens[b] = seq_lens[b] + n_accepted[b].
 *   path       : device int32 [batch, path_len], a row's first n_accepted[b]
 *                entries strictly ascending (a path from the root down is, when
 *                nodes are numbered parents first), each in [0, KVQ_TREE_MAX)
 *   n_accepted : device int32 [batch], in [0, path_len]
 *   new_lens   : device int32 [batch]; may be seq_lens itself
 * Rows that stay in place keep their bytes (values are stored whole 16-byte
 * units at a time, with the bytes of up to three tokens beside a moved one as
 * they were). Entries outside the table or the pool are skipped. */
KVQ_API kvq_status fp8_kv_accept(const fp8_pool* k, const fp8_pool* v, const int32_t* block_table, int32_t batch,
                                 int32_t max_blocks, const int32_t* seq_lens, const int32_t* path, int32_t path_len,
                                 const int32_t* n_accepted, int32_t* new_lens, void* stream);

/* ------------------------------------------------------------------------ */
/* Tree attention                                                            */
/* ------------------------------------------------------------------------ */

/* Workspace of fp8_tree_attention: a status word at offset 0 (as
 * kv_decode_workspace_bytes), and what the call's two kernels hand over: partial
 * results and which of them belong together. Zero it once after allocating it
 * (the status word collects errors until it is cleared). One workspace serves
 * one stream: calls that overlap on the device (two captured graphs among
 * them) must not share it. The size goes by head_dim alone (43 MB at 128, 22 MB
 * at 64: what the blocks of one launch can leave); 0 for shapes the call
 * refuses. */
KVQ_API size_t fp8_tree_workspace_bytes(int32_t batch, int32_t kv_heads, int32_t q_heads, int32_t head_dim,
                                        int32_t max_tree);

/* Attention of a tree of drafted tokens per request over the paged FP8 cache,
 * the tree's own keys and values already appended to it:
 *   q            : device fp16, row n at q + n * q_row_stride is [q_heads, D]
 *   tree_offsets : device int32 [batch + 1]: request b's nodes are rows
 *                  tree_offsets[b] .. tree_offsets[b+1]-1 of q, tree_mask and
 *                  out (at most max_tree of them are used)
 *   seq_lens     : device int32 [batch], the tokens before the tree, 0 or more;
 *                  node j of request b is at position seq_lens[b] + j
 *   tree_mask    : device uint64 [n_tokens, mask_words]: a node sees every
 *                  token before the tree, and node j of its own request where
 *                  bit j % 64 of word j / 64 of its mask is set (its own bit
 *                  included: nothing is implied)
 *   out          : device [n_tokens, q_heads, D], fp32 if out_fp32, else fp16
 *   out[n, hq] = softmax(q . (k_scale K)^T * softmax_scale) (v_scale V) over
 * what node n sees, with kv head hq / (q_heads / kv_heads); zeros for a row
 * that sees nothing. What a row does not see does not reach it, NaN bytes and
 * stale rows behind the last node included. Rows of out behind the last node
 * are left as they are. softmax_scale <= 0 selects 1/sqrt(D).
 * max_seq_len bounds seq_lens[b] + the nodes of b; max_seq_len <= max_blocks *
 * 16. Lengths, offsets and table entries are clamped on the device: a bad one
 * gives wrong numbers, never an access outside the buffers.
 * The softmax weights go into the value product in two fp16 parts (2^-22
 * relative), as fp8_decode_attention's, for fp32 output, for max_tree *
 * (q_heads / kv_heads) <= 16, and for little work altogether (max_seq_len <=
 * 2560, few tiles of 16 rows). Larger calls with fp16 output round them to one
 * (2^-11 relative, as the output itself): two would take them 1.5 to 1.8 times
 * as long. Scores, sums and outputs accumulate in fp32.
 * KVQ_ERR_UNSUPPORTED for max_tree > KVQ_TREE_MAX, batch > KVQ_SPEC_MAX_BATCH
 * or q_heads / kv_heads > KVQ_TREE_MAX_GQA; KVQ_ERR_ARG for mask_words * 64 <
 * max_tree. */
KVQ_API kvq_status fp8_tree_attention(const uint16_t* q, int64_t q_row_stride, int32_t n_tokens, const fp8_pool* k,
                                      const fp8_pool* v, const int32_t* block_table, const int32_t* seq_lens,
                                      const int32_t* tree_offsets, const uint64_t* tree_mask, int32_t mask_words,
                                      int32_t batch, int32_t q_heads, int32_t max_blocks, int32_t max_tree,
                                      int32_t max_seq_len, void* out, int32_t out_fp32, float softmax_scale, void* ws,
                                      size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_SPEC_H_ */
