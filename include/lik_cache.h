/*
 * lik_cache.h -- C ABI of a paged cache of keys and values held in 8 bits
 * (gfx950): its block tables, its writes, and the attention that reads it.
 *
 *   lik_cache_tables      block tables and slot maps from the lengths of the
 *                         requests
 *   lik_cache_append      keys and values of new tokens written to their slots
 *   lik_cache_attention   causal attention of every request's last tokens over
 *                         its cached ones
 *
 * Together with lik_verify_rows (lik_rows.h) they are one step of generation:
 * lengths grow by the drafts, tables give the slots and the offsets of every
 * request's rows, keys and values are appended, attention runs over them, the
 * drafts are verified over the same offsets, and lengths shrink to what was
 * accepted.  A request that the pool has no blocks for is not granted its drafts: it
 * keeps its length, while its rows go through the step with the others'.  Nothing of
 * them is appended, what attention and verification give for them means nothing, and
 * what was accepted must not change its length.
 *
 * The conventions of lik.h hold (memory, stream, errors, determinism,
 * reentrancy), and for every operator here:
 *
 * Cache.  num_blocks blocks of block_size tokens (a power of two, 16 to 256;
 *   num_blocks * block_size < 2^31) for kv_heads heads of dim 64, 128 or 256.
 *   One byte a number, in the format with 4 exponent and 3 mantissa bits and
 *   no infinities (e4m3, largest number 448):
 *     k_cache [num_blocks][kv_heads][block_size][dim]
 *     v_cache [num_blocks][kv_heads][dim][block_size]
 *   (values lie dim by dim, because the product with the weights sums over
 *   tokens), block b at b * k_stride (v_stride) bytes, a multiple of 16 and at
 *   least kv_heads * block_size * dim, the rest dense, 16-byte aligned.
 *     k_scale, v_scale [num_blocks][kv_heads] float32
 *   and a number is its code times the scale of its block and head.  Scales
 *   lie within [2^-40, 2^40] (others count as the nearest of these); a scale
 *   that is NaN makes its block and head NaN.  The codes 0x7f and 0xff, which
 *   are no numbers in the format, must not stand where a request reads.
 * Slots.  Token `o` of block b is slot b * block_size + o.
 * Block tables.  [S][max_blocks] int32 with a row stride of table_ld: the block
 *   of positions i * block_size .. of request s is entry i of row s.  An entry
 *   outside [0, num_blocks) is no block: what would stand there is not read,
 *   not written and not attended to.
 * Lengths.  int32, on the device.  A negative one counts as 0.
 */
#ifndef LIK_CACHE_H_
#define LIK_CACHE_H_

#include "lik.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Block tables and slot maps.  Request s goes from old_len[s] tokens to
 * new_len[s]: blocks that it lacks are taken from the pool of free ones, blocks
 * that it no longer fills are given back, in one call for all requests.
 *
 * The pool is a ring of num_blocks entries of which `count` from `head` on (and
 * round the end) are free blocks; ring_state [4] int32 is {head, count, 0, 0}
 * between calls, at first {0, num_blocks, 0, 0} with every block in the ring.
 * Blocks are taken from the head in the order of the requests and of their
 * positions, and given back to the tail in the same order; what is given back
 * can be taken from the next call on.
 *
 * A request is granted what it asks for unless its table would be longer than
 * max_blocks, or it needs blocks and the requests up to and including it need
 * more than are free.
 *   granted [S]        new_len where granted (a negative one as 0), old_len
 *                      elsewhere (within [0, max_blocks * block_size])
 *   block_table        entries of blocks taken are written, entries of blocks
 *                      given back become -1; others stay
 *   token_offsets [S + 1]  running sum of max(0, new_len - old_len), granted or
 *                      not: where the rows of every request's new tokens lie
 *                      (a sum that passes 2^31 - 1 stays there)
 *   slots [T]          the slot of every new token in that order; -1 for
 *                      those of requests that were not granted, and from
 *                      token_offsets[S] on.  Tokens beyond T have none.
 * Calls on one pool or table must not overlap.  S up to 2^20 and max_blocks *
 * block_size < 2^31 (LIK_ERR_UNSUPPORTED beyond).  The outputs must not overlap the inputs, or each other.  A ring that
 * is not consistent gives wrong blocks, but nothing outside the arrays is read or
 * written.  No workspace; S == 0 sets slots to -1 and token_offsets[0] to 0.
 */
lik_status lik_cache_tables(const int32_t* old_len, const int32_t* new_len,
                            int64_t S, int64_t block_size, int32_t* block_table,
                            int64_t max_blocks, int64_t table_ld, int32_t* ring,
                            int64_t num_blocks, int32_t* ring_state,
                            int32_t* granted, int32_t* token_offsets,
                            int32_t* slots, int64_t T, void* stream);

/*
 * Keys and values of T tokens, k and v [T][kv_heads][dim] in LIK_F16,
 * LIK_BF16 or LIK_F32 with token strides k_ld and v_ld in elements (16-byte
 * aligned, as the strides are), written to slots [T] (int32).  A negative slot,
 * or one past the cache, is left out.
 *
 * A block and head's scale is the smallest power of two, within
 * [2^-40, 2^40], that keeps every number written within 448 times it.  A call
 * that writes a block's first slot starts the block anew: its scale comes from what is
 * written, whatever stood there.  Else the scale grows where what is
 * written needs it (and to a power of two, if it was none), and the codes that stand
 * in the block are rounded again (which changes those alone that leave the
 * format's normal numbers); it never shrinks.  So the tokens of a block are written in the order of their
 * slots, from the first; those behind may be written over, as rejected drafts are.
 * Numbers are rounded to nearest even.  A number that is not finite makes the
 * scale of its block and head NaN, until the block is started anew.
 *
 * Tokens of one block must follow each other in the call (what
 * lik_cache_tables gives does); of two with the same slot the later one stays.
 * T below 2^31 - 2^8 (LIK_ERR_UNSUPPORTED beyond).
 */
lik_status lik_cache_append(const void* k, const void* v, lik_dtype dtype,
                            int64_t T, int64_t k_ld, int64_t v_ld,
                            const int32_t* slots, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, int64_t num_blocks,
                            int64_t kv_heads, int64_t block_size, int64_t dim,
                            int64_t k_stride, int64_t v_stride, void* stream);

/*
 * Workspace bytes of one lik_cache_attention call of the same sizes; 0 for
 * zero-sized ones, SIZE_MAX for sizes that the call refuses.
 */
size_t lik_cache_workspace_bytes(int64_t T, int64_t S, int64_t q_heads,
                                 int64_t kv_heads, int64_t dim, lik_dtype dtype);

/*
 * Attention of T query tokens, q [T][q_heads][dim] in LIK_F16, LIK_BF16 or
 * LIK_F32 with a token stride of q_ld elements.  Request s has the rows
 * q_offsets[s] .. q_offsets[s+1] - 1 (int32 [S + 1], on the device, not
 * decreasing, within [0, T]) as its last tokens: with n rows, row i stands at
 * position kv_len[s] - n + i and attends to the positions up to its own.  Query
 * head h reads head h / (q_heads / kv_heads) of the cache.
 *   out[t, h] = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale q . k_j)
 *   lse[t, h] = log sum_j w_j                (float32 [T][q_heads], or NULL)
 * in q's type with a token stride of out_ld, rounded once.  A row that attends to
 * nothing (a length of 0, no block in its table), and one outside every request, is 0
 * with lse -inf, whatever its query holds; a query that is not finite is NaN, with its
 * lse, where it attends to anything.  kv_len beyond max_blocks * block_size
 * counts as that.
 * Scores, with log2 of their block's v_scale added, and sums are float32; where
 * scale times a query's largest number times a k_scale passes 2^128 the row may be
 * NaN.  A query's numbers are off by up to 2^-39 of its largest (LIK_F32: or 2^-22 of
 * themselves).  A weight w_j is rounded before its product with the values,
 * which sums in float32: to 11 bits (22 with LIK_F32) where
 * w_j times its block's v_scale is above 2^-25 (2^-29) of the largest such product of
 * the row, and by up to 2^-36 (2^-51) of that largest below; scores beyond 2^22, whose
 * differences float32 holds to a quarter, leave 2^-14 and 2^-25 (2^-36) in their place.
 * The weights' own sum is that of the unrounded ones.
 * scale within [2^-64, 2^64].  q and out 16-byte aligned, as their strides are;
 * out must not overlap q.  q_heads a multiple of kv_heads; T * q_heads and
 * max_blocks * block_size below 2^31, S up to 2^20 (LIK_ERR_UNSUPPORTED beyond).
 */
lik_status lik_cache_attention(const void* q, lik_dtype dtype, int64_t T,
                               int64_t q_heads, int64_t q_ld,
                               const int32_t* q_offsets, const int32_t* kv_len,
                               int64_t S, const int32_t* block_table,
                               int64_t max_blocks, int64_t table_ld,
                               const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale,
                               int64_t num_blocks, int64_t kv_heads,
                               int64_t block_size, int64_t dim, int64_t k_stride,
                               int64_t v_stride, float scale, void* out,
                               int64_t out_ld, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIK_CACHE_H_ */
