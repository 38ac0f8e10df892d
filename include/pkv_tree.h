/*
 * pkv_tree.h — C ABI of libpkv.so, speculative decoding with a tree of drafted
 * tokens per row: the drafted tokens are rotated and stored behind the row's
 * context (kv_rope_append, with each token's depth in its position), attended
 * along their branches (paged_tree_attention), and, once the model has accepted
 * one of them, its branch becomes the row's next tokens (kv_tree_commit).
 *
 * Conventions are those of pkv.h and pkv_chunk.h: a row's drafted tokens are its
 * new tokens, entries cu_seqlens[i] .. cu_seqlens[i + 1] - 1 of the token arrays,
 * n_i of them, at the slots C_i .. C_i + n_i - 1 behind its C_i = seq_lens[i] -
 * n_i context tokens.  On top of those:
 *   - parents is a device int32 array [total_tokens]: the parent of a drafted
 *     token, as its index within the row (0 .. n_i - 1), or -1 where it follows
 *     the context.  A parent comes before its children.  Any other value
 *     records PKV_DEV_BAD_TREE and stands for -1.  Several tokens may follow the
 *     context (a forest).
 *   - depth(j) is the number of token j's ancestors, and C_i + depth(j) its
 *     position, which need not be its slot.
 *   - A row with more than PKV_MAX_TREE_TOKENS drafted tokens records
 *     PKV_DEV_BAD_LENGTH and is skipped, as rows of invalid lengths are.
 */
#ifndef PKV_TREE_H
#define PKV_TREE_H

#include "pkv_chunk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_MAX_TREE_TOKENS 1024 /* drafted tokens of a row */

/* paged_tree_attention — attention of the drafted tokens over the paged cache:
 * paged_chunk_attention, but that token j of row i, at position P = C_i +
 * depth(j), attends to
 *     the context tokens t < C_i with t > P - W or t < S, and
 *     of the drafted tokens itself and its ancestors, those at positions p with
 *     p > P - W or p < S
 * under the layer's window W and sinks S (W = 0: to all of these).  So each
 * branch gets what it would get as a row of its own; a chain of parents is
 * paged_chunk_attention, and a single token of parent -1 a decode step.
 * Arguments, types, errors, workspace (paged_chunk_workspace_bytes) and launches
 * are those of paged_chunk_attention, with
 *   parents  int32 [total_tokens], see above
 *   scores   slopes and prefix_lens must be NULL (PKV_ERR_UNSUPPORTED) */
pkv_status paged_tree_attention(const pkv_pool *pool, int layer, const void *q, long long q_stride,
                                pkv_kv_dtype q_dtype, const int32_t *parents, const int32_t *cu_seqlens,
                                int total_tokens, const int32_t *block_table, int bt_stride,
                                const int32_t *seq_lens, int num_rows, int n_q_heads,
                                const pkv_scores *scores, void *out, float *lse, void *workspace,
                                size_t workspace_bytes, int num_chunks, void *stream);

/* kv_tree_commit — keep the branch that ends in the accepted token: with
 * path_0 < path_1 < .. < path_{a-1} = leaves[i] that token and its ancestors, the
 * K and V (all heads, scales included) of slot C_i + path_d are moved to slot
 * C_i + d, in the layers first_layer .. first_layer + num_layers - 1, and
 * new_lens[i] receives C_i + a.  Slots from C_i + a on keep what they held or
 * receive nothing of use: they are the next tokens' to overwrite.
 *   leaves    int32 [num_rows], in [-1, n_i): -1 accepts nothing (a = 0); any other
 *             value records PKV_DEV_BAD_TREE and stands for -1
 *   path      int32 [num_rows][path_stride] or NULL: receives path_d at [i][d], d <
 *             min(a, path_stride); the other entries are left as they are
 *   new_lens  int32 [num_rows].  A skipped row receives its seq_lens[i]
 * path and new_lens are arrays of their own, none of the inputs.  Of the parents,
 * those of the accepted token and its ancestors are looked at.
 * Block-table entries outside the pool record PKV_DEV_BAD_PAGE; the tokens
 * concerned are not moved.  A page behind C_i that two rows of the call share
 * must not be in a path's way.  Every type of pool.  One launch. */
pkv_status kv_tree_commit(const pkv_pool *pool, int first_layer, int num_layers, const int32_t *parents,
                          const int32_t *leaves, const int32_t *cu_seqlens, int total_tokens,
                          const int32_t *block_table, int bt_stride, const int32_t *seq_lens,
                          int num_rows, int32_t *path, int path_stride, int32_t *new_lens,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_TREE_H */
