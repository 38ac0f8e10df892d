/*
 * pkv_chunk.h — C ABI of libpkv.so, the long-prompt operators: a ragged chunk
 * of new tokens per row is rotated and stored in the paged cache
 * (kv_rope_append), attends to the cache (paged_chunk_attention), adds its
 * attention weights to a running weight per cached token
 * (paged_attention_mass), and rows that outgrow their budget keep the tokens
 * of largest weight (kv_evict).
 *
 * Conventions shared by the four calls, next to those of pkv.h (pool, block
 * tables, lengths, alignment, ownership, errors and the status word):
 *   - A chunk.  cu_seqlens is a device int32 array [num_rows + 1]; row i's new
 *     tokens are the entries cu_seqlens[i] .. cu_seqlens[i + 1] - 1 of the token
 *     arrays (q, k, v, out, lse, positions), n_i of them, possibly none.  It
 *     must not decrease and stays within [0, total_tokens]; entries of the
 *     token arrays at or behind cu_seqlens[num_rows] belong to no row and are
 *     neither written nor let into any result.
 *   - Row i holds L_i = seq_lens[i] tokens INCLUDING its n_i new ones: new
 *     token j of the row is the cached token P = L_i - n_i + j.
 *   - Rows with n_i > L_i, L_i < 0, L_i > 16 * bt_stride, or whose cu_seqlens
 *     entries decrease or leave [0, total_tokens], record PKV_DEV_BAD_LENGTH
 *     and are skipped as each call says.
 *   - Element types of token arrays are pkv_kv_dtype values: PKV_KV_F16,
 *     PKV_KV_BF16 or PKV_KV_F32 (PKV_KV_Q8_0 is refused).  A token array of H
 *     heads is [total_tokens][H][128] with `*_stride` elements from one token to
 *     the next (at least 128 H, a multiple of 16 bytes); heads are 128 elements
 *     apart.  q, k and v may therefore be slices of one projection's output.
 *   - total_tokens is at most PKV_MAX_CHUNK_TOKENS, num_rows at most
 *     PKV_MAX_ROWS (PKV_ERR_UNSUPPORTED above).
 *   - Each call is queued on `stream` and returns; nothing is allocated and no
 *     stream is synchronised, so every call may be captured into a graph.
 */
#ifndef PKV_CHUNK_H
#define PKV_CHUNK_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_MAX_CHUNK_TOKENS (1 << 22) /* tokens of a chunk call, all rows together */
#define PKV_MAX_ROPE_AXES 4

/* kv_rope_append — rotate a chunk's queries and keys by their positions, and
 * store its keys and values in the rows' pages (as kv_append encodes them).
 * With R = rot_dim, pair u (0 <= u < R/2) of a head turns by the angle
 *     a = positions[axis(u)][token] * inv_freq[u]
 *     x' = x cos a - y sin a,   y' = x sin a + y cos a
 * where (x, y) are the dims (u, u + R/2), or (2u, 2u + 1) with `interleaved`;
 * dims from R on pass through.  axis(u) is 0 for the first sections[0] pairs,
 * 1 for the next sections[1], and so on: positions of several axes (time,
 * height, width of an image or video token) or of one (text).  The angle is
 * reduced in 64 bits, so far positions keep fp32 accuracy; the rotation is
 * fp32 and rounded once, to the output type or the pool's format.
 *   q            [total_tokens][n_q_heads][128] of in_dtype, or NULL with
 *                n_q_heads = 0
 *   k, v         [total_tokens][n_kv_heads][128] of in_dtype
 *   q_out        contiguous [total_tokens][n_q_heads][128] of q_dtype (f16,
 *                bf16 or f32); it may be q itself where q is contiguous and the
 *                types agree, and must not overlap the inputs otherwise
 *   positions    int32 [num_axes][total_tokens]
 *   inv_freq     fp32 [rot_dim / 2]
 *   sections     HOST int [num_axes], positive, summing to rot_dim / 2
 *   rot_dim      a multiple of 16 in [16, 128]
 * No two new tokens of a call may share a page slot.  A skipped row (see
 * above) stores nothing; its queries are rotated all the same while its
 * cu_seqlens entries are valid.  A block-table entry outside the pool records
 * PKV_DEV_BAD_PAGE and its tokens are not stored.  One launch. */
pkv_status kv_rope_append(const pkv_pool *pool, int layer, const void *q, long long q_stride,
                          const void *k, long long k_stride, const void *v, long long v_stride,
                          pkv_kv_dtype in_dtype, void *q_out, pkv_kv_dtype q_dtype,
                          const int32_t *positions, int num_axes, const int *sections,
                          const float *inv_freq, int rot_dim, int interleaved,
                          const int32_t *cu_seqlens, int total_tokens, const int32_t *block_table,
                          int bt_stride, const int32_t *seq_lens, int num_rows, int n_q_heads,
                          void *stream);

/* How scores are formed, for paged_chunk_attention and paged_attention_mass.
 * Query j of row i sits at P = L_i - n_i + j; for token t and query head g of
 * KV head h = g / G,
 *     s = scale * <q[g], K[h][t]>
 *     softcap > 0:     s = softcap * tanh(s / softcap)
 *     slopes != NULL:  s = s - slopes[g] * |P - t|
 * and the query attends to t in [max(0, P + 1 - W), min(L_i, max(P + 1, F))):
 * causal, but within the row's first F = prefix_lens[i] tokens seen from
 * everywhere (prefix_lens NULL: F = 0), and W the layer's sliding window (0:
 * none).  slopes is fp32 [n_q_heads], prefix_lens int32 [num_rows], both on the
 * device; softcap 0 means none, others are 1e-30 to 1e30. */
typedef struct pkv_scores {
    float scale;
    float softcap;
    const float *slopes;
    const int32_t *prefix_lens;
} pkv_scores;

/* paged_chunk_attention — attention of a ragged chunk over the paged cache
 * (the chunk's K and V stored before, by kv_rope_append or kv_append):
 *     out[j][g] = sum_t softmax_t(s) V[h][t],   lse[j][g] = log sum_t exp(s)
 *   q      [total_tokens][n_q_heads][128] of q_dtype, any token stride
 *   out    contiguous [total_tokens][n_q_heads][128] of q_dtype; it must not
 *          overlap q
 *   lse    fp32 [total_tokens][n_q_heads], or NULL
 * q_dtype is f16 on f16 and q8_0 pools and bf16 on bf16 pools; f32 pools are
 * refused (PKV_ERR_UNSUPPORTED; paged_decode_attention_mq serves them).
 * Products accumulate in fp32; the softmax weights are rounded once to
 * q_dtype before they meet V, and the output once.  Skipped rows get zeros
 * and an lse of -inf (rows with invalid cu_seqlens get nothing).  Values of
 * tokens a query does not attend to never reach its output, whatever they
 * are.  Queries that meet a q8_0 value beyond f16's 65504, and those that share
 * a tile with one that attends to a value that is not finite, take a slow path
 * (a hundred times the time, in fp32).  A
 * block-table entry outside the pool records PKV_DEV_BAD_PAGE and page
 * 0 is read instead.
 *   workspace  paged_chunk_workspace_bytes(pool, n_q_heads, num_chunks) bytes,
 *              256-byte aligned; it needs no initialisation and keeps nothing
 *              from call to call.  Calls that may overlap on the GPU (other
 *              streams, graphs replayed together) need one each.
 *   num_chunks the number of pieces the work is split into, one CTA each (0:
 *              one per SM of the current device).
 * Two launches: the attention, and the merge of the (tile, KV head) segments
 * that were split. */
size_t paged_chunk_workspace_bytes(const pkv_pool *pool, int n_q_heads, int num_chunks);

pkv_status paged_chunk_default_chunks(const pkv_pool *pool, int n_q_heads, int *chunks);

pkv_status paged_chunk_attention(const pkv_pool *pool, int layer, const void *q, long long q_stride,
                                 pkv_kv_dtype q_dtype, const int32_t *cu_seqlens, int total_tokens,
                                 const int32_t *block_table, int bt_stride,
                                 const int32_t *seq_lens, int num_rows, int n_q_heads,
                                 const pkv_scores *scores, void *out, float *lse, void *workspace,
                                 size_t workspace_bytes, int num_chunks, void *stream);

/* paged_attention_mass — the attention weight every cached token has received:
 *     mass_out[i][h][t] = mass_in[i][h][t] (t < L_i - n_i, mass_in != NULL; else 0)
 *                         + sum_j sum_{g of h} exp(s - lse[j][g]),   0 <= t < L_i
 * over the row's queries j (the last last_queries of them; 0: all) that attend
 * to t, with the lse that paged_chunk_attention returned for the same scores.
 * New tokens start at 0, so the array needs no clearing between chunks.
 *   mass_in, mass_out  fp32 [num_rows][n_kv_heads][mass_stride], mass_stride >=
 *                      every L_i (a longer row records PKV_DEV_BAD_LENGTH and is
 *                      skipped); entries from L_i on are left as they are;
 *                      mass_in may be mass_out
 *   q, lse, q_dtype    as in paged_chunk_attention
 * Skipped rows are left as they are, all rows where total_tokens is 0.  A
 * query whose lse is not finite adds nothing.  Sums run in a fixed order: equal
 * calls give equal bits.
 *   workspace, num_chunks  as in paged_chunk_attention, of
 *              paged_attention_mass_workspace_bytes(num_chunks) bytes (the
 *              default chunks are those of paged_chunk_default_chunks)
 * Two launches: the sums, and the merge of the tiles that were split. */
size_t paged_attention_mass_workspace_bytes(int num_chunks);

pkv_status paged_attention_mass(const pkv_pool *pool, int layer, const void *q, long long q_stride,
                                pkv_kv_dtype q_dtype, const float *lse, const int32_t *cu_seqlens,
                                int total_tokens, const int32_t *block_table, int bt_stride,
                                const int32_t *seq_lens, int num_rows, int n_q_heads,
                                const pkv_scores *scores, int last_queries, const float *mass_in,
                                float *mass_out, int mass_stride, void *workspace,
                                size_t workspace_bytes, int num_chunks, void *stream);

/* kv_evict — shorten rows to their budget, per KV head, by attention weight.
 * Row i keeps B_i = min(L_i, keep_lens[i]) tokens of each KV head h: the last
 * min(recent, B_i), the first min(first, what is left), and of the others those
 * of largest mass[i][h][t] (ties: the lowest t; NaN counts below every number),
 * in ascending order of t.  keep_idx[i][h][b] receives the b-th kept t, and the
 * token's K and V (all 128 dims, scales included) are copied to slot b of the
 * row's new pages dst_block_table[i]; dst_mass[i][h][b] (unless NULL) receives
 * its weight and new_lens[i] the new length B_i.
 *   mass             fp32 [num_rows][n_kv_heads][mass_stride]
 *   keep_lens        int32 [num_rows]
 *   dst_block_table  int32 [num_rows][dst_bt_stride]: pages that hold no token
 *                    of the call's rows (take them from the allocator first and
 *                    release the old ones after), or, for a row that keeps all
 *                    its tokens, the same pages as before
 *   keep_idx         int32 [num_rows][n_kv_heads][keep_stride]
 *   dst_mass         fp32 [num_rows][n_kv_heads][keep_stride] or NULL; not mass
 *   new_lens         int32 [num_rows], not seq_lens itself
 * keep_lens below 0, a B_i above what keep_stride and dst_bt_stride hold, and
 * rows with L_i < 0 or beyond bt_stride or mass_stride, record
 * PKV_DEV_BAD_LENGTH and are clamped; keep_lens itself may be any budget.
 * Entries and slots behind B_i are left as they are.  Block table entries
 * outside the pool record PKV_DEV_BAD_PAGE; that token is not copied.  The kept
 * tokens of different heads differ, so slots no longer are positions: distance
 * biases, windows and prefixes do not apply to an evicted row; keys rotated
 * before they were stored keep their angles.
 * Two launches. */
pkv_status kv_evict(const pkv_pool *pool, int layer, const float *mass, int mass_stride,
                    const int32_t *block_table, int bt_stride, const int32_t *seq_lens,
                    int num_rows, const int32_t *keep_lens, int first, int recent,
                    const int32_t *dst_block_table, int dst_bt_stride, int32_t *keep_idx,
                    int keep_stride, float *dst_mass, int32_t *new_lens, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_CHUNK_H */
