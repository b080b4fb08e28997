/*
 * dlrm_history.h -- C ABI of libdlrm_embbag.so, the encoder of a user's event
 * history: instead of summing the rows of a history bag (dlrm_embbag.h), the
 * events are attended to as a sequence. Four operations:
 *   - norms of queries and keys per head with the position rotation in the same
 *     pass, and its backward (training);
 *   - appending keys and values to a paged cache, the norm and rotation applied
 *     on the way (serving);
 *   - attention of the new tokens of many users over that cache (serving: one new
 *     event, a chunk of a history, or candidates to rank).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *   n        number of tokens of the call, 0 <= n < 2^31; with n == 0 nothing is
 *            written but the weight gradients of the backward, which become zero
 *   dim      elements of a head: 32, 64, 128 or 256
 *   dtype    DLRM_F32, DLRM_F16 or DLRM_BF16; the cache and the attention take the
 *            16-bit types
 *   A tensor of heads [n][heads][dim] is given by its address, the elements from
 *   one token to the next and the elements from one head to the next, so that the
 *   slices of one projection's output are passed as they are; the elements of a
 *   head are contiguous. Addresses are aligned to 16 bytes, strides are multiples
 *   of 16 bytes (any sign, 0 for a broadcast input). Outputs are contiguous.
 *
 * Rotation: rot of the dim elements of a head are rotated, rot a multiple of 16
 * (0: no rotation). Pair j of the rot / 2 pairs is (x[j], x[j + rot / 2]), or
 * (x[2 j], x[2 j + 1]) with interleaved != 0. Its angle is
 *     positions[axis(j)][token] * inv_freq[j]   (radians, formed in fp64),
 * where the first sections[0] pairs follow axis 0, the next sections[1] axis 1
 * and so on (the sections sum to rot / 2), and
 *     (a, b) -> (a cos - b sin, a sin + b cos).
 * Norm: x -> w * x / sqrt(mean(x^2) + eps) over the dim elements of a head, before
 * the rotation; w_q and w_k are fp32 [dim], both NULL for no norm.
 *
 * Paged cache: k_cache and v_cache hold num_pages pages; in a page the heads are
 * cache_head_stride elements apart and each head is [page][dim], contiguous; pages
 * are cache_page_stride elements apart (both caches alike). Entry t of sequence s
 * is in page page_table[s * table_stride + t / page], slot t % page; page is a
 * power of two from 16 to 65536.
 *   q_offsets  device int32 [seqs + 1]: the tokens of sequence s are
 *              q_offsets[s] .. q_offsets[s + 1]. Tokens from q_offsets[seqs] on
 *              belong to no sequence (a padded batch): they are not stored and their
 *              attention outputs are not written.
 *   kv_lens    device int32 [seqs]: entries of the history of each sequence, its
 *              new tokens included; token i of m new ones is entry kv_lens[s] - m + i.
 *
 * Limits (DLRM_E_UNSUPPORTED past them): 65535 heads of queries and keys together; at
 * most 2^31 - 2^17 - 1 sequences, entries of a page table's row (table_width * page)
 * and, in the attention, rows (n * q_heads), with 1024 query heads to a cache head.
 *
 * Pointers, ordering and errors are as in dlrm_embbag.h: the caller owns every
 * buffer, the call only enqueues work on `stream`, argument errors are returned
 * before anything is enqueued. Data errors never make a kernel read or write out
 * of bounds; they OR a bit into *status (device int32, may be NULL):
 *   DLRM_STATUS_BAD_OFFSETS  q_offsets decrease or leave [0, n], or kv_lens is
 *                            negative or passes the page table's width. A sequence
 *                            whose own two offsets decrease, or leave [0, n] or
 *                            [q_offsets[0], q_offsets[seqs]], counts as having no
 *                            tokens; the others keep theirs. Where some of those
 *                            overlap, a token they share is stored for one of them,
 *                            and its attention output is that of one of them. The
 *                            attention clamps a length to [0, table_width * page];
 *                            the append stores no token of a sequence whose length is
 *                            bad, and none that would fall before the first entry (a
 *                            history shorter than its new tokens)
 *   DLRM_STATUS_BAD_PAGE     a page number outside [0, num_pages) where an entry is
 *                            needed: the entry is not stored, or takes no part in the
 *                            attention
 */
#ifndef DLRM_HISTORY_H
#define DLRM_HISTORY_H

#include "dlrm_embbag.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DLRM_MAX_AXES 8
#define DLRM_STATUS_BAD_PAGE 4

/*
 * Norm and rotation of queries and keys, one pass.
 *   q, k         [n][q_heads][dim], [n][kv_heads][dim] of dtype, with strides (elements)
 *   positions    device int32 [axes][n], axes pos_stride elements apart
 *   axes, sections  host: number of axes (1 .. DLRM_MAX_AXES) and the pairs of each
 *   inv_freq     device fp32 [rot / 2] (NULL with rot == 0, like positions)
 *   q_out, k_out device, contiguous [n][heads][dim] of dtype
 * Sums, norms and the rotation are in fp32, rounded once at the end.
 */
int dlrm_qk_norm_rope(int64_t n, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot, int32_t dtype,
                      const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                      int64_t k_head_stride, const int32_t* positions, int64_t pos_stride, int32_t axes,
                      const int32_t* sections, const float* inv_freq, const float* w_q, const float* w_k, float eps,
                      int32_t interleaved, void* q_out, void* k_out, void* stream);

/* Workspace of dlrm_qk_norm_rope_bwd (0 without a norm). */
int dlrm_qk_norm_rope_bwd_workspace_bytes(int64_t n, int32_t dim, int32_t norm, size_t* bytes);

/*
 * Backward of dlrm_qk_norm_rope. With g the gradient turned back by the angles,
 * r = 1 / sqrt(mean(x^2) + eps) and u = x r:
 *     dx = r (g w - u mean(g w u)),   dw = sum over tokens and heads of g u
 * (dx = g without a norm).
 *   d_q_out, d_k_out  gradients of the outputs, [n][heads][dim] of dtype with strides
 *   q, k              the forward's inputs (not read without a norm; then they may be NULL)
 *   d_q, d_k          out, contiguous, of dtype
 *   d_w_q, d_w_k      out, fp32 [dim]; NULL without a norm
 *   workspace         device, 256-byte aligned, dlrm_qk_norm_rope_bwd_workspace_bytes
 * The weight gradients are summed in a fixed order: the same call gives the same bits.
 */
int dlrm_qk_norm_rope_bwd(int64_t n, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot, int32_t dtype,
                          const void* d_q_out, int64_t dq_stride, int64_t dq_head_stride, const void* d_k_out,
                          int64_t dk_stride, int64_t dk_head_stride, const void* q, int64_t q_stride,
                          int64_t q_head_stride, const void* k, int64_t k_stride, int64_t k_head_stride,
                          const int32_t* positions, int64_t pos_stride, int32_t axes, const int32_t* sections,
                          const float* inv_freq, const float* w_q, const float* w_k, float eps, int32_t interleaved,
                          void* d_q, void* d_k, float* d_w_q, float* d_w_k, void* workspace, size_t ws_bytes,
                          void* stream);

/*
 * Appends the keys (normed and rotated) and the values (as they are) of the new
 * tokens to the paged cache, and norms and rotates their queries in the same launch.
 *   q, q_out  may both be NULL (then q_heads is 0 and w_q NULL)
 *   k, v      [n][kv_heads][dim] of dtype (DLRM_F16 or DLRM_BF16), with strides
 * The pages of different sequences must be different where new tokens fall.
 */
int dlrm_kv_append(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot, int32_t dtype,
                   const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                   int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride,
                   const int32_t* positions, int64_t pos_stride, int32_t axes, const int32_t* sections,
                   const float* inv_freq, const float* w_q, const float* w_k, float eps, int32_t interleaved,
                   const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* page_table, int64_t table_stride,
                   int32_t table_width, int32_t page, int64_t num_pages, int64_t cache_page_stride,
                   int64_t cache_head_stride, void* k_cache, void* v_cache, void* q_out, int32_t* status,
                   void* stream);

/* Workspace of dlrm_paged_attn for these sizes (0 where no history is split). */
int dlrm_paged_attn_workspace_bytes(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim,
                                    int32_t causal, int32_t window, int32_t max_q, int32_t max_kv, size_t* bytes);

/*
 * Attention of the new tokens over the paged cache. Head h of q reads head
 * h / (q_heads / kv_heads) of the cache. A token that is entry p of its history sees
 *     all kv_lens[s] entries               causal == 0 (window must be 0)
 *     entries t <= p                       causal != 0, window == 0
 *     entries p - window < t <= p          causal != 0, window > 0
 * and   out = sum_t softmax_t(scale q . k_t) v_t,   lse = log sum_t exp(scale q . k_t)
 * (natural logarithm). A token that sees nothing gets out = 0 and lse = -inf. What an
 * entry holds that a token does not see never reaches that token's result, infinities
 * and NaN included.
 *   q       [n][q_heads][dim] of dtype (DLRM_F16 or DLRM_BF16), with strides
 *   scale   positive and finite, usually dim^-0.5
 *   max_q, max_kv  host: the most new tokens and the longest history of a sequence;
 *           they choose how the work is cut. A larger sequence is still computed
 *           right, only slower.
 *   out     device, contiguous [n][q_heads][dim] of dtype
 *   lse     device fp32 [n][q_heads], or NULL
 *   workspace  device, 256-byte aligned, dlrm_paged_attn_workspace_bytes
 * Products are of the 16-bit values, sums and the softmax in fp32; the weights of the
 * values are rounded to dtype before the second product, the result once at the end.
 */
int dlrm_paged_attn(int64_t n, int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t dtype,
                    const void* q, int64_t q_stride, int64_t q_head_stride, const void* k_cache, const void* v_cache,
                    int32_t page, int64_t num_pages, int64_t cache_page_stride, int64_t cache_head_stride,
                    const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* page_table, int64_t table_stride,
                    int32_t table_width, int32_t causal, int32_t window, float scale, int32_t max_q, int32_t max_kv,
                    void* out, float* lse, void* workspace, size_t ws_bytes, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DLRM_HISTORY_H */
