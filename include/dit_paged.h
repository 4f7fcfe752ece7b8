/*
 * dit_paged.h -- C ABI of the operators that serve new tokens over a paged
 * key/value cache, next to the per-token operators of dit_token.h: rotary
 * positions scaled for long contexts, the same on the way into the cache, and
 * attention of a chunk of new tokens over it.
 *
 * A streamed video or a prompt reaches a block in chunks: each chunk's q, k
 * and v rows are packed like every other operator's rows (cu_seqlens,
 * cu_seqlens_padded), its keys and values join the ones that earlier chunks
 * left in the cache, and its queries attend over all of them.  A chunk of one
 * row per sequence is the step that generates single tokens.
 *
 * The conventions of dit_token.h hold (types, pointers, strides, packing,
 * stream, launches, errors), and:
 * Cache       k_cache and v_cache are bf16 pages of page_size tokens.  Head h
 *             of slot s of page g starts at g * page_stride + s * slot_stride
 *             + h * head_stride elements and holds head_dim contiguous
 *             elements; both caches share the strides (multiples of 8), so
 *             [page][slot][head][D] and [page][head][slot][D] are both fine,
 *             and offsets may pass 32 bits.
 * Table       block_table[b * table_stride + i] (device, int32) is the page of
 *             tokens i * page_size .. (i + 1) * page_size - 1 of sequence b,
 *             i < max_pages.  Entries past a sequence's tokens are never read.
 *             The table is trusted but never followed out of bounds: a token
 *             whose entry lies outside [0, num_pages) or past max_pages is
 *             not written by dit_qkv_rope_append; dit_paged_attention reads
 *             zeros as the key and value of a token on such a page, and
 *             never looks past max_pages * page_size tokens.
 * Sharing     pages may be shared between sequences that only read them.  Two
 *             calls that write one token's slot, or write and read it, must be
 *             ordered by the caller (one stream is enough).
 */
#ifndef DIT_PAGED_H
#define DIT_PAGED_H

#include "dit_token.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Frequencies of the rotary pairs, scaled for contexts longer than the ones a
 * model was trained on.  Host only: fills freqs[rotary_dim / 2] (HOST doubles;
 * the caller copies them to the device once) and *attn_scale, the factor on
 * cos and sin.  With f_j = theta^(-2j / R), R = rotary_dim and s = factor >= 1:
 *   NONE    f_j
 *   LINEAR  f_j / s                          (positions compressed s times)
 *   NTK     theta replaced by theta * s^(R / (R - 2))   (R > 2; else f_j)
 *   YARN    f_j / s * r_j + f_j * (1 - r_j), r_j = clamp((j - lo) / max(hi - lo, 0.001), 0, 1),
 *           lo = max(floor(d(beta_fast)), 0), hi = min(ceil(d(beta_slow)), R - 1),
 *           d(t) = R ln(L / (2 pi t)) / (2 ln theta), L = original_len;
 *           *attn_scale = 0.1 ln s + 1       (Peng et al., "YaRN: Efficient Context
 *           Window Extension of Large Language Models", 2023)
 * *attn_scale is 1 but for YARN.  original_len, beta_fast and beta_slow (32
 * and 1 there) are read by YARN only, which needs theta > 1 and
 * 0 < beta_slow <= beta_fast.  rotary_dim: even, > 0 (a table for
 * the calls below needs their rotary_dim; tables of grid sections are built
 * section by section and put one behind the other). */
#define DIT_ROPE_SCALE_NONE 0
#define DIT_ROPE_SCALE_LINEAR 1
#define DIT_ROPE_SCALE_NTK 2
#define DIT_ROPE_SCALE_YARN 3
DIT_API dit_status dit_rope_frequencies(int32_t rotary_dim, double theta, int32_t scaling, double factor,
                                        int64_t original_len, double beta_fast, double beta_slow, double* freqs,
                                        float* attn_scale);

/* Rotary positions of q and k from a table of frequencies, over the first
 * rotary_dim elements of every head, behind an optional per-head RMSNorm.
 *
 * For every valid row and head, with weights
 *   y = x * rsqrt(mean(x^2) + eps) * w       (mean over the whole head)
 * and without (both weights NULL) y = x; then pair j < rotary_dim / 2, whose
 * elements are (2j, 2j + 1) (DIT_ROPE_INTERLEAVED) or (j, j + rotary_dim / 2)
 * (DIT_ROPE_HALF), turns:
 *   (o_a, o_b) = attn_scale * (y_a cos - y_b sin, y_a sin + y_b cos)
 * and elements rotary_dim .. head_dim - 1 keep y (without weights bit for
 * bit).  The angle is p * freqs[j], p = pos_offset[b] + the row's index within
 * its sequence (pos_offset NULL: 0; a negative entry is read as 0); formed
 * and reduced in fp64, so far positions keep their precision.  With rope_grid,
 * rows that lie inside the sequence's T x H x W grid (index p, as in
 * dit_qk_rmsnorm_rope_shard) turn by their t, h or w coordinate times
 * grid_freqs[j]: the first sec_t / 2 pairs are t, the next sec_h / 2 h, the
 * rest w; later rows are 1D, counted from the end of the grid.
 * DIT_ROPE_NONE turns nothing (tables, grid and offsets are ignored).
 *
 * q, k          device bf16, as in dit_qk_rmsnorm_rope (q may be NULL when
 *               num_q_heads is 0, k when num_k_heads is 0)
 * q_out, k_out  where the results go, own row strides; NULL: in place (the
 *               stride is ignored).  Exact aliasing of q_out and q (k_out and
 *               k) is in place too
 * freqs         device fp64 [rotary_dim / 2]; grid_freqs likewise (NULL
 *               without rope_grid); 16-byte aligned
 * rotary_dim    a multiple of 8, 8 <= rotary_dim <= head_dim
 * sec_*         even, >= 0, summing to rotary_dim when rope_grid != NULL
 * head_dim      64, 128 or 256 (else DIT_ERR_UNSUPPORTED)
 */
DIT_API dit_status dit_qk_rope_scaled(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                      void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                      const void* q_weight, const void* k_weight, const int32_t* cu_seqlens,
                                      const int32_t* cu_seqlens_padded, int32_t num_seqs, int64_t num_rows_padded,
                                      int32_t num_q_heads, int32_t num_k_heads, int32_t head_dim,
                                      const double* freqs, int32_t rotary_dim, const int32_t* rope_grid,
                                      const double* grid_freqs, int32_t sec_t, int32_t sec_h, int32_t sec_w,
                                      const int32_t* pos_offset, float attn_scale, float eps, int32_t rope_mode,
                                      void* stream);

/* dit_qk_rope_scaled on the way into a paged cache, in one launch: q as above
 * (to q_out, or in place), k normed and turned into its slots of k_cache, v
 * copied bit for bit into the same slots of v_cache.  Row r of sequence b is
 * the sequence's token cache_lens[b] + r.
 *
 * k, v          device bf16 rows of num_kv_heads heads; read only (neither may
 *               overlap the caches)
 * cache_lens    device int32 [num_seqs]: tokens of each sequence already in the
 *               cache (a negative entry is read as 0); not written -- the caller
 *               advances them, e.g. into the kv_lens of dit_paged_attention
 * pos_offset    rotary position of each sequence's first row; NULL: cache_lens
 * Two rows of one call never share a slot unless the table names one page
 * twice; which of them stays is then not defined.  Slots that no row of the
 * call goes to keep their bits. */
DIT_API dit_status dit_qkv_rope_append(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                       const void* v, int64_t v_row_stride, void* q_out, int64_t q_out_stride,
                                       const void* q_weight, const void* k_weight, void* k_cache, void* v_cache,
                                       int64_t page_stride, int64_t slot_stride, int64_t head_stride,
                                       int32_t num_pages, int32_t page_size, const int32_t* block_table,
                                       int64_t table_stride, int32_t max_pages, const int32_t* cache_lens,
                                       const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded, int32_t num_seqs,
                                       int64_t num_rows_padded, int32_t num_q_heads, int32_t num_kv_heads,
                                       int32_t head_dim, const double* freqs, int32_t rotary_dim,
                                       const int32_t* rope_grid, const double* grid_freqs, int32_t sec_t,
                                       int32_t sec_h, int32_t sec_w, const int32_t* pos_offset, float attn_scale,
                                       float eps, int32_t rope_mode, void* stream);

/* Attention of a chunk of new tokens over a paged cache that holds them.
 *
 * Sequence b has n = cu_seqlens[b + 1] - cu_seqlens[b] queries and kv_lens[b]
 * cached tokens, the last n of which are the chunk's own (append first).
 * Query i sits at position p = kv_lens[b] - n + i and sees the tokens j with
 *   j <= p (causal != 0) or j < kv_lens[b] (causal == 0), and
 *   j > p - window (window > 0; 0 is no window).
 * q head h reads key head h / (num_q_heads / num_kv_heads):
 *   o = sum_j softmax_j(softmax_scale * q . k_j) v_j,  lse = ln sum_j exp(softmax_scale * q . k_j)
 * A query that sees nothing (kv_lens[b] < n, or 0) gives o = 0, lse = -inf.
 * Scores, softmax and sums are fp32; the probabilities are rounded to bf16
 * for their product with v, and o once more to bf16.
 * The slots of tokens >= kv_lens[b] may hold anything, and so may those of
 * tokens that lie before every query's window (their pages may be given
 * away, their table entries be stale or none).  The other cached tokens must be
 * finite, also those a mask hides from some of the queries (a hidden value is
 * multiplied by 0).
 * A chunk kernel whose copies or products do not end within about two seconds
 * (a device fault) gives up: the rows it was computing become NaN in out and in
 * lse; the call itself has returned by then.
 * The result does not depend on what else is in the batch's buffers, and is
 * bitwise reproducible for the same call.
 *
 * q, out        device bf16 [num_rows_padded][num_q_heads * head_dim], own row strides; out
 *               must not overlap q or the caches
 * lse           device fp32 [num_rows_padded][num_q_heads], contiguous, or NULL
 * kv_lens       device int32 [num_seqs]; a negative entry is read as 0
 * num_q_heads   a multiple of num_kv_heads
 * softmax_scale finite, > 0 (usually 1 / sqrt(head_dim))
 * max_pages     max_pages * page_size at most 2^31 - 4097 (else DIT_ERR_UNSUPPORTED)
 * max_chunk     longest chunk of the batch, max_kv_len the longest kv_lens, where the
 *               host knows them (<= 0: num_rows_padded, max_pages * page_size).
 *               They choose kernels and how the key axis is split; the result
 *               is right whatever they say.  A captured call that is replayed
 *               with growing kv_lens gives the largest it will see.
 * workspace     device memory of at least dit_paged_attention_workspace bytes for
 *               the same sizes, 16-byte aligned (NULL if that is 0), used by this
 *               call only until it has run: calls that may run at the same time
 *               (on two streams, or in two graphs) need one each.  Too
 *               small: DIT_ERR_SHAPE.
 */
DIT_API dit_status dit_paged_attention(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                                       int64_t page_stride, int64_t slot_stride, int64_t head_stride,
                                       int32_t num_pages, int32_t page_size, const int32_t* block_table,
                                       int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                                       const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded, int32_t num_seqs,
                                       int64_t num_rows_padded, int32_t num_q_heads, int32_t num_kv_heads,
                                       int32_t head_dim, float softmax_scale, int32_t causal, int32_t window,
                                       int64_t max_chunk, int64_t max_kv_len, void* out, int64_t out_row_stride,
                                       float* lse, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that dit_paged_attention wants for these sizes, under
 * any window and mask (host only; *bytes may be 0).  max_chunk as above;
 * max_kv_len > 0 (the capacity max_pages * page_size where the call passes
 * none; a call with a smaller max_kv_len and the same other sizes is served
 * by the same workspace). */
DIT_API dit_status dit_paged_attention_workspace(int64_t num_rows_padded, int32_t num_seqs, int32_t num_q_heads,
                                                 int32_t num_kv_heads, int32_t head_dim, int64_t max_chunk,
                                                 int64_t max_kv_len, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* DIT_PAGED_H */
