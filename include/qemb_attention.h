/*
 * qemb_attention.h -- C ABI of libqemb_attention: attention over a paged
 * key-value cache on AMD Instinct MI355X (gfx950), for models that keep
 * their keys and values as the embedding tables keep their rows.
 *
 *  - qemb_norm_rope       norms of queries and keys for each head and the
 *                         position rotation in one pass; keys and values are
 *                         appended to the cache
 *  - qemb_prompt_attention  causal attention of prompts, optionally through a
 *                         sliding window with a few first keys (sinks) that
 *                         stay visible
 *  - qemb_decode_attention  attention of one new token over the cache, split
 *                         over the cache's length and joined; optionally adds
 *                         every key's weight to a running mass
 *  - qemb_evict           keeps a budget of rows by accumulated mass and
 *                         copies them to other pages
 *
 * The cache: two arrays (keys, values) of pages,
 *     [pages][kv_heads][page_size][row],
 * page_size a power of two.  A row is `dim` 16-bit values (bits = 16; the
 * queries' type), or a packed row of qemb.h (bits = 8 or 4; INT8 or INT4
 * codes, fp16 scale and bias, the stride qemb_row_stride(dim, bits)).
 * Slot s of a sequence is row s % page_size of page
 * block_table[sequence][s / page_size]; a flat slot is
 * page * page_size + offset.
 *
 * dim (of one head) is a multiple of 8, 8 .. QEMB_MAX_HEAD_DIM; in the
 * attentions q_heads is a multiple of kv_heads, and query head h reads kv head
 * h / (q_heads / kv_heads).  dtype is that of queries, 16-bit rows, weights
 * and outputs.  Sums, softmax statistics and norms are held in binary32; for
 * the second product of the attentions each key's weight is rounded to the
 * 16-bit type, and over packed rows weight times scale to binary16 (and the
 * query, scaled to a largest element of 1 to 2, too: to at most 2^-25), so that
 * an output is off by up to that rounding of its weights and its own.  The
 * scale of the scores is finite, of any sign.
 *
 * Conventions (those of qemb.h): every array is a device pointer owned by
 * the caller; nothing is allocated, kept or synchronized; work goes onto
 * `stream`; errors that the host can see return before anything is enqueued.
 * Bad device data never faults: it is skipped as stated and, where an
 * err_count (nullable, device, caller-zeroed) is taken, counted.  Calls are
 * deterministic: equal calls give equal bits.  (Another batch size or width of
 * the block table moves the borders at which qemb_decode_attention splits its
 * sums, and with them the last bits.)
 */
#ifndef QEMB_ATTENTION_H
#define QEMB_ATTENTION_H

#include "qemb.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QEMB_DTYPE_BF16 0
#define QEMB_DTYPE_FP16 1

#define QEMB_MAX_HEAD_DIM 256

/*
 * Norm, rotation and append.  For every token t and head, in binary32:
 *     y = (x * rsqrt(mean(x^2) + eps)) * weight
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 * over the pairs (i, i + rot_dim/2) (interleaved = 0) or (2i, 2i+1)
 * (interleaved = 1), i < rot_dim/2, with cos = cos_sin[pos][i] and
 * sin = cos_sin[pos][rot_dim/2 + i], pos = positions[t]; elements from
 * rot_dim on are not rotated.  Values are only copied (or packed).  Packed
 * rows hold the binary32 results encoded by the range rule of qemb.h.
 *   q, k, v     [tokens][heads][dim] of dtype, with strides in elements
 *               between tokens and between heads (multiples of 8; a stride
 *               along one token or one head is not read), dim contiguous,
 *               16-byte aligned; v only with pages
 *   positions   [tokens] of index_type, each in [0, places)
 *   cos_sin     [places][rot_dim] fp32; rot_dim a multiple of 16, <= dim
 *   q_weight, k_weight  [dim] of dtype, or NULL for ones
 *   q_out, k_out  [tokens][heads][dim], contiguous; k_out nullable with pages
 *   k_pages, v_pages  the cache, or both NULL
 *   slots       [tokens] int64 flat slots (distinct); a negative slot writes
 *               nothing to the cache
 * A token whose position leaves [0, places) gives zero rows in q_out and
 * k_out and nothing in the cache; a slot past the cache writes nothing there;
 * each is counted once.  q_heads + 2 kv_heads: at most 2^31 - 1024.
 */
int qemb_norm_rope(const void* q, const void* k, const void* v, int64_t tokens, int32_t q_heads,
                   int32_t kv_heads, int32_t dim, int32_t dtype, int64_t q_token_stride,
                   int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                   int64_t v_token_stride, int64_t v_head_stride, const void* positions,
                   int32_t index_type, const float* cos_sin, int64_t places, int32_t rot_dim,
                   int32_t interleaved, const void* q_weight, const void* k_weight, float eps,
                   void* q_out, void* k_out, void* k_pages, void* v_pages, const int64_t* slots,
                   int64_t pages, int32_t page_size, int32_t bits, int32_t* err_count,
                   qemb_stream_t stream);

/*
 * Attention of prompts.  Sequence b has queries [q_offsets[b],
 * q_offsets[b+1]) and keys [k_offsets[b], k_offsets[b+1]); its last query
 * stands at its last key, so query i of nq stands at p = i + nk - nq and sees
 * key j if j <= p and (window == 0 or j > p - window or j < sinks):
 *     out = sum_j softmax_j(scale q.k_j) v_j,  lse = log sum_j exp(scale q.k_j)
 * A query that sees no key gives zeros and lse = -inf.
 *   q        [q_tokens][q_heads][dim], k, v [k_tokens][kv_heads][dim], strided
 *            as in qemb_norm_rope
 *   q_offsets, k_offsets  [batch + 1] int32
 *   max_q    the longest query run expected (a hint for the grid: longer runs
 *            are still computed); 0 = q_tokens, for every sequence, which
 *            launches batch times as many workgroups as have work
 *   window   0 = unlimited; sinks >= 0, read only with a window
 *   out      [q_tokens][q_heads][dim]; lse [q_tokens][q_heads] fp32, nullable
 * Rows that no sequence covers are left as they are.  A sequence whose
 * offsets decrease or leave the arrays is skipped and counted once.
 * A row whose statistics are finite but whose result is not (an infinity or a
 * NaN among the values it sees, or in a tile beside them) is computed again,
 * one key after another: right, but at a small part of the speed.
 * q_tokens (times q_heads / kv_heads) and k_tokens: at most 2^31 - 1024.
 */
int qemb_prompt_attention(const void* q, const void* k, const void* v, int64_t q_tokens,
                          int64_t k_tokens, int32_t batch, int32_t q_heads, int32_t kv_heads,
                          int32_t dim, int32_t dtype, int64_t q_token_stride, int64_t q_head_stride,
                          int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                          int64_t v_head_stride, const int32_t* q_offsets, const int32_t* k_offsets,
                          int64_t max_q, int32_t window, int32_t sinks, float scale, void* out,
                          float* lse, int32_t* err_count, qemb_stream_t stream);

/*
 * Attention of one new token for each sequence over its cached rows (the
 * token's own row among them, the last): p = seq_lens[b] - 1 in the rule of
 * qemb_prompt_attention.
 *   q            [batch][q_heads][dim], contiguous
 *   k_pages, v_pages  the cache of `pages` pages
 *   block_table  [batch][width] int32; width * page_size (or the window, where
 *                it is less) and batch set the split of the work and the
 *                workspace, whatever the lengths are: a table much wider than
 *                the longest sequence costs both
 *   seq_lens     [batch] int32, each in [0, width * page_size]
 *   mass         [batch][kv_heads][mass_len] fp32 or NULL: mass[b][h][j] grows
 *                by the sum over kv head h's query heads of key j's weight
 *                (mass_len >= every length)
 *   out          [batch][q_heads][dim]; lse [batch][q_heads] fp32, nullable
 *   workspace    qemb_decode_workspace_bytes(...) bytes, 16-byte aligned
 *                (NULL where that is 0); contents need not be kept
 * A sequence of length 0 gives zeros and lse = -inf, and so does one whose
 * length leaves its range, which is counted.  The rows of a page outside
 * [0, pages) are taken as not visible and counted (at least once).
 * width * page_size: at most 2^31 - 1024.
 */
size_t qemb_decode_workspace_bytes(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim,
                                   int32_t width, int32_t page_size, int32_t window, int32_t sinks,
                                   int32_t with_mass);

int qemb_decode_attention(const void* q, const void* k_pages, const void* v_pages, int64_t pages,
                          int32_t page_size, int32_t bits, int32_t batch, int32_t q_heads,
                          int32_t kv_heads, int32_t dim, int32_t dtype, const int32_t* block_table,
                          int32_t width, const int32_t* seq_lens, int32_t window, int32_t sinks,
                          float scale, float* mass, int64_t mass_len, void* out, float* lse,
                          void* workspace, int32_t* err_count, qemb_stream_t stream);

/*
 * Eviction.  For every sequence and kv head of length n: all n slots if
 * n <= keep; else the first `sinks`, the last `recent` and, of those between,
 * the keep - sinks - recent with the largest mass (a NaN counts as -inf; ties
 * go to the lower slot).  Their rows are copied in slot order to slots
 * 0, 1, ... of the new pages, which must not overlap the old ones (they may
 * lie in the same arrays).
 *   k_pages, v_pages, pages, block_table [batch][width], seq_lens  the cache
 *   new_k_pages, new_v_pages, new_pages, new_block_table [batch][new_width]
 *            where the rows go, new_width * page_size >= keep
 *   row_bytes  bytes of one row, a multiple of 16
 *   mass     [batch][kv_heads][mass_len] fp32
 *   keep >= 1, sinks >= 0, recent >= 0, sinks + recent <= keep
 *   kept     [batch][kv_heads][keep] int32: the slots kept, -1 past them
 *   new_mass [batch][kv_heads][new_mass_len] fp32, new_mass_len >= keep: the
 *            kept slots' mass, 0 past them; must not overlap mass
 *   new_lens [batch] int32: min(n, keep)
 * A length outside [0, min(width * page_size, mass_len)] is taken as 0 and
 * counted; a row whose old page lies outside its array is copied as zeros, one
 * whose new page does is not copied; both are counted.
 * min(width * page_size, mass_len): at most 2^31 - 1024.
 */
int qemb_evict(const void* k_pages, const void* v_pages, int64_t pages, int32_t page_size,
               int64_t row_bytes, int32_t batch, int32_t kv_heads, const int32_t* block_table,
               int32_t width, const int32_t* seq_lens, const float* mass, int64_t mass_len,
               int32_t keep, int32_t sinks, int32_t recent, void* new_k_pages, void* new_v_pages,
               int64_t new_pages, const int32_t* new_block_table, int32_t new_width, int32_t* kept,
               float* new_mass, int64_t new_mass_len, int32_t* new_lens, int32_t* err_count,
               qemb_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif
