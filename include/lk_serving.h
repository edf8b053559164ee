/*
 * lk_serving.h -- C ABI of the serving operators beside the latent path
 * (liblk.so, sm_100a): layers whose K and V stay dense, with a paged
 * key-value cache, eviction, 4-bit weights and the norms around a block.
 * The conventions of lk.h hold: device pointers owned by the caller, host
 * validation before anything is launched, asynchronous on `stream`.  (No
 * counterpart on the pages, which cache latents only; the dense
 * flash-decoding the pages compare with is lk_dense_decode_attn.)
 */
#ifndef LK_SERVING_H_
#define LK_SERVING_H_

#include "lk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LK_MAX_PAGE_SIZE 1024

/*
 * Paged key-value cache of one layer (caller-owned device memory).  The pool
 * holds n_pages pages; page i, kv head h is page_size consecutive rows
 *   k, v: [n_pages, n_kv_heads, page_size, head_dim]      dtype
 * dtype LK_BF16, LK_F16, or LK_I8: int8 codes, one fp32 scale per row
 *   k_scale, v_scale: fp32 [n_pages, n_kv_heads, page_size]
 * (value = code * scale; rows quantised with lk_quantize_rows_i8's rule).
 * A cache that is evicted from also has, per row,
 *   mass: fp32 [n_pages, n_kv_heads, page_size]  accumulated attention weight
 *   pos:  int32, same shape                      position the token came at
 * page_size: a power of two, at most LK_MAX_PAGE_SIZE.  head_dim: a multiple
 * of 16, at most LK_MAX_HEAD_DIM.  n_pages * n_kv_heads * page_size < 2^31.
 * All pointers 16-byte aligned.
 *
 * A page table, int32 [batch, table_width] on the device, lists each
 * sequence's pages: slot t of sequence b is row t % page_size of page
 * page_table[b * table_width + t / page_size]; table_width * page_size is at
 * most 2^30.  Entries behind a sequence's last page are not read.  A page may
 * be listed by several sequences for reading; a page that is written (append,
 * mass, eviction) must belong to one sequence and be listed once.  The host
 * cannot check page ids: a kernel that meets one outside [0, n_pages) skips its
 * slots (not attended, written or moved) and lk_device_status() reports
 * LK_ERR_DEVICE.  batch is at least 1 in every call.
 */
typedef struct {
  int32_t n_pages, page_size, n_kv_heads, head_dim;
  lk_dtype dtype;
  void* k;
  void* v;
  float* k_scale; /* LK_I8 only, else NULL                                  */
  float* v_scale;
  float* mass; /* NULL: no attention weights are kept                       */
  int32_t* pos; /* NULL exactly if mass is NULL                             */
} lk_paged_cache;

/*
 * Appends up to n_new tokens to every sequence: token i of sequence b goes to
 * slot seq_len[b] + i, for i < min(max(new_len[b], 0), n_new) (new_len NULL:
 * n_new for all; a padded batch passes its counts).
 * k_new, v_new: x_dtype, token (b, i) at element (b * n_new + i) *
 *   token_stride, [n_kv_heads, head_dim] contiguous there (so K and V may be
 *   views of one QKV projection's output); token_stride a multiple of 8.
 *   x_dtype is the cache's dtype; for an int8 cache LK_BF16 or LK_F16.
 * seq_len_out[b] = seq_len[b] + count (may be seq_len itself).
 * A cache with mass also takes next_pos, int32 [batch], the position of each
 *   sequence's next token: the slots get mass 0 and pos next_pos[b] + i, and
 *   next_pos_out[b] = next_pos[b] + count (may be next_pos itself).  Without
 *   mass, next_pos and next_pos_out are NULL.
 * A sequence whose new tokens do not fit in table_width * page_size slots (or
 * whose seq_len is negative) is left as it is, and lk_device_status()
 * reports LK_ERR_DEVICE.
 * One launch for n_new = 1; longer appends advance the lengths in a second.
 */
lk_status lk_paged_append(const lk_paged_cache* cache, const int32_t* page_table, int32_t batch,
                          int32_t table_width, const void* k_new, const void* v_new, lk_dtype x_dtype,
                          int32_t token_stride, int32_t n_new, const int32_t* new_len,
                          const int32_t* seq_len, int32_t* seq_len_out, const int32_t* next_pos,
                          int32_t* next_pos_out, lk_stream_t stream);

/*
 * Attention of one new token per sequence over its pages: for every query
 * head j, with kv head j / (n_heads / n_kv_heads),
 *   out[b, j] = sum_t p_t v_t,  p = softmax over t < seq_len[b] of
 *   softmax_scale * q[b, j] . k_t.
 * q: LK_BF16 or LK_F16 (the cache's dtype; either for an int8 cache), row
 *   (b, j) at element b * q_stride + j * head_dim; q_stride a multiple of 8.
 * out: [batch, n_heads, head_dim] LK_BF16, LK_F16 or LK_F32, not over q.  A
 *   sequence of length 0, and a head whose every score is -infinity, gives
 *   zeros.
 * seq_len: device int32 [batch], clamped to [0, max_seq_len]; max_seq_len:
 *   host bound, at most table_width * page_size.
 * accumulate != 0 (the cache must have mass): mass of slot t of kv head h
 *   grows by the sum of p_t over the heads of h's group.
 * workspace: lk_paged_decode_workspace_bytes(...) bytes, 256-byte aligned,
 *   any contents; calls that may run at the same time need their own.
 * Scores, softmax statistics and the output sum are fp32; the weights p meet
 *   V as a sum of two 16-bit terms (relative rounding at most 2^-16, fp16 and
 *   int8 caches 2^-22 but not below 2^-35 of their sum), for an LK_F32 out of a
 *   bf16 cache of three (2^-24).  An int8 cache's weights carry their V row's
 *   scale, relative to a power of two of at most twice the largest attended
 *   one: beside a row whose v_scale is 2^35 times theirs, others vanish.
 *   Weights are held at up to 2^4 (fp16 and int8 caches: 2^14), and that times
 *   seq_len |v| has to stay in fp32's range; an infinity in an attended V row
 *   makes its dim NaN.
 *   Results do not depend on timing.  One launch for a max_seq_len of up to
 *   512, or up to min(2048, 24 units) where that is more, else two; a unit is a
 *   sequence, a kv head and up to 8 heads of its group (16 of a larger group up
 *   to head_dim 128).  accumulate: one launch only where the group is one unit.
 */
lk_status lk_paged_decode_attn(const lk_paged_cache* cache, const int32_t* page_table, int32_t batch,
                               int32_t table_width, const void* q, lk_dtype q_dtype, int32_t n_heads,
                               int32_t q_stride, const int32_t* seq_len, int32_t max_seq_len,
                               float softmax_scale, int32_t accumulate, void* out, lk_dtype out_dtype,
                               void* workspace, size_t workspace_bytes, lk_stream_t stream);
size_t lk_paged_decode_workspace_bytes(const lk_paged_cache* cache, int32_t batch, int32_t n_heads,
                                       int32_t max_seq_len, int32_t accumulate);

/*
 * Eviction by accumulated attention weight: every sequence longer than
 * `budget` is cut to its `budget` most wanted tokens, per kv head.  Order:
 * tokens with pos < n_sink or pos >= next_pos[b] - window first, then larger
 * mass, then lower slot (NaN counts as the least mass).  Kept tokens stay
 * where they are if their slot is below `budget`; the i-th kept slot at or
 * above it (ascending) moves into the i-th evicted slot below it (K and V
 * rows, scales, mass, pos), so few rows move and slots are then no longer in
 * order of position.  Pages from ceil(budget / page_size) on are free after
 * the call; the slots moved away from are left as they are.
 * mass_out, pos_out: [n_pages, n_kv_heads, page_size]; the kept slots of every
 *   sequence (all of a short one) are written there.  Either both are the
 *   cache's own arrays or neither is.  seq_len_out[b] = min(seq_len[b],
 *   budget) (may be seq_len itself).
 * Lengths are clamped to [0, max_seq_len] first.  The sequences must not share
 * pages.  budget >= 1; window, n_sink >= 0.
 * workspace: lk_paged_evict_workspace_bytes(...) bytes, 256-byte aligned, any
 *   contents; calls that may run at the same time need their own.
 * Two launches, or one where few rows can move (min(budget, max_seq_len -
 * budget) up to 256) and seq_len_out is not seq_len.
 */
lk_status lk_paged_evict(const lk_paged_cache* cache, const int32_t* page_table, int32_t batch,
                         int32_t table_width, const int32_t* seq_len, const int32_t* next_pos,
                         int32_t max_seq_len, int32_t budget, int32_t window, int32_t n_sink, float* mass_out,
                         int32_t* pos_out, int32_t* seq_len_out, void* workspace, size_t workspace_bytes,
                         lk_stream_t stream);
size_t lk_paged_evict_workspace_bytes(const lk_paged_cache* cache, int32_t batch, int32_t max_seq_len,
                                      int32_t budget);

/*
 * 4-bit weights, laid out once for lk_w4_linear.
 * codes: [n_out, k_in / 2] bytes, two's-complement nibbles, low nibble = even
 *   input (as LK_I4 latents); scales: fp16 [n_out, k_in / group];
 *   W[n, k] = code * scale of k's group.  group 32, 64 or 128; k_in a multiple
 *   of group.  codes 4-byte aligned.
 * up_codes, up_scales: NULL, or the up projection of a gated FFN of the same
 *   sizes; the packed weight then holds gate (codes, scales) and up, and
 *   lk_w4_linear computes silu(gate) * up.
 * packed: lk_w4_packed_bytes(...) bytes, 256-byte aligned.
 */
lk_status lk_w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* up_codes,
                     const uint16_t* up_scales, int32_t n_out, int32_t k_in, int32_t group, void* packed,
                     size_t packed_bytes, lk_stream_t stream);
size_t lk_w4_packed_bytes(int32_t n_out, int32_t k_in, int32_t group, int32_t gated);

/*
 * y = x W^T (+ residual), or silu(x Wg^T) * (x Wu^T) for a gated weight, for
 * the few rows of a decode step (any m >= 0; the weights are read once per 32
 * rows).
 * x: [m, k_in] LK_BF16 or LK_F16, row i at element i * x_stride (a multiple of
 *   8); y: [m, n_out] LK_BF16, LK_F16 or LK_F32, contiguous; residual: NULL or
 *   [m, n_out] of x_dtype, contiguous (may be y if the types are the same);
 *   not with a gated weight.
 * Codes and x enter exact products; sums and scales are fp32 (8 |x| summed over
 * a group, before its scale, has to stay in fp32's range); one rounding to y's
 * type.
 */
lk_status lk_w4_linear(const void* packed, int32_t n_out, int32_t k_in, int32_t group, int32_t gated,
                       const void* x, lk_dtype x_dtype, int32_t m, int32_t x_stride, const void* residual,
                       void* y, lk_dtype y_dtype, lk_stream_t stream);

/*
 * The norms around a block, with its gate and residual scale:
 *   x_out = x + scale * gate . (RMSNorm(y) . w_post)
 *   h     = RMSNorm(x_out) . w_pre
 * RMSNorm(v) = v / sqrt(mean(v^2) + eps).  y, x, x_out, h: [m, width] of
 * `dtype` (LK_BF16, LK_F16 or LK_F32), contiguous.  w_post NULL: y enters as it
 * is; gate NULL: 1; gate_per_row 0: [width], 1: [m, width]; w_pre and h both
 * NULL: no second norm.  Weights and gate of `dtype`.  x_out may be x or y, h
 * may be y.  Everything is fp32 inside (a row's sum of squares has to stay in
 * its range); h is taken from x_out before its rounding.  width <= 32768.
 */
lk_status lk_rmsnorm_gate_residual(const void* y, const void* x, const void* w_post, const void* gate,
                                   int32_t gate_per_row, const void* w_pre, lk_dtype dtype, int32_t m,
                                   int32_t width, float scale, float eps, void* x_out, void* h,
                                   lk_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LK_SERVING_H_ */
