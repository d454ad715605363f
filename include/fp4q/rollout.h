/*
 * rollout.h -- C ABI of the operators a 4-bit rollout engine runs between
 * the quantizer's calls (library libfp4q_rollout.so, gfx950):
 *
 *   nvfp4_linear, mxfp4_linear  products with 4-bit weights and group scales
 *   nvfp4_kv_append             keys and values quantized as they are written
 *                               to a paged cache
 *   nvfp4_kv_read               BF16 values of cached rows
 *   nvfp4_kv_attention          softmax attention over that cache, with an
 *                               optional prefix shared by groups of sequences
 *
 * The conventions of fp4q.h hold here as well: device pointers on the
 * stream's device, row-major tensors, asynchronous calls that validate on
 * the host first and launch kernels only, nothing allocated and nothing
 * kept between calls.  A call's scratch memory is the caller's workspace, of
 * at least the size that the call's *_workspace_bytes function returns for
 * the same sizes; its contents on entry are ignored, and calls in flight at
 * the same time must not share one.  For equal inputs and sizes the results
 * are equal bit for bit (no floating-point atomics).
 */
#ifndef FP4Q_ROLLOUT_H
#define FP4Q_ROLLOUT_H

#include "../fp4q.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * nvfp4_linear -- y = x . DQ(W)^T for NVFP4 weights (the outputs of
 * nvfp4_quantize for W): y[m][j] = s_j * sum_i x[m][i] * (+-g(code) * e),
 * products of exact values summed in FP32, rounded once to the output type.
 *
 *   x             BF16 [rows, k], 16-byte aligned.
 *   codes         uint8 [n, k/2] ([num_groups, n, k/2] with groups), 8-byte
 *                 aligned; block_scales uint8 [.., n, k/16] (E4M3FN);
 *                 row_scales float [.., n], 4-byte aligned.
 *   rows          >= 0 (0: nothing is launched); n > 0; k > 0, a multiple of 16, up to 2^26;
 *                 rows and n up to 2^30, and every tensor's elements up to 2^40.
 *   group_offsets NULL, or int64 [num_groups + 1] on the device, 8-byte
 *                 aligned, non-decreasing, within [0, rows]: the rows
 *                 [off[e], off[e+1]) are multiplied with expert e's matrix;
 *                 rows outside [off[0], off[num_groups]) keep their output's
 *                 contents.  Not checked on the host; each range is clamped
 *                 to [0, rows).
 *   num_groups    0 when group_offsets is NULL, else 1 ... 65535.
 *   out_fp32      0: out is BF16 [rows, n], 2-byte aligned; 1: float [rows, n],
 *                 4-byte aligned.  Other values: FP4Q_ERROR_INVALID_ARGUMENT.
 *   workspace     16-byte aligned, workspace_bytes long (may be NULL where
 *                 nvfp4_linear_workspace_bytes returns 0); too short:
 *                 FP4Q_ERROR_INVALID_ARGUMENT.
 */
FP4Q_API fp4q_status nvfp4_linear(const void* x, int64_t rows, const uint8_t* codes,
                                  const uint8_t* block_scales, const float* row_scales,
                                  int64_t n, int64_t k, const int64_t* group_offsets,
                                  int64_t num_groups, int out_fp32, void* out, void* workspace,
                                  int64_t workspace_bytes, void* stream);
FP4Q_API int64_t nvfp4_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k,
                                              int64_t num_groups);

/*
 * mxfp4_linear -- the same product for MXFP4 weights (the primary codes and
 * scales of mxfp4_resq_quantize): w = +-g(code) * 2^(byte - 127).
 *
 *   codes   uint8 [.., n, k/2], 16-byte aligned; scales uint8 [.., n, k/32]
 *           (E8M0): every byte is that power of two, 255 too, also where the
 *           weight itself lies beyond FP32.
 *   k       a multiple of 32, up to 2^26.  Everything else: as for nvfp4_linear.
 */
FP4Q_API fp4q_status mxfp4_linear(const void* x, int64_t rows, const uint8_t* codes,
                                  const uint8_t* scales, int64_t n, int64_t k,
                                  const int64_t* group_offsets, int64_t num_groups, int out_fp32,
                                  void* out, void* workspace, int64_t workspace_bytes,
                                  void* stream);
FP4Q_API int64_t mxfp4_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k,
                                              int64_t num_groups);

/*
 * The paged NVFP4 cache.  One cache row is the head_dim elements of one
 * token and head, quantized as nvfp4_quantize quantizes a row (E2M1 codes,
 * E4M3 scale per 16 elements, one FP32 scale).  Token slot p * page_size + o
 * is place o of page p:
 *   k_codes, v_codes  uint8 [num_pages, kv_heads, page_size, head_dim/2], 16-byte aligned
 *   k_scales          uint8 [num_pages, kv_heads, page_size, head_dim/16], 4-byte aligned
 *   v_scales          uint8 [num_pages, kv_heads, head_dim/16, page_size], 4-byte aligned:
 *                     token innermost, as the value product reads them
 *   k_token_scales, v_token_scales  float [num_pages, kv_heads, page_size], 16-byte aligned
 * num_pages > 0, page_size a positive multiple of 16, kv_heads in
 * 1 ... 65535, head_dim a multiple of 16 up to 512; num_pages * page_size below 2^31.
 */

/*
 * nvfp4_kv_append -- quantize tokens' keys and values into their slots.
 *
 *   k, v      BF16, token t's [kv_heads, head_dim] rows at element
 *             t * k_stride (v_stride): 16-byte aligned, strides multiples
 *             of 8 and at least kv_heads * head_dim (a slice of a fused
 *             projection is taken as it lies).
 *   tokens    >= 0, up to 2^30.
 *   slots     int64 [tokens] on the device, 8-byte aligned; a slot outside
 *             [0, num_pages * page_size) skips its token (padding: -1).  A
 *             slot given twice holds one of the tokens' rows or a mixture.
 *   four_over_six  1 or 0, as for nvfp4_quantize.
 */
FP4Q_API fp4q_status nvfp4_kv_append(uint8_t* k_codes, uint8_t* k_scales, float* k_token_scales,
                                     uint8_t* v_codes, uint8_t* v_scales, float* v_token_scales,
                                     int64_t num_pages, int64_t page_size, int64_t kv_heads,
                                     int64_t head_dim, const void* k, int64_t k_stride,
                                     const void* v, int64_t v_stride, int64_t tokens,
                                     const int64_t* slots, int four_over_six, void* stream);

/*
 * nvfp4_kv_read -- the BF16 values of cached rows, as nvfp4_dequantize
 * gives them: k_out, v_out BF16 [tokens, kv_heads, head_dim], 16-byte
 * aligned.  A slot outside the cache reads as zeros.
 */
FP4Q_API fp4q_status nvfp4_kv_read(const uint8_t* k_codes, const uint8_t* k_scales,
                                   const float* k_token_scales, const uint8_t* v_codes,
                                   const uint8_t* v_scales, const float* v_token_scales,
                                   int64_t num_pages, int64_t page_size, int64_t kv_heads,
                                   int64_t head_dim, const int64_t* slots, int64_t tokens,
                                   void* k_out, void* v_out, void* stream);

/*
 * nvfp4_kv_attention -- softmax(scale * q . K^T) . V over cached tokens.
 *
 * Sequence b's keys are, in order, the prefix of its group (if it is in
 * one) and its own seq_lens[b] tokens.  Its q_tokens queries are its last
 * own tokens: query i sees the whole prefix and the first
 * seq_lens[b] - q_tokens + 1 + i own tokens (none if that is below 1).
 * Query head h reads cache head h / (q_heads / kv_heads).  A query that
 * sees nothing gives zeros, and a log-sum-exp of -infinity.  Keys and values
 * are the exact g * e * s; scores and softmax sums are held in FP32.  Queries
 * enter in FP16 relative to their row's largest element (below 2^-39 of it
 * they count as zero).  Weights, the probabilities times the values' token
 * scales, enter the value product in FP16 relative to the query's largest:
 * those below 2^-23 of it may be lost (where a batch's token scales lie more
 * than 2^100 apart, or scores beyond 2^22, below 2^-23 of the largest scale).
 * Scores up to 2^96 are told apart as FP32 does.  A query that sees a token
 * whose value scale is infinite or NaN gives NaN; others are not touched by it.
 * A NaN among the block scales (nvfp4_kv_append writes none) may reach the
 * queries of its 64 tokens' group that do not see it.
 *
 *   q           BF16: query i of sequence b has its [q_heads, head_dim] rows
 *               at element (b * q_tokens + i) * q_stride; 16-byte aligned,
 *               q_stride a multiple of 8, at least q_heads * head_dim.
 *   q_heads     a positive multiple of kv_heads; head_dim 64, 128, 192 or 256.
 *   batch, q_tokens >= 0 (nothing is launched if either is 0); batch and groups up to 65535,
 *               batch * q_tokens * q_heads below 2^31.
 *   page_size   up to 2^27; max_pages and max_prefix_pages times page_size up to 2^30.
 *               Where contexts are cut into parts (with groups, and for few sequences whose
 *               tables have room for more than 2048 tokens) the room of all tables, in tiles of
 *               64 tokens, times the blocks of 16 or 32 query rows and cache head that read it,
 *               below 2^31.  Beyond these limits: FP4Q_ERROR_INVALID_SHAPE.
 *   page_table  int32 [batch, max_pages] on the device: page of the token
 *               o is page_table[b][o / page_size]; seq_lens int32 [batch],
 *               clamped to [0, max_pages * page_size].  Entries past a
 *               sequence's end are not used; page ids are clamped to the cache.
 *   groups      0 (the four prefix arguments NULL, max_prefix_pages 0), or
 *               the number of groups: sequences [group_offsets[g],
 *               group_offsets[g+1]) share the prefix_lens[g] tokens of the
 *               pages prefix_table[g] (int32 [groups, max_prefix_pages];
 *               lengths clamped likewise).  group_offsets int32 [groups + 1]
 *               on the device, non-decreasing within [0, batch] (clamped);
 *               sequences outside it have no prefix.
 *   scale       the score factor (usually 1/sqrt(head_dim)); finite.
 *   out         BF16 [batch, q_tokens, q_heads, head_dim], 16-byte aligned.
 *   lse         float [batch, q_tokens, q_heads], the natural log-sum-exp of
 *               the scaled scores; or NULL.
 *   workspace   16-byte aligned, as for nvfp4_linear.
 * int32 arrays are 4-byte aligned.
 */
FP4Q_API fp4q_status nvfp4_kv_attention(
    const uint8_t* k_codes, const uint8_t* k_scales, const float* k_token_scales,
    const uint8_t* v_codes, const uint8_t* v_scales, const float* v_token_scales,
    int64_t num_pages, int64_t page_size, int64_t kv_heads, int64_t head_dim, const void* q,
    int64_t q_stride, int64_t batch, int64_t q_tokens, int64_t q_heads, const int32_t* page_table,
    int64_t max_pages, const int32_t* seq_lens, const int32_t* prefix_table,
    int64_t max_prefix_pages, const int32_t* prefix_lens, const int32_t* group_offsets,
    int64_t groups, float scale, void* out, float* lse, void* workspace, int64_t workspace_bytes,
    void* stream);
FP4Q_API int64_t nvfp4_kv_attention_workspace_bytes(int64_t page_size, int64_t kv_heads,
                                                    int64_t head_dim, int64_t batch,
                                                    int64_t q_tokens, int64_t q_heads,
                                                    int64_t max_pages, int64_t max_prefix_pages,
                                                    int64_t groups);

#ifdef __cplusplus
}
#endif
#endif /* FP4Q_ROLLOUT_H */
