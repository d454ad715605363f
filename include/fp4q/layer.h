/*
 * layer.h -- C ABI of the operators that stand between the 4-bit products, the
 * cache and the attention of rollout.h in a layer of a rollout engine (library
 * libfp4q_rollout.so, gfx950):
 *
 *   rotary_embed      rotary positions of queries and keys
 *   prompt_attention  causal attention of packed prompts or chunks in BF16
 *   moe_route         scores of experts: the best of a token, and their weights
 *   moe_dispatch      tokens' rows ordered by expert, with the row offsets that
 *                     nvfp4_linear and mxfp4_linear take
 *   moe_combine       the experts' rows back to their tokens, weighted
 *
 * The conventions of rollout.h hold here as well: device pointers on the
 * stream's device, row-major tensors, asynchronous calls that validate on the
 * host first and launch kernels only, nothing allocated and nothing kept
 * between calls, scratch memory in a caller's workspace that calls in flight
 * at the same time must not share, results equal bit for bit from call to call.
 */
#ifndef FP4Q_LAYER_H
#define FP4Q_LAYER_H

#include "../fp4q.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * rotary_embed -- rotary positions.  Pair i of the first `dims` elements of a
 * head, (x[i], x[i + dims/2]) or, interleaved, (x[2i], x[2i + 1]), is turned by
 * the angle a = positions[t] * frequencies[i] and scaled:
 *   (u, v) -> amplitude * (u cos a - v sin a, v cos a + u sin a)
 * and by -a with inverse = 1 (the transposed map, so also the gradient; with
 * amplitude 1 it undoes the turn).  Elements from dims on are copied.  Sines and
 * cosines are those of the exact product within 2^-23, for angles up to 2^70
 * radians; products are FP32, rounded once to the tensors' type.
 *
 *   q, k          token t's [heads, head_dim] rows at element t * stride
 *                 (a slice of a fused projection is taken as it lies);
 *                 k_heads 0: k, k_out may be NULL.  fp32 0: BF16, 1: float.
 *                 Strides at least heads * head_dim.
 *   q_out, k_out  likewise.  An output may be its input (same stride: turned in
 *                 place); otherwise outputs must not overlap inputs.
 *   tokens        0 ... 2^30 (0: nothing is launched); q_heads 1 ... 65535,
 *                 k_heads 0 ... 65535; head_dim 1 ... 65536; dims even, 2 ... head_dim;
 *                 tokens times a stride up to 2^40.
 *   positions     int64 [tokens], 8-byte aligned; |position| below 2^53.
 *   frequencies   double [dims/2], radians a position, 8-byte aligned; finite.
 *   amplitude     finite.
 * Pointers are aligned to an element (16-byte aligned ones with dims/2,
 * head_dim and strides in whole 16 bytes are read and written 16 bytes at a
 * time).
 */
FP4Q_API fp4q_status rotary_embed(const void* q, int64_t q_stride, int64_t q_heads, const void* k,
                                  int64_t k_stride, int64_t k_heads, int64_t tokens,
                                  int64_t head_dim, int64_t dims, const int64_t* positions,
                                  const double* frequencies, float amplitude, int interleaved,
                                  int inverse, int fp32, void* q_out, int64_t q_out_stride,
                                  void* k_out, int64_t k_out_stride, void* stream);

/*
 * prompt_attention -- softmax(scale * q . K^T) . V, causal, over packed
 * sequences: sequence b has the queries [q_offsets[b], q_offsets[b + 1]) and
 * the keys [k_offsets[b], k_offsets[b + 1]); its queries are the last of its
 * keys, so that with m queries and n keys query i sees the keys up to
 * n - m + i (none, if that is negative).  Query head h reads key head
 * h / (q_heads / kv_heads).  A query that sees nothing gives zeros, and a
 * log-sum-exp of -infinity; so does one whose visible scores are all
 * -infinity, where the values it sees are finite.  Rows outside [q_offsets[0], q_offsets[batch]) are left as they
 * are.  Scores, maxima, sums and outputs are held in FP32; probabilities
 * enter the value product in BF16, relative to the row's largest (up to 2^12
 * of an earlier largest, so that 2^12 times the sum of a row's values has to
 * stay within FP32), and are divided by their sum as rounded; the log-sum-exp
 * takes them before rounding.  Keys and values that a query does not see have no
 * effect on any bit of it, infinities and NaN among them; a value that is not
 * finite, where a query sees it with a score above -infinity, makes that element
 * of its output infinite or NaN (with one of -infinity, that or nothing).
 *
 *   q            BF16: token t's [q_heads, head_dim] rows at element t * q_stride.
 *   k, v         BF16 [.., kv_heads, head_dim] rows likewise.  16-byte aligned,
 *                strides multiples of 8, at least heads * head_dim, up to 2^24.
 *   q_tokens     rows of q (and out), k_tokens rows of k and v: 0 ... 2^30.  Keys
 *                are cut into parts by k_tokens / batch, so of a long buffer
 *                pass the rows in use.
 *   q_heads      a positive multiple of kv_heads (up to 65535); head_dim 64,
 *                128, 192 or 256; q_tokens * (q_heads / kv_heads) and
 *                q_tokens * q_heads / 32 + batch * kv_heads below 2^31.
 *   q_offsets,   int32 [batch + 1] on the device, 4-byte aligned, non-decreasing
 *   k_offsets    within [0, q_tokens] and [0, k_tokens] (clamped); k_offsets may
 *                be q_offsets.
 *   batch        0 ... 65535.
 *   scale        finite, up to 2^100 in magnitude.
 *   out          BF16 [q_tokens, q_heads, head_dim], 16-byte aligned.
 *   lse          float [q_tokens, q_heads], the natural log-sum-exp of the
 *                scaled scores; or NULL.
 *   workspace    16-byte aligned, at least prompt_attention_workspace_bytes
 *                long (may be NULL where that is 0).
 */
FP4Q_API fp4q_status prompt_attention(const void* q, int64_t q_stride, int64_t q_tokens,
                                      int64_t q_heads, const void* k, int64_t k_stride,
                                      const void* v, int64_t v_stride, int64_t k_tokens,
                                      int64_t kv_heads, int64_t head_dim, const int32_t* q_offsets,
                                      const int32_t* k_offsets, int64_t batch, float scale,
                                      void* out, float* lse, void* workspace,
                                      int64_t workspace_bytes, void* stream);
FP4Q_API int64_t prompt_attention_workspace_bytes(int64_t q_tokens, int64_t q_heads,
                                                  int64_t k_tokens, int64_t kv_heads,
                                                  int64_t head_dim, int64_t batch);

/*
 * moe_route -- the top_k experts of every token and their weights.
 *
 *   score   softmax of a token's logits over all experts (scoring 0) or the
 *           sigmoid of each (scoring 1)
 *   key     score + bias[expert]; without a bias the logit itself (the scores'
 *           order, unrounded).  The bias has no part in the weights.
 *   groups  above 1: experts are in that many equal groups of neighbours, a
 *           group's mark is the sum of the two largest keys in it (without a
 *           bias: scores; of the one, in groups of one), and only the experts
 *           of the top_groups groups with the largest marks can be chosen
 *   chosen  the top_k largest keys, in falling order; of equal keys or marks
 *           the lower index comes first
 *   weight  the chosen score, with renormalize divided by the sum of the chosen
 *           scores (0 where all their logits are -infinity), times scale; renormalized
 *           weights are formed relative to the largest, so that scores below
 *           FP32's range keep their shares
 *
 * Keys with a bias, and marks, are formed in FP64 and compared to 42 bits behind
 * the leading one.  A NaN key ranks behind every other, and the weights of a
 * token with a NaN logit may be NaN; the chosen experts are always distinct and
 * in range.  A token whose logits are all -infinity has weights of 0.
 *
 *   logits   BF16 (fp32 0) or float (1) [tokens, experts], aligned to an element.
 *   tokens   0 ... 2^30; experts 1 ... 1024; top_k 1 ... 64, at most
 *            top_groups * experts / groups; groups 1 ... 64, dividing experts;
 *            top_groups 1 ... groups.
 *   bias     float [experts], or NULL; finite.
 *   active   uint8 [tokens], or NULL: tokens whose byte is 0 (a batch's
 *            padding) have the experts -1 and weights 0.
 *   scale    finite.
 *   weights  float [tokens, top_k]; chosen int32 [tokens, top_k].
 */
FP4Q_API fp4q_status moe_route(const void* logits, int fp32, int64_t tokens, int64_t experts,
                               int64_t top_k, const float* bias, int scoring, int64_t groups,
                               int64_t top_groups, int renormalize, float scale,
                               const uint8_t* active, float* weights, int32_t* chosen,
                               void* stream);

/*
 * moe_dispatch -- every token's row once for each of its experts, ordered by
 * expert, then token, then choice: rows[place[t][j]] = x[t] for the expert
 * chosen[t][j], and expert e's rows are [offsets[e], offsets[e + 1]).  A chosen
 * expert outside [0, experts) (padding: -1) gets no row and the place -1; rows
 * from offsets[experts] on are left as they are.
 *
 *   x          BF16 [tokens, hidden]; rows BF16 [tokens * top_k, hidden]; 2-byte
 *              aligned (16-byte aligned with hidden a multiple of 8: moved 16
 *              bytes at a time).  hidden 1 ... 2^30.
 *   chosen     int32 [tokens, top_k]; top_k 1 ... 64; tokens >= 0, tokens *
 *              top_k below 2^31; experts 1 ... 1024.
 *   offsets    int64 [experts + 1], 8-byte aligned (written also for no
 *              tokens); place int32 [tokens, top_k].
 *   workspace  16-byte aligned, moe_dispatch_workspace_bytes long at least (may
 *              be NULL where that is 0).
 */
FP4Q_API fp4q_status moe_dispatch(const void* x, int64_t tokens, int64_t hidden,
                                  const int32_t* chosen, int64_t top_k, int64_t experts,
                                  void* rows, int64_t* offsets, int32_t* place, void* workspace,
                                  int64_t workspace_bytes, void* stream);
FP4Q_API int64_t moe_dispatch_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts);

/*
 * moe_combine -- out[t] = add[t] + sum over j of weights[t][j] * y[place[t][j]],
 * summed in FP32 in that order and rounded once.  A place outside [0, y_rows)
 * adds nothing, whatever its weight.
 *
 *   y        BF16 (y_fp32 0) or float (1) [y_rows, n]; place, weights [tokens, top_k].
 *   add      BF16 [tokens, n], or NULL (a residual, or a shared expert's output);
 *            may be out, if that is BF16.
 *   out      BF16 (out_fp32 0) or float (1) [tokens, n].
 *   tokens   0 ... 2^30; top_k 1 ... 64; n 1 ... 2^30; y_rows below 2^31.
 * Aligned to an element (all 16-byte aligned with n a multiple of 8: read and
 * written 8 elements at a time).
 */
FP4Q_API fp4q_status moe_combine(const void* y, int y_fp32, int64_t y_rows, const int32_t* place,
                                 const float* weights, const void* add, int64_t tokens,
                                 int64_t top_k, int64_t n, int out_fp32, void* out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4Q_LAYER_H */
