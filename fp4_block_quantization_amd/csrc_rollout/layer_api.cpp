// layer_api.cpp -- the C ABI declared in include/fp4q/layer.h: host-side
// argument validation, then the kernel launches of the call on the caller's
// stream.  Validation touches no HIP API, so a rejected call returns its
// status even on a machine without a GPU.
#include <hip/hip_runtime.h>

#include <cmath>

#include "fp4q/layer.h"
#include "layer_launch.h"

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxElements = (int64_t)1 << 40;
constexpr int64_t kMaxInt = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxHeads = 65535;
constexpr int64_t kMaxStride = (int64_t)1 << 24;  // 64 rows of keys within 32-bit offsets
constexpr int64_t kMaxExperts = 1024, kMaxChoices = 64, kMaxExpertGroups = 64;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool fits(int64_t a, int64_t b) { return b == 0 || a <= kMaxElements / b; }

bool within(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

bool flag(int v) { return v == 0 || v == 1; }

fp4q_status launched(hipError_t e) { return e == hipSuccess ? FP4Q_SUCCESS : FP4Q_ERROR_LAUNCH; }

bool prompt_shape_ok(int64_t q_tokens, int64_t q_heads, int64_t k_tokens, int64_t kv_heads,
                     int64_t head_dim, int64_t batch) {
  if (!within(q_tokens, 0, kMaxRows) || !within(k_tokens, 0, kMaxRows) ||
      !within(kv_heads, 1, kMaxHeads) || !within(q_heads, 1, kMaxHeads) ||
      !within(batch, 0, kMaxHeads))
    return false;
  if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256) return false;
  // query rows of a key head, and workgroups, are numbered in 31 bits
  return q_heads % kv_heads == 0 &&
         (q_tokens == 0 || q_heads / kv_heads <= kMaxInt / q_tokens) &&
         q_tokens * q_heads / 32 + batch * kv_heads <= kMaxInt;
}

}  // namespace

extern "C" {

fp4q_status rotary_embed(const void* q, int64_t q_stride, int64_t q_heads, const void* k,
                         int64_t k_stride, int64_t k_heads, int64_t tokens, int64_t head_dim,
                         int64_t dims, const int64_t* positions, const double* frequencies,
                         float amplitude, int interleaved, int inverse, int fp32, void* q_out,
                         int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  if (!within(tokens, 0, kMaxRows) || !within(q_heads, 1, kMaxHeads) ||
      !within(k_heads, 0, kMaxHeads) || !within(head_dim, 1, 65536) ||
      !within(dims, 2, head_dim) || dims % 2 != 0)
    return FP4Q_ERROR_INVALID_SHAPE;
  for (int64_t s : {q_stride, q_out_stride})
    if (s < q_heads * head_dim || !fits(tokens, s)) return FP4Q_ERROR_INVALID_SHAPE;
  for (int64_t s : {k_stride, k_out_stride})
    if (k_heads > 0 && (s < k_heads * head_dim || !fits(tokens, s)))
      return FP4Q_ERROR_INVALID_SHAPE;
  if (!flag(interleaved) || !flag(inverse) || !flag(fp32) || !std::isfinite(amplitude))
    return FP4Q_ERROR_INVALID_ARGUMENT;
  if (tokens == 0) return FP4Q_SUCCESS;
  if (!q || !q_out || !positions || !frequencies || (k_heads > 0 && (!k || !k_out)))
    return FP4Q_ERROR_NULL_POINTER;
  const uintptr_t size = fp32 ? 4 : 2;
  if (!aligned(q, size) || !aligned(q_out, size) || !aligned(positions, 8) ||
      !aligned(frequencies, 8) || (k_heads > 0 && (!aligned(k, size) || !aligned(k_out, size))))
    return FP4Q_ERROR_MISALIGNED;
  if ((q == q_out && q_stride != q_out_stride) ||
      (k_heads > 0 && k == k_out && k_stride != k_out_stride))
    return FP4Q_ERROR_INVALID_ARGUMENT;
  const fp4q::RotaryArgs a{{q, k},      {q_out, k_out}, {q_stride, k_stride},
                           {q_out_stride, k_out_stride}, {q_heads, k_heads},
                           tokens,      head_dim,       dims,
                           positions,   frequencies,    amplitude,
                           interleaved != 0, inverse != 0, fp32 != 0};
  return launched(fp4q::rotary_launch(a, (hipStream_t)stream));
}

fp4q_status prompt_attention(const void* q, int64_t q_stride, int64_t q_tokens, int64_t q_heads,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             int64_t k_tokens, int64_t kv_heads, int64_t head_dim,
                             const int32_t* q_offsets, const int32_t* k_offsets, int64_t batch,
                             float scale, void* out, float* lse, void* workspace,
                             int64_t workspace_bytes, void* stream) {
  if (!prompt_shape_ok(q_tokens, q_heads, k_tokens, kv_heads, head_dim, batch))
    return FP4Q_ERROR_INVALID_SHAPE;
  if (q_stride < q_heads * head_dim || q_stride > kMaxStride || q_stride % 8 != 0 ||
      !fits(q_tokens, q_stride))
    return FP4Q_ERROR_INVALID_SHAPE;
  for (int64_t s : {k_stride, v_stride})
    if (s < kv_heads * head_dim || s > kMaxStride || s % 8 != 0 || !fits(k_tokens, s))
      return FP4Q_ERROR_INVALID_SHAPE;
  if (!(std::fabs(scale) <= 0x1p100f)) return FP4Q_ERROR_INVALID_ARGUMENT;
  if (batch == 0 || q_tokens == 0) return FP4Q_SUCCESS;
  const int64_t need =
      fp4q::prompt_workspace_bytes(q_tokens, q_heads, k_tokens, kv_heads, head_dim, batch);
  if (!q || !q_offsets || !k_offsets || !out || (k_tokens > 0 && (!k || !v)) ||
      (need > 0 && !workspace))
    return FP4Q_ERROR_NULL_POINTER;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(q_offsets, 4) || !aligned(k_offsets, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return FP4Q_ERROR_MISALIGNED;
  if (workspace_bytes < need) return FP4Q_ERROR_INVALID_ARGUMENT;
  const fp4q::PromptArgs a{q,        k,        v,       q_stride,  k_stride,  v_stride, q_tokens,
                           k_tokens, q_heads,  kv_heads, head_dim, q_offsets, k_offsets, batch,
                           scale,    out,      lse,     workspace};
  return launched(fp4q::prompt_launch(a, (hipStream_t)stream));
}

int64_t prompt_attention_workspace_bytes(int64_t q_tokens, int64_t q_heads, int64_t k_tokens,
                                         int64_t kv_heads, int64_t head_dim, int64_t batch) {
  if (!prompt_shape_ok(q_tokens, q_heads, k_tokens, kv_heads, head_dim, batch) || batch == 0 ||
      q_tokens == 0)
    return 0;
  return fp4q::prompt_workspace_bytes(q_tokens, q_heads, k_tokens, kv_heads, head_dim, batch);
}

fp4q_status moe_route(const void* logits, int fp32, int64_t tokens, int64_t experts,
                      int64_t top_k, const float* bias, int scoring, int64_t groups,
                      int64_t top_groups, int renormalize, float scale, const uint8_t* active,
                      float* weights, int32_t* chosen, void* stream) {
  if (!within(tokens, 0, kMaxRows) || !within(experts, 1, kMaxExperts) ||
      !within(groups, 1, kMaxExpertGroups) || experts % groups != 0 ||
      !within(top_groups, 1, groups) || !within(top_k, 1, kMaxChoices) ||
      top_k > experts / groups * top_groups)
    return FP4Q_ERROR_INVALID_SHAPE;
  if (!flag(fp32) || !flag(scoring) || !flag(renormalize) || !std::isfinite(scale))
    return FP4Q_ERROR_INVALID_ARGUMENT;
  if (tokens == 0) return FP4Q_SUCCESS;
  if (!logits || !weights || !chosen) return FP4Q_ERROR_NULL_POINTER;
  if (!aligned(logits, fp32 ? 4 : 2) || !aligned(bias, 4) || !aligned(weights, 4) ||
      !aligned(chosen, 4))
    return FP4Q_ERROR_MISALIGNED;
  const fp4q::RouteArgs a{logits,     fp32 != 0,   tokens, experts, top_k,   bias,
                          scoring == 1, groups,    top_groups, renormalize != 0, scale,
                          active,     weights,     chosen};
  return launched(fp4q::route_launch(a, (hipStream_t)stream));
}

fp4q_status moe_dispatch(const void* x, int64_t tokens, int64_t hidden, const int32_t* chosen,
                         int64_t top_k, int64_t experts, void* rows, int64_t* offsets,
                         int32_t* place, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  if (!within(tokens, 0, kMaxRows) || !within(hidden, 1, kMaxRows) ||
      !within(top_k, 1, kMaxChoices) || !within(experts, 1, kMaxExperts) ||
      tokens > kMaxInt / top_k || !fits(tokens * top_k, hidden))
    return FP4Q_ERROR_INVALID_SHAPE;
  const int64_t need = fp4q::dispatch_workspace_bytes(tokens, top_k, experts);
  if (!offsets || (tokens > 0 && (!x || !chosen || !rows || !place)) || (need > 0 && !workspace))
    return FP4Q_ERROR_NULL_POINTER;
  if (!aligned(x, 2) || !aligned(chosen, 4) || !aligned(rows, 2) || !aligned(offsets, 8) ||
      !aligned(place, 4) || !aligned(workspace, 16))
    return FP4Q_ERROR_MISALIGNED;
  if (workspace_bytes < need) return FP4Q_ERROR_INVALID_ARGUMENT;
  const fp4q::DispatchArgs a{x,    tokens,  hidden, chosen,   top_k, experts,
                             rows, offsets, place,  workspace};
  return launched(fp4q::dispatch_launch(a, (hipStream_t)stream));
}

int64_t moe_dispatch_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts) {
  if (!within(tokens, 0, kMaxRows) || !within(top_k, 1, kMaxChoices) ||
      !within(experts, 1, kMaxExperts) || tokens > kMaxInt / top_k)
    return 0;
  return fp4q::dispatch_workspace_bytes(tokens, top_k, experts);
}

fp4q_status moe_combine(const void* y, int y_fp32, int64_t y_rows, const int32_t* place,
                        const float* weights, const void* add, int64_t tokens, int64_t top_k,
                        int64_t n, int out_fp32, void* out, void* stream) {
  if (!within(tokens, 0, kMaxRows) || !within(y_rows, 0, kMaxInt) ||
      !within(top_k, 1, kMaxChoices) || !within(n, 1, kMaxRows) || !fits(tokens, n) ||
      !fits(y_rows, n))
    return FP4Q_ERROR_INVALID_SHAPE;
  if (!flag(y_fp32) || !flag(out_fp32)) return FP4Q_ERROR_INVALID_ARGUMENT;
  if (tokens == 0) return FP4Q_SUCCESS;
  if (!out || !place || !weights || (y_rows > 0 && !y)) return FP4Q_ERROR_NULL_POINTER;
  if (!aligned(y, y_fp32 ? 4 : 2) || !aligned(add, 2) || !aligned(out, out_fp32 ? 4 : 2) ||
      !aligned(place, 4) || !aligned(weights, 4))
    return FP4Q_ERROR_MISALIGNED;
  if (out_fp32 && add == out) return FP4Q_ERROR_INVALID_ARGUMENT;
  const fp4q::CombineArgs a{y,      y_fp32 != 0, y_rows, place, weights, add,
                            tokens, top_k,       n,      out_fp32 != 0, out};
  return launched(fp4q::combine_launch(a, (hipStream_t)stream));
}

}  // extern "C"
