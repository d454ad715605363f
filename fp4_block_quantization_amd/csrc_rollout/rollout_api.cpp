// rollout_api.cpp -- the C ABI declared in include/fp4q/rollout.h:
// host-side argument validation, then the kernel launches of the call on the
// caller's stream.  Validation touches no HIP API, so a rejected call
// returns its status even on a machine without a GPU.
#include <hip/hip_runtime.h>

#include <cmath>

#include "fp4q/rollout.h"
#include "rollout_launch.h"

namespace {

// Largest sizes accepted: every element count fits in 2^40, every extent
// that a kernel holds in an int in 2^30.
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxDepth = (int64_t)1 << 26;  // 32 rows of weights within 32-bit offsets
constexpr int64_t kMaxExtent = (int64_t)1 << 30;
constexpr int64_t kMaxElements = (int64_t)1 << 40;
constexpr int64_t kMaxGroups = 65535;
constexpr int64_t kMaxSlots = ((int64_t)1 << 31) - 1;
// Attention: a context's positions and a page's value scales are reached by 32-bit offsets.
constexpr int64_t kMaxContext = (int64_t)1 << 30;
constexpr int64_t kMaxPage = (int64_t)1 << 27;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool fits(int64_t a, int64_t b) { return b == 0 || a <= kMaxElements / b; }

fp4q_status launched(hipError_t e) { return e == hipSuccess ? FP4Q_SUCCESS : FP4Q_ERROR_LAUNCH; }

bool linear_shape_ok(int64_t rows, int64_t n, int64_t k, int64_t groups, int64_t block) {
  return rows >= 0 && rows <= kMaxRows && n > 0 && n <= kMaxExtent && k > 0 && k <= kMaxDepth &&
         k % block == 0 && groups >= 0 && groups <= kMaxGroups && fits(rows, k) &&
         fits(rows, n) && fits(n, k) && (groups == 0 || fits(n * k, groups));
}

fp4q_status linear(bool mx, const fp4q::LinearArgs& a, int64_t workspace_bytes, void* stream) {
  if (!linear_shape_ok(a.rows, a.n, a.k, a.groups, mx ? 32 : 16)) return FP4Q_ERROR_INVALID_SHAPE;
  if (a.out_fp32 != 0 && a.out_fp32 != 1) return FP4Q_ERROR_INVALID_ARGUMENT;
  if (a.groups == 0 && a.offsets != nullptr) return FP4Q_ERROR_INVALID_SHAPE;
  if (a.groups > 0 && a.offsets == nullptr) return FP4Q_ERROR_NULL_POINTER;
  if (a.rows == 0) return FP4Q_SUCCESS;
  if (!a.x || !a.codes || !a.scales || !a.out || (!mx && !a.row_scales))
    return FP4Q_ERROR_NULL_POINTER;
  const int64_t need = fp4q::linear_workspace_bytes(mx, a.rows, a.n, a.k, a.groups);
  if (need > 0 && !a.workspace) return FP4Q_ERROR_NULL_POINTER;
  if (!aligned(a.x, 16) || !aligned(a.codes, mx ? 16 : 8) || !aligned(a.row_scales, 4) ||
      !aligned(a.offsets, 8) || !aligned(a.out, a.out_fp32 ? 4 : 2) || !aligned(a.workspace, 16))
    return FP4Q_ERROR_MISALIGNED;
  if (workspace_bytes < need) return FP4Q_ERROR_INVALID_ARGUMENT;
  return launched(fp4q::linear_launch(mx, a, (hipStream_t)stream));
}

fp4q_status check_cache(const fp4q::KvCache& c) {
  if (c.num_pages <= 0 || c.page_size <= 0 || c.page_size % 16 != 0 || c.kv_heads <= 0 ||
      c.head_dim <= 0 || c.head_dim % 16 != 0 || c.head_dim > 512)
    return FP4Q_ERROR_INVALID_SHAPE;
  if (c.page_size > kMaxSlots || c.num_pages > kMaxSlots / c.page_size ||
      c.kv_heads > kMaxGroups || !fits(c.num_pages * c.page_size, c.kv_heads * c.head_dim))
    return FP4Q_ERROR_INVALID_SHAPE;
  return FP4Q_SUCCESS;
}

fp4q_status check_cache_pointers(const fp4q::KvCache& c) {
  for (int i = 0; i < 2; ++i) {
    if (!c.codes[i] || !c.scales[i] || !c.token_scales[i]) return FP4Q_ERROR_NULL_POINTER;
  }
  for (int i = 0; i < 2; ++i) {
    if (!aligned(c.codes[i], 16) || !aligned(c.scales[i], 4) || !aligned(c.token_scales[i], 16))
      return FP4Q_ERROR_MISALIGNED;
  }
  return FP4Q_SUCCESS;
}

fp4q::KvCache cache_of(const uint8_t* kc, const uint8_t* ks, const float* kt, const uint8_t* vc,
                       const uint8_t* vs, const float* vt, int64_t pages, int64_t page,
                       int64_t heads, int64_t dim) {
  return fp4q::KvCache{{(uint8_t*)kc, (uint8_t*)vc},
                       {(uint8_t*)ks, (uint8_t*)vs},
                       {(float*)kt, (float*)vt},
                       pages,
                       page,
                       heads,
                       dim};
}

bool attention_shape_ok(int64_t page_size, int64_t kv_heads, int64_t head_dim, int64_t batch,
                        int64_t q_tokens, int64_t q_heads, int64_t max_pages,
                        int64_t max_prefix_pages, int64_t groups) {
  if (page_size <= 0 || page_size % 16 != 0 || kv_heads <= 0 || batch < 0 || q_tokens < 0 ||
      q_heads <= 0 || max_pages < 0 || max_prefix_pages < 0 || groups < 0)
    return false;
  if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256) return false;
  if (q_heads % kv_heads != 0 || kv_heads > kMaxGroups || q_heads > kMaxExtent / 512) return false;
  if (batch > kMaxGroups || groups > kMaxGroups || q_tokens > kMaxExtent) return false;
  if (page_size > kMaxPage || max_pages > kMaxContext / page_size ||
      max_prefix_pages > kMaxContext / page_size)
    return false;
  // query rows are numbered in 31 bits
  if (q_tokens > 0 && batch * q_heads > kMaxSlots / q_tokens) return false;
  return batch == 0 || q_tokens == 0 ||
         fp4q::kv_attention_fits(page_size, kv_heads, head_dim, batch, q_tokens, q_heads,
                                 max_pages, max_prefix_pages, groups);
}

}  // namespace

extern "C" {

fp4q_status nvfp4_linear(const void* x, int64_t rows, const uint8_t* codes,
                         const uint8_t* block_scales, const float* row_scales, int64_t n,
                         int64_t k, const int64_t* group_offsets, int64_t num_groups,
                         int out_fp32, void* out, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  const fp4q::LinearArgs a{x,          rows,          n,          k,        codes, block_scales,
                           row_scales, group_offsets, num_groups, out_fp32, out,   workspace};
  return linear(false, a, workspace_bytes, stream);
}

int64_t nvfp4_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k, int64_t num_groups) {
  if (!linear_shape_ok(rows, n, k, num_groups, 16) || rows == 0) return 0;
  return fp4q::linear_workspace_bytes(false, rows, n, k, num_groups);
}

fp4q_status mxfp4_linear(const void* x, int64_t rows, const uint8_t* codes,
                         const uint8_t* scales, int64_t n, int64_t k,
                         const int64_t* group_offsets, int64_t num_groups, int out_fp32,
                         void* out, void* workspace, int64_t workspace_bytes, void* stream) {
  const fp4q::LinearArgs a{x,       rows,          n,          k,        codes, scales,
                           nullptr, group_offsets, num_groups, out_fp32, out,   workspace};
  return linear(true, a, workspace_bytes, stream);
}

int64_t mxfp4_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k, int64_t num_groups) {
  if (!linear_shape_ok(rows, n, k, num_groups, 32) || rows == 0) return 0;
  return fp4q::linear_workspace_bytes(true, rows, n, k, num_groups);
}

fp4q_status nvfp4_kv_append(uint8_t* k_codes, uint8_t* k_scales, float* k_token_scales,
                            uint8_t* v_codes, uint8_t* v_scales, float* v_token_scales,
                            int64_t num_pages, int64_t page_size, int64_t kv_heads,
                            int64_t head_dim, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, int64_t tokens, const int64_t* slots,
                            int four_over_six, void* stream) {
  const fp4q::KvCache c = cache_of(k_codes, k_scales, k_token_scales, v_codes, v_scales,
                                   v_token_scales, num_pages, page_size, kv_heads, head_dim);
  fp4q_status st = check_cache(c);
  if (st != FP4Q_SUCCESS) return st;
  if (tokens < 0 || tokens > kMaxRows || k_stride % 8 != 0 || v_stride % 8 != 0 ||
      k_stride < kv_heads * head_dim || v_stride < kv_heads * head_dim || !fits(tokens, k_stride) ||
      !fits(tokens, v_stride))
    return FP4Q_ERROR_INVALID_SHAPE;
  if (four_over_six != 0 && four_over_six != 1) return FP4Q_ERROR_INVALID_ARGUMENT;
  if (tokens == 0) return FP4Q_SUCCESS;
  if ((st = check_cache_pointers(c)) == FP4Q_ERROR_NULL_POINTER || !k || !v || !slots)
    return FP4Q_ERROR_NULL_POINTER;
  if (st != FP4Q_SUCCESS || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return FP4Q_ERROR_MISALIGNED;
  return launched(fp4q::kv_append_launch(c, k, k_stride, v, v_stride, tokens, slots,
                                         four_over_six, (hipStream_t)stream));
}

fp4q_status nvfp4_kv_read(const uint8_t* k_codes, const uint8_t* k_scales,
                          const float* k_token_scales, const uint8_t* v_codes,
                          const uint8_t* v_scales, const float* v_token_scales,
                          int64_t num_pages, int64_t page_size, int64_t kv_heads,
                          int64_t head_dim, const int64_t* slots, int64_t tokens, void* k_out,
                          void* v_out, void* stream) {
  const fp4q::KvCache c = cache_of(k_codes, k_scales, k_token_scales, v_codes, v_scales,
                                   v_token_scales, num_pages, page_size, kv_heads, head_dim);
  fp4q_status st = check_cache(c);
  if (st != FP4Q_SUCCESS) return st;
  if (tokens < 0 || tokens > kMaxRows || !fits(tokens, kv_heads * head_dim))
    return FP4Q_ERROR_INVALID_SHAPE;
  if (tokens == 0) return FP4Q_SUCCESS;
  if ((st = check_cache_pointers(c)) == FP4Q_ERROR_NULL_POINTER || !slots || !k_out || !v_out)
    return FP4Q_ERROR_NULL_POINTER;
  if (st != FP4Q_SUCCESS || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(slots, 8))
    return FP4Q_ERROR_MISALIGNED;
  return launched(
      fp4q::kv_read_launch(c, slots, tokens, k_out, v_out, (hipStream_t)stream));
}

fp4q_status nvfp4_kv_attention(
    const uint8_t* k_codes, const uint8_t* k_scales, const float* k_token_scales,
    const uint8_t* v_codes, const uint8_t* v_scales, const float* v_token_scales,
    int64_t num_pages, int64_t page_size, int64_t kv_heads, int64_t head_dim, const void* q,
    int64_t q_stride, int64_t batch, int64_t q_tokens, int64_t q_heads, const int32_t* page_table,
    int64_t max_pages, const int32_t* seq_lens, const int32_t* prefix_table,
    int64_t max_prefix_pages, const int32_t* prefix_lens, const int32_t* group_offsets,
    int64_t groups, float scale, void* out, float* lse, void* workspace, int64_t workspace_bytes,
    void* stream) {
  const fp4q::KvCache c = cache_of(k_codes, k_scales, k_token_scales, v_codes, v_scales,
                                   v_token_scales, num_pages, page_size, kv_heads, head_dim);
  fp4q_status st = check_cache(c);
  if (st != FP4Q_SUCCESS) return st;
  if (!attention_shape_ok(page_size, kv_heads, head_dim, batch, q_tokens, q_heads, max_pages,
                          max_prefix_pages, groups) ||
      q_stride % 8 != 0 || q_stride < q_heads * head_dim || !fits(batch * q_tokens, q_stride))
    return FP4Q_ERROR_INVALID_SHAPE;
  if (groups == 0 && (max_prefix_pages != 0 || prefix_table || prefix_lens || group_offsets))
    return FP4Q_ERROR_INVALID_SHAPE;
  if (!std::isfinite(scale)) return FP4Q_ERROR_INVALID_ARGUMENT;
  if (batch == 0 || q_tokens == 0) return FP4Q_SUCCESS;
  const int64_t need = fp4q::kv_attention_workspace_bytes(
      page_size, kv_heads, head_dim, batch, q_tokens, q_heads, max_pages, max_prefix_pages, groups);
  if ((st = check_cache_pointers(c)) == FP4Q_ERROR_NULL_POINTER || !q || !seq_lens || !out ||
      (max_pages > 0 && !page_table) || (groups > 0 && (!prefix_lens || !group_offsets)) ||
      (max_prefix_pages > 0 && !prefix_table) || (need > 0 && !workspace))
    return FP4Q_ERROR_NULL_POINTER;
  if (st != FP4Q_SUCCESS || !aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(prefix_table, 4) || !aligned(prefix_lens, 4) ||
      !aligned(group_offsets, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
    return FP4Q_ERROR_MISALIGNED;
  if (workspace_bytes < need) return FP4Q_ERROR_INVALID_ARGUMENT;
  const fp4q::AttentionArgs a{q,           q_stride,         batch,        q_tokens,
                              q_heads,     page_table,       max_pages,    seq_lens,
                              prefix_table, max_prefix_pages, prefix_lens, group_offsets,
                              groups,      scale,            out,          lse,
                              workspace};
  return launched(fp4q::kv_attention_launch(c, a, (hipStream_t)stream));
}

int64_t nvfp4_kv_attention_workspace_bytes(int64_t page_size, int64_t kv_heads, int64_t head_dim,
                                           int64_t batch, int64_t q_tokens, int64_t q_heads,
                                           int64_t max_pages, int64_t max_prefix_pages,
                                           int64_t groups) {
  if (!attention_shape_ok(page_size, kv_heads, head_dim, batch, q_tokens, q_heads, max_pages,
                          max_prefix_pages, groups) ||
      batch == 0 || q_tokens == 0)
    return 0;
  return fp4q::kv_attention_workspace_bytes(page_size, kv_heads, head_dim, batch, q_tokens,
                                            q_heads, max_pages, max_prefix_pages, groups);
}

}  // extern "C"
