// rollout_launch.h -- internal launchers behind include/fp4q/rollout.h.
// Arguments reaching these have already been validated on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q/rollout.h"

namespace fp4q {

struct LinearArgs {
  const void* x;
  int64_t rows, n, k;
  const uint8_t* codes;
  const uint8_t* scales;    // E4M3 per 16 (NVFP4) or E8M0 per 32 (MXFP4)
  const float* row_scales;  // NVFP4 only
  const int64_t* offsets;
  int64_t groups;
  int out_fp32;
  void* out;
  void* workspace;
};

int64_t linear_workspace_bytes(bool mx, int64_t rows, int64_t n, int64_t k, int64_t groups);
hipError_t linear_launch(bool mx, const LinearArgs& a, hipStream_t stream);

struct KvCache {
  uint8_t* codes[2];  // keys, values
  uint8_t* scales[2];
  float* token_scales[2];
  int64_t num_pages, page_size, kv_heads, head_dim;
};

hipError_t kv_append_launch(const KvCache& c, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, int64_t tokens, const int64_t* slots,
                            int four_over_six, hipStream_t stream);
hipError_t kv_read_launch(const KvCache& c, const int64_t* slots, int64_t tokens, void* k_out,
                          void* v_out, hipStream_t stream);

struct AttentionArgs {
  const void* q;
  int64_t q_stride, batch, q_tokens, q_heads;
  const int32_t* page_table;
  int64_t max_pages;
  const int32_t* seq_lens;
  const int32_t* prefix_table;
  int64_t max_prefix_pages;
  const int32_t* prefix_lens;
  const int32_t* group_offsets;
  int64_t groups;
  float scale;
  void* out;
  float* lse;
  void* workspace;
};

// Whether a call's workgroups and the tiles that its tables have room for are counted in 31
// bits, as the kernels count them.
bool kv_attention_fits(int64_t page_size, int64_t kv_heads, int64_t head_dim, int64_t batch,
                       int64_t q_tokens, int64_t q_heads, int64_t max_pages,
                       int64_t max_prefix_pages, int64_t groups);
int64_t kv_attention_workspace_bytes(int64_t page_size, int64_t kv_heads, int64_t head_dim,
                                     int64_t batch, int64_t q_tokens, int64_t q_heads,
                                     int64_t max_pages, int64_t max_prefix_pages, int64_t groups);
hipError_t kv_attention_launch(const KvCache& c, const AttentionArgs& a, hipStream_t stream);

}  // namespace fp4q
