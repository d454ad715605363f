// layer_launch.h -- internal launchers behind include/fp4q/layer.h.
// Arguments reaching these have already been validated on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q/layer.h"

namespace fp4q {

struct RotaryArgs {
  const void* in[2];  // queries, keys
  void* out[2];
  int64_t in_stride[2], out_stride[2], heads[2];
  int64_t tokens, head_dim, dims;
  const int64_t* positions;
  const double* frequencies;
  float amplitude;
  bool interleaved, inverse, fp32;
};
hipError_t rotary_launch(const RotaryArgs& a, hipStream_t stream);

struct PromptArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int64_t q_tokens, k_tokens, q_heads, kv_heads, head_dim;
  const int32_t *q_offsets, *k_offsets;
  int64_t batch;
  float scale;
  void* out;
  float* lse;
  void* workspace;
};
int64_t prompt_workspace_bytes(int64_t q_tokens, int64_t q_heads, int64_t k_tokens,
                               int64_t kv_heads, int64_t head_dim, int64_t batch);
hipError_t prompt_launch(const PromptArgs& a, hipStream_t stream);

struct RouteArgs {
  const void* logits;
  bool fp32;
  int64_t tokens, experts, top_k;
  const float* bias;
  bool sigmoid;
  int64_t groups, top_groups;
  bool renormalize;
  float scale;
  const uint8_t* active;
  float* weights;
  int32_t* chosen;
};
hipError_t route_launch(const RouteArgs& a, hipStream_t stream);

struct DispatchArgs {
  const void* x;
  int64_t tokens, hidden;
  const int32_t* chosen;
  int64_t top_k, experts;
  void* rows;
  int64_t* offsets;
  int32_t* place;
  void* workspace;
};
int64_t dispatch_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts);
hipError_t dispatch_launch(const DispatchArgs& a, hipStream_t stream);

struct CombineArgs {
  const void* y;
  bool y_fp32;
  int64_t y_rows;
  const int32_t* place;
  const float* weights;
  const void* add;
  int64_t tokens, top_k, n;
  bool out_fp32;
  void* out;
};
hipError_t combine_launch(const CombineArgs& a, hipStream_t stream);

}  // namespace fp4q
