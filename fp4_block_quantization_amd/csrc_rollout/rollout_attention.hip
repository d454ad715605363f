// rollout_attention.hip -- softmax attention over the paged NVFP4 cache,
// with a prefix shared by groups of sequences (definitions in
// include/fp4q/rollout.h).
#include "fp4q_device.h"
#include "rollout_launch.h"

namespace fp4q {
namespace {

__device__ __forceinline__ int32_t clamp_id(int32_t v, int64_t count) {
  return v < 0 ? 0 : v >= count ? (int32_t)(count - 1) : v;
}

// One wavefront per query row, one token at a time: the scores' running
// maximum m and sum l, and the value sum, rescaled when m grows.
template <int D>
__global__ __launch_bounds__(64) void attention_kernel(KvCache c, AttentionArgs a) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x;
  const int64_t head = blockIdx.x % a.q_heads, bt = blockIdx.x / a.q_heads;
  const int64_t b = bt / a.q_tokens, i = bt - b * a.q_tokens;
  const int64_t kvh = head / (a.q_heads / c.kv_heads);
  float q[E], o[E];
  for (int j = 0; j < E; ++j) {
    const uint16_t* src = (const uint16_t*)a.q + bt * a.q_stride + head * D;
    q[j] = __uint_as_float((uint32_t)src[lane * E + j] << 16) * a.scale;
    o[j] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  auto run = [&](const int32_t* table, int64_t count) {
    for (int64_t t = 0; t < count; ++t) {
      const int64_t page = clamp_id(table[t / c.page_size], c.num_pages), at = t % c.page_size;
      const int64_t ph = page * c.kv_heads + kvh, row = ph * c.page_size + at;
      float dot = 0.0f, v[E];
      for (int j = 0; j < E; ++j) {
        const int64_t el = row * D + lane * E + j;
        const int block = (lane * E + j) / 16;
        const float ke = e4m3_decode(c.scales[0][row * (D / 16) + block]) * c.token_scales[0][row];
        const float ve = e4m3_decode(c.scales[1][(ph * (D / 16) + block) * c.page_size + at]) *
                         c.token_scales[1][row];
        const uint32_t kq = c.codes[0][el / 2] >> (4 * (el & 1)) & 15u;
        const uint32_t vq = c.codes[1][el / 2] >> (4 * (el & 1)) & 15u;
        const float kg = e2m1_value(kq & 7u), vg = e2m1_value(vq & 7u);
        dot = __builtin_fmaf(q[j], ((kq & 8u) ? -kg : kg) * ke, dot);
        v[j] = ((vq & 8u) ? -vg : vg) * ve;
      }
      for (int step = 32; step > 0; step >>= 1) dot += __shfl_xor(dot, step);
      const float top = fmaxf(m, dot), keep = expf(m - top), p = expf(dot - top);
      l = l * keep + p;
      for (int j = 0; j < E; ++j) o[j] = o[j] * keep + p * v[j];
      m = top;
    }
  };
  for (int64_t g = 0; g < a.groups; ++g) {
    const int64_t lo = max(a.group_offsets[g], 0), hi = a.group_offsets[g + 1];
    if (b >= lo && b < hi) {
      run(a.prefix_table + g * a.max_prefix_pages,
          min((int64_t)max(a.prefix_lens[g], 0), a.max_prefix_pages * c.page_size));
      break;
    }
  }
  const int64_t len = min((int64_t)max(a.seq_lens[b], 0), a.max_pages * c.page_size);
  run(a.page_table + b * a.max_pages, max(len - a.q_tokens + 1 + i, (int64_t)0));
  for (int j = 0; j < E; ++j)
    ((__bf16*)a.out)[(int64_t)blockIdx.x * D + lane * E + j] =
        (__bf16)(l == 0.0f ? 0.0f : o[j] / l);
  if (a.lse && lane == 0) a.lse[blockIdx.x] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

int64_t kv_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                                     int64_t, int64_t, int64_t) {
  return 0;
}

hipError_t kv_attention_launch(const KvCache& c, const AttentionArgs& a, hipStream_t stream) {
  const uint32_t grid = (uint32_t)(a.batch * a.q_tokens * a.q_heads);
  switch (c.head_dim) {
    case 64: attention_kernel<64><<<grid, 64, 0, stream>>>(c, a); break;
    case 128: attention_kernel<128><<<grid, 64, 0, stream>>>(c, a); break;
    case 192: attention_kernel<192><<<grid, 64, 0, stream>>>(c, a); break;
    case 256: attention_kernel<256><<<grid, 64, 0, stream>>>(c, a); break;
  }
  return hipGetLastError();
}

}  // namespace fp4q
