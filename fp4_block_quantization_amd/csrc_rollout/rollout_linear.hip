// rollout_linear.hip -- products with 4-bit weights and group scales
// (definitions in include/fp4q/rollout.h).
#include "fp4q_device.h"
#include "rollout_launch.h"

namespace fp4q {
namespace {

// One wavefront per output column n of one group: its lanes take the
// column's scale blocks in turn, once per row.
template <bool MX>
__global__ __launch_bounds__(256) void linear_kernel(LinearArgs a) {
  constexpr int BLOCK = MX ? 32 : 16;
  const int64_t n = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int lane = threadIdx.x % 64;
  const int64_t group = blockIdx.y;
  if (n >= a.n) return;
  int64_t first = 0, last = a.rows;
  if (a.offsets) {
    first = min(max(a.offsets[group], (int64_t)0), a.rows);
    last = min(max(a.offsets[group + 1], (int64_t)0), a.rows);
  }
  const int64_t col = group * a.n + n, blocks = a.k / BLOCK;
  const uint8_t* codes = a.codes + col * (a.k / 2);
  const uint8_t* scales = a.scales + col * blocks;
  const float s = MX ? 1.0f : a.row_scales[col];
  for (int64_t m = first; m < last; ++m) {
    const uint16_t* x = (const uint16_t*)a.x + m * a.k;
    float sum = 0.0f;
    for (int64_t b = lane; b < blocks; b += 64) {
      float part = 0.0f;
      for (int i = 0; i < BLOCK / 2; ++i) {
        const uint32_t byte = codes[b * (BLOCK / 2) + i];
        const float lo = e2m1_value(byte & 7u), hi = e2m1_value(byte >> 4 & 7u);
        const float x0 = __uint_as_float((uint32_t)x[b * BLOCK + 2 * i] << 16);
        const float x1 = __uint_as_float((uint32_t)x[b * BLOCK + 2 * i + 1] << 16);
        part = __builtin_fmaf((byte & 8u) ? -lo : lo, x0, part);
        part = __builtin_fmaf((byte & 0x80u) ? -hi : hi, x1, part);
      }
      const float e = MX ? __builtin_ldexpf(1.0f, (int)scales[b] - 127) : e4m3_decode(scales[b]);
      sum = __builtin_fmaf(part, e, sum);
    }
    for (int step = 32; step > 0; step >>= 1) sum += __shfl_xor(sum, step);
    sum *= s;
    if (lane == 0) {
      if (a.out_fp32)
        ((float*)a.out)[m * a.n + n] = sum;
      else
        ((__bf16*)a.out)[m * a.n + n] = (__bf16)sum;
    }
  }
}

}  // namespace

int64_t linear_workspace_bytes(bool, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t linear_launch(bool mx, const LinearArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)((a.n + 3) / 4), (uint32_t)(a.groups ? a.groups : 1));
  if (mx)
    linear_kernel<true><<<grid, 256, 0, stream>>>(a);
  else
    linear_kernel<false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace fp4q
