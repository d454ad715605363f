// rollout_cache.hip -- writing and reading the paged NVFP4 key/value cache
// (layout and definitions in include/fp4q/rollout.h).
//
// A cache row (one token, one head) is quantized exactly as nvfp4_quantize
// quantizes a row of head_dim elements: s = amax / C, per 16-element block
// and candidate k in {6, 4}: e = E4M3(b / (k s)), codes E2M1(|x| / (e s)),
// values g e s, the candidate with the lower squared error.  Every step is
// one IEEE binary32 operation, in the definition's order, so the cache holds
// the very bytes that nvfp4_quantize gives for the same rows.
//
// Both kernels only move data: one lane per 16-element block, a row's
// blocks in neighbouring lanes, so a wavefront reads (or writes) 2 KiB of
// consecutive BF16 and as many consecutive codes as the rows allow.
#include "fp4q_device.h"
#include "rollout_launch.h"

namespace fp4q {
namespace {

struct CacheView {
  uint8_t* codes[2];
  uint8_t* scales[2];
  float* token_scales[2];
  int64_t slots;  // num_pages * page_size
  int32_t page_size, heads, blocks;  // blocks: head_dim / 16
};

CacheView view_of(const KvCache& c) {
  CacheView v;
  for (int i = 0; i < 2; ++i) {
    v.codes[i] = c.codes[i];
    v.scales[i] = c.scales[i];
    v.token_scales[i] = c.token_scales[i];
  }
  v.slots = c.num_pages * c.page_size;
  v.page_size = (int32_t)c.page_size;
  v.heads = (int32_t)c.kv_heads;
  v.blocks = (int32_t)(c.head_dim / 16);
  return v;
}

struct Place {
  int64_t row;       // index of the cache row: codes at row * d/2, scale at row
  int64_t key_byte;  // of this lane's block scale in k_scales
  int64_t val_byte;  // and in v_scales
};

__device__ __forceinline__ Place place_of(const CacheView& c, uint32_t slot, int head, int block) {
  const uint32_t page = slot / (uint32_t)c.page_size, at = slot - page * (uint32_t)c.page_size;
  const int64_t ph = (int64_t)page * c.heads + head;
  Place p;
  p.row = ph * c.page_size + at;
  p.key_byte = p.row * c.blocks + block;
  p.val_byte = (ph * c.blocks + block) * c.page_size + at;
  return p;
}

// One candidate of a block: its scale byte, codes and squared error.
struct Candidate {
  uint32_t e_byte, lo, hi;
  float err;
};

__device__ __forceinline__ Candidate candidate(const float* x, float b, float s, float k) {
  Candidate c;
  float e;
  c.e_byte = e4m3_encode(b / (k * s), e);
  const float d = e * s;
  const float r = d > 0.0f ? 1.0f / d : 0.0f;
  uint32_t w[2] = {0u, 0u};
  float err = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float g;
    const uint32_t code = e2m1_code_sw(__builtin_fabsf(x[i]) * r, g);
    const uint32_t sign = __float_as_uint(x[i]) >> 31;
    w[i >> 3] |= (code | sign << 3) << (4 * (i & 7));
    const float v = (g * e) * s;
    const float diff = x[i] - (sign ? -v : v);
    err = err + diff * diff;
  }
  c.lo = w[0];
  c.hi = w[1];
  c.err = err;
  return c;
}

// Lanes per row: the blocks of a row rounded up to a power of two (LANES),
// so that a row's maximum is a butterfly within its lanes.
template <int LANES>
__global__ __launch_bounds__(256) void kv_append_kernel(CacheView c, const uint16_t* k,
                                                        int64_t k_stride, const uint16_t* v,
                                                        int64_t v_stride, int64_t tokens,
                                                        const int64_t* slots, int fos) {
  const int which = blockIdx.y;
  const int64_t unit = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int block = threadIdx.x % LANES;
  const int64_t token = unit / c.heads;
  const int head = (int)(unit - token * c.heads);
  const bool live = token < tokens && block < c.blocks;
  const int64_t slot = token < tokens ? slots[token] : -1;
  float x[16];
  float b = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  if (live) {
    const uint16_t* src = (which ? v + token * v_stride : k + token * k_stride) +
                          (int64_t)head * c.blocks * 16 + block * 16;
    const uint4 a = ((const uint4*)src)[0], z = ((const uint4*)src)[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, z.x, z.y, z.z, z.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
      b = fmaxf(b, fmaxf(__builtin_fabsf(x[2 * i]), __builtin_fabsf(x[2 * i + 1])));
    }
  }
  float amax = b;
#pragma unroll
  for (int step = LANES / 2; step > 0; step >>= 1) amax = fmaxf(amax, __shfl_xor(amax, step));
  const float s = amax / (fos ? 1536.0f : 2688.0f);
  Candidate q = candidate(x, b, s, 6.0f);
  if (fos) {
    const Candidate q4 = candidate(x, b, s, 4.0f);
    if (q4.err < q.err) q = q4;
  }
  if (!live || slot < 0 || slot >= c.slots) return;
  const Place p = place_of(c, (uint32_t)slot, head, block);
  ((uint2*)c.codes[which])[p.row * c.blocks + block] = make_uint2(q.lo, q.hi);
  c.scales[which][which ? p.val_byte : p.key_byte] = (uint8_t)q.e_byte;
  if (block == 0) c.token_scales[which][p.row] = s;
}

__global__ __launch_bounds__(256) void kv_read_kernel(CacheView c, const int64_t* slots,
                                                      int64_t tokens, uint4* k_out,
                                                      uint4* v_out) {
  const int which = blockIdx.y;
  const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x;  // a 16-element block
  const int64_t row = unit / c.blocks;
  const int block = (int)(unit - row * c.blocks);
  const int64_t token = row / c.heads;
  if (token >= tokens) return;
  const int head = (int)(row - token * c.heads);
  const int64_t slot = slots[token];
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0u;
  if (slot >= 0 && slot < c.slots) {
    const Place p = place_of(c, (uint32_t)slot, head, block);
    const uint2 q = ((const uint2*)c.codes[which])[p.row * c.blocks + block];
    const float e = e4m3_decode(c.scales[which][which ? p.val_byte : p.key_byte]);
    const float s = c.token_scales[which][p.row];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = (i < 4 ? q.x : q.y) >> (8 * (i & 3));
      const float a = (e2m1_value(byte & 7u) * e) * s, z = (e2m1_value(byte >> 4 & 7u) * e) * s;
      w[i] = cvt_bf16x2((byte & 8u) ? -a : a, (byte & 0x80u) ? -z : z);
    }
  }
  uint4* out = (which ? v_out : k_out) + unit * 2;
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

}  // namespace

// The dispatch packet counts work-items in 32 bits: longer calls go in several
// launches over consecutive tokens.
static int64_t tokens_per_launch(int64_t lanes_per_token) {
  const int64_t n = ((int64_t)1 << 30) / lanes_per_token;
  return n < 1 ? 1 : n;
}

hipError_t kv_append_launch(const KvCache& cache, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, int64_t tokens, const int64_t* slots,
                            int four_over_six, hipStream_t stream) {
  const CacheView c = view_of(cache);
  int lanes = 1;
  while (lanes < c.blocks) lanes *= 2;
  const int64_t per = 256 / lanes, step = tokens_per_launch(lanes * cache.kv_heads);
  for (int64_t t0 = 0; t0 < tokens; t0 += step) {
    const int64_t n = tokens - t0 < step ? tokens - t0 : step;
    const dim3 g((uint32_t)((n * c.heads + per - 1) / per), 2);
    const uint16_t* kt = (const uint16_t*)k + t0 * k_stride;
    const uint16_t* vt = (const uint16_t*)v + t0 * v_stride;
#define FP4Q_APPEND(L)                                                                       \
  case L:                                                                                    \
    kv_append_kernel<L><<<g, 256, 0, stream>>>(c, kt, k_stride, vt, v_stride, n, slots + t0, \
                                               four_over_six);                               \
    break;
    switch (lanes) {
      FP4Q_APPEND(1)
      FP4Q_APPEND(2)
      FP4Q_APPEND(4)
      FP4Q_APPEND(8)
      FP4Q_APPEND(16)
      FP4Q_APPEND(32)
    }
#undef FP4Q_APPEND
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t kv_read_launch(const KvCache& cache, const int64_t* slots, int64_t tokens, void* k_out,
                          void* v_out, hipStream_t stream) {
  const CacheView c = view_of(cache);
  const int64_t per_token = (int64_t)c.heads * c.blocks, step = tokens_per_launch(per_token);
  for (int64_t t0 = 0; t0 < tokens; t0 += step) {
    const int64_t n = tokens - t0 < step ? tokens - t0 : step;
    const dim3 g((uint32_t)((n * per_token + 255) / 256), 2);
    kv_read_kernel<<<g, 256, 0, stream>>>(c, slots + t0, n, (uint4*)k_out + t0 * per_token * 2,
                                          (uint4*)v_out + t0 * per_token * 2);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp4q
