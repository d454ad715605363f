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
// One lane per 16-element block, a row's blocks in neighbouring lanes: a
// wavefront reads (or writes) 2 KiB of consecutive BF16, and whole rows of
// codes.  Reading is bound by memory: 32k tokens of 8 heads of 128 take 30
// us, 5.6 TB/s.  8k such tokens are written in 12.4 us, 3.5 TB/s (13.3 with
// the errors of every block by the definition): memory takes 7 of them, the
// rest are the launch, loads behind loads in wavefronts that do one block a
// lane, and the value scales' single bytes (1 us).
#include "fp4q_device.h"
#include "rollout_divisor.h"
#include "rollout_launch.h"

namespace fp4q {
namespace {

struct CacheView {
  uint8_t* codes[2];
  uint8_t* scales[2];
  float* token_scales[2];
  int64_t slots;  // num_pages * page_size
  Divisor page_size, heads;
  int32_t blocks;  // head_dim / 16
};

CacheView view_of(const KvCache& c) {
  CacheView v;
  for (int i = 0; i < 2; ++i) {
    v.codes[i] = c.codes[i];
    v.scales[i] = c.scales[i];
    v.token_scales[i] = c.token_scales[i];
  }
  v.slots = c.num_pages * c.page_size;
  v.page_size = divisor_of((uint32_t)c.page_size);
  v.heads = divisor_of((uint32_t)c.kv_heads);
  v.blocks = (int32_t)(c.head_dim / 16);
  return v;
}

struct Place {
  int64_t row;    // index of the cache row: codes at row * d/2, scale at row
  int64_t scale;  // of this lane's block among the block scales
};

__device__ __forceinline__ Place place_of(const CacheView& c, uint32_t slot, uint32_t head,
                                          int block, int which) {
  const uint32_t page = quotient(slot, c.page_size), at = slot - page * c.page_size.d;
  const int64_t ph = (int64_t)page * c.heads.d + head;
  Place p;
  p.row = ph * c.page_size.d + at;
  p.scale = which ? (ph * c.blocks + block) * c.page_size.d + at : p.row * c.blocks + block;
  return p;
}

// One candidate of a block: its scale byte, codes and squared error; of a
// row with 2^-50 <= s <= 2^40 first only a, the error in units of the decode
// step d = e s, and d^2.
struct Candidate {
  uint32_t e_byte;
  uint32_t word[2];
  float err, a, d2;
};

// The scale byte of one candidate.  A zero row (s = 0) has zero scales; the quotient rounds to
// at most 448.
__device__ __forceinline__ uint32_t scale_byte(float b, float s, float k) {
  const float t = s > 0.0f ? fminf(b / (k * s), 448.0f) : 0.0f;
  return cvt_e4m3x2(t, t) & 0xFFu;
}

__device__ __forceinline__ void encode(const float* x, float b, float s, float k, Candidate& c) {
  c.e_byte = scale_byte(b, s, k);
  const float d = e4m3_value<0>(c.e_byte) * s;
  const float r = d == 0.0f ? 0.0f : recip_normal(d);
  c.a = 0.0f;
  c.d2 = d * d;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[8 * w + i] * r;
    uint32_t q = cvt_e2m1x2<0>(any_word(), v[0], v[1]);
    q = cvt_e2m1x2<1>(q, v[2], v[3]);
    q = cvt_e2m1x2<2>(q, v[4], v[5]);
    q = cvt_e2m1x2<3>(q, v[6], v[7]);
    c.word[w] = q;
    const float2v g[4] = {e2m1x2_values<0>(q), e2m1x2_values<1>(q), e2m1x2_values<2>(q),
                          e2m1x2_values<3>(q)};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float diff = v[i] - g[i / 2][i % 2];
      c.a = __builtin_fmaf(diff, diff, c.a);
    }
  }
}

// The definition's squared error of a candidate's codes.
__device__ __forceinline__ float error_of(const float* x, const Candidate& c, float s) {
  const float e = e4m3_value<0>(c.e_byte);
  float err = 0.0f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t q = c.word[w];
    const float2v g[4] = {e2m1x2_values<0>(q), e2m1x2_values<1>(q), e2m1x2_values<2>(q),
                          e2m1x2_values<3>(q)};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float diff = x[8 * w + i] - (g[i / 2][i % 2] * e) * s;
      err = err + diff * diff;
    }
  }
  return err;
}

// Whether the candidate for 4 has the lower error, as far as a and d^2 tell.  With u = 2^-24,
// |v| < 10 and |g| <= 6, each x - c of the definition is within 32.2 u d of d (v - g), and its
// sum of squares, summed in FP32, within d^2 (163.4 u a + 129.3 u) of d^2 a (nvfp4_quantize's
// kernel derives it); the differences, sums and margin below are within 2.1 u of theirs.  So
// twice that margin decides, and what it leaves open the errors by the definition do.
__device__ __forceinline__ bool four_is_lower(const Candidate& six, const Candidate& four,
                                              bool& sure) {
  constexpr float u = 0x1p-24f;
  const float p = four.d2 * four.a, q = six.d2 * six.a, diff = q - p;
  const float margin = __builtin_fmaf(p + q, 330.0f * u, (four.d2 + six.d2) * (260.0f * u));
  sure = __builtin_fabsf(diff) > margin && six.e_byte != 0;
  return diff > margin;
}

__device__ __forceinline__ Candidate candidate(const float* x, float b, float s, float k) {
  Candidate c;
  c.e_byte = scale_byte(b, s, k);
  const float e = e4m3_value<0>(c.e_byte), d = e * s;
  c.err = 0.0f;
  if (d >= 0x1p-126f || d == 0.0f) {
    // d = 0: every code is a zero with the element's sign
    const float r = d == 0.0f ? 0.0f : recip_normal(d);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float* v = x + 8 * w;
      uint32_t q = cvt_e2m1x2<0>(any_word(), v[0] * r, v[1] * r);
      q = cvt_e2m1x2<1>(q, v[2] * r, v[3] * r);
      q = cvt_e2m1x2<2>(q, v[4] * r, v[5] * r);
      q = cvt_e2m1x2<3>(q, v[6] * r, v[7] * r);
      c.word[w] = q;
      const float2v g[4] = {e2m1x2_values<0>(q), e2m1x2_values<1>(q), e2m1x2_values<2>(q),
                            e2m1x2_values<3>(q)};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float diff = v[i] - (g[i / 2][i % 2] * e) * s;
        c.err = c.err + diff * diff;
      }
    }
    return c;
  }
  // a subnormal step, whose reciprocal may be infinite: the conversions' domain ends here
  const float r = 1.0f / d;
  c.word[0] = c.word[1] = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float g;
    const uint32_t code = e2m1_code_sw(__builtin_fabsf(x[i]) * r, g);
    const uint32_t sign = __float_as_uint(x[i]) >> 31;
    c.word[i >> 3] |= (code | sign << 3) << (4 * (i & 7));
    const float v = (g * e) * s;
    const float diff = x[i] - (sign ? -v : v);
    c.err = c.err + diff * diff;
  }
  return c;
}

// Lanes per row: the blocks of a row rounded up to a power of two (LANES),
// so that a row's maximum is a butterfly within its lanes.
template <int LANES>
__global__ __launch_bounds__(256) void kv_append_kernel(CacheView c, const uint16_t* k,
                                                        int64_t k_stride, const uint16_t* v,
                                                        int64_t v_stride, uint32_t rows,
                                                        const int64_t* slots, int fos) {
  const int which = blockIdx.y;
  const uint32_t row = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int block = threadIdx.x % LANES;
  const uint32_t token = quotient(row, c.heads), head = row - token * c.heads.d;
  const bool live = row < rows && block < c.blocks;
  const int64_t slot = row < rows ? slots[token] : -1;
  float x[16];
  float b = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  if (live) {
    const uint16_t* src = (which ? v + token * v_stride : k + token * k_stride) +
                          (int64_t)head * c.blocks * 16 + block * 16;
    const u32x4v a = ((const u32x4v*)src)[0], z = ((const u32x4v*)src)[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = i < 4 ? a[i] : z[i - 4];
      x[2 * i] = bf16_lo(w);
      x[2 * i + 1] = bf16_hi(w);
      b = fmaxf(b, fmaxf(__builtin_fabsf(x[2 * i]), __builtin_fabsf(x[2 * i + 1])));
    }
  }
  float amax = b;
#pragma unroll
  for (int step = LANES / 2; step > 0; step >>= 1) amax = fmaxf(amax, __shfl_xor(amax, step));
  const float s = amax_over_c(amax, fos != 0);
  Candidate q;
  if (__all(s >= 0x1p-50f && s <= 0x1p40f)) {
    encode(x, b, s, 6.0f, q);
    if (fos) {
      Candidate q4;
      encode(x, b, s, 4.0f, q4);
      bool sure, four = four_is_lower(q, q4, sure);
      if (!sure) four = error_of(x, q4, s) < error_of(x, q, s);
      if (four) q = q4;
    }
  } else {
    q = candidate(x, b, s, 6.0f);
    if (fos) {
      const Candidate q4 = candidate(x, b, s, 4.0f);
      if (q4.err < q.err) q = q4;
    }
  }
  if (!live || slot < 0 || slot >= c.slots) return;
  const Place p = place_of(c, (uint32_t)slot, head, block, which);
  ((u32x2v*)c.codes[which])[p.row * c.blocks + block] = (u32x2v){q.word[0], q.word[1]};
  c.scales[which][p.scale] = (uint8_t)q.e_byte;
  if (block == 0) c.token_scales[which][p.row] = s;
}

// PIECES half blocks (8 elements) a thread, 256 apart: a wavefront's stores
// are 1 KiB of consecutive BF16 each, and several loads, each behind that of
// its slot, are in flight.  Non-temporal stores: 32k tokens of 8 heads of 128
// take 31 us (5.5 TB/s), 42 with plain ones, and 47 with a whole block a
// thread, whose stores fill every line in two instructions.
template <int PIECES>
__global__ __launch_bounds__(256) void kv_read_kernel(CacheView c, Divisor row_pieces,
                                                      const int64_t* slots, uint32_t pieces,
                                                      u32x4v* k_out, u32x4v* v_out) {
  const int which = blockIdx.y;
  const uint32_t piece0 = blockIdx.x * (256 * PIECES) + threadIdx.x;
  uint32_t q[PIECES], e[PIECES];
  float s[PIECES];
  int64_t slot[PIECES];
  uint32_t row[PIECES], token[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    row[i] = quotient(min(piece0 + i * 256, pieces - 1), row_pieces);
    token[i] = quotient(row[i], c.heads);
    slot[i] = slots[token[i]];
  }
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int in_row = (int)(min(piece0 + i * 256, pieces - 1) - row[i] * row_pieces.d);
    const bool held = slot[i] >= 0 && slot[i] < c.slots;  // else zeros, from slot 0's place
    const Place p = place_of(c, held ? (uint32_t)slot[i] : 0u, row[i] - token[i] * c.heads.d,
                             in_row / 2, which);
    q[i] = ((const uint32_t*)c.codes[which])[p.row * row_pieces.d + in_row];
    e[i] = c.scales[which][p.scale];
    s[i] = c.token_scales[which][p.row];
    if (!held) q[i] = 0, e[i] = 0, s[i] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const uint32_t piece = piece0 + i * 256;
    if (piece >= pieces) return;
    const float f = e4m3_value<0>(e[i]);
    const float2v g[4] = {e2m1x2_values<0>(q[i]), e2m1x2_values<1>(q[i]),
                          e2m1x2_values<2>(q[i]), e2m1x2_values<3>(q[i])};
    u32x4v w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = cvt_bf16x2((g[j][0] * f) * s[i], (g[j][1] * f) * s[i]);
    __builtin_nontemporal_store(w, (which ? v_out : k_out) + piece);
  }
}

}  // namespace

// Work-items of a launch are counted in 31 bits: longer calls go in several
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
    const int64_t n = tokens - t0 < step ? tokens - t0 : step, rows = n * cache.kv_heads;
    const dim3 g((uint32_t)((rows + per - 1) / per), 2);
    const uint16_t* kt = (const uint16_t*)k + t0 * k_stride;
    const uint16_t* vt = (const uint16_t*)v + t0 * v_stride;
#define FP4Q_APPEND(L)                                                                     \
  case L:                                                                                  \
    kv_append_kernel<L><<<g, 256, 0, stream>>>(c, kt, k_stride, vt, v_stride,              \
                                               (uint32_t)rows, slots + t0, four_over_six); \
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
  const int64_t per_token = cache.kv_heads * c.blocks * 2, step = tokens_per_launch(per_token);
  const Divisor row_pieces = divisor_of((uint32_t)c.blocks * 2);
  for (int64_t t0 = 0; t0 < tokens; t0 += step) {
    const int64_t pieces = (tokens - t0 < step ? tokens - t0 : step) * per_token;
    u32x4v* ko = (u32x4v*)k_out + t0 * per_token;
    u32x4v* vo = (u32x4v*)v_out + t0 * per_token;
    // 32k tokens of 8 heads of 128: 31 us with 4 pieces a thread, 33 with 2, 56 with 1; 64
    // tokens (with their append): 5.9, 5.3 and 5.4
    const int each = pieces >= ((int64_t)1 << 19) ? 4 : 2;
    const dim3 g((uint32_t)((pieces + 256 * each - 1) / (256 * each)), 2);
    if (each == 4)
      kv_read_kernel<4>
          <<<g, 256, 0, stream>>>(c, row_pieces, slots + t0, (uint32_t)pieces, ko, vo);
    else
      kv_read_kernel<2>
          <<<g, 256, 0, stream>>>(c, row_pieces, slots + t0, (uint32_t)pieces, ko, vo);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp4q
