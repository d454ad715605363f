// rollout_linear.hip -- products with 4-bit weights and group scales
// (definitions in include/fp4q/rollout.h).
//
// All forms read every weight byte once per 16 * RT (or ROWS) rows of x
// and are bound by that read: 0.5625 bytes a weight (NVFP4), 0.53 (MXFP4).
// 65536 x 7168 (264 MB): one row 52 us (5.1 TB/s), 16 rows 65 (66 to 71 on other
// boxes), 64 rows 100 (0.6 PFLOP/s).
//
// One or two rows (dot form).  A wavefront takes NC output columns; a lane
// takes 32 consecutive weights of a column at a time (16 bytes of codes, so a
// load covers 1 KiB of a column) and multiplies them with BF16 dot products:
//   y = s sum_b e_b (sum_{i in b} g_i x_i), the inner sum over raw codes,
// so a scale costs one FMA per 16 weights and row.
//
// More rows (matrix form).  Weights are the rows of a 16x16x32 matrix
// instruction, activations its columns.  A weight enters as an exact BF16
// number: g e of NVFP4 has at most 6 significant bits, g 2^E of MXFP4 (times
// 2^-3) at most 2 (the conversion's own scale operand gives it), and the
// activations enter as they are.  Widening to FP16 instead takes half the vector
// instructions an NVFP4 weight (packed products), but then the activations
// have to be brought into FP16's range by a kernel before, which costs more
// than it gives.  Large matrices: slabs of the activations are copied to
// LDS, once for the workgroup's four wavefronts, and the weights to
// registers, one slab ahead of their use.  Small ones: the wavefronts of a
// workgroup share 16 columns and divide k, so that even a few columns make
// enough wavefronts without a second kernel to join them.
#include <type_traits>

#include "fp4q_device.h"
#include "rollout_launch.h"

namespace fp4q {
namespace {

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef short short2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));

struct Range {
  int64_t first, last;
};

__device__ __forceinline__ Range rows_of(const LinearArgs& a, int64_t group) {
  if (!a.offsets) return {0, a.rows};
  const int64_t lo = min(max(a.offsets[group], (int64_t)0), a.rows);
  return {lo, min(max(a.offsets[group + 1], (int64_t)0), a.rows)};
}

__device__ __forceinline__ void put_out(const LinearArgs& a, int64_t at, float v) {
  if (a.out_fp32)
    ((float*)a.out)[at] = v;
  else
    ((__bf16*)a.out)[at] = (__bf16)v;
}

template <int SEL>
__device__ __forceinline__ bf16x2v e2m1_bf16x2(uint32_t w, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL);
}

__device__ __forceinline__ float dot2(bf16x2v a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(short2v, a),
                                         __builtin_bit_cast(short2v, b), c, false);
}

// ---- one or two rows -----------------------------------------------------------------

// WAVES wavefronts of NC columns each share the activations in LDS, a chunk
// of KC elements of k at a time: read from global memory by the lanes that
// need them, 64 bytes apart, they took more of the load path than the weights.
template <bool MX, int ROWS, int NC, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void linear_dot(LinearArgs a, int64_t x0) {
  constexpr int KC = 8192 / ROWS;  // 16 KiB
  __shared__ alignas(16) uint8_t xs[ROWS][KC * 2];
  const int lane = threadIdx.x % 64;
  const int64_t n0 = ((x0 + blockIdx.x) * WAVES + threadIdx.x / 64) * NC;
  const int64_t k = a.k;
  const uint8_t* codes[NC];
  const uint8_t* scales[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t n = min(n0 + c, a.n - 1);
    codes[c] = a.codes + n * (k / 2) + lane * 16;
    scales[c] = a.scales + n * (k / (MX ? 32 : 16)) + lane * (MX ? 1 : 2);
  }
  float sum[NC][ROWS];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) sum[c][r] = 0.0f;

  u32x4v w[NC];
  uint32_t e[NC];
  auto load = [&](int64_t k0) {  // weights k0 + 32 lane ... of each column
    const int64_t left = k - k0 - lane * 32;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      w[c] = (u32x4v){0, 0, 0, 0};
      e[c] = 0;
      const uint8_t* from = codes[c] + k0 / 2;
      const uint8_t* scale = scales[c] + k0 / (MX ? 32 : 16);
      if (left >= 32) {
        w[c] = __builtin_nontemporal_load((const u32x4v*)from);
        if constexpr (MX)
          e[c] = *scale;
        else
          e[c] = *(const uint16_t*)scale;
      } else if (!MX && left >= 16) {  // the column ends after 16: k is a multiple of 16
        const u32x2v half = *(const u32x2v*)from;
        w[c] = (u32x4v){half[0], half[1], 0, 0};
        e[c] = *scale;
      }
    }
  };
  load(0);
  for (int64_t c0 = 0; c0 < k; c0 += KC) {
    // The lane's four 16-byte pieces of a step lie at piece ^ (lane / 4 mod 4), so that 16
    // lanes' reads, 64 bytes apart, meet all banks once; pieces past k are zeros.
    const int pieces = (int)min((int64_t)KC / 8, (k - c0) / 8), steps = (pieces + 255) / 256;
    if (c0 > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const uint16_t* x = (const uint16_t*)a.x + min((int64_t)r, a.rows - 1) * k + c0;
      for (int i = threadIdx.x; i < steps * 256; i += 64 * WAVES) {
        u32x4v v = *(const u32x4v*)(x + min(i, pieces - 1) * 8);
        if (i >= pieces) v = (u32x4v){0, 0, 0, 0};
        *(u32x4v*)&xs[r][(i ^ (i / 16 % 4)) * 16] = v;
      }
    }
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
      u32x4v now[NC];
      uint32_t e_now[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) now[c] = w[c], e_now[c] = e[c];
      const int64_t next = c0 + (s + 1) * 2048;
      if (next < k) load(next);
      u32x4v xv[ROWS][4];
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          xv[r][i] = *(const u32x4v*)&xs[r][(s * 256 + lane * 4 + (i ^ (lane / 4 % 4))) * 16];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float part[2][ROWS];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int r = 0; r < ROWS; ++r) part[h][r] = 0.0f;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t word = now[c][2 * h + q];
            const bf16x2v g[4] = {e2m1_bf16x2<0>(word, 1.0f), e2m1_bf16x2<1>(word, 1.0f),
                                  e2m1_bf16x2<2>(word, 1.0f), e2m1_bf16x2<3>(word, 1.0f)};
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                part[h][r] = dot2(g[i], xv[r][2 * h + q][i], part[h][r]);
          }
        }
        if constexpr (MX) {
          // (a power of two of its own would leave FP32 at the highest byte)
#pragma unroll
          for (int r = 0; r < ROWS; ++r)
            sum[c][r] += __builtin_ldexpf(part[0][r] + part[1][r], (int)e_now[c] - 127);
        } else {
          const float f0 = e4m3_value<0>(e_now[c]), f1 = e4m3_value<1>(e_now[c]);
#pragma unroll
          for (int r = 0; r < ROWS; ++r)
            sum[c][r] = __builtin_fmaf(part[1][r], f1, __builtin_fmaf(part[0][r], f0, sum[c][r]));
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
#pragma unroll
      for (int s = 32; s > 0; s >>= 1) sum[c][r] += __shfl_xor(sum[c][r], s);
    }
  if (lane == 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (n0 + c >= a.n) break;
      const float s = MX ? 1.0f : a.row_scales[n0 + c];
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (r < a.rows) put_out(a, r * a.n + n0 + c, sum[c][r] * s);
    }
  }
}

// ---- more rows ----------------------------------------------------------------

// MXFP4 weights reach 6 * 2^128: the matrix forms take them times 2^-3, so that all are BF16
// numbers, and scale the sums back.  The three lowest bytes leave the conversions' scale operand
// then: slabs that have them are decoded by careful_weights, by which the small form decodes
// all of them (testing for them took as long).
constexpr uint32_t kMxDown = 3;
constexpr float kMxUp = 8.0f;

__device__ __forceinline__ float power_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight weights of a word of codes as BF16, exact.  f: MXFP4's power of two,
// or NVFP4's block scale.
template <bool MX>
__device__ __forceinline__ bf16x8v weights_of(uint32_t word, float f) {
  if constexpr (MX) {
    const bf16x2v a = e2m1_bf16x2<0>(word, f), b = e2m1_bf16x2<1>(word, f);
    const bf16x2v c = e2m1_bf16x2<2>(word, f), d = e2m1_bf16x2<3>(word, f);
    return (bf16x8v){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const float2v a = e2m1x2_values<0>(word), b = e2m1x2_values<1>(word);
    const float2v c = e2m1x2_values<2>(word), d = e2m1x2_values<3>(word);
    const u32x4v w = {cvt_bf16x2(a[0] * f, a[1] * f), cvt_bf16x2(b[0] * f, b[1] * f),
                      cvt_bf16x2(c[0] * f, c[1] * f), cvt_bf16x2(d[0] * f, d[1] * f)};
    return __builtin_bit_cast(bf16x8v, w);
  }
}

// The same for any E8M0 byte, f = power_of(byte): times 2^-3.
template <bool MX>
__device__ __forceinline__ bf16x8v careful_weights(uint32_t word, float f) {
  if constexpr (!MX) {
    return weights_of<MX>(word, f);
  } else {
    const uint32_t byte = __float_as_uint(f) >> 23;
    const float base = power_of(max(byte, kMxDown) - kMxDown);
    const float rest = byte < kMxDown ? __builtin_ldexpf(1.0f, (int)byte - (int)kMxDown) : 1.0f;
    const float2v a = e2m1x2_values_scaled<0>(word, base), b = e2m1x2_values_scaled<1>(word, base);
    const float2v c = e2m1x2_values_scaled<2>(word, base), d = e2m1x2_values_scaled<3>(word, base);
    const u32x4v w = {cvt_bf16x2(a[0] * rest, a[1] * rest), cvt_bf16x2(b[0] * rest, b[1] * rest),
                      cvt_bf16x2(c[0] * rest, c[1] * rest), cvt_bf16x2(d[0] * rest, d[1] * rest)};
    return __builtin_bit_cast(bf16x8v, w);
  }
}

__device__ __forceinline__ float4v product(bf16x8v w, u32x4v x, float4v acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8v, x), acc, 0, 0, 0);
}

// Small matrices.  Wavefront w of WAVES takes the steps of 128 elements of k
// w, w + WAVES, ... for 16 columns and up to 16 * RT rows; activations come
// straight from global memory (the cache serves the workgroups' repeats).
template <bool MX, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void linear_small(LinearArgs a) {
  constexpr int RB = 16 * RT;
  __shared__ float sums[WAVES][RB][17];
  const int lane = threadIdx.x % 64, col = lane % 16, grp = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t k = a.k, n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * RB;
  const int64_t n = min(n0 + col, a.n - 1), steps = (k + 127) / 128;
  const uint8_t* codes = a.codes + n * (k / 2) + grp * 16;
  const uint8_t* scales = a.scales + n * (k / (MX ? 32 : 16)) + grp * (MX ? 1 : 2);
  const uint16_t* x[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    x[r] = (const uint16_t*)a.x + min(m0 + r * 16 + col, a.rows - 1) * k;

  struct Step {
    u32x4v w, x[RT][4];
    uint32_t e;
  };
  auto load = [&](int64_t step, Step& s) {
    const int64_t k0 = step * 128 + grp * 32;
    s.w = (u32x4v){0, 0, 0, 0};
    s.e = 0;
    if (k0 + 32 <= k) {
      s.w = *(const u32x4v*)(codes + step * 64);
      if constexpr (MX)
        s.e = scales[step * 4];
      else
        s.e = *(const uint16_t*)(scales + step * 8);
    } else if (!MX && k0 + 16 <= k) {
      const u32x2v half = *(const u32x2v*)(codes + step * 64);
      s.w = (u32x4v){half[0], half[1], 0, 0};
      s.e = scales[step * 8];
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        s.x[r][q] = *(const u32x4v*)(x[r] + min(k0 + q * 8, k - 8));
    if (step * 128 + 128 > k) {
      // pieces past k are zeros: a weight of zero alone does not take an infinity away
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (k0 + q * 8 >= k) {
#pragma unroll
          for (int r = 0; r < RT; ++r) s.x[r][q] = (u32x4v){0, 0, 0, 0};
        }
    }
  };
  float4v acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  Step next;
  if (wave < steps) load(wave, next);
  for (int64_t step = wave; step < steps; step += WAVES) {
    const Step now = next;
    if (step + WAVES < steps) load(step + WAVES, next);
    const float f0 = MX ? power_of(now.e) : e4m3_value<0>(now.e);
    const float f1 = MX ? f0 : e4m3_value<1>(now.e);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bf16x8v w = careful_weights<MX>(now.w[q], q < 2 ? f0 : f1);
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = product(w, now.x[r][q], acc[r]);
    }
  }
  // lane (col, grp) holds columns n0 + 4 grp + i of row m0 + 16 r + col
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[wave][r * 16 + col][grp * 4 + i] = acc[r][i];
  __syncthreads();
  for (int at = threadIdx.x; at < RB * 16; at += 64 * WAVES) {
    const int64_t m = m0 + at / 16, to = n0 + at % 16;
    if (m >= a.rows || to >= a.n) continue;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += sums[w][at / 16][at % 16];
    put_out(a, m * a.n + to, sum * (MX ? kMxUp : a.row_scales[to]));
  }
}

typedef __attribute__((address_space(3))) void lds_void;

// A lane's scale bytes in a slab: those of its own elements, neighbours in memory.
template <bool MX, int KS>
struct ScaleLoad {
  static constexpr int BYTES = KS / (MX ? 32 : 16) / 4;  // 8, 4 or 2 a lane
  static constexpr int STEPS = KS / 128;
  uint32_t w[BYTES == 8 ? 2 : 1];

  __device__ __forceinline__ void whole(const uint8_t* p) {
    if constexpr (BYTES == 8) {
      const u32x2v v = *(const u32x2v*)p;
      w[0] = v[0], w[1] = v[1];
    } else if constexpr (BYTES == 4) {
      w[0] = *(const uint32_t*)p;
    } else {
      w[0] = *(const uint16_t*)p;
    }
  }
  // the first n of them, the others zero
  __device__ __forceinline__ void some(const uint8_t* p, int n) {
#pragma unroll
    for (int i = 0; i < (BYTES + 3) / 4; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < BYTES; ++i)
      if (i < n) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  }
  // MXFP4: whether a byte is below kMxDown, and all of them less kMxDown (if none is)
  static constexpr uint32_t kDown = kMxDown * (BYTES == 2 ? 0x0101u : 0x01010101u);
  __device__ __forceinline__ bool low() const {
    return ((w[0] - kDown) & ~w[0] & (BYTES == 2 ? 0x8080u : 0x80808080u)) != 0;
  }
  __device__ __forceinline__ void lower() { w[0] -= kDown; }
  // The scale of the first (H = 0) and second 16 elements of step S; MXFP4's power of two, an
  // FP32 pattern of which the conversions read the exponent field alone (so 0, 2^-127, works
  // too), for both.
  template <int S, int H>
  __device__ __forceinline__ float value() const {
    if constexpr (MX)
      return power_of(w[S / 4] >> (8 * (S % 4)) & 255u);
    else
      return e4m3_value<(2 * S + H) % 4>(w[S / 2]);
  }
};

// The matrix instruction wants a column a lane, but loaded so every lane's 16 bytes are an
// access of their own, 64 a load.  So N neighbouring lanes read N * 16 consecutive bytes of one column, for N columns in turn, and this
// is the transposition: w[r] of lane b of N becomes what lane r had in w[b].  (32 experts x 8 rows
// 67 -> 61 us, 65536 x 7168 by 16 rows 71 -> 63; exchanged through LDS 63 and 64; two slabs of
// weights ahead instead of one 62 and 65.)
template <int N>
__device__ __forceinline__ void turn(u32x4v (&w)[N], int lane) {
  auto swap = [&](u32x4v& lo, u32x4v& hi, bool odd, auto from) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = lo[i], b = hi[i], fa = from(a), fb = from(b);
      lo[i] = odd ? fb : a;
      hi[i] = odd ? b : fa;
    }
  };
  auto by_1 = [](uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);
  };
  auto by_2 = [](uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);
  };
#pragma unroll
  for (int i = 0; i < N; i += 2) swap(w[i], w[i + 1], lane & 1, by_1);
  if constexpr (N == 4) {
    swap(w[0], w[2], lane & 2, by_2);
    swap(w[1], w[3], lane & 2, by_2);
  }
}

// One workgroup: 64 * NT columns (tile x0 + blockIdx.x), 16 * RT rows (block
// y0 + blockIdx.y; with groups, all rows of that group in turn), and the
// blockIdx.z-th share of k's slabs of KS elements; with several shares the
// sums go to `partial`.
template <bool MX, int RT, int NT>
__global__ __launch_bounds__(256, RT == 1 ? 4 : 2) void linear_large(LinearArgs a, int64_t x0,
                                                                     int64_t y0, float* partial) {
  constexpr int KS = RT == 1 ? 512 : 256, STEPS = KS / 128, RB = 16 * RT;
  constexpr int PIECES = KS / 8, PER_COPY = 64 / PIECES;  // 16-byte pieces a row; rows a copy
  // A copy's rows lie together, 1 KiB, and 16 bytes after them stay unused; the second of two
  // rows has its pieces 8 apart exchanged: so 16 rows' reads of a piece meet all banks once.
  constexpr int COPY = 1024 + 16;
  __shared__ alignas(16) uint8_t xs[2][RB / PER_COPY * COPY];
  const int lane = threadIdx.x % 64, col = lane % 16, grp = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t k = a.k, y = y0 + blockIdx.y;
  const uint16_t* x = (const uint16_t*)a.x;
  const int64_t splits = gridDim.z, split = blockIdx.z;
  const Range range = a.offsets ? rows_of(a, y) : Range{y * RB, a.rows};
  const int64_t matrix = a.offsets ? y : 0;
  // whole slabs [slab_lo, slab_whole), and after them perhaps k's last part
  const int slabs = (int)((k + KS - 1) / KS);
  const int slab_lo = (int)(slabs * split / splits), slab_hi = (int)(slabs * (split + 1) / splits);
  const int slab_whole = min(slab_hi, (int)(k / KS));
  const int64_t n0 = ((x0 + blockIdx.x) * 4 + wave) * 16 * NT;
  // Lane (col, grp) multiplies the elements [grp KS/4, (grp + 1) KS/4) of a slab, 32 a step, of
  // column n0 + 16 t + col; it loads, as w[r], the (col mod STEPS)-th 16 bytes of them of column
  // n0 + 16 t + col - col mod STEPS + r.
  const int first = __builtin_amdgcn_readfirstlane((int)min(n0, a.n - 1));
  const uint8_t* codes = a.codes + (matrix * a.n + first) * (k / 2);
  const uint32_t row_bytes = (uint32_t)(k / 2);
  uint32_t code_at[NT][STEPS], own_at[NT];
  const uint8_t* scales[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    auto column = [&](int c) { return (uint32_t)(min(n0 + t * 16 + c, a.n - 1) - first); };
#pragma unroll
    for (int r = 0; r < STEPS; ++r)
      code_at[t][r] = column(col / STEPS * STEPS + r) * row_bytes + grp * (KS / 8) + col % STEPS * 16;
    own_at[t] = column(col) * row_bytes + grp * (KS / 8);
    scales[t] = a.scales + (matrix * a.n + first + column(col)) * (k / (MX ? 32 : 16)) +
                grp * ScaleLoad<MX, KS>::BYTES;
  }
  // the lane's first piece in LDS; its others follow
  const uint32_t at_piece =
      (uint32_t)(col / PER_COPY * COPY +
                 (PER_COPY == 1 ? grp * 16 : col % 2 * 32 + ((grp * 8) ^ (col % 2 * 8))) * 16);

  for (int64_t m0 = range.first; m0 < range.last; m0 += RB) {
    const int rows = (int)min((int64_t)RB, range.last - m0);
    u32x4v w[NT][STEPS], w_next[NT][STEPS];
    ScaleLoad<MX, KS> e_next[NT];
    float4v acc[NT][RT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[t][r] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};

    // a slab's activations: a copy fills 64 pieces; rows past the last are left as they are
    // (their columns of the result are not stored), pieces past k repeat the last one and are
    // not multiplied
    auto copy = [&](int slab) {
      const int64_t piece0 = (int64_t)slab * PIECES, last = k / 8 - 1;
#pragma unroll
      for (int i = 0; i < RB / PER_COPY / 4; ++i) {
        const int row0 = (i * 4 + wave) * PER_COPY;
        if (row0 < rows) {
          const int r = row0 + lane / PIECES;
          const int64_t piece = min(piece0 + ((lane % PIECES) ^ (lane / PIECES * 8)), last);
          __builtin_amdgcn_global_load_lds(x + (m0 + min(r, rows - 1)) * k + piece * 8,
                                           (lds_void*)(xs[slab & 1] + row0 / PER_COPY * COPY), 16,
                                           0, 0);
        }
      }
    };
    auto load = [&](int slab) {
      copy(slab);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint8_t* c = codes + (int64_t)slab * (KS / 2);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) w_next[t][s] = *(const u32x4v*)(c + code_at[t][s]);
        e_next[t].whole(scales[t] + (int64_t)slab * (KS / (MX ? 32 : 16)));
      }
    };
    // the slab of w, of which k has `left` elements; with care, these may be less than all of
    // them, and scale bytes may be any
    auto multiply = [&](int slab, float (&f)[NT][STEPS][2], auto care, int left) {
      constexpr bool CARE = decltype(care)::value;
      const uint8_t* xb = xs[slab & 1] + at_piece;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u32x4v xv[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r)
            if (r == 0 || r * 16 < rows)
              xv[r] = *(const u32x4v*)(xb + r * 16 / PER_COPY * COPY + s * 64 + q * 16);
          if constexpr (CARE) {
            // (a weight of zero alone does not take an infinity away)
#pragma unroll
            for (int r = 0; r < RT; ++r)
              if (grp * (KS / 4) + s * 32 + q * 8 >= left) xv[r] = (u32x4v){0, 0, 0, 0};
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float fv = f[t][s][MX ? 0 : q / 2];
            const bf16x8v wv =
                CARE ? careful_weights<MX>(w[t][s][q], fv) : weights_of<MX>(w[t][s][q], fv);
#pragma unroll
            for (int r = 0; r < RT; ++r)
              if (r == 0 || r * 16 < rows) acc[t][r] = product(wv, xv[r], acc[t][r]);
          }
        }
      }
    };
    // returns whether the slab needs care
    auto begin = [&](bool turned, bool care, float (&f)[NT][STEPS][2]) {
      __builtin_amdgcn_s_waitcnt(0);  // this wavefront's copies and weights have landed
      if constexpr (MX) {
        bool low = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) low |= e_next[t].low();
        care = care || __any(low);
        if (!care) {
#pragma unroll
          for (int t = 0; t < NT; ++t) e_next[t].lower();
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) w[t][s] = w_next[t][s];
        if (!turned) turn<STEPS>(w[t], lane);
        f[t][0][0] = e_next[t].template value<0, 0>();
        f[t][0][1] = e_next[t].template value<0, 1>();
        f[t][1][0] = e_next[t].template value<1, 0>();
        f[t][1][1] = e_next[t].template value<1, 1>();
        if constexpr (STEPS == 4) {
          f[t][2][0] = e_next[t].template value<2, 0>();
          f[t][2][1] = e_next[t].template value<2, 1>();
          f[t][3][0] = e_next[t].template value<3, 0>();
          f[t][3][1] = e_next[t].template value<3, 1>();
        }
      }
      __syncthreads();  // the other wavefronts' copies too; the slab before is read
      return care;
    };

    if (m0 != range.first) __syncthreads();  // the last rows' slabs are read
    if (slab_lo < slab_whole) load(slab_lo);
    for (int slab = slab_lo; slab < slab_whole; ++slab) {
      float f[NT][STEPS][2];
      const bool care = begin(false, false, f);
      if (slab + 1 < slab_whole) load(slab + 1);
      if (MX && care)
        multiply(slab, f, std::true_type(), KS);
      else
        multiply(slab, f, std::false_type(), KS);
    }
    if (slab_whole < slab_hi) {
      const int left = (int)(k - (int64_t)slab_whole * KS);
      copy(slab_whole);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint8_t* c = codes + (int64_t)slab_whole * (KS / 2) + own_at[t];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int at = grp * (KS / 4) + s * 32;
          w_next[t][s] = (u32x4v){0, 0, 0, 0};
          if (at + 32 <= left) {
            w_next[t][s] = *(const u32x4v*)(c + s * 16);
          } else if (!MX && at + 16 <= left) {
            const u32x2v half = *(const u32x2v*)(c + s * 16);
            w_next[t][s] = (u32x4v){half[0], half[1], 0, 0};
          }
        }
        e_next[t].some(scales[t] + (int64_t)slab_whole * (KS / (MX ? 32 : 16)),
                       left / (MX ? 32 : 16) - grp * ScaleLoad<MX, KS>::BYTES);
      }
      float f[NT][STEPS][2];
      begin(true, true, f);
      multiply(slab_whole, f, std::true_type(), left);
    }

    // lane (col, grp) holds columns n0 + 16 t + 4 grp + i of row m0 + 16 r + col
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int64_t m = m0 + r * 16 + col;
      if (r * 16 + col >= rows) continue;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int64_t n = n0 + t * 16 + grp * 4;
        if (partial) {
          float* to = partial + (split * a.rows + m) * a.n + n;
          if (n + 4 <= a.n && a.n % 4 == 0) {
            *(float4v*)to = acc[t][r];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n + i < a.n) to[i] = acc[t][r][i];
          }
          continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < a.n) {
            const float s = MX ? kMxUp : a.row_scales[matrix * a.n + n + i];
            put_out(a, m * a.n + n + i, acc[t][r][i] * s);
          }
      }
    }
    if (!a.offsets) break;
  }
}

// The splits' partial sums added in order, times the row scale.
template <bool MX>
__global__ __launch_bounds__(256) void linear_join(LinearArgs a, int splits,
                                                   const float* partial) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, all = a.rows * a.n;
  if (at >= all) return;
  float sum = 0.0f;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) sum += partial[s * all + at];
  put_out(a, at, sum * (MX ? kMxUp : a.row_scales[at % a.n]));
}

// ---- shape of a call ------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

enum class Form { kDot, kSmall, kLarge };

struct Plan {
  Form form;
  int rows;  // rows a workgroup takes: 1, 2 (dot), 16, 32, 64
  int nt;    // column tiles a wavefront takes: 1, 2
  int64_t splits;
};

// The forms' times below are for NVFP4, on the device, in us.
Plan plan_of(int64_t rows, int64_t n, int64_t k, int64_t groups) {
  Plan p{Form::kLarge, 16, 1, 1};
  if (groups == 0 && rows <= 2) {
    p.form = Form::kDot;
    p.rows = (int)rows;
    // one column a wavefront fills the chip best (2048 x 7168: 5.2, 5.8 with two); where
    // columns abound, two share the activations' reads (65536 x 7168: 52, 56 with one)
    p.nt = rows == 2 || n >= 16384 ? 2 : 1;
    return p;
  }
  // with groups, enough rows for most of them in one pass over their weights: routing leaves
  // a group's share mostly below its mean and twice the mean's root
  int64_t each = groups ? ceil_div(rows, groups) : rows, root = 1;
  while (root * root < each) ++root;
  if (groups) each = each + 2 * root < rows ? each + 2 * root : rows;
  p.rows = each <= 16 ? 16 : each <= 32 ? 32 : 64;
  if (groups) {
    p.nt = p.rows == 16 ? 1 : 2;
    return p;
  }
  // Each wavefront of the small form goes through k / 1024 steps a row tile on its own, and
  // reads all activations: 8 rows, 4096 x 4096 6.7 (large form 8.8), 2048 x 2048 4.4 (7.9),
  // but 1024 x 7168 9.1 (8.5), 16384 x 2048 11.2 (11.4); 24 rows, 2048 x 2048 6.2 (7.0), but
  // 7168 x 2048 10.4 (9.3)
  const int64_t row_tiles = ceil_div(rows, 16);
  if (k * row_tiles <= 4096 && n * k * row_tiles <= ((int64_t)1 << 24)) {
    p.form = Form::kSmall;
    return p;
  }
  // above 16 rows, two column tiles a wavefront halve the activations' reads from LDS where
  // enough workgroups remain (64 rows, 65536 x 7168: 99, 124 with one; 8192 x 7168: 24.2, 22.0)
  p.nt = p.rows > 16 && n >= 16384 ? 2 : 1;
  // k divided over enough workgroups to fill the chip twice, each two slabs at least
  const int64_t tiles = ceil_div(n, 64 * p.nt) * ceil_div(rows, p.rows);
  const int64_t slabs = ceil_div(k, p.rows == 16 ? 512 : 256);
  p.splits = ceil_div(512, tiles);
  if (p.splits > slabs / 2) p.splits = slabs / 2;
  if (p.splits > 16) p.splits = 16;
  if (p.splits < 1) p.splits = 1;
  return p;
}

// The dispatch packet counts work-items in 32 bits, and the second grid
// dimension 16: larger calls go in several launches.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 31) / 512;

template <bool MX, int ROWS, int NC, int WAVES>
hipError_t dot(const LinearArgs& a, hipStream_t stream) {
  const int64_t blocks = ceil_div(a.n, WAVES * NC);
  for (int64_t x0 = 0; x0 < blocks; x0 += kMaxBlocks) {
    const int64_t n = blocks - x0 < kMaxBlocks ? blocks - x0 : kMaxBlocks;
    linear_dot<MX, ROWS, NC, WAVES><<<(uint32_t)n, 64 * WAVES, 0, stream>>>(a, x0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool MX, int RT, int WAVES>
hipError_t small(const LinearArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)ceil_div(a.n, 16), (uint32_t)ceil_div(a.rows, 16 * RT));
  linear_small<MX, RT, WAVES><<<grid, 64 * WAVES, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool MX, int RT, int NT>
hipError_t large(const LinearArgs& a, const Plan& p, hipStream_t stream) {
  float* partial = p.splits > 1 ? (float*)a.workspace : nullptr;
  const int64_t xs = ceil_div(a.n, 64 * NT);
  const int64_t ys = a.groups ? a.groups : ceil_div(a.rows, 16 * RT);
  const int64_t dx = xs < kMaxBlocks / p.splits ? xs : kMaxBlocks / p.splits;
  int64_t dy = kMaxBlocks / (dx * p.splits);
  if (dy > 65535) dy = 65535;
  for (int64_t y0 = 0; y0 < ys; y0 += dy)
    for (int64_t x0 = 0; x0 < xs; x0 += dx) {
      const dim3 grid((uint32_t)(xs - x0 < dx ? xs - x0 : dx),
                      (uint32_t)(ys - y0 < dy ? ys - y0 : dy), (uint32_t)p.splits);
      linear_large<MX, RT, NT><<<grid, 256, 0, stream>>>(a, x0, y0, partial);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  if (!partial) return hipSuccess;
  // several splits: fewer than 512 tiles of at most 64 rows and 128 columns
  linear_join<MX><<<(uint32_t)ceil_div(a.rows * a.n, 256), 256, 0, stream>>>(a, (int)p.splits,
                                                                             partial);
  return hipGetLastError();
}

template <bool MX>
hipError_t launch(const LinearArgs& a, hipStream_t stream) {
  const Plan p = plan_of(a.rows, a.n, a.k, a.groups);
  switch (p.form) {
    case Form::kDot:
      if (p.rows == 2) return dot<MX, 2, 2, 4>(a, stream);
      return p.nt == 2 ? dot<MX, 1, 2, 4>(a, stream) : dot<MX, 1, 1, 8>(a, stream);
    case Form::kSmall:
      if (p.rows == 16) return small<MX, 1, 8>(a, stream);
      if (p.rows == 32) return small<MX, 2, 8>(a, stream);
      return small<MX, 4, 8>(a, stream);
    default:
      if (p.rows == 16) return large<MX, 1, 1>(a, p, stream);
      if (p.rows == 32)
        return p.nt == 2 ? large<MX, 2, 2>(a, p, stream) : large<MX, 2, 1>(a, p, stream);
      return p.nt == 2 ? large<MX, 4, 2>(a, p, stream) : large<MX, 4, 1>(a, p, stream);
  }
}

}  // namespace

int64_t linear_workspace_bytes(bool, int64_t rows, int64_t n, int64_t k, int64_t groups) {
  const Plan p = plan_of(rows, n, k, groups);
  return p.splits > 1 ? p.splits * rows * n * 4 : 0;
}

hipError_t linear_launch(bool mx, const LinearArgs& a, hipStream_t stream) {
  return mx ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace fp4q
