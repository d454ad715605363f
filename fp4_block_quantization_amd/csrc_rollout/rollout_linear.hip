// rollout_linear.hip -- products with 4-bit weights and group scales
// (definitions in include/fp4q/rollout.h).
//
// Both forms read every weight byte once per 16 * RT (or ROWS) rows of x
// and are bound by that read: 0.5625 bytes a weight (NVFP4), 0.53 (MXFP4).
//
// Few rows (dot form).  A wavefront takes NC output columns; a lane takes 32
// consecutive weights of a column at a time (16 bytes of codes, so a load
// covers 1 KiB of a column) and multiplies them with BF16 dot products:
//   y = s sum_b e_b (sum_{i in b} g_i x_i), the inner sum over raw codes,
// so a scale costs one FMA per 16 weights and row.
//
// More rows (matrix form).  Weights are the rows of a 16x16x32 matrix
// instruction, activations its columns.  An NVFP4 weight enters as g e, an
// exact FP16 number (one conversion and one packed product per two weights),
// the activations as FP16 scaled by a power of two per row (exact for
// elements within 2^29 of the row's largest), converted by a small kernel
// before; an MXFP4 weight is an exact BF16 number that the conversion's own
// scale operand gives, and the activations stay as they are.  Slabs of the
// activations are copied to LDS, once for the workgroup's four wavefronts,
// and the weights to registers, one slab ahead of their use.
#include "fp4q_device.h"
#include "rollout_launch.h"

namespace fp4q {
namespace {

typedef _Float16 half8v __attribute__((ext_vector_type(8)));
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

// The two E4M3 bytes of a word's low (0) or high (1) half as FP16, exact.
template <int SEL>
__device__ __forceinline__ half2v e4m3_f16x2(uint32_t w) {
  return __builtin_bit_cast(half2v,
                            __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, SEL != 0));
}

template <int SEL>
__device__ __forceinline__ bf16x2v e2m1_bf16x2(uint32_t w, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL);
}

__device__ __forceinline__ float dot2(bf16x2v a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(short2v, a),
                                         __builtin_bit_cast(short2v, b), c, false);
}

// ---- few rows -----------------------------------------------------------------

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
    // lanes' reads, 64 bytes apart, meet all banks once; pieces past k repeat the last.
    const int pieces = (int)min((int64_t)KC / 8, (k - c0) / 8), steps = (pieces + 255) / 256;
    if (c0 > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const uint16_t* x = (const uint16_t*)a.x + min((int64_t)r, a.rows - 1) * k + c0;
      for (int i = threadIdx.x; i < steps * 256; i += 64 * WAVES)
        *(u32x4v*)&xs[r][(i ^ (i / 16 % 4)) * 16] = *(const u32x4v*)(x + min(i, pieces - 1) * 8);
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
          const float f = __builtin_ldexpf(1.0f, (int)e_now[c] - 127);
#pragma unroll
          for (int r = 0; r < ROWS; ++r)
            sum[c][r] = __builtin_fmaf(part[0][r] + part[1][r], f, sum[c][r]);
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

// Rows of x as FP16 times a power of two that takes the row's largest
// element to [2^14, 2^15), and the power's inverse.  Zeros, and rows with a
// NaN or infinity, stay as they are.
__global__ __launch_bounds__(256) void linear_convert(LinearArgs a, int64_t row0, uint16_t* to,
                                                      float* scale) {
  __shared__ uint32_t tops[4];
  const int64_t row = row0 + blockIdx.x, pieces = a.k / 8;
  const u32x4v* x = (const u32x4v*)((const uint16_t*)a.x + row * a.k);
  uint32_t top = 0;
  for (int64_t i = threadIdx.x; i < pieces; i += 256) {
    const u32x4v v = x[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max(v[j] & 0x7FFFu, v[j] >> 16 & 0x7FFFu));
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, s));
  if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const int field = (int)(top >> 7);
  const int ex = top == 0 || field == 255 ? 0 : 14 + 127 - max(field, 1);
  for (int64_t i = threadIdx.x; i < pieces; i += 256) {
    u32x4v v = x[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const half2v h = {(_Float16)__builtin_ldexpf(bf16_lo(v[j]), ex),
                        (_Float16)__builtin_ldexpf(bf16_hi(v[j]), ex)};
      v[j] = __builtin_bit_cast(uint32_t, h);
    }
    ((u32x4v*)(to + row * a.k))[i] = v;
  }
  if (threadIdx.x == 0) scale[row] = __builtin_ldexpf(1.0f, -ex);
}

typedef __attribute__((address_space(3))) void lds_void;

// The scale bytes of a wavefront's 16 columns over a slab.  A step's scales
// are two bytes a lane (NVFP4; one, MXFP4) out of 8 (4) consecutive ones of
// each column: loaded so, four narrow loads a slab took 40% of the kernel's
// time.  Instead lane (col, grp) loads the grp-th quarter of its column's
// bytes in the slab at once, and the four lanes of a column exchange them.
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
  // NVFP4: the two bytes of step s in the low (s < 2) or high half of e[s % 2]; MXFP4: in
  // e[s] the FP32 pattern of step s's power of two (the conversions read the exponent field
  // alone, so byte 0, 2^-127, works too).
  __device__ __forceinline__ void exchange(int col, int grp, uint32_t (&e)[STEPS]) const {
    if constexpr (BYTES == 8) {
      // lane group g holds, of step g, the pairs for groups 0 ... 3; a 4 x 4 transposition
      const auto h = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
      const uint32_t lo = __builtin_amdgcn_perm(h[1], h[0], 0x05040100u);
      const uint32_t hi = __builtin_amdgcn_perm(h[1], h[0], 0x07060302u);
      const auto r = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
      e[0] = r[0], e[1] = r[1];
    } else if constexpr (!MX) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        e[s] = (uint32_t)__shfl((int)w[0], col + 16 * (2 * s + grp / 2)) >> (16 * (grp % 2));
    } else if constexpr (BYTES == 4) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        e[s] = ((uint32_t)__shfl((int)w[0], col + 16 * s) >> (8 * grp) & 255u) << 23;
    } else {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        e[s] = ((uint32_t)__shfl((int)w[0], col + 16 * (2 * s + grp / 2)) >> (8 * (grp % 2)) &
                255u)
               << 23;
    }
  }
};

// One workgroup: 64 * NT columns (tile x0 + blockIdx.x), 16 * RT rows (block
// y0 + blockIdx.y; with groups, all rows of that group in turn), split
// blockIdx.z of the slabs of KS elements of k.  x: the activations as the
// matrix instruction takes them, x_scale: NVFP4's inverse row scales.
template <bool MX, int RT, int NT>
__global__ __launch_bounds__(256) void linear_mfma(LinearArgs a, const uint16_t* x,
                                                   const float* x_scale, int64_t x0, int64_t y0,
                                                   int splits, float* partial) {
  constexpr int KS = RT == 1 ? 512 : 256, STEPS = KS / 128, RB = 16 * RT;
  constexpr int PIECES = KS / 8, PER_COPY = 64 / PIECES;  // 16-byte pieces a row; rows a copy
  __shared__ alignas(16) uint8_t xs[2][RB * KS * 2];
  const int lane = threadIdx.x % 64, col = lane % 16, grp = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t k = a.k, y = y0 + blockIdx.y;
  const int split = blockIdx.z;
  const Range range = a.offsets ? rows_of(a, y) : Range{y * RB, a.rows};
  const int64_t matrix = a.offsets ? y : 0;
  const int64_t slabs = (k + KS - 1) / KS;
  const int64_t slab_lo = slabs * split / splits, slab_hi = slabs * (split + 1) / splits;
  const int64_t n0 = (x0 + blockIdx.x) * 64 * NT + wave * 16 * NT;
  const uint8_t* codes[NT];
  const uint8_t* scales[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t n = matrix * a.n + min(n0 + t * 16 + col, a.n - 1);
    codes[t] = a.codes + n * (k / 2) + grp * 16;
    scales[t] = a.scales + n * (k / (MX ? 32 : 16)) + grp * ScaleLoad<MX, KS>::BYTES;
  }
  // where the lane's four 8-element pieces of a step lie in LDS: the pieces of row m are
  // stored in the order piece ^ (m mod 16), so that 16 rows' reads meet all banks once
  uint32_t at_piece[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) at_piece[q] = (uint32_t)(col * KS * 2 + ((grp * 4 + q) ^ col) * 16);

  for (int64_t m0 = range.first; m0 < range.last; m0 += RB) {
    const int rows = (int)min((int64_t)RB, range.last - m0);
    u32x4v w[NT][STEPS], w_next[NT][STEPS];
    ScaleLoad<MX, KS> e_next[NT];
    uint32_t e[NT][STEPS];
    auto load = [&](int64_t slab, u32x4v (&wv)[NT][STEPS], ScaleLoad<MX, KS> (&ev)[NT]) {
      const int64_t k0 = slab * KS;
      // activations: a copy fills 64 pieces; rows past the last are left as they are (their
      // columns of the result are not stored), pieces past k repeat the last (times weights 0)
#pragma unroll
      for (int i = 0; i < RB / PER_COPY / 4; ++i) {
        const int first = (i * 4 + wave) * PER_COPY;
        if (first < rows) {
          const int r = first + lane / PIECES;
          const int64_t piece = min(k0 / 8 + ((lane % PIECES) ^ (r & 15)), k / 8 - 1);
          __builtin_amdgcn_global_load_lds(
              x + (m0 + min(r, rows - 1)) * k + piece * 8,
              (lds_void*)(xs[slab & 1] + first * KS * 2), 16, 0, 0);
        }
      }
      const int left = (int)min((int64_t)KS, k - k0);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint8_t* c = codes[t] + k0 / 2;
        const uint8_t* b = scales[t] + k0 / (MX ? 32 : 16);
        if (left == KS) {
#pragma unroll
          for (int s = 0; s < STEPS; ++s) wv[t][s] = *(const u32x4v*)(c + s * 64);
          ev[t].whole(b);
        } else {
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const int at = s * 128 + grp * 32;
            wv[t][s] = (u32x4v){0, 0, 0, 0};
            if (at + 32 <= left) {
              wv[t][s] = *(const u32x4v*)(c + s * 64);
            } else if (!MX && at + 16 <= left) {
              const u32x2v half = *(const u32x2v*)(c + s * 64);
              wv[t][s] = (u32x4v){half[0], half[1], 0, 0};
            }
          }
          ev[t].some(b, left / (MX ? 32 : 16) - grp * ScaleLoad<MX, KS>::BYTES);
        }
      }
    };
    float4v acc[NT][RT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[t][r] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};

    if (m0 != range.first) __syncthreads();  // the last rows' slabs are read
    if (slab_lo < slab_hi) load(slab_lo, w_next, e_next);
    for (int64_t slab = slab_lo; slab < slab_hi; ++slab) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < STEPS; ++s) w[t][s] = w_next[t][s];
      __builtin_amdgcn_s_waitcnt(0);  // this wavefront's copies of the slab have landed
#pragma unroll
      for (int t = 0; t < NT; ++t) e_next[t].exchange(col, grp, e[t]);
      __syncthreads();                // and the others'; the slab before is read
      if (slab + 1 < slab_hi) load(slab + 1, w_next, e_next);
      const uint8_t* xb = xs[slab & 1];
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u32x4v xv[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r)
            if (r == 0 || r * 16 < rows)
              xv[r] = *(const u32x4v*)(xb + at_piece[q] + r * 16 * KS * 2 + s * 256);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t word = w[t][s][q];
            if constexpr (MX) {
              const float sc = __uint_as_float(e[t][s]);
              const bf16x2v b0 = e2m1_bf16x2<0>(word, sc), b1 = e2m1_bf16x2<1>(word, sc);
              const bf16x2v b2 = e2m1_bf16x2<2>(word, sc), b3 = e2m1_bf16x2<3>(word, sc);
              const bf16x8v wv = {b0[0], b0[1], b1[0], b1[1], b2[0], b2[1], b3[0], b3[1]};
#pragma unroll
              for (int r = 0; r < RT; ++r)
                if (r == 0 || r * 16 < rows)
                  acc[t][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                      wv, __builtin_bit_cast(bf16x8v, xv[r]), acc[t][r], 0, 0, 0);
            } else {
              const half2v both =
                  STEPS == 4 && s >= 2 ? e4m3_f16x2<1>(e[t][s % 2]) : e4m3_f16x2<0>(e[t][s % 2]);
              const half2v sc = {both[q / 2], both[q / 2]};
              const half2v h0 = e2m1x2_values_f16<0>(word) * sc;
              const half2v h1 = e2m1x2_values_f16<1>(word) * sc;
              const half2v h2 = e2m1x2_values_f16<2>(word) * sc;
              const half2v h3 = e2m1x2_values_f16<3>(word) * sc;
              const half8v wv = {h0[0], h0[1], h1[0], h1[1], h2[0], h2[1], h3[0], h3[1]};
#pragma unroll
              for (int r = 0; r < RT; ++r)
                if (r == 0 || r * 16 < rows)
                  acc[t][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                      wv, __builtin_bit_cast(half8v, xv[r]), acc[t][r], 0, 0, 0);
            }
          }
        }
      }
    }

    // lane (col, grp) holds columns n0 + 16 t + 4 grp + i of row m0 + 16 r + col
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int64_t m = m0 + r * 16 + col;
      if (r * 16 + col >= rows) continue;
      const float xs_inv = MX ? 1.0f : x_scale[m];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int64_t n = n0 + t * 16 + grp * 4;
        if (partial) {
          float* to = partial + ((int64_t)split * a.rows + m) * a.n + n;
          const float4v v = acc[t][r] * xs_inv;
          if (n + 4 <= a.n && a.n % 4 == 0) {
            *(float4v*)to = v;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n + i < a.n) to[i] = v[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < a.n) {
              const float s = MX ? 1.0f : a.row_scales[matrix * a.n + n + i];
              put_out(a, m * a.n + n + i, acc[t][r][i] * xs_inv * s);
            }
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
  for (int s = 0; s < splits; ++s) sum += partial[s * all + at];
  put_out(a, at, MX ? sum : sum * a.row_scales[at % a.n]);
}

// ---- shape of a call ------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  int dot_rows;  // rows of the dot form (1, 2, 4), 0: the matrix form
  int rt, nt;
  int64_t splits;
};

#ifndef DOT_W
#define DOT_W 4
#endif
#ifndef DOT_NC1
#define DOT_NC1 2
#endif
#ifndef LIN_TARGET
#define LIN_TARGET 512
#endif
#ifndef LIN_NT1
#define LIN_NT1 1
#endif

Plan plan_of(int64_t rows, int64_t n, int64_t k, int64_t groups) {
  Plan p{0, 1, 1, 1};
  if (groups == 0 && rows <= 4) {
    p.dot_rows = rows <= 2 ? (int)rows : 4;
    return p;
  }
  const int64_t each = groups ? ceil_div(rows, groups) : rows;
  p.rt = each <= 16 ? 1 : each <= 32 ? 2 : 4;
  p.nt = p.rt == 1 ? LIN_NT1 : 2;
  if (groups == 0) {
    const int64_t tiles = ceil_div(n, 64 * p.nt) * ceil_div(rows, 16 * p.rt);
    const int64_t slabs = ceil_div(k, p.rt == 1 ? 512 : 256);
    p.splits = ceil_div(LIN_TARGET, tiles);
    if (p.splits > slabs) p.splits = slabs;
    if (p.splits > 16) p.splits = 16;
  }
  return p;
}

// Workspace: NVFP4's converted activations and their scales, then the
// splits' partial sums, each from a 16-byte boundary.
int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

struct Space {
  int64_t scale, partial, bytes;
};

Space space_of(bool mx, const Plan& p, int64_t rows, int64_t n, int64_t k) {
  Space s{0, 0, 0};
  if (p.dot_rows) return s;
  s.scale = mx ? 0 : round16(rows * k * 2);
  s.partial = mx ? 0 : s.scale + round16(rows * 4);
  s.bytes = s.partial + (p.splits > 1 ? p.splits * rows * n * 4 : 0);
  return s;
}

// The dispatch packet counts work-items in 32 bits, and the second grid
// dimension 16: larger calls go in several launches.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 31) / 256;

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

template <bool MX, int RT, int NT>
hipError_t mfma(const LinearArgs& a, const Plan& p, hipStream_t stream) {
  const Space space = space_of(MX, p, a.rows, a.n, a.k);
  uint8_t* ws = (uint8_t*)a.workspace;
  const uint16_t* x = MX ? (const uint16_t*)a.x : (const uint16_t*)ws;
  float* x_scale = MX ? nullptr : (float*)(ws + space.scale);
  if (!MX) {
    for (int64_t r0 = 0; r0 < a.rows; r0 += kMaxBlocks) {
      const int64_t n = a.rows - r0 < kMaxBlocks ? a.rows - r0 : kMaxBlocks;
      linear_convert<<<(uint32_t)n, 256, 0, stream>>>(a, r0, (uint16_t*)ws, x_scale);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  float* partial = p.splits > 1 ? (float*)(ws + space.partial) : nullptr;
  const int64_t xs = ceil_div(a.n, 64 * NT);
  const int64_t ys = a.groups ? a.groups : ceil_div(a.rows, 16 * RT);
  const int64_t dx = xs < kMaxBlocks / p.splits ? xs : kMaxBlocks / p.splits;
  int64_t dy = kMaxBlocks / (dx * p.splits);
  if (dy > 65535) dy = 65535;
  for (int64_t y0 = 0; y0 < ys; y0 += dy)
    for (int64_t x0 = 0; x0 < xs; x0 += dx) {
      const dim3 grid((uint32_t)(xs - x0 < dx ? xs - x0 : dx),
                      (uint32_t)(ys - y0 < dy ? ys - y0 : dy), (uint32_t)p.splits);
      linear_mfma<MX, RT, NT><<<grid, 256, 0, stream>>>(a, x, x_scale, x0, y0, (int)p.splits,
                                                        partial);
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
  if (p.dot_rows == 1) return dot<MX, 1, DOT_NC1, DOT_W>(a, stream);
  if (p.dot_rows == 2) return dot<MX, 2, 2, DOT_W>(a, stream);
  if (p.dot_rows == 4) return dot<MX, 4, 2, DOT_W>(a, stream);
  if (p.rt == 1) return mfma<MX, 1, LIN_NT1>(a, p, stream);
  if (p.rt == 2) return mfma<MX, 2, 2>(a, p, stream);
  return mfma<MX, 4, 2>(a, p, stream);
}

}  // namespace

int64_t linear_workspace_bytes(bool mx, int64_t rows, int64_t n, int64_t k, int64_t groups) {
  return space_of(mx, plan_of(rows, n, k, groups), rows, n, k).bytes;
}

hipError_t linear_launch(bool mx, const LinearArgs& a, hipStream_t stream) {
  return mx ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace fp4q
