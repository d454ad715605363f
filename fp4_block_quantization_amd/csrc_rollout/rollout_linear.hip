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
// the activations as FP16 scaled by a power of two per row and slab of k
// (exact for elements within 2^29 of the row's largest there); an MXFP4
// weight is an exact BF16 number that the conversion's own scale operand
// gives, and the activations stay BF16.  A slab of activations is converted
// once per workgroup into LDS and shared by its four wavefronts.
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

// The FP32 pattern of an E8M0 byte's power of two; the conversions read the
// exponent field alone, so byte 0 (2^-127) works too.
__device__ __forceinline__ float e8m0_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

template <int SEL>
__device__ __forceinline__ bf16x2v e2m1_bf16x2(uint32_t w, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL);
}

__device__ __forceinline__ float dot2(bf16x2v a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(short2v, a),
                                         __builtin_bit_cast(short2v, b), c, false);
}

// ---- few rows -----------------------------------------------------------------

template <bool MX, int ROWS, int NC>
__global__ __launch_bounds__(256) void linear_dot(LinearArgs a, int64_t x0) {
  const int lane = threadIdx.x % 64;
  const int64_t n0 = ((x0 + blockIdx.x) * 4 + threadIdx.x / 64) * NC;
  if (n0 >= a.n) return;
  const int64_t k = a.k;
  const uint8_t* codes[NC];
  const uint8_t* scales[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t n = min(n0 + c, a.n - 1);
    codes[c] = a.codes + n * (k / 2);
    scales[c] = a.scales + n * (k / (MX ? 32 : 16));
  }
  const uint16_t* x[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) x[r] = (const uint16_t*)a.x + min((int64_t)r, a.rows - 1) * k;
  float sum[NC][ROWS];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) sum[c][r] = 0.0f;

  for (int64_t k0 = lane * 32; k0 < k; k0 += 2048) {
    const bool whole = k0 + 32 <= k;  // else the column ends after 16 (k is a multiple of 16)
    u32x4v w[NC], xv[ROWS][4];
    uint32_t e[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (whole) {
        w[c] = __builtin_nontemporal_load((const u32x4v*)(codes[c] + k0 / 2));
      } else {
        const u32x2v half = *(const u32x2v*)(codes[c] + k0 / 2);
        w[c] = (u32x4v){half[0], half[1], 0, 0};
      }
      if constexpr (MX) {
        e[c] = scales[c][k0 / 32];
      } else {
        e[c] = scales[c][k0 / 16];
        if (whole) e[c] |= (uint32_t)scales[c][k0 / 16 + 1] << 8;
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xv[r][i] = whole || i < 2 ? *(const u32x4v*)(x[r] + k0 + i * 8) : (u32x4v){0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float part[2][ROWS];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) part[h][r] = 0.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t word = w[c][2 * h + q];
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
        const float s = __builtin_ldexpf(1.0f, (int)e[c] - 127);
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
          sum[c][r] = __builtin_fmaf(part[0][r] + part[1][r], s, sum[c][r]);
      } else {
        const float s0 = e4m3_value<0>(e[c]), s1 = e4m3_value<1>(e[c]);
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
          sum[c][r] = __builtin_fmaf(part[1][r], s1, __builtin_fmaf(part[0][r], s0, sum[c][r]));
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

// One workgroup: 64 * NT columns (tile x0 + blockIdx.x), 16 * RT rows (block
// y0 + blockIdx.y; with groups, all rows of that group in turn), split
// blockIdx.z of the slabs of KS elements of k.
template <bool MX, int RT, int NT>
__global__ __launch_bounds__(256) void linear_mfma(LinearArgs a, int64_t x0, int64_t y0,
                                                   int splits, float* partial) {
  constexpr int KS = 1024 / RT, STEPS = KS / 128, RB = 16 * RT;
  constexpr int PITCH = KS + 8;  // LDS row in elements: neighbouring rows 4 banks apart
  __shared__ alignas(16) uint16_t xs[RB * PITCH];
  __shared__ float slab_scale[RB];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, col = lane % 16, grp = lane / 16;
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
    scales[t] = a.scales + n * (k / (MX ? 32 : 16)) + grp * (MX ? 1 : 2);
  }

  for (int64_t m0 = range.first; m0 < range.last; m0 += RB) {
    const int rows = (int)min((int64_t)RB, range.last - m0);
    float4v acc[NT][RT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[t][r] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};

    for (int64_t slab = slab_lo; slab < slab_hi; ++slab) {
      const int64_t k0 = slab * KS;
      const int left = (int)min((int64_t)KS, k - k0);  // elements of k in this slab
      // weights of the slab
      u32x4v w[NT][STEPS];
      uint32_t e[NT][STEPS];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int at = s * 128 + grp * 32;
          const uint8_t* c = codes[t] + k0 / 2 + s * 64;
          const uint8_t* b = scales[t] + (MX ? k0 / 32 + s * 4 : k0 / 16 + s * 8);
          if (at + 32 <= left) {
            w[t][s] = *(const u32x4v*)c;
            if constexpr (MX)
              e[t][s] = *b;
            else
              e[t][s] = b[0] | (uint32_t)b[1] << 8;
          } else if (!MX && at + 16 <= left) {
            const u32x2v half = *(const u32x2v*)c;
            w[t][s] = (u32x4v){half[0], half[1], 0, 0};
            e[t][s] = b[0];
          } else {
            w[t][s] = (u32x4v){0, 0, 0, 0};
            e[t][s] = 0;
          }
        }
      // activations of the slab into LDS, 256 / RB threads to a row
      {
        constexpr int TPR = 256 / RB, PIECES = KS / 8 / TPR;  // 16-byte pieces per thread
        const int r = threadIdx.x / TPR, part = threadIdx.x % TPR;
        u32x4v v[PIECES];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const int at = (i * TPR + part) * 8;
          v[i] = r < rows && at < left
                     ? *(const u32x4v*)((const uint16_t*)a.x + (m0 + r) * k + k0 + at)
                     : (u32x4v){0, 0, 0, 0};
        }
        if constexpr (!MX) {
#pragma unroll
          for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              top = max(top, max(v[i][j] & 0x7FFFu, v[i][j] >> 16 & 0x7FFFu));
#pragma unroll
          for (int s = TPR / 2; s > 0; s >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, s));
          const int field = (int)(top >> 7);
          // the largest element lands in [2^14, 2^15); zeros, NaN and infinity stay
          const int ex = top == 0 || field == 255 ? 0 : 14 + 127 - max(field, 1);
#pragma unroll
          for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const half2v h = {(_Float16)__builtin_ldexpf(bf16_lo(v[i][j]), ex),
                                (_Float16)__builtin_ldexpf(bf16_hi(v[i][j]), ex)};
              v[i][j] = __builtin_bit_cast(uint32_t, h);
            }
          if (slab != slab_lo || m0 != range.first) __syncthreads();
          if (part == 0) slab_scale[r] = __builtin_ldexpf(1.0f, -ex);
        } else {
          if (slab != slab_lo || m0 != range.first) __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          *(u32x4v*)&xs[r * PITCH + (i * TPR + part) * 8] = v[i];
      }
      __syncthreads();

      float4v slab_acc[NT][RT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < RT; ++r)
          slab_acc[t][r] = MX ? acc[t][r] : (float4v){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u32x4v xv[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r)
            xv[r] = *(const u32x4v*)&xs[(r * 16 + col) * PITCH + s * 128 + grp * 32 + q * 8];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t word = w[t][s][q];
            if constexpr (MX) {
              const float sc = e8m0_scale(e[t][s]);
              const bf16x2v b0 = e2m1_bf16x2<0>(word, sc), b1 = e2m1_bf16x2<1>(word, sc);
              const bf16x2v b2 = e2m1_bf16x2<2>(word, sc), b3 = e2m1_bf16x2<3>(word, sc);
              const bf16x8v wv = {b0[0], b0[1], b1[0], b1[1], b2[0], b2[1], b3[0], b3[1]};
#pragma unroll
              for (int r = 0; r < RT; ++r)
                slab_acc[t][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    wv, __builtin_bit_cast(bf16x8v, xv[r]), slab_acc[t][r], 0, 0, 0);
            } else {
              const half2v both = __builtin_bit_cast(
                  half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)e[t][s], 1.0f, false));
              const half2v sc = {both[q / 2], both[q / 2]};
              const half2v h0 = e2m1x2_values_f16<0>(word) * sc, h1 = e2m1x2_values_f16<1>(word) * sc;
              const half2v h2 = e2m1x2_values_f16<2>(word) * sc, h3 = e2m1x2_values_f16<3>(word) * sc;
              const half8v wv = {h0[0], h0[1], h1[0], h1[1], h2[0], h2[1], h3[0], h3[1]};
#pragma unroll
              for (int r = 0; r < RT; ++r)
                slab_acc[t][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    wv, __builtin_bit_cast(half8v, xv[r]), slab_acc[t][r], 0, 0, 0);
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if constexpr (MX)
            acc[t][r] = slab_acc[t][r];
          else
            acc[t][r] += slab_acc[t][r] * slab_scale[r * 16 + col];
        }
    }

    // lane (col, grp) holds columns n0 + 16 t + 4 grp + i of row m0 + 16 r + col
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t n = n0 + t * 16 + grp * 4;
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[i] = MX || partial || n + i >= a.n ? 1.0f : a.row_scales[matrix * a.n + n + i];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int64_t m = m0 + r * 16 + col;
        if (r * 16 + col >= rows) continue;
        if (partial) {
          float* to = partial + ((int64_t)split * a.rows + m) * a.n + n;
          if (n + 4 <= a.n && a.n % 4 == 0) {
            *(float4v*)to = acc[t][r];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n + i < a.n) to[i] = acc[t][r][i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < a.n) put_out(a, m * a.n + n + i, acc[t][r][i] * s[i]);
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

Plan plan_of(int64_t rows, int64_t n, int64_t k, int64_t groups) {
  Plan p{0, 1, 1, 1};
  if (groups == 0 && rows <= 4) {
    p.dot_rows = rows <= 2 ? (int)rows : 4;
    return p;
  }
  const int64_t each = groups ? ceil_div(rows, groups) : rows;
  p.rt = each <= 16 ? 1 : each <= 32 ? 2 : 4;
  p.nt = p.rt == 1 ? 1 : 2;
  if (groups == 0) {
    const int64_t tiles = ceil_div(n, 64 * p.nt) * ceil_div(rows, 16 * p.rt);
    const int64_t slabs = ceil_div(k, 1024 / p.rt);
    p.splits = ceil_div(512, tiles);
    if (p.splits > slabs) p.splits = slabs;
    if (p.splits > 16) p.splits = 16;
  }
  return p;
}

// The dispatch packet counts work-items in 32 bits, and the second grid
// dimension 16: larger calls go in several launches.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 31) / 256;

template <bool MX, int ROWS, int NC>
hipError_t dot(const LinearArgs& a, hipStream_t stream) {
  const int64_t blocks = ceil_div(a.n, 4 * NC);
  for (int64_t x0 = 0; x0 < blocks; x0 += kMaxBlocks) {
    const int64_t n = blocks - x0 < kMaxBlocks ? blocks - x0 : kMaxBlocks;
    linear_dot<MX, ROWS, NC><<<(uint32_t)n, 256, 0, stream>>>(a, x0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool MX, int RT, int NT>
hipError_t mfma(const LinearArgs& a, const Plan& p, hipStream_t stream) {
  const int64_t xs = ceil_div(a.n, 64 * NT);
  const int64_t ys = a.groups ? a.groups : ceil_div(a.rows, 16 * RT);
  const int64_t dx = xs < kMaxBlocks / p.splits ? xs : kMaxBlocks / p.splits;
  int64_t dy = kMaxBlocks / (dx * p.splits);
  if (dy > 65535) dy = 65535;
  for (int64_t y0 = 0; y0 < ys; y0 += dy)
    for (int64_t x0 = 0; x0 < xs; x0 += dx) {
      const dim3 grid((uint32_t)(xs - x0 < dx ? xs - x0 : dx),
                      (uint32_t)(ys - y0 < dy ? ys - y0 : dy), (uint32_t)p.splits);
      linear_mfma<MX, RT, NT><<<grid, 256, 0, stream>>>(
          a, x0, y0, (int)p.splits, p.splits > 1 ? (float*)a.workspace : nullptr);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

template <bool MX>
hipError_t launch(const LinearArgs& a, hipStream_t stream) {
  const Plan p = plan_of(a.rows, a.n, a.k, a.groups);
  if (p.dot_rows == 1) return dot<MX, 1, 2>(a, stream);
  if (p.dot_rows == 2) return dot<MX, 2, 2>(a, stream);
  if (p.dot_rows == 4) return dot<MX, 4, 4>(a, stream);
  const hipError_t e = p.rt == 1   ? mfma<MX, 1, 1>(a, p, stream)
                       : p.rt == 2 ? mfma<MX, 2, 2>(a, p, stream)
                                   : mfma<MX, 4, 2>(a, p, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  // several splits: fewer than 512 tiles of at most 64 rows and 128 columns
  linear_join<MX><<<(uint32_t)ceil_div(a.rows * a.n, 256), 256, 0, stream>>>(
      a, (int)p.splits, (const float*)a.workspace);
  return hipGetLastError();
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
