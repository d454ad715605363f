// rollout_attention.hip -- softmax attention over the paged NVFP4 cache,
// with a prefix shared by groups of sequences (definitions in
// include/fp4q/rollout.h).
//
// Mathematics.  With cached rows k_t = s_t (e g)_t and v_t = s'_t (e' g')_t,
// the products g e are FP16 numbers (at most 6 significant bits, 2^-10 to
// 2688), so the matrix units take them as they are:
//   S[t][q] = sum_d (g e)[t][d] q[d]       q scaled by a power of two into
//                                          FP16's range, exactly
//   x = S s_t c_q                          c_q: scale, log2(e), q's power of two
//   p = 2^(x - m), l += p, m the running maximum of x
//   O[d][q] += sum_t (g' e')[t][d] w,  w = FP16(p s'_t / b)
// with b a power of two at or above every s'_t met so far times 2^-15: token
// scales differ by orders of magnitude, and w keeps FP16's full precision
// over 29 binades below the largest (probabilities are rounded to 11 bits;
// BF16, with 8, is what the output holds).  The scales s and s' cost one
// multiplication per score instead of one per element.
//
// Layout.  S is computed transposed (keys as rows of the 16x16x32 matrix
// instruction, queries as columns): a lane then holds, for one query, four
// consecutive tokens of every 16, and that is already the operand layout of
// the value product when the values' token order is permuted alike.  The
// values, stored token by token, are turned by the LDS's 4-bit transposing
// read, codes still packed; the block scales of the values are stored token
// innermost so that a lane's four tokens are one word.
//
// Work.  One wavefront takes a tile of 64 tokens at a time and up to
// 16 * RT query rows of one cache head (a sequence's queries and the heads
// that share the cache head; for a prefix, those of all sequences of the
// group, so that the prefix is read once per 16 * RT of them).  The WAVES
// wavefronts of a workgroup take tiles in turn and merge their (m, l, O)
// through LDS; a long context is split over several workgroups, whose
// partial results a second kernel joins in a fixed order.
#include "fp4q_device.h"
#include "rollout_launch.h"

namespace fp4q {
namespace {

typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef int int2v __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr int kTile = 64;  // tokens per step of a wavefront

struct Params {
  const uint8_t* codes[2];  // keys, values
  const uint8_t* scales[2];
  const float* token_scales[2];
  const uint16_t* q;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* prefix_table;
  const int32_t* prefix_lens;
  const int32_t* group_offsets;
  uint16_t* out;
  float* lse;
  float* part_o;   // [splits][rows][D]
  float2* part_ml; // [splits][rows]
  int64_t q_stride, rows;
  int32_t num_pages, page_size, page_groups, kv_heads, per_head;  // per_head: q_heads / kv_heads
  int32_t batch, q_tokens, q_heads, max_pages, max_prefix_pages, groups;
  int32_t own_blocks, own_splits, prefix_blocks, prefix_splits;
  float scale;
};

__device__ __forceinline__ float max_of_halves(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_of_groups(float x) {  // over lanes l, l^16, l^32, l^48
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return max_of_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_of_groups(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float y = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const uint32_t w = __float_as_uint(y);
  const auto h = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}

// The two E4M3 bytes of a word's low (0) or high (1) half as FP16, exact.
template <int SEL>
__device__ __forceinline__ half2v e4m3_f16x2(uint32_t w) {
  return __builtin_bit_cast(half2v,
                            __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, SEL != 0));
}

// 8 codes of one word times one scale pair per two codes.
__device__ __forceinline__ half8v decode8(uint32_t w, half2v e0, half2v e1, half2v e2, half2v e3) {
  const half2v a = e2m1x2_values_f16<0>(w) * e0, b = e2m1x2_values_f16<1>(w) * e1;
  const half2v c = e2m1x2_values_f16<2>(w) * e2, d = e2m1x2_values_f16<3>(w) * e3;
  return (half8v){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float factor(float m, float top) {  // 2^(m - top), 0 for m = -inf
  return __builtin_amdgcn_exp2f(m - top);
}

// What a workgroup works on: a block of query rows of one cache head, and
// the tokens [0, len) of one page-table row.
struct Job {
  const int32_t* table;
  int32_t len;       // tokens any row of the block sees
  int32_t floor;     // tokens every row of the block sees
  int32_t first_b;   // row r belongs to sequence first_b + r / (T * per_head)
  int32_t row0;      // first row of the block, counted from first_b's first
  int32_t rows;      // rows in the block
  int32_t own_len;   // own tokens: the limit of row r is own_len - T + 1 + t (prefix: len)
  int32_t kvh, split, splits, part;  // part: index of this split's partial result
  bool prefix;
};

__device__ __forceinline__ int64_t global_row(const Params& p, const Job& j, int r) {
  const int per_seq = p.q_tokens * p.per_head;
  const int rr = j.row0 + r, b = rr / per_seq, in = rr - b * per_seq;
  const int t = in / p.per_head, g = in - t * p.per_head;
  return ((int64_t)(j.first_b + b) * p.q_tokens + t) * p.q_heads + j.kvh * p.per_head + g;
}

// The job of workgroup `block`; false: none.  The prefix's workgroups come
// first (they are the longest), then the sequences' own.
template <int RB>
__device__ __forceinline__ bool job_of(const Params& p, int64_t block, Job& j) {
  const int per_seq = p.q_tokens * p.per_head;
  const int64_t prefix_jobs = (int64_t)p.prefix_blocks * p.kv_heads * p.prefix_splits;
  j.prefix = block < prefix_jobs;
  if (j.prefix) {
    // row blocks innermost, 8 apart: those of one head and split run together on one of the
    // 8 dies, whose cache then holds the tokens they share
    const int64_t pairs = (int64_t)p.kv_heads * p.prefix_splits;
    const int pair = (int)(block % pairs), slot = (int)(block / pairs);
    j.kvh = pair / p.prefix_splits;
    j.split = pair - j.kvh * p.prefix_splits;
    j.splits = p.prefix_splits;
    j.part = j.split;
    // the slot-th row block over all groups: each lane counts one group's blocks
    const int lane = threadIdx.x % 64;
    int before = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 64) {
      const int g = g0 + lane;
      int lo = 0, hi = 0;
      if (g < p.groups) {
        lo = min(max(p.group_offsets[g], 0), p.batch);
        hi = min(max(p.group_offsets[g + 1], lo), p.batch);
      }
      const int rows = (hi - lo) * per_seq, n = (rows + RB - 1) / RB;
      int upto = n;
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const int other = __shfl_up(upto, s);
        if (lane >= s) upto += other;
      }
      const uint64_t past = __ballot(before + upto > slot);
      if (past != 0) {
        const int at = __builtin_ctzll(past);
        const int block_in = slot - before - (__shfl(upto, at) - __shfl(n, at));
        j.first_b = __builtin_amdgcn_readfirstlane(__shfl(lo, at));
        j.row0 = __builtin_amdgcn_readfirstlane(block_in) * RB;
        j.rows = min(RB, __builtin_amdgcn_readfirstlane(__shfl(rows, at)) - j.row0);
        const int group = g0 + at;
        j.table = p.prefix_table + (int64_t)group * p.max_prefix_pages;
        j.len = min(max(p.prefix_lens[group], 0), p.max_prefix_pages * p.page_size);
        j.len = __builtin_amdgcn_readfirstlane(j.len);
        j.floor = j.own_len = j.len;
        return true;
      }
      before += __shfl(upto, 63);
    }
    return false;
  }
  block -= prefix_jobs;
  j.split = (int)(block % p.own_splits);
  block /= p.own_splits;
  j.kvh = (int)(block % p.kv_heads);
  block /= p.kv_heads;
  const int rb = (int)(block % p.own_blocks);
  j.first_b = (int)(block / p.own_blocks);
  j.splits = p.own_splits;
  j.part = p.prefix_splits + j.split;
  j.row0 = rb * RB;
  j.rows = min(RB, per_seq - j.row0);
  j.table = p.page_table + (int64_t)j.first_b * p.max_pages;
  j.own_len = min(max(p.seq_lens[j.first_b], 0), p.max_pages * p.page_size);
  const int first = j.own_len - p.q_tokens + 1;  // the limit of query 0
  j.len = max(0, first + (j.row0 + j.rows - 1) / p.per_head);
  j.floor = max(0, first + j.row0 / p.per_head);
  return true;
}

template <int D, int RT, int WAVES>
struct Shared {
  static constexpr int kVRow = D / 2 + 16;  // padded: neighbouring rows start 16 banks on
  struct Tile {
    alignas(16) uint8_t codes[kTile * kVRow];
    alignas(16) uint8_t scales[D / 16][kTile];  // [block][4 (t/4 % 4)][t / 16][t % 4]
    alignas(16) float k_scale[kTile];
    alignas(16) float v_scale[kTile];
  };
  struct Merge {
    float o[WAVES][16][D + 4];
    float2 ml[WAVES][16];
  };
  union {
    Tile tile[WAVES];
    Merge merge;
  };
};

template <int D, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, RT == 2 && D > 128 ? 1 : 2) void attention_kernel(Params p) {
  constexpr int DT = D / 16, NK = D / 32, KS = D / 64, VL = D / 32;
  constexpr int EU = (DT * 8 + 63) / 64;  // 8-token pieces of value scales per lane
  constexpr int RB = 16 * RT;
  __shared__ Shared<D, RT, WAVES> sh;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int col = lane % 16, grp = lane / 16;
  Job job;
  if (!job_of<RB>(p, blockIdx.x, job)) return;

  const int tiles = (job.len + kTile - 1) / kTile;
  const int tile_lo = (int)((int64_t)tiles * job.split / job.splits);
  const int tile_hi = (int)((int64_t)tiles * (job.split + 1) / job.splits);
  const int steps = max(0, (tile_hi - tile_lo - wave + WAVES - 1) / WAVES);
  const int last_group = (job.len - 1) / 16;

  // queries: lane (col, grp) holds row col's elements [grp * D/4, (grp + 1) * D/4)
  half8v q[RT][NK];
  float c_q[RT];
  int limit[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = rt * 16 + col;
    const bool live = r < job.rows;
    const int rr = job.row0 + (live ? r : 0);
    limit[rt] = job.prefix ? job.len
                           : job.own_len - p.q_tokens + 1 + rr / p.per_head;
    u32x4v raw[NK];
    const int64_t row = global_row(p, job, live ? r : 0);
    const int64_t bt = row / p.q_heads;
    const uint16_t* src = p.q + bt * p.q_stride + (row - bt * p.q_heads) * D + grp * (D / 4);
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      raw[k] = live ? ((const u32x4v*)src)[k] : (u32x4v){0, 0, 0, 0};
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, w[i] >> 16 & 0x7FFFu));
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    // 2^ex: the row's largest element lands in [2^14, 2^15).  A row of zeros, or one
    // with a NaN or infinity, stays as it is
    const int field = (int)(top >> 7);
    const int ex = top == 0 || field == 255 ? 0 : 14 + 127 - max(field, 1);
    const float sign = p.scale < 0.0f ? -1.0f : 1.0f;
    c_q[rt] = __builtin_ldexpf(__builtin_fabsf(p.scale) * kLog2e, -ex);
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[rt][k][2 * i] = (_Float16)__builtin_ldexpf(bf16_lo(w[i]) * sign, ex);
        q[rt][k][2 * i + 1] = (_Float16)__builtin_ldexpf(bf16_hi(w[i]) * sign, ex);
      }
    }
  }

  float4v o[RT][DT];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY;
    l[rt] = 0.0f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[rt][dt] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  }
  // value scales up to `bound` times `norm` reach 2^15
  float bound = 0.0f, norm = 1.0f;

  // Pages: lane 4 k + j holds the place of the 16 tokens j of step 16 n + k.
  int64_t page_head = 0;  // page * kv_heads + head
  int32_t page_at = 0;    // first token's place in the page
  auto load_pages = [&](int first_step) {
    const int tile = tile_lo + wave + (first_step + lane / 4) * WAVES;
    const int g = min(tile * 4 + lane % 4, last_group);
    const int page = g / p.page_groups;
    const int id = min(max(job.table[page], 0), p.num_pages - 1);
    page_head = (int64_t)id * p.kv_heads + job.kvh;
    page_at = (g - page * p.page_groups) * 16;
  };
  int64_t at_ph[4];  // of the step being loaded: page and head, and place, of its 16-token groups
  int32_t at_place[4];
  auto locate = [&](int step) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int from = (step % 16) * 4 + j;
      at_ph[j] = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)page_head, from) |
                              (uint64_t)(uint32_t)__builtin_amdgcn_readlane(
                                  (int)(page_head >> 32), from)
                                  << 32);
      at_place[j] = __builtin_amdgcn_readlane(page_at, from);
    }
  };
#define FP4Q_PICK(v, j) ((j) == 0 ? v[0] : (j) == 1 ? v[1] : (j) == 2 ? v[2] : v[3])

  uint32_t kw[4][NK];     // key codes: token 16 j + col, elements grp * D/4 ...
  uint32_t ks[4];         // their block scales
  u32x4v vw[VL];          // value codes, 16-byte pieces in memory order
  u32x2v ve[EU];          // value block scales, 8 tokens each
  float kt = 0.0f, vt = 0.0f;
  auto load_values = [&]() {
    int64_t row[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) row[j] = at_ph[j] * p.page_size + at_place[j];
#pragma unroll
    for (int r = 0; r < VL; ++r) {
      const int piece = r * 64 + lane, t = piece / VL, in = piece - t * VL;
      vw[r] = *(const u32x4v*)(p.codes[1] + (FP4Q_PICK(row, t / 16) + t % 16) * (D / 2) + in * 16);
    }
#pragma unroll
    for (int r = 0; r < EU; ++r) {
      const int u = r * 64 + lane, dt = u / 8, j = u / 2 % 4;
      const int64_t at = FP4Q_PICK(at_place, j) + u % 2 * 8;
      if (DT * 8 % 64 == 0 || u < DT * 8)
        ve[r] = *(const u32x2v*)(p.scales[1] + (FP4Q_PICK(at_ph, j) * DT + dt) * p.page_size + at);
    }
    const int64_t mine = FP4Q_PICK(row, lane / 16) + col;
    kt = p.token_scales[0][mine];
    vt = p.token_scales[1][mine];
  };
  auto load_keys = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = at_ph[j] * p.page_size + at_place[j] + col;
      const uint8_t* src = p.codes[0] + row * (D / 2) + grp * (D / 8);
      if constexpr (NK % 4 == 0) {
#pragma unroll
        for (int k = 0; k < NK; k += 4) {
          const uint4 w = *(const uint4*)(src + k * 4);
          kw[j][k] = w.x, kw[j][k + 1] = w.y, kw[j][k + 2] = w.z, kw[j][k + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < NK; k += 2) {
          const uint2 w = *(const uint2*)(src + k * 4);
          kw[j][k] = w.x, kw[j][k + 1] = w.y;
        }
      }
      const uint8_t* sc = p.scales[0] + row * DT + grp * KS;
      if constexpr (KS == 4)
        ks[j] = *(const uint32_t*)sc;
      else if constexpr (KS == 2)
        ks[j] = *(const uint16_t*)sc;
      else if constexpr (KS == 1)
        ks[j] = *sc;
      else
        ks[j] = sc[0] | sc[1] << 8 | sc[2] << 16;
    }
  };

#undef FP4Q_PICK

  auto& tile = sh.tile[wave];
  if (steps > 0) {
    load_pages(0);
    locate(0);
    load_values();
    load_keys();
  }
  for (int step = 0; step < steps; ++step) {
    const int t0 = (tile_lo + wave + step * WAVES) * kTile;
    const int left = job.len - t0;  // tokens of this tile that exist
    // values and scales into LDS; scales of tokens past the end become zero, so that
    // whatever lies there adds nothing
#pragma unroll
    for (int r = 0; r < VL; ++r) {
      const int piece = r * 64 + lane, t = piece / VL, in = piece - t * VL;
      *(u32x4v*)(tile.codes + t * Shared<D, RT, WAVES>::kVRow + in * 16) = vw[r];
    }
#pragma unroll
    for (int r = 0; r < EU; ++r) {
      const int u = r * 64 + lane, dt = u / 8, j = u / 2 % 4, half = u % 2;
      u32x2v e = ve[r];
      if (left < kTile) {
        const int n = min(max(left - 16 * j - 8 * half, 0), 8);  // of these 8 tokens
        const uint64_t keep = n == 0 ? 0 : ~(uint64_t)0 >> (64 - 8 * n);
        e.x &= (uint32_t)keep;
        e.y &= (uint32_t)(keep >> 32);
      }
      if (DT * 8 % 64 == 0 || u < DT * 8) {
        *(uint32_t*)&tile.scales[dt][(2 * half) * 16 + j * 4] = e.x;
        *(uint32_t*)&tile.scales[dt][(2 * half + 1) * 16 + j * 4] = e.y;
      }
    }
    const float vt_live = lane < left ? vt : 0.0f;
    if (__any(vt_live > bound)) {
      // a larger value scale than any before: a new power of two, with room for 8 times more
      const float top = max_of_groups(vt_live);
      float all = top;
#pragma unroll
      for (int s = 8; s > 0; s /= 2) all = fmaxf(all, __shfl_xor(all, s));
      const int ex = min(max(((int)(__float_as_uint(all) >> 23) & 255) - 126, -90) + 3, 120);
      const float grown = __builtin_ldexpf(1.0f, ex);
      const float shrink = bound == 0.0f ? 1.0f : bound / grown;
      bound = grown;
      norm = __builtin_ldexpf(1.0f, 15 - ex);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[rt][dt] *= shrink;
    }
    tile.k_scale[lane] = kt;
    tile.v_scale[lane] = vt_live * norm;
    if (step + 1 < steps) {
      if ((step + 1) % 16 == 0) load_pages(step + 1);
      locate(step + 1);
      load_values();
    }

    // scores
    float4v s[RT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
      const half2v e01 = e4m3_f16x2<0>(ks[j]), e23 = e4m3_f16x2<1>(ks[j]);
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int b = k / 2;  // 16-element block of the lane's range
        const _Float16 e1 = b < 2 ? e01[b % 2] : e23[b % 2];
        const half2v e = {e1, e1};
        const half8v key = decode8(kw[j][k], e, e, e, e);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          if (rt == 0 || rt * 16 < job.rows)
            s[rt][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[rt][k], s[rt][j], 0, 0, 0);
      }
    }
    if (step + 1 < steps) load_keys();

    // softmax
    half8v w[RT][2];
    const bool edge = t0 + kTile > job.floor;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt > 0 && rt * 16 >= job.rows) continue;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4v sc = *(const float4v*)&tile.k_scale[16 * j + 4 * grp];
        s[rt][j] *= sc;
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t0 + 16 * j + 4 * grp + i >= limit[rt]) s[rt][j][i] = -INFINITY;
        }
        top = fmaxf(top, fmaxf(fmaxf(s[rt][j][0], s[rt][j][1]), fmaxf(s[rt][j][2], s[rt][j][3])));
      }
      top = max_of_groups(top);
      top = top == -INFINITY ? top : top * c_q[rt];
      if (__any(top > m[rt])) {
        const float grown = fmaxf(m[rt], top);
        const float keep = m[rt] == -INFINITY ? 1.0f : factor(m[rt], grown);
        m[rt] = grown;
        l[rt] *= keep;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[rt][dt] *= keep;
      }
      const float base = m[rt] == -INFINITY ? 0.0f : m[rt];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4v sc = *(const float4v*)&tile.v_scale[16 * j + 4 * grp];
        float4v e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][j][i], c_q[rt], -base));
          if (edge && t0 + 16 * j + 4 * grp + i >= limit[rt]) e[i] = 0.0f;
          l[rt] += e[i];
        }
        e *= sc;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[rt][j / 2][j % 2 * 4 + i] = (_Float16)e[i];
      }
    }

    // values
    const int turned = 16 * (col / 4) + 4 * grp + col % 4;  // the token whose row this lane names
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const int2v c = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
          (__attribute__((address_space(3))) int2v*)(tile.codes +
                                                     turned * Shared<D, RT, WAVES>::kVRow +
                                                     dt * 8));
      const uint4 e = *(const uint4*)&tile.scales[dt][grp * 16];
      const half8v v0 = decode8((uint32_t)c[0], e4m3_f16x2<0>(e.x), e4m3_f16x2<1>(e.x),
                                e4m3_f16x2<0>(e.y), e4m3_f16x2<1>(e.y));
      const half8v v1 = decode8((uint32_t)c[1], e4m3_f16x2<0>(e.z), e4m3_f16x2<1>(e.z),
                                e4m3_f16x2<0>(e.w), e4m3_f16x2<1>(e.w));
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (rt > 0 && rt * 16 >= job.rows) continue;
        o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w[rt][0], o[rt][dt], 0, 0, 0);
        o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w[rt][1], o[rt][dt], 0, 0, 0);
      }
    }
  }

  // the wavefronts' results joined, 16 rows at a time; each thread takes pairs of one row
  const float unscale = bound == 0.0f ? 0.0f : 1.0f / norm;
  const int tid = threadIdx.x, row_in = tid / (WAVES * 4), sub = tid % (WAVES * 4);
  const bool direct = p.part_o == nullptr;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (rt * 16 >= job.rows) break;
    __syncthreads();
    const float sum = sum_of_groups(l[rt]);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
      *(float4v*)&sh.merge.o[wave][col][dt * 16 + grp * 4] = o[rt][dt] * unscale;
    if (grp == 0) sh.merge.ml[wave][col] = make_float2(m[rt], sum);
    __syncthreads();
    const int r = rt * 16 + row_in;
    if (r < job.rows) {
      float top = -INFINITY, total = 0.0f, f[WAVES];
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sh.merge.ml[w][row_in].x);
      const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        f[w] = factor(sh.merge.ml[w][row_in].x, base);
        total += f[w] * sh.merge.ml[w][row_in].y;
      }
      const int64_t row = global_row(p, job, r);
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
      for (int c = 0; c < D / (WAVES * 8); ++c) {
        const int d = (c * WAVES * 4 + sub) * 2;
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
          const float2 v = *(const float2*)&sh.merge.o[w][row_in][d];
          a = __builtin_fmaf(f[w], v.x, a);
          b = __builtin_fmaf(f[w], v.y, b);
        }
        if (direct)
          *(uint32_t*)(p.out + row * D + d) = cvt_bf16x2(a * inv, b * inv);
        else
          *(float2*)(p.part_o + ((int64_t)job.part * p.rows + row) * D + d) = make_float2(a, b);
      }
      if (sub == 0) {
        if (!direct)
          p.part_ml[(int64_t)job.part * p.rows + row] = make_float2(top, total);
        else if (p.lse)
          p.lse[row] = total == 0.0f ? -INFINITY : (base + __builtin_log2f(total)) * kLn2;
      }
    }
  }
}

// The partial results of one query row joined, in the order of their tokens:
// prefix, then own.  D / 4 threads per row.
template <int D>
__global__ __launch_bounds__(256) void attention_join(Params p) {
  constexpr int PER = 256 / (D / 4);
  const int64_t row = (int64_t)blockIdx.x * PER + threadIdx.x / (D / 4);
  if (threadIdx.x / (D / 4) >= PER || row >= p.rows) return;
  const int d = threadIdx.x % (D / 4) * 4;
  int first = p.prefix_splits;
  if (p.groups > 0) {
    // the last group that starts at or before this row's sequence
    const int b = (int)(row / ((int64_t)p.q_tokens * p.q_heads));
    int lo = 0, hi = p.groups;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.group_offsets[mid] <= b)
        lo = mid + 1;
      else
        hi = mid;
    }
    if (lo > 0 && b < p.group_offsets[lo]) first = 0;
  }
  const int parts = p.prefix_splits + p.own_splits;
  float top = -INFINITY;
  for (int i = first; i < parts; ++i) top = fmaxf(top, p.part_ml[(int64_t)i * p.rows + row].x);
  const float base = top == -INFINITY ? 0.0f : top;
  float total = 0.0f;
  float4v acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = first; i < parts; ++i) {
    const float2 ml = p.part_ml[(int64_t)i * p.rows + row];
    const float f = factor(ml.x, base);
    total += f * ml.y;
    acc += f * *(const float4v*)(p.part_o + ((int64_t)i * p.rows + row) * D + d);
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  *(uint2*)(p.out + row * D + d) = make_uint2(cvt_bf16x2(acc[0] * inv, acc[1] * inv),
                                              cvt_bf16x2(acc[2] * inv, acc[3] * inv));
  if (d == 0 && p.lse)
    p.lse[row] = total == 0.0f ? -INFINITY : (base + __builtin_log2f(total)) * kLn2;
}

// ---- shape of a call --------------------------------------------------------

struct Plan {
  int rt;  // 16-row tiles of queries per wavefront
  int64_t own_blocks, own_splits, prefix_blocks, prefix_splits, rows;
  bool direct;  // one part only: the first kernel writes the output
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// Workgroups to aim for: 256 CUs with two of 8 wavefronts each, twice over,
// so that contexts of unequal length even out.
constexpr int64_t kTargetGroups = 1024;

Plan plan_of(int64_t page_size, int64_t kv_heads, int64_t head_dim, int64_t batch,
             int64_t q_tokens, int64_t q_heads, int64_t max_pages, int64_t max_prefix_pages,
             int64_t groups) {
  Plan p;
  const int64_t per_seq = q_tokens * (q_heads / kv_heads);
  p.rt = groups == 0 && per_seq <= 16 ? 1 : 2;
  const int64_t rb = 16 * p.rt, waves = p.rt == 1 ? 8 : 4;
  p.rows = batch * q_tokens * q_heads;
  p.own_blocks = ceil_div(per_seq, rb);
  p.prefix_blocks = groups ? batch * per_seq / rb + groups : 0;
  // a part per workgroup: enough of them to fill the chip, each at least two rounds of its
  // wavefronts' tiles long
  const int64_t own_tokens = max_pages * page_size, prefix_tokens = max_prefix_pages * page_size;
  p.own_splits = clamp64(ceil_div(kTargetGroups, batch * kv_heads * p.own_blocks), 1,
                         clamp64(own_tokens / (2 * waves * kTile), 1, 64));
  p.prefix_splits =
      groups ? clamp64(ceil_div(kTargetGroups,
                                clamp64(batch * per_seq / rb, 1, p.prefix_blocks) * kv_heads),
                       1, clamp64(prefix_tokens / (2 * waves * kTile), 1, 64))
             : 0;
  p.direct = p.own_splits + p.prefix_splits == 1;
  return p;
}

template <int D>
hipError_t launch(const Params& p, const Plan& plan, hipStream_t stream) {
  const int64_t grid = plan.prefix_blocks * p.kv_heads * plan.prefix_splits +
                       (int64_t)p.batch * plan.own_blocks * p.kv_heads * plan.own_splits;
  if (grid > ((int64_t)1 << 31) / 512) return hipErrorInvalidValue;
  if (plan.rt == 1)
    attention_kernel<D, 1, 8><<<(uint32_t)grid, 512, 0, stream>>>(p);
  else
    attention_kernel<D, 2, 4><<<(uint32_t)grid, 256, 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.direct) return e;
  const int64_t per = 256 / (D / 4);
  attention_join<D><<<(uint32_t)ceil_div(plan.rows, per), 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

int64_t kv_attention_workspace_bytes(int64_t page_size, int64_t kv_heads, int64_t head_dim,
                                     int64_t batch, int64_t q_tokens, int64_t q_heads,
                                     int64_t max_pages, int64_t max_prefix_pages,
                                     int64_t groups) {
  const Plan p = plan_of(page_size, kv_heads, head_dim, batch, q_tokens, q_heads, max_pages,
                         max_prefix_pages, groups);
  return p.direct ? 0 : (p.own_splits + p.prefix_splits) * p.rows * (head_dim * 4 + 8);
}

hipError_t kv_attention_launch(const KvCache& c, const AttentionArgs& a, hipStream_t stream) {
  const Plan plan = plan_of(c.page_size, c.kv_heads, c.head_dim, a.batch, a.q_tokens, a.q_heads,
                            a.max_pages, a.max_prefix_pages, a.groups);
  Params p;
  for (int i = 0; i < 2; ++i) {
    p.codes[i] = c.codes[i];
    p.scales[i] = c.scales[i];
    p.token_scales[i] = c.token_scales[i];
  }
  p.q = (const uint16_t*)a.q;
  p.page_table = a.page_table;
  p.seq_lens = a.seq_lens;
  p.prefix_table = a.prefix_table;
  p.prefix_lens = a.prefix_lens;
  p.group_offsets = a.group_offsets;
  p.out = (uint16_t*)a.out;
  p.lse = a.lse;
  const int64_t parts = plan.own_splits + plan.prefix_splits;
  p.part_o = plan.direct ? nullptr : (float*)a.workspace;
  p.part_ml =
      plan.direct ? nullptr : (float2*)((float*)a.workspace + parts * plan.rows * c.head_dim);
  p.q_stride = a.q_stride;
  p.rows = plan.rows;
  p.num_pages = (int32_t)c.num_pages;
  p.page_size = (int32_t)c.page_size;
  p.page_groups = (int32_t)(c.page_size / 16);
  p.kv_heads = (int32_t)c.kv_heads;
  p.per_head = (int32_t)(a.q_heads / c.kv_heads);
  p.batch = (int32_t)a.batch;
  p.q_tokens = (int32_t)a.q_tokens;
  p.q_heads = (int32_t)a.q_heads;
  p.max_pages = (int32_t)a.max_pages;
  p.max_prefix_pages = (int32_t)a.max_prefix_pages;
  p.groups = (int32_t)a.groups;
  p.own_blocks = (int32_t)plan.own_blocks;
  p.own_splits = (int32_t)plan.own_splits;
  p.prefix_blocks = (int32_t)plan.prefix_blocks;
  p.prefix_splits = (int32_t)plan.prefix_splits;
  p.scale = a.scale;
  switch (c.head_dim) {
    case 64: return launch<64>(p, plan, stream);
    case 128: return launch<128>(p, plan, stream);
    case 192: return launch<192>(p, plan, stream);
    default: return launch<256>(p, plan, stream);
  }
}

}  // namespace fp4q
