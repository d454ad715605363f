// layer_prompt.hip -- causal attention of packed sequences in BF16
// (definition in include/fp4q/layer.h).
//
// Mathematics.  With c = |scale| log2(e) (queries take the scale's sign) and m
// a row's running maximum of its scores s:
//   p = 2^(s c - m c), l += p, O += p v;  out = O / l, lse = (m c + log2 l) ln 2
// p enters the value product in BF16, as the operands of the matrix instruction
// are (half a step is 2^-8 of it or less, and a row's errors are averaged over
// its keys); s, m, l and O are FP32.  l sums p as it is rounded, so that a row's
// weights add up to one: 512 tokens are off by 0.0018 of their size, 0.0017 of it
// the result's own rounding, and by 0.0020 with the sum of p before rounding.
// The log-sum-exp takes that one, which is kept where it is asked for (8192
// tokens 511 us without, 530 with it).
// m is moved only when a score passes it by 12 / c: until then p is at most
// 2^12, and BF16 holds that as well as 1, while a move costs a pass over O, of
// all rows of a wavefront, each of which moves for its own scores: with 8 / c
// 4096 tokens of heads of 256 take 314 us instead of 299.
// Where |m c| passes 2^20, s c - m c would lose more than 2^-4 to cancellation
// and is formed as (s - m) c, in steps of their own (and of the rows where it does).
//
// Layout.  Scores are computed transposed, S^T = K Q^T (32 x 32 x 16 matrix
// instructions): a lane holds 16 keys' scores of one query of every 32 keys,
// so maxima and sums are its own but for one exchange between the halves of
// the wavefront, and the probabilities of 16 keys, rounded to BF16, are the
// operand of O^T = V^T P^T as they lie when the values' keys are taken in the
// same order; the LDS's transposing read turns the values.  Keys and values go
// to LDS without passing registers, 64 keys a step, in two tiles each: while a
// step's keys or values are read the next one's arrive.  Their 16-byte pieces
// are permuted within 128 bytes so that neither read has bank conflicts.
//
// Work.  A workgroup takes the rows (query, head of those that share a key
// head) of one sequence and key head, 32 a wavefront: the heads that share
// keys share their loads as well, and few queries fill a tile.  Workgroup
// numbers run over key heads first, so that a key head's workgroups meet in
// the same dies' L2.  The last rows of a sequence, which see the most keys,
// start first, and the longest sequences where there are workgroups that wait;
// few rows behind many keys are cut along the keys and joined by a second
// kernel (parts_of).
//
// Bounds.  A step of 32 rows by 64 keys of 128 is 32 matrix instructions of 32
// cycles and, of every lane, 32 scores at about 20 cycles of vector work (an
// exponential is 8), 48 reads of LDS and some 100 scalar instructions.  `both`
// places them beside one another by hand.  Counted for one sequence of 8192
// tokens, 32 heads on 8 of 128 (502 to 522 us by card, 1095 to 1050 TFLOP/s, at
// 1.8 GHz, which power leaves; a large product of the library reaches 1420 to
// 1470): a SIMD's matrix unit works 58% of the time, its vector unit 48, the LDS
// 58, and some instruction starts in 76: with two wavefronts a SIMD it is the
// starts that bound.  (Heads of 192 and 256 have moves between the two halves of
// the registers in that loop as well, 64 and 294 a step, and 256 spills 11;
// heads of 64 have 169 registers, for two wavefronts a SIMD.)  There is one copy of the code of each kind of step, for a
// workgroup of few steps waits for its instructions from memory: 16 sequences
// of up to 2048 tokens took 273 us with the steps written out, and take 240 now
// (800 TFLOP/s).  There four tenths of a workgroup's time go outside whole
// steps: its block's search, the first copies and the queries, three steps one
// after the other, the output.
// Measured and not taken, for 8192 tokens when this took 526 to 539 us: 64 rows a
// wavefront 615 us (its accumulators pass through the other half of the
// registers), two wavefronts that share rows and take every other step 635,
// three steps' copies in flight 695; at 508, workgroups that stay and take one
// block after the other 524 (and the 16 sequences 257 for 240).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "layer_launch.h"
#include "rollout_divisor.h"

namespace fp4q {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kKeys = 64;  // of a step
constexpr int kWaves = 4, kRows = 32 * kWaves;  // of a workgroup
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kSlack = 12.0f;      // powers of two by which scores may pass m
constexpr float kLarge = 0x1p20f;    // |m c| from which exponents are formed as (s - m) c

// The same value in every lane, said so.
__device__ __forceinline__ int32_t same(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

struct Params {
  const uint16_t *q, *k, *v;
  const int32_t *q_offsets, *k_offsets;
  uint16_t* out;
  float* lse;
  int64_t q_stride, k_stride, v_stride;
  int32_t q_tokens, k_tokens, q_heads, batch;
  Divisor kv_heads;
  Divisor per_head;  // query heads of a key head
  int32_t blocks;    // of a key head: room for all sequences' row blocks
  int32_t by_length;  // the order of the blocks
  Divisor parts;     // that a block's steps are cut into
  float* part_o;     // [parts][q_tokens][q_heads][D], where there are several
  float2* part_ml;   // m and l of each, and l before rounding
  float* part_sum;
  uint32_t first_block;
  float c;           // |scale| log2(e)
  uint32_t sign;     // 0x80008000 for a negative scale
};

// A sequence's rows and keys.
struct Sequence {
  int32_t q0, m, k0, n;
};

__device__ __forceinline__ Sequence sequence(const Params& p, int b) {
  Sequence s;
  s.q0 = min(max(p.q_offsets[b], 0), p.q_tokens);
  s.m = min(max(p.q_offsets[b + 1], s.q0), p.q_tokens) - s.q0;
  s.k0 = min(max(p.k_offsets[b], 0), p.k_tokens);
  s.n = min(max(p.k_offsets[b + 1], s.k0), p.k_tokens) - s.k0;
  return s;
}

// A block of rows of a sequence (block < 0 or past the last: none).
struct Block {
  Sequence s;
  int block;
};

// Blocks in the sequences' order: sequence b's are numbered from q_offsets[b] * per_head / kRows +
// b on, which leaves room for all of them: rows / kRows, rounded up, is at most one more than the
// difference of that quotient.
__device__ __forceinline__ Block block_by_place(const Params& p, int w) {
  const int lane = threadIdx.x % 64;
  auto first_of = [&](int b) {
    const int32_t q0 = min(max(p.q_offsets[b], 0), p.q_tokens);
    return (int)((uint32_t)q0 * p.per_head.d / kRows) + b;
  };
  // the last sequence whose first number is at most w, 64 candidates at a time: one of
  // [lo, lo + count), lo's number is at most w, or lo is 0
  int lo = 0, count = p.batch;
  while (count > 1) {
    const int step = (count + 63) / 64;
    const int at = lo + lane * step;
    const bool below = at < lo + count && first_of(at) <= w;
    const uint64_t set = __ballot(below);
    const int last = set == 0 ? 0 : 63 - __builtin_clzll(set);
    count = min(step, lo + count - (lo + last * step));
    lo += last * step;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  return Block{sequence(p, lo), w - first_of(lo)};
}

// Blocks in falling order of their sequences' keys, and from the last to the first of a sequence:
// a lane a sequence, up to 64 of them.  What starts last is short; and a sequence's blocks are
// neighbours, so that its keys are met in L2.
__device__ __forceinline__ Block block_by_length(const Params& p, int w) {
  const int lane = threadIdx.x % 64;
  Sequence s{0, 0, 0, 0};
  if (lane < p.batch) s = sequence(p, lane);
  const int blocks = (int)(((uint32_t)s.m * p.per_head.d + kRows - 1) / kRows);
  // (lanes without a sequence have no blocks)
  int before = 0;
  for (int i0 = 0; i0 < p.batch; i0 += 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j;
      const int n = __builtin_amdgcn_readlane(s.n, i), c = __builtin_amdgcn_readlane(blocks, i);
      before += n > s.n || (n == s.n && i < lane) ? c : 0;
    }
  }
  const uint64_t is = __ballot(lane < p.batch && w >= before && w < before + blocks);
  if (is == 0) return Block{{0, 0, 0, 0}, -1};
  const int b = __builtin_ctzll(is);
  auto of = [&](int v) { return __builtin_amdgcn_readlane(v, b); };
  return Block{{of(s.q0), of(s.m), of(s.k0), of(s.n)}, of(before + blocks) - 1 - w};
}

// 16 bytes a lane, from base + scalar + lane's offset to lds + 16 * lane.  (Written out: the
// compiler would wait for all copies in flight before the next transposing read, whatever it
// reads.  Nothing is returned to registers; the callers wait for vmcnt before the tiles are read.
// m0 holds nothing of the compiler's here.)
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t base, uint32_t lane, uint32_t scalar,
                                       uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "{m0}"(lds), "v"(lane), "s"(base), "s"(scalar)
               : "memory");
}

__device__ __forceinline__ float other_half(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(threadIdx.x % 64 < 32 ? r[1] : r[0]);
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// sum + both of w's BF16 numbers.
__device__ __forceinline__ float add_pair(float sum, uint32_t w) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), ones, sum, false);
}

// The places of a row's 16-byte pieces are exchanged so that no two lanes of a read meet in a
// bank.  LDS has 64 banks of 4 bytes: 16 lanes read 16 bytes each, of 16 neighbouring keys at the
// same place, at once; these have to lie differently in 256 bytes.  A transposing read takes 8
// bytes of 16 lanes, 32 bytes of four neighbouring keys.
__device__ __forceinline__ int turned(int key) { return (key & 3) << 1 | (key >> 2 & 1); }

// Two BF16 numbers with zeros for infinities and NaN.
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) |
         ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
}

template <int D>
struct Tiles {  // one step's in use, the next one's in flight
  alignas(16) uint8_t k[2][kKeys * D * 2];
  alignas(16) uint8_t v[2][kKeys * D * 2];
};

// LSE: probabilities are summed before they are rounded as well, for the log-sum-exp.
template <int D, bool LSE>
__global__ __launch_bounds__(64 * kWaves, D <= 128 ? 2 : 1) void prompt_kernel(const Params p) {
  // whether the next step's scores may be masked where they are computed beside the values'
  // product (heads of 256 have no registers for it: 583 us instead of 331 for 4096 tokens)
  constexpr bool kMaskNext = D < 256;
  constexpr int NK = D / 16, DT = D / 32, kRow = 2 * D;
  __shared__ Tiles<D> tiles;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int col = lane % 32, half = lane / 32;

  // numbers: key heads first, then parts, then blocks
  const uint32_t id = p.first_block + blockIdx.x;
  uint32_t w = quotient(id, p.kv_heads);
  const int kvh = (int)(id - w * p.kv_heads.d);
  const uint32_t nth = quotient(w, p.parts);
  const int part = (int)(w - nth * p.parts.d);
  const Block at = p.by_length ? block_by_length(p, (int)nth)
                               : block_by_place(p, p.blocks - 1 - (int)nth);
  const Sequence s{same(at.s.q0), same(at.s.m), same(at.s.k0), same(at.s.n)};
  const int rows = (int)((uint32_t)s.m * p.per_head.d);
  const int64_t row0 = (int64_t)same(at.block) * kRows;
  if (at.block < 0 || row0 >= rows) return;

  // rows past the last are the last once more, and not stored
  auto limit_of = [&](int r) {  // keys that row r sees
    return max(0, s.n - s.m + 1 + (int)quotient((uint32_t)min(r, rows - 1), p.per_head));
  };
  const int first = (int)row0 + wave * 32, r = min(first + col, rows - 1);
  const int token = (int)quotient((uint32_t)r, p.per_head);
  const int head = kvh * (int)p.per_head.d + r - token * (int)p.per_head.d;
  const int limit = limit_of(r);
  const int block_limit = limit_of((int)row0 + kRows - 1);
  const int wave_limit = first < rows ? limit_of(first + 31) : 0;  // the most any row sees,
  const int all_see = limit_of(first);                             // and the least
  // the part's steps
  const int all_steps = (block_limit + kKeys - 1) / kKeys;
  const int share = (int)quotient((uint32_t)all_steps + p.parts.d - 1, p.parts);
  const int begin_step = part * share, steps = min(begin_step + share, all_steps);

  // A step's copies: this wavefront's keys are the 16 from wave * 16 on, D / 64 copies for every
  // eight of them; the pieces' order comes again with these.
  constexpr int kPeriod = D / 64, kLoads = kKeys / kWaves / 8 * kPeriod;
  const char* k_base = (const char*)(p.k + (int64_t)s.k0 * p.k_stride + kvh * D);
  const char* v_base = (const char*)(p.v + (int64_t)s.k0 * p.v_stride + kvh * D);
  const uint32_t k_row = (uint32_t)p.k_stride * 2, v_row = (uint32_t)p.v_stride * 2;  // bytes
  auto piece_of = [&](int n, int& key, uint32_t& in_row) {  // this lane's of the n-th copy
    const int piece = n * 64 + lane;
    key = wave * (kKeys / kWaves) + piece / (D / 8);
    in_row = (uint32_t)(piece % (D / 8) ^ turned(key)) * 16;
  };
  uint32_t k_from[kPeriod], v_from[kPeriod];
#pragma unroll
  for (int n = 0; n < kPeriod; ++n) {
    int key;
    uint32_t in_row;
    piece_of(n, key, in_row);
    k_from[n] = key * k_row + in_row;
    v_from[n] = key * v_row + in_row;
  }
  auto buffer = [&](const char* at) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)at, 0, -1, 0x20000);
  };
  auto source = [&](const char* base, uint32_t row, int step) {
    return buffer(base + (int64_t)step * kKeys * row);
  };
  // (offsets in LDS as numbers: a generic pointer is checked for null at every copy)
  constexpr uint32_t kTile = kKeys * D * 2;
  const uint32_t own_k = (uint32_t)same((int32_t)(uint32_t)(uintptr_t)(lds_void*)tiles.k) +
                         wave * kLoads * 1024;
  const uint32_t own_v = own_k + (uint32_t)offsetof(Tiles<D>, v);
  auto copy_one = [&](int n, uint32_t to, __amdgpu_buffer_rsrc_t at, uint32_t row,
                      const uint32_t (&from)[kPeriod]) {
    to_lds(at, from[n % kPeriod], n / kPeriod * 8 * row, to + n * 1024);
  };
  // a step's keys (or values) to tile step % 2
  auto copy = [&](int step, const char* base, uint32_t row, const uint32_t (&from)[kPeriod],
                  uint32_t tile) {
    if (step >= steps) return;
    const auto at = source(base, row, step);
    const uint32_t to = tile + (step & 1) * kTile;
    if (step * kKeys + kKeys <= s.n) {
#pragma unroll
      for (int n = 0; n < kLoads; ++n) copy_one(n, to, at, row, from);
    } else {
      // keys past the sequence's end are its last once more
#pragma unroll 1
      for (int n = 0; n < kLoads; ++n) {
        int key;
        uint32_t in_row;
        piece_of(n, key, in_row);
        to_lds(at, (uint32_t)min(key, s.n - 1 - step * kKeys) * row + in_row, 0,
               to + n * 1024);
      }
    }
  };
  // Copies go in pairs, a step's values and the next one's keys, one step ahead.
  auto copy_pair = [&](int step) {
    copy(step, v_base, v_row, v_from, own_v);
    copy(step + 1, k_base, k_row, k_from, own_k);
  };

  int step = begin_step;
  copy(step, k_base, k_row, k_from, own_k);
  // queries, as the scores' second operand
  bf16x8 q[NK];
  {
    const uint16_t* from = p.q + (int64_t)(s.q0 + token) * p.q_stride + head * D + half * 8;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      uint4v u = *(const uint4v*)(from + i * 16);
      u ^= p.sign;
      q[i] = __builtin_bit_cast(bf16x8, u);
    }
  }

  float16v o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = (float16v)0.0f;
  float m = -INFINITY, mc = 0.0f, l = 0.0f, sum = 0.0f;  // (sum: l before rounding)
  bool large = false, any_dirty = false;

  // where this lane's keys and values lie
  int k_at[4], v_at[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) k_at[i] = col * kRow + ((2 * i + half) ^ turned(col)) * 16;
  {
    const int i = lane % 16, key = 4 * half + i / 4;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      v_at[j] = key * kRow + ((4 * j + 2 * (lane / 16 % 2) + i % 4 / 2) ^ turned(key)) * 16 +
                i % 2 * 8;
  }

  // 16 bytes of this lane's key: the first operand of the i-th product of the kb-th 32 keys
  auto key_part = [&](const uint8_t* t, int kb, int i) {
    return *(const bf16x8*)(t + k_at[i % 4] + i / 4 * 128 + kb * 32 * kRow);
  };
  // that of the d-th 32 elements and the j-th 16 keys of the values
  auto value_part = [&](const uint8_t* t, int j, int d) {
    uint4v a;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* at = t + v_at[d % 2] + d / 2 * 128 + (j * 16 + i * 8) * kRow;
      const uint2v u = __builtin_bit_cast(
          uint2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                      (__attribute__((address_space(3))) short4v*)at));
      a[2 * i] = u[0];
      a[2 * i + 1] = u[1];
    }
    return a;
  };
  // m and what hangs on it, for a step whose largest score of this lane's keys is top.  A row's m
  // moves by its own scores alone: a key that other rows of the wavefront see changes none of its bits.
  auto renew = [&](float top) {
    top = __builtin_fmaxf(top, other_half(top));
    const bool moves = (top - m) * p.c > kSlack;
    if (__any(moves)) {
      const float next = moves ? top : m;
      const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - next) * p.c);
      m = next;
      mc = m == -INFINITY ? 0.0f : m * p.c;
      l *= f;
      if constexpr (LSE) sum *= f;
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i] *= f;
      large = __any(__builtin_fabsf(mc) >= kLarge);
    }
  };
  auto masked = [&](int step) { return step * kKeys + kKeys > all_see; };
  auto mask = [&](int step, float16v (&sc)[2]) {
    const int seen = limit - step * kKeys - 4 * half;  // this lane's keys below that count
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i / 16 * 32 + i % 16 / 4 * 8 + i % 4 >= seen) sc[i / 16][i % 16] = -INFINITY;
  };
  auto largest = [&](const float16v (&sc)[2]) {
    float top = sc[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) top = __builtin_fmaxf(top, sc[i / 16][i % 16]);
    return top;
  };
  // scores to the exponents of their probabilities
  auto exponents = [&](const float16v (&sc)[2], float16v (&to)[2]) {
    if (large) {
      const bool far = __builtin_fabsf(mc) >= kLarge;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = sc[i / 16][i % 16];
        to[i / 16][i % 16] = far ? (x - m) * p.c : __builtin_fmaf(x, p.c, -mc);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        to[i / 16][i % 16] = __builtin_fmaf(sc[i / 16][i % 16], p.c, -mc);
    }
  };
  // a step's scores, masked, m for them, and the exponents
  auto score = [&](int step, float16v (&sc)[2]) {
    const uint8_t* t = tiles.k[step & 1];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      sc[kb] = (float16v)0.0f;
#pragma unroll
      for (int i = 0; i < NK; ++i)
        sc[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_part(t, kb, i), q[i], sc[kb], 0, 0, 0);
    }
    if (masked(step)) mask(step, sc);
    renew(largest(sc));
    exponents(sc, sc);
  };
  // The i-th of a step's probabilities and the next one, rounded: the i / 2-th word of the weights.
  auto weigh = [&](const float16v (&sc)[2], int i, uint4v (&weights)[4]) {
    const float a = sc[i / 16][i % 16], b = sc[i / 16][i % 16 + 1];
    weights[i / 8][i % 8 / 2] = pack(a, b);
    if constexpr (LSE) {
      sum += a;
      sum += b;
    }
  };
  // a step's probabilities, from their exponents, and their product with the values
  auto add_values = [&](int step, float16v (&sc)[2]) {
    const uint8_t* t = tiles.v[step & 1];
#pragma unroll
    for (int i = 0; i < 32; ++i) sc[i / 16][i % 16] = __builtin_amdgcn_exp2f(sc[i / 16][i % 16]);
    uint4v weights[4];  // 16 keys each
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      weigh(sc, i, weights);
      l = add_pair(l, weights[i / 8][i % 8 / 2]);
    }
    auto product = [&](auto clean) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          uint4v a = value_part(t, j, d);
          if constexpr (decltype(clean)::value) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = finite_part(a[i]);
          }
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                         __builtin_bit_cast(bf16x8, weights[j]),
                                                         o[d], 0, 0, 0);
        }
    };
    // A weight of zero does not take out an infinity or NaN: where a step that not every row sees
    // whole has one, it is left out here and added behind the loop.
    bool dirty = false;
    if (masked(step)) {
      // an exponent of ones overflows to the sign when one is added to it
      uint32_t bad = 0;
#pragma unroll 4
      for (int i = lane * 16; i < kKeys * kRow; i += 1024) {
        const uint4v u = *(const uint4v*)(t + i);
#pragma unroll
        for (int x = 0; x < 4; ++x) bad |= (u[x] & 0x7f807f80u) + 0x00800080u;
      }
      bad &= 0x80008000u;
      dirty = __any(bad != 0);
    }
    if (dirty) {
      any_dirty = true;
      product(std::true_type{});
    } else {
      product(std::false_type{});
    }
  };
  // Both at once, add_values(step, sc) and score(step + 1, next) but for the exponents, for a step
  // that every row sees whole: the matrix units do the next step's scores, then this one's values,
  // and beside each of their instructions stand a few of the others' -- the probabilities in the
  // first half (the last quarter in the second), the next step's maximum in the second -- and the
  // reads of operands two instructions ahead.
  auto both = [&](int step, float16v (&sc)[2], float16v (&next)[2], auto copies) {
    constexpr int kSlots = 2 * NK;  // matrix instructions of a half (4 * DT as well)
    const uint8_t *kt = tiles.k[(step + 1) & 1], *vt = tiles.v[step & 1];
    uint4v weights[4];
    auto packed = [&](int i) {  // (a pair later: what follows an exponential at once waits for it)
      weigh(sc, i, weights);
      if (i > 0) l = add_pair(l, weights[(i - 2) / 8][(i - 2) % 8 / 2]);  // (another pair later)
      if (i == 30) l = add_pair(l, weights[3][3]);
    };
    auto probability = [&](int i) {
      const float x = __builtin_amdgcn_exp2f(sc[i / 16][i % 16]);
      if (i % 2 == 0 && i > 0) packed(i - 2);
      sc[i / 16][i % 16] = x;
    };
    auto fetch = [&](int n) {  // the operand of the n-th instruction of both halves
      return n < kSlots ? key_part(kt, n % 2, n / 2)
                        : __builtin_bit_cast(bf16x8, value_part(vt, (n - kSlots) / DT,
                                                                (n - kSlots) % DT));
    };
    bf16x8 ring[4];  // before an instruction of even number, the operands of the next pair
    auto fetch_pair = [&](int n) {
      if (n % 2 == 0 && n < 2 * kSlots) {
        ring[n % 4] = fetch(n);
        ring[n % 4 + 1] = fetch(n + 1);
      }
    };
    fetch_pair(0);
    next[0] = next[1] = (float16v)0.0f;
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
      fetch_pair(n + 2);
      next[n % 2] =
          __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[n % 4], q[n / 2], next[n % 2], 0, 0, 0);
      copies(n);
#pragma unroll
      for (int i = n * 24 / kSlots; i < (n + 1) * 24 / kSlots; ++i) probability(i);
      __builtin_amdgcn_sched_barrier(0);
    }
    float top = next[0][0];
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
      fetch_pair(n + kSlots + 2);
      const int j = n / DT, d = n % DT;
      o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          ring[n % 4], __builtin_bit_cast(bf16x8, weights[j]), o[d], 0, 0, 0);
      if (n < kSlots / 2) {
#pragma unroll
        for (int i = 24 + n * 16 / kSlots; i < 24 + (n + 1) * 16 / kSlots; ++i) probability(i);
        if (n == kSlots / 2 - 1) packed(30);
      } else {
#pragma unroll
        for (int i = (n - kSlots / 2) * 64 / kSlots; i < (n + 1 - kSlots / 2) * 64 / kSlots; ++i)
          top = __builtin_fmaxf(top, next[i / 16][i % 16]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kMaskNext) {
      if (masked(step + 1)) {
        mask(step + 1, next);
        top = largest(next);
      }
    }
    renew(top);
  };

  // A step's pair is there, and every wavefront is done with the tiles that come next.
  auto begin = [&]() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };
  const int own_steps = min((wave_limit + kKeys - 1) / kKeys, steps);  // this wavefront's end
  const int whole_steps = min(all_see / kKeys, steps);  // end of those that all its rows see whole
  const int last_whole = min(whole_steps, kMaskNext ? own_steps - 1 : own_steps) - !kMaskNext;
  // (one copy of the code of each kind of step: a workgroup of few steps waits for instructions)
  // The pairs copied in the inner loop have to exist to their last key (behind the last step keys
  // are copied as well, once more the last step's, and not used).
  const int fast_end = min(last_whole, s.n / kKeys >= steps ? steps : s.n / kKeys - 2);
  float16v sc[2];
#pragma unroll 1
  for (--step; step < steps; ++step) {
    begin();
    copy_pair(step + 1);
    if (step >= begin_step && step < own_steps) add_values(step, sc);
    if (step + 1 < own_steps) score(step + 1, sc);
    const char *v_from_step = v_base + (int64_t)(step + 2) * kKeys * v_row;
    const char *k_from_step = k_base + (int64_t)min(step + 3, steps - 1) * kKeys * k_row;
#pragma unroll 1
    for (; step + 1 < fast_end && !large; ++step) {
      float16v next[2];
      begin();
      const auto values = buffer(v_from_step), keys = buffer(k_from_step);
      v_from_step += kKeys * v_row;
      k_from_step += step + 4 < steps ? kKeys * k_row : 0;  // (the last step's once more)
      const uint32_t to_v = own_v + (step & 1) * kTile, to_k = own_k + (step + 1 & 1) * kTile;
      both(step + 1, sc, next, [&](int n) {
        if (n < kLoads)
          copy_one(n, to_v, values, v_row, v_from);
        else if (n < 2 * kLoads)
          copy_one(n - kLoads, to_k, keys, k_row, k_from);
      });
      exponents(next, sc);  // (to sc's registers, which saves a copy)
    }
  }

  if (any_dirty) {
    // values that are not finite, of the steps that were masked, to the rows that see them
    const int from_key = max(all_see / kKeys, begin_step) * kKeys;
    const int to_key = min(wave_limit, steps * kKeys);
    const char* from = v_base + (int64_t)from_key * v_row + 8 * half;
#pragma unroll 1
    for (int key = from_key; key < to_key; ++key, from += v_row) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2v u = *(const uint2v*)(from + d * 64 + i * 16);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t bits = x % 2 ? u[x / 2] & 0xffff0000u : u[x / 2] << 16;
            if ((bits & 0x7f800000u) == 0x7f800000u && key < limit)
              o[d][4 * i + x] += __uint_as_float(bits);
          }
        }
    }
  }

  l += other_half(l);
  if constexpr (LSE) sum += other_half(sum);
  if (first + col >= rows) return;
  const int64_t row = (int64_t)(s.q0 + token) * p.q_heads + head;
  if (p.parts.d > 1) {
    const int64_t at_part = part * (int64_t)p.q_tokens * p.q_heads + row;
    if (half == 0) p.part_ml[at_part] = make_float2(m, l);
    if (LSE && half == 0) p.part_sum[at_part] = sum;
    if (l == 0.0f) return;
    float* to = p.part_o + at_part * D + 4 * half;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(float4*)(to + d * 32 + i * 8) =
            make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]);
    return;
  }
  const float each = l == 0.0f ? 0.0f : 1.0f / l;
  // the two halves hold every other four elements: exchanged, a lane has eight neighbours
  uint16_t* to = p.out + row * D + 8 * half;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      uint4v u;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int e = 4 * i + 2 * x;
        const auto r = __builtin_amdgcn_permlane32_swap(
            pack(o[d][e] * each, o[d][e + 1] * each),
            pack(o[d][e + 4] * each, o[d][e + 5] * each), false, false);
        u[x] = r[0];
        u[2 + x] = r[1];
      }
      *(uint4v*)(to + d * 32 + i * 8) = u;
    }
  if (LSE && half == 0)
    p.lse[row] = l == 0.0f ? -INFINITY : (mc + __builtin_amdgcn_logf(sum)) * kLn2;
}

// The parts of a row to its output, in order.  A wavefront takes a row, a lane D / 64 elements.
template <int D>
__global__ __launch_bounds__(256) void prompt_join(const Params p) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x % 64;
  const int64_t all = (int64_t)p.q_tokens * p.q_heads;
  const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (row >= all) return;
  // rows of no sequence are left as they are
  const int64_t lo = min(max(p.q_offsets[0], 0), p.q_tokens);
  const int64_t hi = min(max(p.q_offsets[p.batch], 0), p.q_tokens);
  if (row < lo * p.q_heads || row >= hi * p.q_heads) return;
  const int parts = (int)p.parts.d;
  float top = -INFINITY;
  for (int i = 0; i < parts; ++i) {
    const float2 ml = p.part_ml[i * all + row];
    if (ml.y != 0.0f) top = __builtin_fmaxf(top, ml.x);
  }
  float l = 0.0f, sum = 0.0f, o[E] = {};
  for (int i = 0; i < parts; ++i) {
    const float2 ml = p.part_ml[i * all + row];
    if (ml.y == 0.0f) continue;  // (nothing was written)
    const float f = __builtin_amdgcn_exp2f((ml.x - top) * p.c);
    l = __builtin_fmaf(ml.y, f, l);
    if (p.lse) sum = __builtin_fmaf(p.part_sum[i * all + row], f, sum);
    const float* from = p.part_o + (i * all + row) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(from[e], f, o[e]);
  }
  const float each = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.out[row * D + lane * E + e] = (uint16_t)(pack(o[e] * each, 0.0f) & 0xffffu);
  if (p.lse && lane == 0)
    p.lse[row] = l == 0.0f ? -INFINITY : (top * p.c + __builtin_amdgcn_logf(sum)) * kLn2;
}

}  // namespace

namespace {

// Parts that the steps of every block are cut into.  A step takes about D / 128 us, however few
// blocks there are; a part costs its rows' sums, written and read in FP32 (3 TB/s), and 0.5 us, and
// the join 4 us.  So the steps are cut in the square root of their time by a part's, up to two
// workgroups a compute unit, where there are 12 us of them.  Measured, with 32 heads on 8 of 128
// but for the last, whole and in 2, 4, 8 and 16 parts (the rule's number first):
//   16 queries behind 8000 keys  (13) 117, 67, 39, 27, 25 us
//   64 behind 2000                (5) 37, 26, 20, 18, 23
//   256 behind 4000               (4) 68, 45, 34, 37, 50
//   8 times 16 behind 1000        (2) 22, 20, 19, 21, 30
//   512 behind 16000              (3) 238, 150, 142, 154, 184
//   512 behind 512                (1) 22, 24, 27, 42, 68
//   512, 8 heads on 2 of 256, behind 4000  (6) 121, 76, 53, 46, 61
// The lengths are on the device; what the host knows is how many rows of keys there are.  Where most
// are in no sequence there are too many parts: 16 queries behind 100 keys take 25 us in a buffer of
// 131072 rows (55 parts) and 8 with its first 100 alone; behind 2000 of 32768 21 and 15.
int64_t parts_of(int64_t q_tokens, int64_t q_heads, int64_t k_tokens, int64_t kv_heads,
                 int64_t head_dim, int64_t batch) {
  const int64_t groups = (q_tokens * (q_heads / kv_heads) / kRows + batch) * kv_heads;
  const double steps = (double)k_tokens / batch / kKeys * head_dim / 128;  // us
  const double part = 0.5 + (double)q_tokens * q_heads * head_dim * 8 / 3e6;
  if (steps < 12) return 1;
  const int64_t parts = std::min((int64_t)std::sqrt(steps / part), 512 / groups);
  return std::min(std::max(parts, (int64_t)1), (int64_t)64);
}

}  // namespace

int64_t prompt_workspace_bytes(int64_t q_tokens, int64_t q_heads, int64_t k_tokens,
                               int64_t kv_heads, int64_t head_dim, int64_t batch) {
  const int64_t parts = parts_of(q_tokens, q_heads, k_tokens, kv_heads, head_dim, batch);
  return parts == 1 ? 0 : parts * q_tokens * q_heads * (head_dim + 3) * 4;
}

hipError_t prompt_launch(const PromptArgs& a, hipStream_t stream) {
  Params p{};
  p.q = (const uint16_t*)a.q;
  p.k = (const uint16_t*)a.k;
  p.v = (const uint16_t*)a.v;
  p.q_offsets = a.q_offsets;
  p.k_offsets = a.k_offsets;
  p.out = (uint16_t*)a.out;
  p.lse = a.lse;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_tokens = (int32_t)a.q_tokens;
  p.k_tokens = (int32_t)a.k_tokens;
  p.q_heads = (int32_t)a.q_heads;
  p.batch = (int32_t)a.batch;
  p.kv_heads = divisor_of((uint32_t)a.kv_heads);
  p.per_head = divisor_of((uint32_t)(a.q_heads / a.kv_heads));
  const float c = __builtin_fabsf(a.scale) * kLog2e;
  // (zero times an infinite score would be NaN; this leaves less than 2^-20 of any finite one)
  p.c = c > 0.0f ? c : 0x1p-149f;
  p.sign = a.scale < 0.0f ? 0x80008000u : 0u;
  const int64_t parts = parts_of(a.q_tokens, a.q_heads, a.k_tokens, a.kv_heads,
                                 a.head_dim, a.batch);
  p.parts = divisor_of((uint32_t)parts);
  p.part_o = (float*)a.workspace;
  if (parts > 1) {
    const int64_t all = parts * a.q_tokens * a.q_heads;
    p.part_ml = (float2*)(p.part_o + all * a.head_dim);
    p.part_sum = (float*)(p.part_ml + all);
  }
  p.blocks = (int32_t)(a.q_tokens * p.per_head.d / kRows + a.batch);
  auto launch = [&](const void* kernel, const void* join) {
    const int64_t total = (int64_t)p.blocks * a.kv_heads * parts;
    // By place, numbers without a block lie between the others, and workgroups go round the compute
    // units by number: where there are more than one each (two fit), some units have two and others
    // none.  By length they come last, and the order is right where workgroups wait for others; but
    // finding a block takes longer, the more sequences the longer.  By place and by length: 4 times
    // 32 queries behind 4000 keys, in 5 parts, 34.7 and 26.8 us, 8 times 16 behind 2000, in 4, 28.1
    // and 23.2; whole, 6 of 200 to 300 18.9 and 16.7, 20 of 20 to 80 10.9 and 11.3, 40 of 10 to 60
    // 11.1 and 12.9; where all have a unit, 13 of up to 300 10.1 and 10.8, one of 512 14.8 and
    // 15.4; where some wait, 4 times 512 behind up to 8192 192 and 188.
    const int64_t alone = a.batch <= 16 ? 256 : 512;
    p.by_length = a.batch > 1 && a.batch <= 64 && (parts > 1 || total > alone);
    const int64_t most = ((int64_t)1 << 32) / (64 * kWaves) - 1;  // (a launch holds 2^32 threads)
    void* args[] = {&p};
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < total && e == hipSuccess; first += most) {
      p.first_block = (uint32_t)first;
      const uint32_t grid = (uint32_t)(total - first < most ? total - first : most);
      e = hipLaunchKernel(kernel, dim3(grid), dim3(64 * kWaves), args, 0, stream);
    }
    if (parts > 1 && e == hipSuccess)
      e = hipLaunchKernel(join, dim3((uint32_t)((a.q_tokens * a.q_heads + 3) / 4)), dim3(256), args,
                          0, stream);
    return e;
  };
  auto sized = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    return launch(a.lse ? (void*)prompt_kernel<D, true> : (void*)prompt_kernel<D, false>,
                  (void*)prompt_join<D>);
  };
  switch (a.head_dim) {
    case 64: return sized(std::integral_constant<int, 64>{});
    case 128: return sized(std::integral_constant<int, 128>{});
    case 192: return sized(std::integral_constant<int, 192>{});
    default: return sized(std::integral_constant<int, 256>{});
  }
}

}  // namespace fp4q
