// rollout_attention.hip -- softmax attention over the paged NVFP4 cache,
// with a prefix shared by groups of sequences (definitions in
// include/fp4q/rollout.h).
//
// Mathematics.  With cached rows k_t = s_t (e g)_t and v_t = s'_t (e' g')_t,
// the products g e are FP16 numbers (at most 6 significant bits, 2^-10 to
// 2688), so the matrix units take them as they are:
//   S[t][q] = sum_d (g e)[t][d] q[d]       q scaled by a power of two into
//                                          FP16's range
//   x = (S (s_t f)) c_q                    scale log2(e) = f 2^n; c_q: 2^n, q's power of two
//   p = 2^(x - m), l += p, m the running maximum of x
//   O[d][q] += sum_t (g' e')[t][d] w,  w = FP16(p s'_t / b)
// with b a power of two at or above every s'_t met so far times 2^-14.  Where
// token scales are within 2^14 of each other, w keeps 11 bits for every token
// whose p s' is within 2^12 of the row's largest, and an error of 2^-23 of that
// below (the output holds 8 bits).  Where they lie further apart, large ones
// may have no weight in a row: then m is lowered row by row until its largest
// w is near 2^14.  The scales s and s' cost one multiplication per score
// instead of one per element.  FP16 queries lose what is below 2^-39 of their
// row's largest element, and bits from 2^-29 on.
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
// group, so that the prefix is read and decoded once per 16 * RT of them).  The WAVES
// wavefronts of a workgroup take an item's tiles in turn and merge their
// (m, l, O) through LDS.  Short contexts take one workgroup per item.  Longer
// ones are cut into parts of about equal length, one for each workgroup: the
// part's length follows from the lengths on the device, so that a batch of
// unequal contexts fills the chip as an equal one does.  A second kernel
// joins the parts of an item in a fixed order.
//
// What bounds it.  Long contexts: the cache's bytes.  64 sequences of 64
// heads over 8 of 128 take 90 us with 5120 tokens each and 164 with 10240: 84%
// of a copy's rate, and 16 us for the launch, the first loads (length, table and
// queries, tokens, each behind the one before), the last parts and the join.
// 2048 to 8192 tokens (400 MB as well) take 97 us, as unequal contexts' parts are
// unequal too.  Prompts shared by 16 sequences: decoding, repeated for each 16
// rows (49 us; one read of the bytes would take 12).  Small batches: some 7 us for
// a context of one tile, and 3 for each further step of a wavefront, whose chain
// of scores, softmax and values few wavefronts do not cover (777 tokens 10.7).
#include "fp4q_device.h"
#include "rollout_divisor.h"
#include "rollout_launch.h"

namespace fp4q {
namespace {

typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef _Float16 half4v __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef int int2v __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr int kTile = 64;  // tokens per step of a wavefront
constexpr float kFar = 0x1p14f;  // ratio of value scales from which they count as far apart

// Beside the sums of a row's first part: m and l, where the item's further
// parts are, and how many there are (-1: none, and the output is written).
struct First {
  float m, l;
  int32_t next, more;
};

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
  // partial results (unscaled sums, and m and l): of an item's first part by query row, for
  // own items and prefix ones; of further parts by their number and the row of the block
  float* first_o[2];   // [own, prefix][rows][D]
  First* first[2];
  float* next_o;       // [parts][16 * RT][D]
  float2* next_ml;
  int64_t q_stride, rows;
  Divisor page_groups;  // 16-token groups of a page
  Divisor per_head;     // q_heads / kv_heads
  Divisor per_seq;      // query rows of a sequence and cache head: q_tokens * per_head
  int32_t num_pages, page_size, kv_heads;
  int32_t batch, q_tokens, q_heads, max_pages, max_prefix_pages, groups;
  int32_t blocks;  // row blocks of a sequence's own items
  int32_t parts;   // parts to cut all items into, about; 0: one workgroup per item
  uint32_t first_block;  // number of the launch's first workgroup: a call may take several
  float scale;
};

// Over lanes l, l ^ 16, l ^ 32, l ^ 48: maximum (NaN if one is) and sum.
__device__ __forceinline__ float max_of_groups(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t w = __float_as_uint(
      __builtin_elementwise_maximum(__uint_as_float(r[0]), __uint_as_float(r[1])));
  const auto h = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __builtin_elementwise_maximum(__uint_as_float(h[0]), __uint_as_float(h[1]));
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

// Lane `from`'s value, for every lane.
__device__ __forceinline__ int64_t lane_value(int64_t v, int from) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)v, from);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), from);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// An item: a block of query rows of one cache head, and the tokens [0, len)
// of one page-table row that they see.
struct Item {
  const int32_t* table;
  int32_t pages;    // entries of that row
  int32_t len;      // tokens any row of the block sees
  int32_t floor;    // tokens every row of the block sees
  int32_t first_b;  // row r belongs to sequence first_b + (row0 + r) / (T * per_head)
  int32_t row0;     // first row of the block, counted from first_b's first
  int32_t rows;     // rows in the block
  int32_t own_len;  // own tokens: the limit of query t is own_len - T + 1 + t (prefix: len)
  int32_t kvh;
  bool prefix;
};

struct Row {
  int64_t token;  // b * q_tokens + t
  int t, head;
};

__device__ __forceinline__ Row row_of(const Params& p, const Item& j, int r) {
  const uint32_t rr = j.row0 + r, b = quotient(rr, p.per_seq), in = rr - b * p.per_seq.d;
  const uint32_t t = quotient(in, p.per_head);
  return Row{(int64_t)(j.first_b + (int)b) * p.q_tokens + t, (int)t,
             j.kvh * (int)p.per_head.d + (int)(in - t * p.per_head.d)};
}

__device__ __forceinline__ int tiles_of(int len) { return (int)((uint32_t)(len + kTile - 1) / kTile); }

__device__ __forceinline__ int32_t own_length(const Params& p, int b) {
  return min(max(p.seq_lens[b], 0), p.max_pages * p.page_size);
}

// Tokens that row block rb of a sequence of own_len tokens sees.
template <int RB>
__device__ __forceinline__ int seen_by(const Params& p, int own_len, int rb) {
  const uint32_t last = min((uint32_t)(rb + 1) * RB, p.per_seq.d) - 1;
  return max(0, own_len - p.q_tokens + 1 + (int)quotient(last, p.per_head));
}

struct Members {
  int lo, hi;  // sequences [lo, hi) of a group
};

__device__ __forceinline__ Members members_of(const Params& p, int g) {
  Members m;
  m.lo = min(max(p.group_offsets[g], 0), p.batch);
  m.hi = min(max(p.group_offsets[g + 1], m.lo), p.batch);
  return m;
}

__device__ __forceinline__ int32_t prefix_length(const Params& p, int g) {
  return min(max(p.prefix_lens[g], 0), p.max_prefix_pages * p.page_size);
}

// Entries are the groups' prefixes, then the sequences.  An entry's items:
// f(number of items, tiles of each), row block by row block.  A sequence's
// item has one tile even if it sees nothing (its zeros have to be written), a
// prefix's may have none.
template <int RB, class F>
__device__ __forceinline__ void items_of(const Params& p, int entry, F f) {
  if (entry < p.groups) {
    const Members m = members_of(p, entry);
    const int rows = (m.hi - m.lo) * (int)p.per_seq.d;
    const int tiles = tiles_of(prefix_length(p, entry));
    if (tiles > 0) f((rows + RB - 1) / RB * p.kv_heads, tiles);
    return;
  }
  const int len = own_length(p, entry - p.groups);
  for (int rb = 0; rb < p.blocks; ++rb) f(p.kv_heads, max(1, tiles_of(seen_by<RB>(p, len, rb))));
}

// Tiles of a part: an equal share, in whole rounds of four wavefronts, two
// rounds at least (a shorter part costs more to start than it gives).
__device__ __forceinline__ int part_tiles(uint32_t total, uint32_t parts) {
  return (int)max(((total + parts - 1) / parts + 3) / 4 * 4, 8u);
}

__device__ __forceinline__ int parts_of(int tiles, int share) {
  return (int)((uint32_t)(tiles + share - 1) / (uint32_t)share);
}

struct Spot {
  int entry;           // where a workgroup's part lies; -1: no such part
  int parts_before;    // parts of the entries before it
  int further_before;  // of those, the ones that are not an item's first
  int share;
};

// The entry of this workgroup's part: the tiles of all entries are summed, which
// gives the parts' length, and then the entries' counts of parts are scanned.
// All sums fit in 31 bits (the host's check).  Up to 64 entries, one a lane,
// every wavefront does it by itself: this stands before anything else that a
// workgroup does, and a barrier costs more than the repetition.
template <int RB>
__device__ __forceinline__ Spot find_part(const Params& p, int (&shared)[16]) {
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int entries = p.groups + p.batch, want = (int)(p.first_block + blockIdx.x);
  Spot spot;
  int parts = 0, items = 0;
  auto count = [&](int n, int each_tiles) {
    parts += n * parts_of(each_tiles, spot.share);
    items += n;
  };
  auto scan = [&](int& parts_upto, int& items_upto) {
    parts_upto = parts, items_upto = items;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const int a = __shfl_up(parts_upto, s), b = __shfl_up(items_upto, s);
      if (lane >= s) {
        parts_upto += a;
        items_upto += b;
      }
    }
  };
  auto sum_tiles = [&](int lo, int hi) {
    int tiles = 0;
    for (int e = lo; e < hi; ++e)
      items_of<RB>(p, e, [&](int n, int each_tiles) { tiles += n * each_tiles; });
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) tiles += __shfl_xor(tiles, s);
    return tiles;
  };
  int parts_upto, items_upto;
  if (entries <= 64) {
    const int lo = min(lane, entries), hi = min(lane + 1, entries);
    spot.share = part_tiles((uint32_t)sum_tiles(lo, hi), (uint32_t)p.parts);
    if (lo < hi) items_of<RB>(p, lo, count);
    scan(parts_upto, items_upto);
    const uint64_t past = __ballot(parts_upto > want);
    if (past == 0) {
      spot.entry = -1;
      return spot;
    }
    spot.entry = __builtin_ctzll(past);
    spot.parts_before = __builtin_amdgcn_readlane(parts_upto - parts, spot.entry);
    spot.further_before =
        spot.parts_before - __builtin_amdgcn_readlane(items_upto - items, spot.entry);
    return spot;
  }
  const int each = (entries + 255) / 256;
  const int lo = min(tid * each, entries), hi = min(lo + each, entries);
  const int tiles = sum_tiles(lo, hi);
  if (lane == 0) shared[wave] = tiles;
  __syncthreads();
  spot.share = part_tiles((uint32_t)(shared[0] + shared[1] + shared[2] + shared[3]),
                          (uint32_t)p.parts);
  for (int e = lo; e < hi; ++e) items_of<RB>(p, e, count);
  scan(parts_upto, items_upto);
  if (lane == 63) {
    shared[4 + wave] = parts_upto;
    shared[8 + wave] = items_upto;
  }
  if (tid == 0) shared[12] = -1;
  __syncthreads();
  int before = parts_upto - parts, items_before = items_upto - items;
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    if (w < wave) {
      before += shared[4 + w];
      items_before += shared[8 + w];
    }
  }
  if (want >= before && want < before + parts) {
    int e = lo;
    for (;; ++e) {
      parts = items = 0;
      items_of<RB>(p, e, count);
      if (want < before + parts) break;
      before += parts;
      items_before += items;
    }
    shared[12] = e;
    shared[13] = before;
    shared[14] = before - items_before;
  }
  __syncthreads();
  spot.entry = shared[12];
  spot.parts_before = shared[13];
  spot.further_before = shared[14];
  return spot;
}

template <int D, int RT, int WAVES>
struct Shared {
  static constexpr int kVRow = D / 2 + 16;  // padded against bank conflicts
  struct Tile {
    alignas(16) uint8_t codes[kTile * kVRow];
    alignas(16) _Float16 scales[D / 16][4][16];  // [block][t / 4 % 4][t / 16 * 4 + t % 4]
    alignas(16) float k_scale[kTile];
    alignas(16) float v_scale[kTile];
    float largest[16 * RT];  // of a row's weights, where the value scales are far apart
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

// Workgroups of four wavefronts that a CU holds (by registers).
constexpr int groups_per_cu(int d, int rt) {
  return rt == 1 && d <= 128 ? (d == 64 ? 4 : 3) : 2;
}

// The same value in every lane, said so: descriptors and branches come from it.
__device__ __forceinline__ int32_t same(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// Tiles [tile_lo, tile_hi) of an item; results to the output (more < 0: the
// item is whole) or as a partial result (tile_lo 0: by row; else as further
// part `next`).
template <int D, int RT, int WAVES>
__device__ __forceinline__ void attend(const Params& p, const Item& job, int tile_lo, int tile_hi,
                                       int next_part, int more, Shared<D, RT, WAVES>& sh) {
  constexpr int DT = D / 16, NK = D / 32, KS = D / 64;
  constexpr int KSW = KS == 3 ? 2 : 1;
  constexpr int VA = D / 128;          // 16-byte pieces of 16 tokens' value codes per lane,
  constexpr bool VB = D % 128 != 0;    // and one of 8 bytes
  constexpr int kVRow = Shared<D, RT, WAVES>::kVRow;
  constexpr int RB = 16 * RT;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int col = lane % 16, grp = lane / 16;
  const int steps = max(0, min(tile_hi, tiles_of(job.len)) - tile_lo - wave + WAVES - 1) / WAVES;
  float4v o[RT][DT];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY;
    l[rt] = 0.0f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[rt][dt] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  }
  // Value scales are held times 2^v_exp: up to `bound` they reach 2^14.  Once some lie far apart
  // from others, or are not finite, `apart` is set, and every step takes care of each row.  (At
  // every step without that flag it cost 1 to 3% of long contexts and 8% of many queries; so, up to
  // 1% and 2%.)
  float bound = 0.0f;
  int v_exp = 0;
  bool apart = false;

  // Pages: lane 4 k + j holds, for the 16 tokens j of step 16 n + k, the index of their first
  // cache row and of their first byte among the value scales of block 0.
  int64_t page_row = 0, page_scale = 0;
  auto load_pages = [&](int first_step) {
    const int tile = tile_lo + wave + (first_step + lane / 4) * WAVES;
    // (past the context's end: whatever the table holds there, clamped, and masked later; so
    // the first load need not wait for the context's length)
    const uint32_t g = min((uint32_t)tile * 4 + lane % 4, (uint32_t)job.pages * p.page_groups.d - 1);
    const uint32_t page = quotient(g, p.page_groups);
    const int at = (int)(g - page * p.page_groups.d) * 16;
    const int id = min(max(job.table[page], 0), p.num_pages - 1);
    const int64_t head = ((int64_t)id * p.kv_heads + job.kvh) * p.page_size;
    page_row = head + at;
    page_scale = head * DT + at;
  };
  int64_t row[4], vscale[4];  // of the step being loaded
  auto locate = [&](int step) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int from = (step % 16) * 4 + j;
      row[j] = lane_value(page_row, from);
      vscale[j] = lane_value(page_scale, from);
    }
  };

  // A lane's share of the 16 tokens j: 16 bytes of value codes (8 for 64-element heads; 192:
  // 16 and 8), one word of value scales (4 tokens of a block), and the key codes of token col
  // that its queries' elements meet.  Loaded through descriptors at the 16 tokens' first byte:
  // the lane's offset never changes, so a load takes no address arithmetic, and one past the
  // last step takes an empty descriptor instead of a branch.
  uint32_t kw[4][NK], ve[4];
  uint32_t ks[4][KSW];  // the words that hold the lane's KS key scale bytes
  u32x4v vw[4][VA ? VA : 1];
  u32x2v vh[4];
  float kt = 0.0f, vt = 0.0f;
  const uint32_t e_lane = (uint32_t)min(lane, DT * 4 - 1);
  const uint32_t e_at = e_lane / 4 * p.page_size + e_lane % 4 * 4;
  const uint32_t key_at = (uint32_t)(col * (D / 2) + grp * (D / 8));
  const uint32_t key_scale_word = KSW == 2 ? grp / 2 * 4 : grp * KS / 4 * 4;
  const uint32_t key_scale_at = (uint32_t)(col * DT) + key_scale_word;
  const uint32_t key_scale_shift = 8 * (grp * KS - key_scale_word);
  auto load_values = [&](int step) {
    const int bytes = __builtin_amdgcn_readfirstlane(step < steps ? -1 : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const auto c = __builtin_amdgcn_make_buffer_rsrc((void*)(p.codes[1] + row[j] * (D / 2)), 0,
                                                       bytes, 0x20000);
      const auto e =
          __builtin_amdgcn_make_buffer_rsrc((void*)(p.scales[1] + vscale[j]), 0, bytes, 0x20000);
#pragma unroll
      for (int r = 0; r < VA; ++r)
        vw[j][r] = __builtin_amdgcn_raw_buffer_load_b128(c, lane * 16, r * 1024, 0);
      if constexpr (VB) vh[j] = __builtin_amdgcn_raw_buffer_load_b64(c, lane * 8, VA * 1024, 0);
      ve[j] = __builtin_amdgcn_raw_buffer_load_b32(e, e_at, 0, 0);
    }
    if (step < steps) {
      const int from = step % 16 * 4 + grp;  // the lane that holds this lane's tokens' place
      const int64_t mine = __shfl(page_row, from) + col;
      kt = p.token_scales[0][mine];
      vt = p.token_scales[1][mine];
    }
  };
  auto load_keys = [&](int step) {
    const int bytes = __builtin_amdgcn_readfirstlane(step < steps ? -1 : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const auto c = __builtin_amdgcn_make_buffer_rsrc((void*)(p.codes[0] + row[j] * (D / 2)), 0,
                                                       bytes, 0x20000);
      const auto e =
          __builtin_amdgcn_make_buffer_rsrc((void*)(p.scales[0] + row[j] * DT), 0, bytes, 0x20000);
      if constexpr (NK % 4 == 0) {
#pragma unroll
        for (int k = 0; k < NK; k += 4) {
          const u32x4v w = __builtin_amdgcn_raw_buffer_load_b128(c, key_at, k * 4, 0);
          kw[j][k] = w[0], kw[j][k + 1] = w[1], kw[j][k + 2] = w[2], kw[j][k + 3] = w[3];
        }
      } else {
#pragma unroll
        for (int k = 0; k < NK; k += 2) {
          const u32x2v w = __builtin_amdgcn_raw_buffer_load_b64(c, key_at, k * 4, 0);
          kw[j][k] = w[0], kw[j][k + 1] = w[1];
        }
      }
      // whole words: a byte or half-word load would be widened, and so waited for, at once
      if constexpr (KSW == 1) {
        ks[j][0] = __builtin_amdgcn_raw_buffer_load_b32(e, key_scale_at, 0, 0);
      } else {
        const u32x2v w = __builtin_amdgcn_raw_buffer_load_b64(e, key_scale_at, 0, 0);
        ks[j][0] = w[0], ks[j][1] = w[1];
      }
    }
  };

  auto& tile = sh.tile[wave];
  const int turned = 16 * (col / 4) + 4 * grp + col % 4;  // the token whose row this lane names
  auto turned_codes = [&](int dt) {
    return __builtin_amdgcn_ds_read_tr4_b64_v2i32(
        (__attribute__((address_space(3))) int2v*)(tile.codes + turned * kVRow + dt * 8));
  };
  // The page table, then the queries, then the first tile are asked for (each waits for the one
  // before: the table entry is made into addresses at once, and a row that does not exist is a
  // branch).  Queries: lane (col, grp) holds row col's elements [grp D/4, (grp + 1) D/4).
  u32x4v raw[RT][NK];
  int limit[RT];
  if (job.pages > 0) load_pages(0);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const bool live = rt * 16 + col < job.rows;
    const int r = live ? rt * 16 + col : 0;
    const Row row = row_of(p, job, r);
    const uint16_t* src = p.q + row.token * p.q_stride + (int64_t)row.head * D + grp * (D / 4);
    limit[rt] = job.prefix ? job.len : job.own_len - p.q_tokens + 1 + row.t;
#pragma unroll
    for (int k = 0; k < NK; ++k) raw[rt][k] = live ? ((const u32x4v*)src)[k] : (u32x4v){0, 0, 0, 0};
  }
  if (steps > 0) {
    locate(0);
    load_values(0);
    load_keys(0);
  }
  half8v q[RT][NK];
  float c_q[RT];
  // The score factor of a row, scale log2(e) 2^-ex, leaves FP32's range where tiny queries meet
  // a small scale, or huge ones a large one.  Then it is held times 2^lift, and the token scales
  // divided by that, with the lift that brings the largest factor of the wavefront's rows to
  // [0.5, 1): the others are smaller as their queries are.  (Ordinary rows, whose factors lie
  // around 2^-16, keep 0: without the reduction over the rows, which takes 0.2 us.)  The factor's
  // mantissa, the same for all rows, goes with the token scales, so that c_q is a power of two:
  // its products are exact, and so is their difference to m, however large the scores are.
  const float factor_part = __builtin_amdgcn_frexp_mantf(__builtin_fabsf(p.scale) * kLog2e);
  const int factor_exp = __builtin_amdgcn_frexp_expf(__builtin_fabsf(p.scale) * kLog2e);
  constexpr int kNone = -100000;
  int c_exp[RT], lift = 0;
  bool far = false;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = max(top, max(raw[rt][k][i] & 0x7FFFu, raw[rt][k][i] >> 16 & 0x7FFFu));
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    // 2^ex: the row's largest element lands in [2^14, 2^15).  A row of zeros, or one
    // with a NaN or infinity, stays as it is
    const int field = (int)(top >> 7);
    const int ex = top == 0 || field == 255 ? 0 : 14 + 127 - max(field, 1);
    const float sign = p.scale < 0.0f ? -1.0f : 1.0f;
    c_exp[rt] = top == 0 || p.scale == 0.0f ? kNone : factor_exp - ex;
    far |= c_exp[rt] != kNone && (c_exp[rt] < -32 || c_exp[rt] > 64);
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[rt][k][2 * i] = (_Float16)__builtin_ldexpf(bf16_lo(raw[rt][k][i]) * sign, ex);
        q[rt][k][2 * i + 1] = (_Float16)__builtin_ldexpf(bf16_hi(raw[rt][k][i]) * sign, ex);
      }
  }
  if (__any(far)) {
    int most = kNone;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) most = max(most, c_exp[rt]);
#pragma unroll
    for (int s = 8; s > 0; s /= 2) most = max(most, __shfl_xor(most, s));
    lift = -most;
  }
  // (never 0, so that a masked score's -infinity stays one)
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    c_q[rt] = fmaxf(__builtin_ldexpf(1.0f, c_exp[rt] + lift), 0x1p-149f);
  for (int step = 0; step < steps; ++step) {
    const int t0 = (tile_lo + wave + step * WAVES) * kTile;
    const int left = job.len - t0;  // tokens of this tile that exist
    // values and scales into LDS; scales of tokens past the end become zero, so that
    // whatever lies there adds nothing
    if (left < kTile) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = min(max(left - 16 * j - 4 * (int)(e_lane % 4), 0), 4);  // of these 4 tokens
        ve[j] = n == 0 ? 0 : ve[j] & (~0u >> (32 - 8 * n));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int r = 0; r < VA; ++r) {
        const int byte = r * 1024 + lane * 16;
        *(u32x4v*)(tile.codes + (16 * j + byte / (D / 2)) * kVRow + byte % (D / 2)) = vw[j][r];
      }
      if constexpr (VB) {
        const int byte = VA * 1024 + lane * 8;
        *(u32x2v*)(tile.codes + (16 * j + byte / (D / 2)) * kVRow + byte % (D / 2)) = vh[j];
      }
      const half2v a = e4m3_f16x2<0>(ve[j]), b = e4m3_f16x2<1>(ve[j]);
      *(half4v*)&tile.scales[e_lane / 4][e_lane % 4][j * 4] = (half4v){a[0], a[1], b[0], b[1]};
    }
    float vt_live = lane < left ? vt : 0.0f;
    uint64_t broken = 0;  // tokens whose value scale is infinite or NaN
    if (__any(!(vt_live <= bound) || (vt_live * kFar < bound && vt_live != 0.0f))) {
      broken = __ballot(!(vt_live < INFINITY));
      if (!(vt_live < INFINITY)) vt_live = 0.0f;
      const float top = max_of_groups(vt_live);
      float all = top;
#pragma unroll
      for (int s = 8; s > 0; s /= 2) all = fmaxf(all, __shfl_xor(all, s));
      const bool before = apart;
      int down = 0;
      if (all > bound) {
        // a larger value scale than any before: a new power of two, with room for 8 times more
        const int ex = min(__builtin_amdgcn_frexp_expf(all) + 3, 127);
        const float grown = __builtin_ldexpf(1.0f, ex);
        if (__any(bound == 0.0f)) {  // the first
          if (!apart) tile.largest[0] = grown;
        } else {
          down = 14 - ex - v_exp;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[rt][dt][i] = __builtin_ldexpf(o[rt][dt][i], down);
          apart = apart || __any(tile.largest[0] * 0x1p6f < grown);
        }
        bound = grown;
        v_exp = 14 - ex;
      }
      // Scales within 2^14 of the bound, or 2^20 of a later one, leave the weights of every row
      // 2^23 of precision.  Any further apart, rows are kept apart as well (below).
      apart = apart || broken != 0 || __any(vt_live * kFar < bound && vt_live != 0.0f);
      if (apart) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          tile.largest[rt * 16 + col] = __builtin_ldexpf(
              before ? tile.largest[rt * 16 + col] : m[rt] == -INFINITY ? 0.0f : 0x1p14f, down);
      }
    }
    tile.k_scale[lane] = __builtin_ldexpf(kt * factor_part, -lift);
    tile.v_scale[lane] = __builtin_ldexpf(vt_live, v_exp);
    if ((step + 1) % 16 == 0) load_pages(step + 1);
    locate(step + 1);
    load_values(step + 1);

    // scores
    float4v s[RT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
      uint32_t e_bytes = ks[j][0];
      if constexpr (KSW == 2)
        e_bytes = (uint32_t)(((uint64_t)ks[j][1] << 32 | ks[j][0]) >> key_scale_shift);
      else if constexpr (KS < 4)
        e_bytes >>= key_scale_shift;
      const half2v e01 = e4m3_f16x2<0>(e_bytes), e23 = e4m3_f16x2<1>(e_bytes);
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
    load_keys(step + 1);

    // softmax
    half8v w[RT][2];
    const bool edge = t0 + kTile > job.floor;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt > 0 && rt * 16 >= job.rows) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) s[rt][j] *= *(const float4v*)&tile.k_scale[16 * j + 4 * grp];
      if (edge) {
        asm volatile("");  // keeps this a branch: most tiles have no edge
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t0 + 16 * j + 4 * grp + i >= limit[rt]) s[rt][j][i] = -INFINITY;
      }
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        top = __builtin_elementwise_maximum(
            __builtin_elementwise_maximum(top, s[rt][j][0]), s[rt][j][1]);
        top = __builtin_elementwise_maximum(
            __builtin_elementwise_maximum(top, s[rt][j][2]), s[rt][j][3]);
      }
      top = max_of_groups(top) * c_q[rt];
      if (__any(!(top <= m[rt])) || apart) {
        const float grown = __builtin_elementwise_maximum(m[rt], top);
        const float keep = m[rt] == -INFINITY ? 1.0f : factor(m[rt], grown);
        m[rt] = grown;
        l[rt] *= keep;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[rt][dt] *= keep;
        if (apart) {
          // The larger value scales may have no weight in this row, or not be seen by it: m is
          // lowered until the row's largest weight is near 2^14, as far as l has room for that
          // (2^100: sums of l over wavefronts and parts stay within FP32).  A row that sees an
          // infinite or NaN scale becomes NaN.
          const float from = m[rt] == -INFINITY ? 0.0f : m[rt];
          float largest = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int token = 16 * j + 4 * grp + i;
              const float e =
                  __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][j][i], c_q[rt], -from));
              largest = fmaxf(largest, e * tile.v_scale[token]);
            }
          const int seen = limit[rt] - t0;
          const bool bad = seen > 0 && (broken << (64 - min(seen, 64))) != 0;
          largest = fmaxf(max_of_groups(largest), tile.largest[rt * 16 + col] * keep);
          int up = min(14 - __builtin_amdgcn_frexp_expf(largest),
                       100 - __builtin_amdgcn_frexp_expf(max_of_groups(l[rt])));
          // (past 2^22 a difference of 1 would be lost)
          if (!(largest > 0.0f) || !(__builtin_fabsf(from) < 0x1p22f)) up = 0;
          m[rt] -= up;
          l[rt] = __builtin_ldexpf(l[rt], up);
          tile.largest[rt * 16 + col] = __builtin_ldexpf(largest, up);
          const float poison = bad ? __builtin_nanf("") : 0.0f;
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[rt][dt][i] = __builtin_ldexpf(o[rt][dt][i], up) + poison;
        }
      }
      const float base = m[rt] == -INFINITY ? 0.0f : m[rt];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4v e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][j][i], c_q[rt], -base));
          l[rt] += e[i];
        }
        e *= *(const float4v*)&tile.v_scale[16 * j + 4 * grp];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[rt][j / 2][j % 2 * 4 + i] = (_Float16)e[i];
      }
    }

    // values, the next 16 columns' codes and scales read while these are multiplied
    int2v c = turned_codes(0);
    half8v e0 = *(const half8v*)&tile.scales[0][grp][0], e1 = *(const half8v*)&tile.scales[0][grp][8];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      int2v c_next = c;
      half8v e0_next = e0, e1_next = e1;
      if (dt + 1 < DT) {
        c_next = turned_codes(dt + 1);
        e0_next = *(const half8v*)&tile.scales[dt + 1][grp][0];
        e1_next = *(const half8v*)&tile.scales[dt + 1][grp][8];
      }
      const half8v v0 = decode8((uint32_t)c[0], (half2v){e0[0], e0[1]}, (half2v){e0[2], e0[3]},
                                (half2v){e0[4], e0[5]}, (half2v){e0[6], e0[7]});
      const half8v v1 = decode8((uint32_t)c[1], (half2v){e1[0], e1[1]}, (half2v){e1[2], e1[3]},
                                (half2v){e1[4], e1[5]}, (half2v){e1[6], e1[7]});
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (rt > 0 && rt * 16 >= job.rows) continue;
        o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w[rt][0], o[rt][dt], 0, 0, 0);
        o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w[rt][1], o[rt][dt], 0, 0, 0);
      }
      c = c_next;
      e0 = e0_next;
      e1 = e1_next;
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // the wavefronts' results joined, 16 rows at a time; each thread takes pairs of one row
  const int tid = threadIdx.x, row_in = tid / (WAVES * 4), sub = tid % (WAVES * 4);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (rt * 16 >= job.rows) break;
    __syncthreads();
    const float sum = sum_of_groups(l[rt]);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
      *(float4v*)&sh.merge.o[wave][col][dt * 16 + grp * 4] =
          (float4v){__builtin_ldexpf(o[rt][dt][0], -v_exp), __builtin_ldexpf(o[rt][dt][1], -v_exp),
                    __builtin_ldexpf(o[rt][dt][2], -v_exp), __builtin_ldexpf(o[rt][dt][3], -v_exp)};
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
      const Row of = row_of(p, job, r);
      const int64_t row = of.token * p.q_heads + of.head;
      const int64_t next = (int64_t)next_part * RB + r;
      float* to = tile_lo > 0 ? p.next_o + next * D : p.first_o[job.prefix] + row * D;
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
        if (more < 0)
          *(uint32_t*)(p.out + row * D + d) = cvt_bf16x2(a * inv, b * inv);
        else
          *(float2*)(to + d) = make_float2(a, b);
      }
      if (sub == 0) {
        if (tile_lo > 0)
          p.next_ml[next] = make_float2(top, total);
        else if (p.parts > 0)
          p.first[job.prefix][row] = First{top, total, next_part, more};
        if (more < 0 && p.lse)
          p.lse[row] = total == 0.0f ? -INFINITY : (base + __builtin_log2f(total)) * kLn2;
      }
    }
  }
}

template <int RB>
__device__ __forceinline__ void own_item(const Params& p, int b, int rb, Item& j) {
  j.prefix = false;
  j.first_b = b;
  j.row0 = rb * RB;
  j.rows = min(RB, (int)p.per_seq.d - j.row0);
  j.table = p.page_table + (int64_t)b * p.max_pages;
  j.pages = p.max_pages;
  j.own_len = own_length(p, b);
  j.len = seen_by<RB>(p, j.own_len, rb);
  j.floor = max(0, j.own_len - p.q_tokens + 1 + (int)quotient(j.row0, p.per_head));
}

__device__ __forceinline__ void make_uniform(Item& j) {
  j.len = same(j.len);
  j.floor = same(j.floor);
  j.first_b = same(j.first_b);
  j.row0 = same(j.row0);
  j.rows = same(j.rows);
  j.own_len = same(j.own_len);
  j.kvh = same(j.kvh);
}

// One workgroup per own item.
template <int D, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES == 4 ? groups_per_cu(D, RT)
                                         : D == 64  ? 4
                                                    : 2) void attention_items(Params p) {
  __shared__ Shared<D, RT, WAVES> sh;
  const uint32_t block = p.first_block + blockIdx.x, pair = block / (uint32_t)p.kv_heads;
  Item job;
  own_item<16 * RT>(p, (int)(pair / (uint32_t)p.blocks), (int)(pair % (uint32_t)p.blocks), job);
  job.kvh = (int)(block % (uint32_t)p.kv_heads);
  make_uniform(job);
  attend<D, RT, WAVES>(p, job, 0, tiles_of(job.len), 0, -1, sh);
}

// One workgroup per part.
template <int D, int RT>
__global__ __launch_bounds__(256, groups_per_cu(D, RT)) void attention_parts(Params p) {
  constexpr int RB = 16 * RT;
  __shared__ Shared<D, RT, 4> sh;
  __shared__ int scratch[16];
  const Spot spot = find_part<RB>(p, scratch);
  const int entry = same(spot.entry), share = same(spot.share);
  if (entry < 0) return;
  int at = (int)(p.first_block + blockIdx.x) - same(spot.parts_before);  // the part's number in its entry
  int further = same(spot.further_before);
  Item job;
  int tiles, item, n;
  if (entry < p.groups) {
    const Members m = members_of(p, entry);
    const int rows = (m.hi - m.lo) * (int)p.per_seq.d, blocks = (rows + RB - 1) / RB;
    job.prefix = true;
    job.table = p.prefix_table + (int64_t)entry * p.max_prefix_pages;
    job.pages = p.max_prefix_pages;
    job.len = job.floor = job.own_len = prefix_length(p, entry);
    tiles = tiles_of(job.len);
    n = parts_of(tiles, share);
    item = at / n;
    // heads outside, row blocks inside: a head's blocks share their tokens
    job.kvh = item / blocks;
    job.first_b = m.lo;
    job.row0 = (item - job.kvh * blocks) * RB;
    job.rows = min(RB, rows - job.row0);
  } else {
    int rb = 0;
    for (;; ++rb) {
      own_item<RB>(p, entry - p.groups, rb, job);
      tiles = max(1, tiles_of(job.len));
      n = parts_of(tiles, share);
      if (at < n * p.kv_heads) break;
      at -= n * p.kv_heads;
      further += (n - 1) * p.kv_heads;
    }
    item = job.kvh = at / n;
  }
  make_uniform(job);
  tiles = same(tiles);
  n = same(n);
  item = same(item);
  const int part = at - item * n;
  further += item * (n - 1);
  // n parts of equal length, to a tile
  const int lo = same((int)((int64_t)tiles * part / n));
  const int hi = same((int)((int64_t)tiles * (part + 1) / n));
  // (group offsets that overlap, against the definition, could ask for more than there are)
  if (lo > 0 && (uint32_t)(further + part - 1) >= (uint32_t)p.parts) return;
  attend<D, RT, 4>(p, job, lo, hi, further + max(part - 1, 0),
                   p.groups == 0 && n == 1 ? -1 : n - 1, sh);
}

// The partial results of query rows joined, in the order of their tokens:
// prefix, then own.  A workgroup takes ROWS heads of one token (1, or all
// that its threads have room for); D / 4 threads hold a row's elements, and
// with ROWS 1 the others share the row's parts.
template <int D, int RT, bool ONE>
__global__ __launch_bounds__(256) void attention_join(Params p) {
  constexpr int RB = 16 * RT, COLS = D / 4, LANES = 256 / COLS;
  __shared__ float4v acc_of[LANES][COLS];
  __shared__ float top_of[LANES], total_of[LANES];
  const int lane = threadIdx.x / COLS, d = threadIdx.x % COLS * 4;
  const int64_t per = ONE ? p.q_heads : (p.q_heads + LANES - 1) / LANES;
  const uint32_t block = p.first_block + blockIdx.x;
  const int64_t bt = block / (uint32_t)per;
  const int head = (int)(block - bt * per) * (ONE ? 1 : LANES) + (ONE ? 0 : lane);
  if (!ONE && (lane >= LANES || head >= p.q_heads)) return;
  const int64_t row = bt * p.q_heads + head;
  const First own = p.first[0][row];
  if (own.more < 0) return;  // written whole
  const int b = (int)(bt / p.q_tokens), t = (int)(bt - (int64_t)b * p.q_tokens);
  const int kvh = (int)quotient(head, p.per_head);
  const int in_seq = (t - kvh) * (int)p.per_head.d + head;

  float top = -INFINITY, total = 0.0f;
  float4v acc = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](float m, float l, float4v v) {
    const float grown = m > top ? m : top;  // a NaN in l and O stays one in the sums
    const float base = grown == -INFINITY ? 0.0f : grown;
    const float keep = factor(top, base), f = factor(m, base);
    total = total * keep + f * l;
    acc = acc * keep + f * v;
    top = grown;
  };
  // r: the row's number in its item's block
  auto gather = [&](const First& first, const float* o, int r) {
    const float4v v = *(const float4v*)(o + d);
    // (within the workspace, whatever overlapping groups have left unwritten)
    const int more =
        (uint32_t)first.next < (uint32_t)p.parts ? min(first.more, p.parts - first.next) : 0;
    // some parts at a time, so that their loads are in flight together (one context of 32k
    // tokens 19.7 us, one part at a time 21.1)
    constexpr int STEP = ONE ? LANES : 1, MANY = 4;
    for (int i = ONE ? lane : 0; i < more; i += STEP * MANY) {
      float2 ml[MANY];
      float4v part[MANY];
#pragma unroll
      for (int j = 0; j < MANY; ++j) {
        const int64_t at = (int64_t)(first.next + min(i + j * STEP, more - 1)) * RB + r;
        ml[j] = p.next_ml[at];
        part[j] = *(const float4v*)(p.next_o + at * D + d);
      }
      if (i == 0) add(first.m, first.l, v);
#pragma unroll
      for (int j = 0; j < MANY; ++j)
        if (i + j * STEP < more) add(ml[j].x, ml[j].y, part[j]);
    }
    if (more <= 0 && (!ONE || lane == 0)) add(first.m, first.l, v);
  };
  if (p.groups > 0) {
    // the last group that starts at or before this row's sequence
    int lo = 0, hi = p.groups;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.group_offsets[mid] <= b)
        lo = mid + 1;
      else
        hi = mid;
    }
    if (lo > 0) {
      const Members m = members_of(p, lo - 1);
      if (b >= m.lo && b < m.hi && prefix_length(p, lo - 1) > 0)
        gather(p.first[1][row], p.first_o[1] + row * D,
               ((b - m.lo) * (int)p.per_seq.d + in_seq) % RB);
    }
  }
  gather(own, p.first_o[0] + row * D, in_seq % RB);
  if constexpr (ONE) {
    if (lane < LANES) {
      acc_of[lane][d / 4] = acc;
      if (d == 0) {
        top_of[lane] = top;
        total_of[lane] = total;
      }
    }
    __syncthreads();
    if (lane != 0) return;
    for (int i = 1; i < LANES; ++i) top = top_of[i] > top ? top_of[i] : top;
    const float base = top == -INFINITY ? 0.0f : top;
    total = 0.0f;
    acc = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < LANES; ++i) {
      const float f = factor(top_of[i], base);
      total += f * total_of[i];
      acc += f * acc_of[i][d / 4];
    }
  }
  const float base = top == -INFINITY ? 0.0f : top;
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  *(uint2*)(p.out + row * D + d) = make_uint2(cvt_bf16x2(acc[0] * inv, acc[1] * inv),
                                              cvt_bf16x2(acc[2] * inv, acc[3] * inv));
  if (d == 0 && p.lse)
    p.lse[row] = total == 0.0f ? -INFINITY : (base + __builtin_log2f(total)) * kLn2;
}

// ---- shape of a call --------------------------------------------------------

struct Plan {
  int rt;  // 16-row tiles of queries per wavefront
  bool wide;  // items: eight wavefronts a workgroup, not four
  int64_t blocks, items, rows;
  int64_t parts;   // 0: one workgroup per item
  int64_t groups;  // workgroups
  bool fits;       // workgroups and tiles within 31 bits
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

Plan plan_of(int64_t page_size, int64_t kv_heads, int64_t head_dim, int64_t batch,
             int64_t q_tokens, int64_t q_heads, int64_t max_pages, int64_t max_prefix_pages,
             int64_t groups) {
  Plan p;
  const int64_t per_seq = q_tokens * (q_heads / kv_heads);
  const int64_t rows_each = groups ? batch * per_seq / groups : per_seq;
  // One row tile a workgroup, or two that share what they decode.  Two from heads of 192 on would
  // take 416 registers and more: one workgroup per CU (16 sequences a prompt of 8192, heads of
  // 256: 80 us with one, 116 with two).  Groups: one up to 256 rows each (4 x 64 rows x 8192 tokens
  // 49 us with one, 52 with two; 4 x 512 rows x 16384 318 and 276).  Without groups: two where
  // a tile would not hold a sequence's and twos are enough for all CUs (64 sequences x 64 rows x
  // 512-2000 tokens 66 us with two, 75 with one; 4 such sequences 27 and 17)
  const bool two = groups ? rows_each > 256
                          : per_seq > 16 && batch * ceil_div(per_seq, 32) * kv_heads >= 256;
  p.rt = head_dim <= 128 && two ? 2 : 1;
  p.blocks = ceil_div(per_seq, 16 * p.rt);
  p.rows = batch * q_tokens * q_heads;
  p.items = batch * p.blocks * kv_heads;
  const int64_t held = 256 * groups_per_cu((int)head_dim, p.rt);
  const int64_t tokens = max_pages * page_size;
  // One row tile: eight wavefronts a workgroup where the chip holds all of them at once (128
  // items of heads of 128, 100-700 tokens: 9.7 us with eight, 11.1 with four), else four
  // (512 items of 512 tokens 19.8 and 14.2, 2048 of 30-500 60 and 34)
  p.wide = p.rt == 1 && p.items <= (head_dim == 64 ? 512 : 256);
  // One workgroup per item where the contexts are short (777 tokens 10.8 us so, 13.4 cut), also
  // longer ones where items keep all CUs busy (512 of 2000-4000 tokens 56 and 65, 256 of 1000-4000
  // 30 and 37; but 64 of 2000-4000 27 and 19, and 8 of such a length among 56 of 300 tokens 23 and
  // 14), or the items so many that their unequal lengths even out.  Else as many parts as the chip
  // holds workgroups; twice as many where one tile holds a sequence's rows (64 x 2048-8192 tokens:
  // 97 us, 101 with one); two a CU with groups, whose rows are many to join (4 x 256 rows x 8192
  // tokens 63 us, 73 with one a CU, 64 with three; 4 x 64 rows 50, 46 and 50; the same with heads
  // of 64 34, 37 and 37)
  p.parts = groups ? 512
            : tokens <= (p.items >= 256 ? 4096 : 2048) || p.items >= 8 * held ? 0
            : per_seq <= 16 ? 2 * held : held;
  // row blocks of all groups at most, and so parts at most: each cut adds one to an item's first
  const int64_t prefix_items = groups ? (batch * per_seq / (16 * p.rt) + groups) * kv_heads : 0;
  p.groups = p.items + (p.parts ? p.parts + prefix_items : 0);
  const double tiles = (double)p.items * (double)ceil_div(tokens, kTile) +
                       (double)prefix_items * (double)ceil_div(max_prefix_pages * page_size, kTile);
  p.fits = p.groups < ((int64_t)1 << 31) && (p.parts == 0 || tiles < 2147483648.0);
  return p;
}

int64_t first_parts(int64_t groups) { return groups ? 2 : 1; }

// The dispatch packet counts work-items in 32 bits: larger calls go in several launches.
constexpr int64_t kMaxItems = (int64_t)1 << 31;

template <class F>
hipError_t in_launches(Params& p, int64_t blocks, int threads, F launch_blocks) {
  const int64_t step = kMaxItems / threads;
  for (int64_t b0 = 0; b0 < blocks; b0 += step) {
    p.first_block = (uint32_t)b0;
    launch_blocks((uint32_t)(blocks - b0 < step ? blocks - b0 : step));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int D, int RT>
hipError_t join(Params& p, const Plan& plan, hipStream_t stream) {
  constexpr int64_t lanes = 256 / (D / 4);
  // few rows: a workgroup for each, whose threads share its parts
  if (plan.rows < 1024)
    return in_launches(p, plan.rows, 256, [&](uint32_t grid) {
      attention_join<D, RT, true><<<grid, 256, 0, stream>>>(p);
    });
  return in_launches(p, plan.rows / p.q_heads * ceil_div(p.q_heads, lanes), 256,
                     [&](uint32_t grid) {
                       attention_join<D, RT, false><<<grid, 256, 0, stream>>>(p);
                     });
}

template <int D, int RT>
hipError_t launch(Params& p, const Plan& plan, hipStream_t stream) {
  if (plan.parts == 0) {
    if constexpr (RT == 1) {
      if (plan.wide)
        return in_launches(p, plan.groups, 512, [&](uint32_t grid) {
          attention_items<D, RT, 8><<<grid, 512, 0, stream>>>(p);
        });
    }
    return in_launches(p, plan.groups, 256, [&](uint32_t grid) {
      attention_items<D, RT, 4><<<grid, 256, 0, stream>>>(p);
    });
  }
  const hipError_t e = in_launches(p, plan.groups, 256, [&](uint32_t grid) {
    attention_parts<D, RT><<<grid, 256, 0, stream>>>(p);
  });
  return e != hipSuccess ? e : join<D, RT>(p, plan, stream);
}

}  // namespace

bool kv_attention_fits(int64_t page_size, int64_t kv_heads, int64_t head_dim, int64_t batch,
                       int64_t q_tokens, int64_t q_heads, int64_t max_pages,
                       int64_t max_prefix_pages, int64_t groups) {
  return plan_of(page_size, kv_heads, head_dim, batch, q_tokens, q_heads, max_pages,
                 max_prefix_pages, groups)
      .fits;
}

int64_t kv_attention_workspace_bytes(int64_t page_size, int64_t kv_heads, int64_t head_dim,
                                     int64_t batch, int64_t q_tokens, int64_t q_heads,
                                     int64_t max_pages, int64_t max_prefix_pages,
                                     int64_t groups) {
  const Plan p = plan_of(page_size, kv_heads, head_dim, batch, q_tokens, q_heads, max_pages,
                         max_prefix_pages, groups);
  return p.parts == 0
             ? 0
             : first_parts(groups) * p.rows * (head_dim * 4 + (int64_t)sizeof(First)) +
                   p.parts * 16 * p.rt * (head_dim * 4 + 8);
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
  // sums, then the 16-byte and the 8-byte records
  const int64_t parts = first_parts(a.groups), next = plan.parts * 16 * plan.rt;
  float* o = (float*)a.workspace;
  First* first = (First*)(o + (parts * plan.rows + next) * c.head_dim);
  for (int i = 0; i < 2; ++i) {
    const int64_t at = i < parts ? i * plan.rows : 0;
    p.first_o[i] = o + at * c.head_dim;
    p.first[i] = first + at;
  }
  p.next_o = o + parts * plan.rows * c.head_dim;
  p.next_ml = (float2*)(first + parts * plan.rows);
  p.q_stride = a.q_stride;
  p.rows = plan.rows;
  p.num_pages = (int32_t)c.num_pages;
  p.page_size = (int32_t)c.page_size;
  p.kv_heads = (int32_t)c.kv_heads;
  p.page_groups = divisor_of((uint32_t)(c.page_size / 16));
  p.per_head = divisor_of((uint32_t)(a.q_heads / c.kv_heads));
  p.per_seq = divisor_of((uint32_t)(a.q_tokens * (a.q_heads / c.kv_heads)));
  p.batch = (int32_t)a.batch;
  p.q_tokens = (int32_t)a.q_tokens;
  p.q_heads = (int32_t)a.q_heads;
  p.max_pages = (int32_t)a.max_pages;
  p.max_prefix_pages = (int32_t)a.max_prefix_pages;
  p.groups = (int32_t)a.groups;
  p.blocks = (int32_t)plan.blocks;
  p.parts = (int32_t)plan.parts;
  p.scale = a.scale;
  switch (c.head_dim) {
    case 64: return plan.rt == 1 ? launch<64, 1>(p, plan, stream) : launch<64, 2>(p, plan, stream);
    case 128:
      return plan.rt == 1 ? launch<128, 1>(p, plan, stream) : launch<128, 2>(p, plan, stream);
    case 192: return launch<192, 1>(p, plan, stream);
    default: return launch<256, 1>(p, plan, stream);
  }
}

}  // namespace fp4q
