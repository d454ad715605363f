// layer_rows.hip -- tokens' rows to their experts' places, and the weighted
// sums back (definitions in include/fp4q/layer.h).
//
// Mathematics.  A stable counting sort of the tokens * top_k choices by
// expert: a choice's place is the number of choices of lower experts, plus
// those of the same expert before it.  Whole numbers throughout, so the order
// of additions does not matter; places are the same from call to call.
//
// Work.  Few choices: every workgroup counts them all and copies its tokens'
// rows, one launch.  Many: counts per chunk of choices; places from the counts
// of the chunks before; then the rows, each token's read once and written to
// its places.  The sums back read every row once.
//
// Bounds.  Launches, while there are few rows: 64 tokens of 8 rows of 7168
// take 4.3 us on the device and their sums 3.5, where a launch that does
// nothing is about 2.  Memory, when there are many: 8192 tokens of 8 rows of
// 2048, 302 MB there and 336 back, take 120 us together, 5.3 TB/s, where a
// large copy reaches 5.6 to 6.4; of these the places are 10 us.
#include <algorithm>

#include "layer_launch.h"
#include "rollout_divisor.h"

namespace fp4q {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPass = 1024;         // choices that a workgroup counts or places at a time
constexpr int kMaxChunks = 256;     // workgroups of a call: every one reads all their counts
// Choices up to which one launch does everything: 512 tokens of 8 rows of 2048 take 8.4 us in one
// and 13.6 in three, 64 of 7168 4.7 and 17.2; 1024 of 8 rows 16.0 and 17.4, 4096 of one of 1024 8.3
// and 11.3, 1024 of 8 11.0 and 14.2; 2048 of 8 rows 30.4 and 23.8.
constexpr int64_t kFew = 8192;
constexpr int kMaxExperts = 1024, kMaxChoices = 64;
constexpr int64_t kLastLevel = 256 << 20;  // bytes of the cache in front of memory

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

struct Params {
  const char* x;
  char* rows;
  const int32_t* chosen;
  int64_t* offsets;
  int32_t* place;
  int32_t* counts;  // [chunks][experts]
  int64_t hidden;
  Divisor top_k;
  int32_t entries, experts;
  int32_t chunks, chunk;  // and the choices of one, whole passes
  int64_t tokens;
  int32_t each;  // tokens of a workgroup, where one launch does everything
};

// counts[e] -> their sums before e, for threads of one workgroup; the sum of all is returned.
__device__ __forceinline__ int scan_counts(int* counts, int experts, int (&shared)[kWaves]) {
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int each = (experts + kThreads - 1) / kThreads;
  const int lo = min(tid * each, experts), hi = min(lo + each, experts);
  int own = 0;
  for (int e = lo; e < hi; ++e) own += counts[e];
  int upto = own;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const int o = __shfl_up(upto, s);
    if (lane >= s) upto += o;
  }
  if (lane == 63) shared[wave] = upto;
  __syncthreads();
  int before = upto - own, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += shared[w];
    all += shared[w];
  }
  for (int e = lo; e < hi; ++e) {
    const int n = counts[e];
    counts[e] = before;
    before += n;
  }
  __syncthreads();
  return all;
}

// One V at a time from a token's row to the places of its choices, RUN of them, `step` apart, to
// one place before the next.  ONCE: past the caches.
template <class V, int RUN, bool ONCE>
__device__ __forceinline__ void copy_row(const Params& p, int64_t token, const int* place,
                                         int64_t first, int step) {
  const int64_t bytes = p.hidden * 2, pieces = bytes / (int64_t)sizeof(V);
  const V* from = (const V*)(p.x + token * bytes);
  for (int64_t i = first; i < pieces; i += RUN * step) {
    V v[RUN];
#pragma unroll
    for (int r = 0; r < RUN; ++r) v[r] = from[min(i + r * step, pieces - 1)];
    for (int j = 0; j < (int)p.top_k.d; ++j) {
      if (place[j] < 0) continue;
      V* to = (V*)(p.rows + (int64_t)place[j] * bytes);
#pragma unroll
      for (int r = 0; r < RUN; ++r) {
        if (i + r * step >= pieces) break;
        if constexpr (ONCE)
          __builtin_nontemporal_store(v[r], to + i + r * step);
        else
          to[i + r * step] = v[r];
      }
    }
  }
}

// One workgroup a token, or SEVERAL, one after the other, and part of their rows; every one counts
// all choices.
template <class V, bool SEVERAL>
__global__ __launch_bounds__(kThreads) void dispatch_few(const Params p) {
  __shared__ int total[kMaxExperts], before[kMaxExperts], sums[kWaves], places[kMaxChoices];
  const int tid = threadIdx.x, k = (int)p.top_k.d;
  for (int e = tid; e < p.experts; e += kThreads) total[e] = before[e] = 0;
  __syncthreads();
  const int from = (int)blockIdx.x * (SEVERAL ? p.each : 1);  // the first token
  const int to = min(from + (SEVERAL ? p.each : 1), (int)p.tokens), own = from * k;
#pragma unroll SEVERAL ? 4 : 1
  for (int i = tid; i < p.entries; i += kThreads) {
    const int e = p.chosen[i];
    if ((uint32_t)e >= (uint32_t)p.experts) continue;
    atomicAdd(&total[e], 1);
    if (i < own) atomicAdd(&before[e], 1);
  }
  __syncthreads();
  const int all = scan_counts(total, p.experts, sums);
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int e = tid; e < p.experts; e += kThreads) p.offsets[e] = total[e];
    if (tid == 0) p.offsets[p.experts] = all;
  }
  for (int t = from; t < to; ++t) {
    if (tid < k) {
      const int e = p.chosen[t * k + tid];
      int at = -1;
      if ((uint32_t)e < (uint32_t)p.experts) {
        at = total[e] + before[e];
        for (int j = 0; j < tid; ++j) at += p.chosen[t * k + j] == e;
      }
      places[tid] = at;
      if (blockIdx.y == 0) p.place[t * k + tid] = at;
    }
    __syncthreads();
    copy_row<V, 1, false>(p, t, places, blockIdx.y * kThreads + tid, gridDim.y * kThreads);
    if (!SEVERAL || t + 1 == to) break;
    if (tid < k) {
      const int e = p.chosen[t * k + tid];
      if ((uint32_t)e < (uint32_t)p.experts) atomicAdd(&before[e], 1);
    }
    __syncthreads();  // (the places have been read, too)
  }
}

__global__ __launch_bounds__(kThreads) void count_chunks(const Params p) {
  __shared__ int count[kMaxExperts];
  const int tid = threadIdx.x;
  for (int e = tid; e < p.experts; e += kThreads) count[e] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * p.chunk;
  const int64_t hi = min(lo + p.chunk, (int64_t)p.entries);
  for (int64_t i = lo + tid; i < hi; i += kThreads) {
    const int e = p.chosen[i];
    if ((uint32_t)e < (uint32_t)p.experts) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < p.experts; e += kThreads)
    p.counts[(int64_t)blockIdx.x * p.experts + e] = count[e];
}

// Places of a chunk's choices, a pass at a time.  A wavefront takes a quarter of a pass, 64 at a
// time in order; next[wave][e] is the place of the next choice of e that the wavefront meets, and
// base[e] that of the pass.
__global__ __launch_bounds__(kThreads) void place_chunks(const Params p) {
  __shared__ int base[kMaxExperts], next[kWaves][kMaxExperts], sums[kWaves];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, chunk = blockIdx.x;
  constexpr int kEach = kMaxExperts / kThreads;  // experts of a thread: tid, tid + kThreads, ..
  int before[kEach];                             // their choices in chunks before
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = j * kThreads + tid;
    before[j] = 0;
    if (e >= p.experts) continue;
    int all = 0;
#pragma unroll 32
    for (int c = 0; c < p.chunks; ++c) {
      const int n = p.counts[(int64_t)c * p.experts + e];
      all += n;
      before[j] += c < chunk ? n : 0;
    }
    base[e] = all;
  }
  __syncthreads();
  const int all = scan_counts(base, p.experts, sums);
  if (chunk == 0) {
    for (int e = tid; e < p.experts; e += kThreads) p.offsets[e] = base[e];
    if (tid == 0) p.offsets[p.experts] = all;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = j * kThreads + tid;
    if (e < p.experts) base[e] += before[j];
  }
  const int bits = 32 - __builtin_clz(p.experts);  // experts, and one number for none
  const int64_t from = (int64_t)chunk * p.chunk;
  const int64_t to = min(from + p.chunk, (int64_t)p.entries);
  for (int64_t pass = from; pass < to; pass += kPass) {
    __syncthreads();  // (the pass before is done with its places)
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int e = j * kThreads + tid;
      if (e < p.experts)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) next[w][e] = 0;
    }
    __syncthreads();
    constexpr int kShare = kPass / kWaves, kRounds = kShare / 64;
    const int64_t lo = pass + wave * kShare + lane;
    int own[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      own[r] = lo + r * 64 < to ? p.chosen[lo + r * 64] : -1;
      if ((uint32_t)own[r] >= (uint32_t)p.experts) own[r] = -1;
      if (own[r] >= 0) atomicAdd(&next[wave][own[r]], 1);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int e = j * kThreads + tid;
      if (e >= p.experts) continue;
      int at = base[e];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int n = next[w][e];
        next[w][e] = at;
        at += n;
      }
      base[e] = at;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int e = own[r] >= 0 ? own[r] : p.experts;
      uint64_t peers = ~0ull;  // lanes with the same expert
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((e >> b) & 1);
        peers &= (e >> b) & 1 ? set : ~set;
      }
      int at = -1;
      if (own[r] >= 0) at = next[wave][e] + __popcll(peers & ((1ull << lane) - 1));
      // every lane has read its expert's number before the last of them moves it on
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (own[r] >= 0 && (peers >> lane) == 1) next[wave][e] = at + 1;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lo + r * 64 < to) p.place[lo + r * 64] = at;
    }
  }
}

// A wavefront a token at a time.
template <class V, bool ONCE>
__global__ __launch_bounds__(kThreads) void copy_rows(const Params p) {
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < p.tokens;
       t += (int64_t)gridDim.x * kWaves)
    copy_row<V, 4, ONCE>(p, t, p.place + t * p.top_k.d, lane, 64);
}

struct Sums {
  const char* y;
  const int32_t* place;
  const float* weights;
  const char* add;
  char* out;
  int64_t tokens, n, y_rows;
  int32_t top_k;
};

template <class T, int N, bool ONCE = false>
__device__ __forceinline__ void load_run(const char* base, int64_t at, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = (float)((const T*)base)[at];
  } else {
    // 16 bytes at a time
    constexpr int E = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(E)));
#pragma unroll
    for (int i = 0; i < N / E; ++i) {
      const vec* from = (const vec*)((const T*)base + at + i * E);
      const vec w = ONCE ? __builtin_nontemporal_load(from) : *from;
#pragma unroll
      for (int j = 0; j < E; ++j) v[i * E + j] = (float)w[j];
    }
  }
}

template <class T, int N>
__device__ __forceinline__ void store_run(char* base, int64_t at, const float (&v)[N]) {
  if constexpr (N == 1) {
    ((T*)base)[at] = (T)v[0];
  } else {
    constexpr int E = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(E)));
#pragma unroll
    for (int i = 0; i < N / E; ++i) {
      vec w;
#pragma unroll
      for (int j = 0; j < E; ++j) w[j] = (T)v[i * E + j];
      *(vec*)((T*)base + at + i * E) = w;
    }
  }
}

// A workgroup takes a token and a part of its columns; a thread N of them.  The rows of eight
// choices are asked for at once (with a branch at each, one at a time): a choice without a row
// reads row 0, and takes nothing of it.
template <class T, class O, int N, bool ONCE>
__global__ __launch_bounds__(kThreads) void combine_kernel(const Sums p) {
  constexpr int kBatch = 8;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const int32_t* place = p.place + t * p.top_k;
    const float* weights = p.weights + t * p.top_k;
    for (int64_t c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * N; c < p.n;
         c += (int64_t)gridDim.y * kThreads * N) {
      float sum[N];
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] = 0.0f;
      if (p.add) load_run<__bf16, N>(p.add, t * p.n + c, sum);
      for (int j0 = 0; j0 < p.top_k && p.y_rows > 0; j0 += kBatch) {
        float v[kBatch][N], w[kBatch];
        bool has[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int choice = min(j0 + j, p.top_k - 1), at = place[choice];
          has[j] = j0 + j < p.top_k && at >= 0 && at < p.y_rows;
          w[j] = weights[choice];
          load_run<T, N, ONCE>(p.y, (has[j] ? at : 0) * p.n + c, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i)
            sum[i] = has[j] ? __builtin_fmaf(w[j], v[j][i], sum[i]) : sum[i];
      }
      store_run<O, N>(p.out, t * p.n + c, sum);
    }
  }
}

// The launch's own error: hipGetLastError would report, and clear, what another call has left.
template <class P>
hipError_t launch(void* kernel, dim3 grid, P p, hipStream_t stream) {
  void* args[] = {&p};
  return hipLaunchKernel(kernel, grid, dim3(kThreads), args, 0, stream);
}

struct Chunks {
  int64_t count, each;
};

Chunks chunks_of(int64_t entries) {
  const int64_t passes = entries > 0 ? (entries + kPass - 1) / kPass : 1;
  const int64_t each = (passes + kMaxChunks - 1) / kMaxChunks * kPass;
  return Chunks{(entries + each - 1) / each, each};
}

}  // namespace

int64_t dispatch_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts) {
  const int64_t entries = tokens * top_k;
  return entries <= kFew ? 0 : chunks_of(entries).count * experts * 4;
}

hipError_t dispatch_launch(const DispatchArgs& a, hipStream_t stream) {
  Params p{};
  p.x = (const char*)a.x;
  p.rows = (char*)a.rows;
  p.chosen = a.chosen;
  p.offsets = a.offsets;
  p.place = a.place;
  p.counts = (int32_t*)a.workspace;
  p.hidden = a.hidden;
  p.top_k = divisor_of((uint32_t)a.top_k);
  p.entries = (int32_t)(a.tokens * a.top_k);
  p.experts = (int32_t)a.experts;
  const Chunks chunks = chunks_of(p.entries);
  p.chunks = (int32_t)chunks.count;
  p.chunk = (int32_t)chunks.each;
  p.tokens = a.tokens;
  const bool wide = a.hidden % 8 == 0 && ((uintptr_t)a.x | (uintptr_t)a.rows) % 16 == 0;
  const int64_t pieces = wide ? a.hidden / 8 : a.hidden;
  if (p.entries <= kFew) {
    // Up to four workgroups for each of the chip's 256 compute units, of a piece a thread at least.
    // (With the loop over several tokens, 64 tokens of 8 rows of 7168 take 4.9 us instead of 4.7.)
    p.each = (int32_t)std::max((a.tokens + 1023) / 1024, (int64_t)1);
    const int64_t blocks = std::max((a.tokens + p.each - 1) / p.each, (int64_t)1);
    const int64_t most = (pieces + kThreads - 1) / kThreads;
    const dim3 grid((uint32_t)blocks, (uint32_t)std::min((511 + blocks) / blocks, most));
    void* kernel = p.each > 1 ? (wide ? (void*)dispatch_few<uint4v, true>
                                      : (void*)dispatch_few<uint16_t, true>)
                              : (wide ? (void*)dispatch_few<uint4v, false>
                                      : (void*)dispatch_few<uint16_t, false>);
    return launch(kernel, grid, p, stream);
  }
  hipError_t e = launch((void*)count_chunks, p.chunks, p, stream);
  if (e == hipSuccess) e = launch((void*)place_chunks, p.chunks, p, stream);
  if (e != hipSuccess) return e;
  const int64_t blocks = (a.tokens + kWaves - 1) / kWaves;
  const uint32_t grid = (uint32_t)(blocks < (1 << 20) ? blocks : (1 << 20));
  // Rows that the last-level cache does not hold go past it: what reads them next finds most of
  // them evicted either way, and lines that are still to be written slow it down.  Dispatch and a
  // pass that reads its rows, past the caches and through them: 67 MB 42 and 37 us, 134 MB 74 and
  // 71, 268 MB 141 and 143, 1.9 GB 913 and 929; and a pass that reads other memory: 39 and 48, 74
  // and 81, 141 and 158, 915 and 929.
  const bool once = (int64_t)p.entries * a.hidden * 2 >= kLastLevel;
  void* kernel = !wide  ? (void*)copy_rows<uint16_t, false>
                 : once ? (void*)copy_rows<uint4v, true>
                        : (void*)copy_rows<uint4v, false>;
  return launch(kernel, grid, p, stream);
}

hipError_t combine_launch(const CombineArgs& a, hipStream_t stream) {
  const Sums p{(const char*)a.y, a.place, a.weights, (const char*)a.add, (char*)a.out, a.tokens,
               a.n,              a.y_rows, (int32_t)a.top_k};
  const bool wide = a.n % 8 == 0 &&
                    ((uintptr_t)a.y | (uintptr_t)a.out | (uintptr_t)a.add) % 16 == 0;
  const int64_t parts = (a.n / (wide ? 8 : 1) + kThreads - 1) / kThreads;
  const dim3 grid((uint32_t)(a.tokens < (1 << 20) ? a.tokens : (1 << 20)),
                  (uint32_t)(parts < 1 ? 1 : parts < 8 ? parts : 8));
  // Rows that take a quarter of the last-level cache or more are read past it, so that they evict
  // nothing: after the dispatch that wrote them, through the caches and past them, 67 MB 38.2 and
  // 38.8 us, 117 MB 59.7 and 54.9, 268 MB 137 and 124; after another pass 48 and 41, 71 and 63, 136
  // and 123.  7 MB, just written, 5.2 and 6.2 us.
  const bool once = a.y_rows * a.n * (a.y_fp32 ? 4 : 2) >= kLastLevel / 4;
  auto go = [&](auto t, auto o) {
    using T = decltype(t);
    using O = decltype(o);
    void* kernel = !wide  ? (void*)combine_kernel<T, O, 1, false>
                   : once ? (void*)combine_kernel<T, O, 8, true>
                          : (void*)combine_kernel<T, O, 8, false>;
    return launch(kernel, grid, p, stream);
  };
  if (a.y_fp32) return a.out_fp32 ? go(0.0f, 0.0f) : go(0.0f, __bf16{});
  return a.out_fp32 ? go(__bf16{}, 0.0f) : go(__bf16{}, __bf16{});
}

}  // namespace fp4q
