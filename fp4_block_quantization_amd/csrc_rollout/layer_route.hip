// layer_route.hip -- scores of experts, the best of every token and their
// weights (definition in include/fp4q/layer.h).
//
// Mathematics.  A key becomes an unsigned integer in the keys' order.  Without
// a bias the scores' order is the logits', and 32 bits hold it exactly.  A
// bias makes the order depend on roundings of the scores: keys are FP64 then,
// of which 42 bits behind the leading one are compared, so that two experts
// change places only where their keys agree to 2^-42; the expert's number,
// turned round, stands in the bits below, so that the largest is the best
// expert, the lowest of equal ones.  Groups' marks are sums of two FP64
// numbers for the same reason.
// Weights decide nothing and are formed in FP32: they are off by 6e-8 of their
// size, 3e-8 of it their own rounding.
//
// Work.  One wavefront takes a token; a lane holds the experts lane, lane +
// 64, and so on.  The best are taken one at a time: a maximum over the lane's
// own and one over the lanes (data-parallel moves, no LDS).  Of 32-bit keys
// the expert is found from ballots: with the number in 64 bits as well, 8192
// tokens of 128 experts take 6.9 us instead of 6.5.  64-bit keys are sorted in
// each lane first, and of its best the upper half goes over the lanes; with
// both halves of the lane's largest, 8192 tokens of 256 experts with a bias and
// groups take 16.1 us instead of 13.5, 64 of them 6.0 instead of 5.8, and 8192
// of 1024 with a bias 34 instead of 31 (22 instead of 26 for the one best).
//
// Bounds.  The chain of these steps, of which each of the best waits for the
// one before: 64 tokens of 256 experts take 3.5 us on the device for 8 of
// them, 2.4 for one (a launch that does nothing is about 2), 4.7 with a bias,
// 5.8 with groups as well; 8192 tokens of 128 experts 6.6 us, of 4.7 MB.
#include "layer_lanes.h"
#include "layer_launch.h"
#include "rollout_divisor.h"

namespace fp4q {
namespace {

constexpr int kWaves = 4;

struct Params {
  const void* logits;
  const float* bias;
  const uint8_t* active;
  float* weights;
  int32_t* chosen;
  int64_t tokens;
  int32_t experts, top_k, groups, top_groups;
  Divisor per_group;
  float scale;
};

constexpr uint32_t kNumbers = 1024;  // of experts

// Ordered integers: NaN comes first.  0 stands for an expert that is not there, or not any more.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // (-0 counts as 0)
  const uint32_t o = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return x != x ? 1u : o;
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  const uint64_t o = u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
  return x != x ? kNumbers : o & ~(uint64_t)(kNumbers - 1);
}

template <class K>
__device__ __forceinline__ K larger(K a, K b) {
  return a > b ? a : b;
}

// Takes the best out of the keys; its expert.
template <int S>
__device__ __forceinline__ int take_best(uint32_t (&key)[S], int lane) {
  uint32_t top = key[0];
#pragma unroll
  for (int j = 1; j < S; ++j) top = larger(key[j], top);
  top = over_lanes(top, larger<uint32_t>);
  int expert = 0;
#pragma unroll
  for (int j = S - 1; j >= 0; --j) {
    const uint64_t with = __ballot(key[j] == top);
    expert = with != 0 ? j * 64 + __builtin_ctzll(with) : expert;
  }
#pragma unroll
  for (int j = 0; j < S; ++j) key[j] = j * 64 + lane == expert ? 0 : key[j];
  return expert;
}
// A lane's keys into falling order (Batcher's network of merges).
template <int S>
__device__ __forceinline__ void sort_lane(uint64_t (&key)[S]) {
#pragma unroll
  for (int p = 1; p < S; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int i = 0; i + k < S; ++i) {
        if (i < k % p || (i - k % p) / k % 2 != 0 || i / (2 * p) != (i + k) / (2 * p)) continue;
        const uint64_t a = key[i], b = key[i + k];
        key[i] = b > a ? b : a;
        key[i + k] = b > a ? a : b;
      }
}

// Takes the best out of sorted 64-bit keys.  The lower halves are looked at only where lanes'
// upper ones are equal.
template <int S>
__device__ __forceinline__ int take_best(uint64_t (&key)[S], int) {
  const uint32_t high = (uint32_t)(key[0] >> 32), low = (uint32_t)key[0];
  const uint32_t top = over_lanes(high, larger<uint32_t>);
  bool best = high == top;
  uint64_t with = __ballot(best);
  if (with & (with - 1)) {
    const uint32_t most = over_lanes(best ? low : 0, larger<uint32_t>);
    best = best && low == most;
    with = __ballot(best);
  }
#pragma unroll
  for (int j = 0; j < S; ++j) key[j] = !best ? key[j] : j + 1 < S ? key[j + 1] : 0;
  const uint32_t number = __builtin_amdgcn_readlane((int)low, __builtin_ctzll(with));
  return (int)(kNumbers - 1 - (number & (kNumbers - 1)));
}

// The two largest of some numbers.
struct Two {
  double first, second;
  __device__ __forceinline__ void take(double v) {
    const bool up = v > first;
    second = up ? first : (v > second ? v : second);
    first = up ? v : first;
  }
};

// Over groups of `share` neighbouring lanes, a power of two.
__device__ __forceinline__ Two over_share(Two t, int share) {
  auto step = [&](auto move) {
    uint32_t w[4], m[4];
    __builtin_memcpy(w, &t, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = move(w[i]);
    Two o;
    __builtin_memcpy(&o, m, 16);
    t.take(o.first);
    t.take(o.second);
  };
  // (in each step both sides' lanes hold the same two already)
  if (share > 1) step([](uint32_t x) { return moved<kSwap1>(x); });
  if (share > 2) step([](uint32_t x) { return moved<kSwap2>(x); });
  if (share > 4) step([](uint32_t x) { return moved<kHalfMirror>(x); });
  if (share > 8) step([](uint32_t x) { return moved<kMirror>(x); });
  for (int s = 16; s < share; s *= 2)
    step([&](uint32_t x) { return (uint32_t)__shfl_xor((int)x, s); });
  return t;
}

__device__ __forceinline__ uint64_t lane_value(uint64_t v, int from) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, from);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), from);
  return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ void own_lds_done() {  // a wavefront's LDS accesses are in order
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// S: experts of a lane.  WIDE: keys in FP64 (a bias, or groups).
template <class T, int S, bool WIDE>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const Params p, const bool sigmoid,
                                                            const bool renormalize) {
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t token = (int64_t)blockIdx.x * kWaves + wave;
  if (token >= p.tokens) return;
  const int64_t at = token * p.top_k;
  if (p.active && p.active[token] == 0) {
    if (lane < p.top_k) {
      p.weights[at + lane] = 0.0f;
      p.chosen[at + lane] = -1;
    }
    return;
  }
  float x[S];
  typename std::conditional<WIDE, uint64_t, uint32_t>::type key[S];
  const T* row = (const T*)p.logits + token * p.experts;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int e = j * 64 + lane;
    x[j] = e < p.experts ? (float)row[e] : -INFINITY;
  }
  float top = x[0];
#pragma unroll
  for (int j = 1; j < S; ++j) top = __builtin_fmaxf(top, x[j]);
  top = over_lanes(top, [](float a, float b) { return __builtin_fmaxf(a, b); });
  if constexpr (WIDE) {
    double score[S];
    if (sigmoid) {
#pragma unroll
      for (int j = 0; j < S; ++j) score[j] = 1.0 / (1.0 + exp(-(double)x[j]));
    } else {
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < S; ++j) {
        // (a row of -infinity only has no scores: zeros)
        score[j] = top == -INFINITY ? 0.0 : exp((double)x[j] - (double)top);
        sum += score[j];
      }
      sum = over_lanes(sum, [](double a, double b) { return a + b; });
      const double each = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
      for (int j = 0; j < S; ++j) score[j] *= each;
    }
    double mark[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int e = j * 64 + lane;
      if (p.bias) {
        mark[j] = score[j] + (double)p.bias[e < p.experts ? e : 0];
        key[j] = ordered(mark[j]);
      } else {
        mark[j] = score[j];
        key[j] = (uint64_t)ordered(x[j]) << 32;
      }
    }
    if (p.groups > 1) {
      __shared__ double marks[kWaves][S * 64];
#pragma unroll
      for (int j = 0; j < S; ++j) marks[wave][j * 64 + lane] = mark[j];
      own_lds_done();
      // `share` lanes a group, a power of two
      int share = 64;
      while (share * p.groups > 64) share /= 2;
      const int g = lane / share;
      Two two{-INFINITY, -INFINITY};
      if (g < p.groups)
        for (int i = lane % share; i < (int)p.per_group.d; i += share)
          two.take(marks[wave][g * (int)p.per_group.d + i]);
      two = over_share(two, share);
      // (groups of one expert have no second)
      const double sum = p.per_group.d > 1 ? two.first + two.second : two.first;
      const uint64_t own = g < p.groups ? ordered(sum) : 0;
      int ahead = 0;  // groups that come before this lane's
      for (int i = 0; i < p.groups; ++i) {
        const uint64_t other = lane_value(own, i * share);
        ahead += other > own || (other == own && i < g);
      }
      const uint64_t open = __ballot(ahead < p.top_groups && g < p.groups);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const uint32_t of = quotient(min(j * 64 + lane, p.experts - 1), p.per_group);
        if (!(open >> (of * share) & 1)) key[j] = 0;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < S; ++j) key[j] = ordered(x[j]);
  }
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const uint32_t e = j * 64 + lane;
    if ((int)e >= p.experts || key[j] == 0)
      key[j] = 0;
    else if constexpr (WIDE)
      key[j] |= kNumbers - 1 - e;
  }
  if constexpr (WIDE) sort_lane(key);
  __shared__ float all[kWaves][S * 64];
#pragma unroll
  for (int j = 0; j < S; ++j) all[wave][j * 64 + lane] = x[j];
  own_lds_done();
  int expert = 0;  // the lane-th choice
  for (int i = 0; i < p.top_k; ++i) {
    const int best = take_best<S>(key, lane);
    expert = lane == i ? best : expert;
  }
  const float logit = lane < p.top_k ? all[wave][expert] : 0.0f;
  float w = 0.0f;
  auto add = [](float a, float b) { return a + b; };
  auto most = [](float a, float b) { return __builtin_fmaxf(a, b); };
  if (sigmoid) {
    // e^min(x, 0) / (1 + e^-|x|), which no exponential overflows in; to be renormalized, where every
    // chosen logit is below zero, relative to the largest numerator, or all might underflow
    const float e = expf(-__builtin_fabsf(logit));
    float part = logit < 0.0f ? e : 1.0f;
    if (renormalize && !__any(lane < p.top_k && logit >= 0.0f)) {
      const float base = over_lanes(lane < p.top_k ? logit : -INFINITY, most);
      part = base == -INFINITY ? 0.0f : expf(logit - base);
    }
    if (lane < p.top_k) w = part / (1.0f + e);
    if (renormalize) {
      const float sum = over_lanes(w, add);
      w = sum == 0.0f ? 0.0f : w / sum;
    }
  } else if (renormalize) {
    // relative to the largest chosen: what the others add to the sum cancels
    const float base = over_lanes(lane < p.top_k ? logit : -INFINITY, most);
    if (lane < p.top_k && base != -INFINITY) w = expf(logit - base);
    const float sum = over_lanes(w, add);
    w = sum == 0.0f ? 0.0f : w / sum;
  } else {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < S; ++j) sum += top == -INFINITY ? 0.0f : expf(x[j] - top);
    sum = over_lanes(sum, add);
    if (lane < p.top_k && top != -INFINITY) w = expf(logit - top) / sum;
  }
  if (lane < p.top_k) {
    p.weights[at + lane] = w * p.scale;
    p.chosen[at + lane] = expert;
  }
}

template <class T, bool WIDE>
void* kernel_of(int64_t experts) {
  const int64_t s = (experts + 63) / 64;
  if (s <= 1) return (void*)route_kernel<T, 1, WIDE>;
  if (s <= 2) return (void*)route_kernel<T, 2, WIDE>;
  if (s <= 4) return (void*)route_kernel<T, 4, WIDE>;
  if (s <= 8) return (void*)route_kernel<T, 8, WIDE>;
  return (void*)route_kernel<T, 16, WIDE>;
}

}  // namespace

hipError_t route_launch(const RouteArgs& a, hipStream_t stream) {
  Params p{a.logits, a.bias, a.active, a.weights, a.chosen, a.tokens, (int32_t)a.experts,
           (int32_t)a.top_k, (int32_t)a.groups, (int32_t)a.top_groups,
           divisor_of((uint32_t)(a.experts / a.groups)), a.scale};
  const bool wide = a.bias || a.groups > 1;
  void* kernel = a.fp32 ? (wide ? kernel_of<float, true>(a.experts)
                                : kernel_of<float, false>(a.experts))
                        : (wide ? kernel_of<__bf16, true>(a.experts)
                                : kernel_of<__bf16, false>(a.experts));
  bool sigmoid = a.sigmoid, renormalize = a.renormalize;
  // (a launch holds 2^32 threads)
  const int64_t step = (int64_t)kWaves << 23;
  for (int64_t first = 0; first < a.tokens; first += step) {
    p.tokens = a.tokens - first < step ? a.tokens - first : step;
    void* args[] = {&p, &sigmoid, &renormalize};
    const hipError_t e = hipLaunchKernel(kernel, dim3((uint32_t)((p.tokens + kWaves - 1) / kWaves)),
                                         dim3(64 * kWaves), args, 0, stream);
    if (e != hipSuccess) return e;
    p.logits = (const char*)p.logits + p.tokens * p.experts * (a.fp32 ? 4 : 2);
    if (p.active) p.active += p.tokens;
    p.weights += p.tokens * p.top_k;
    p.chosen += p.tokens * p.top_k;
  }
  return hipSuccess;
}

}  // namespace fp4q
