// layer_rotary.hip -- rotary positions (definition in include/fp4q/layer.h).
//
// Mathematics.  The angle p f is reduced in FP64 to quarter turns and a rest
// of at most an eighth of a turn either way, whose sine and cosine are their
// Taylor polynomials (degrees 9 and 10: 2e-9 off at the ends).  FP32 would lose
// the angle of far positions: 10^6 radians have 2^-4 as their last place there.  Of
// 2^22 quarter turns and more the low parts of the products are kept, too, in a
// second pass (in one for all angles, 8192 tokens of 40 heads of 128 take 0.5 us
// more, 777 of FP32 0.3).
//
// Work.  A thread owns some pairs of one token (16 bytes of a head, or two
// times 16 where the halves lie apart), computes their sines and cosines once
// and applies them to every HS-th head of the queries and keys.
//
// Bounds.  Every element is read and written once: 8192 tokens of 40 heads of
// 128 are 168 MB, 28.9 us, 5.8 TB/s, where a large copy reaches 5.3 to 6.4.
// 64 tokens take 2.9 us on the device, of which a launch that does nothing is
// 2.4.
#include <type_traits>

#include "layer_launch.h"
#include "rollout_divisor.h"

namespace fp4q {
namespace {

constexpr int kThreads = 256;
// Threads wanted, so that a token's angles serve few heads of many tokens: 8192 tokens of 40 heads
// of 128 take 42.9 us with 131072, 31.3 with twice that, 29.1, and 28.4 with this many.
constexpr int64_t kWanted = 1048576;

// Quarter turns from which angles are formed once more with the low parts of their products.  Up to
// there an angle is off by 2^-28, far behind by no small part of a turn.
constexpr double kFar = 0x1p22;

struct Params {
  const char* in[2];
  char* out[2];
  int64_t in_stride[2], out_stride[2];  // elements
  const int64_t* positions;
  const double* frequencies;
  int64_t first_token;  // of this launch
  int32_t heads[2];
  int32_t head_dim, dims;
  int32_t pair_units;  // of a head's units those that turn; the rest copies
  Divisor units;
  Divisor slots;       // threads that share a token's unit, each every slots-th head
  float amplitude;
  uint32_t threads;    // tokens * slots * units, below 2^31
};

struct Turn {
  float c, s;
};

// Sine and cosine of position * frequency; `most` takes the largest size of x so far, whose three
// roundings lose 2^-51 of it.  FAR: with the products' low parts.
template <bool FAR>
__device__ __forceinline__ Turn turn_of(double position, double frequency, double& most) {
  // 2 / pi in two words, so that x counts quarter turns
  constexpr double kFirst = 0.63661977236758134308, kSecond = -3.9357353350364971764e-17;
  auto mod4 = [](double v) { return (int)(v - 4.0 * __builtin_floor(v * 0.25)); };  // (past an int)
  const double angle = position * frequency, x = angle * kFirst, n = __builtin_rint(x);
  double rest = x - n;
  int quarter = mod4(n);
  if constexpr (FAR) {
    rest += __builtin_fma(angle, kFirst, -x) +
            (angle * kSecond + __builtin_fma(position, frequency, -angle) * kFirst);
    const double more = __builtin_rint(rest);  // (the low parts may be quarters, too)
    rest -= more;
    quarter = (quarter + mod4(more)) & 3;
  } else {
    most = __builtin_fmax(most, __builtin_fabs(x));
  }
  const float r = (float)(rest * 1.57079632679489661923);
  const float r2 = r * r;
  float s = 2.7557319223985893e-6f;  // 1 / 9!
  s = __builtin_fmaf(s, r2, -1.9841269841269841e-4f);
  s = __builtin_fmaf(s, r2, 8.3333333333333333e-3f);
  s = __builtin_fmaf(s, r2, -1.6666666666666667e-1f);
  s = __builtin_fmaf(s * r2, r, r);
  float c = -2.7557319223985888e-7f;  // -1 / 10!
  c = __builtin_fmaf(c, r2, 2.4801587301587302e-5f);
  c = __builtin_fmaf(c, r2, -1.3888888888888889e-3f);
  c = __builtin_fmaf(c, r2, 4.1666666666666667e-2f);
  c = __builtin_fmaf(c, r2, -0.5f);
  c = __builtin_fmaf(c, r2, 1.0f);
  const bool odd = quarter & 1;
  const float a = odd ? s : c, b = odd ? c : s;
  return Turn{quarter == 1 || quarter == 2 ? -a : a, quarter >= 2 ? -b : b};
}

template <class T>
struct Element;
template <>
struct Element<float> {
  static constexpr int kVec = 4;  // elements of 16 bytes
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Element<__bf16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(__bf16 v) { return (float)v; }
  static __device__ __forceinline__ __bf16 put(float v) { return (__bf16)v; }
};

// N consecutive elements (N 1: at their own alignment; else 16 bytes).
template <class T, int N>
struct Run {
  typedef T vec __attribute__((ext_vector_type(N)));
  T v[N];
  // ONCE: past the caches
  template <bool ONCE>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (N == 1) {
      v[0] = *p;
    } else {
      const vec w = ONCE ? __builtin_nontemporal_load((const vec*)p) : *(const vec*)p;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = w[i];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (N == 1) {
      *p = v[0];
    } else {
      vec w;
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = v[i];
      *(vec*)p = w;
    }
  }
};

// WIDE: units of 16 bytes (two of them where halves lie apart); else of a pair, or an element.
// ONCE: inputs are read past the caches.
template <class T, bool WIDE, bool INTERLEAVED, bool INVERSE, bool ONCE>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const Params p) {
  using E = Element<T>;
  // elements of a run, and pairs of a unit
  constexpr int N = WIDE ? E::kVec : 1;
  constexpr int PAIRS = WIDE && INTERLEAVED ? N / 2 : N;
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
  if (id >= p.threads) return;
  const uint32_t rest = quotient(id, p.units);
  const int unit = (int)(id - rest * p.units.d);
  const uint32_t nth = quotient(rest, p.slots);
  const int slot = (int)(rest - nth * p.slots.d);
  const int64_t token = p.first_token + nth;
  const int all = p.heads[0] + p.heads[1];
  const bool turns = unit < p.pair_units;
  // where the unit's runs are within a head
  const int first = !turns ? p.dims + (unit - p.pair_units) * N
                           : (INTERLEAVED ? 2 * PAIRS : N) * unit;
  const int second = INTERLEAVED ? first + 1 : first + p.dims / 2;
  float c[PAIRS], s[PAIRS];
  if (turns) {
    const double position = (double)p.positions[token];
    double most = 0.0;
    auto turn = [&](auto far) {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const Turn t = turn_of<decltype(far)::value>(position, p.frequencies[unit * PAIRS + i], most);
        c[i] = t.c * p.amplitude;
        s[i] = (INVERSE ? -t.s : t.s) * p.amplitude;
      }
    };
    turn(std::false_type{});
    if (most >= kFar) turn(std::true_type{});
  }
  for (int h = slot; h < all; h += (int)p.slots.d) {
    const int which = h >= p.heads[0];
    const int64_t at = (int64_t)(which ? h - p.heads[0] : h) * p.head_dim;
    const T* in = (const T*)p.in[which] + token * p.in_stride[which] + at;
    T* out = (T*)p.out[which] + token * p.out_stride[which] + at;
    if (!turns) {
      if (in == out) continue;
      Run<T, N> r;
      r.template load<ONCE>(in + first);
      r.store(out + first);
    } else if constexpr (WIDE && INTERLEAVED) {
      Run<T, N> r;
      r.template load<ONCE>(in + first);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const float u = E::get(r.v[2 * i]), v = E::get(r.v[2 * i + 1]);
        r.v[2 * i] = E::put(__builtin_fmaf(u, c[i], -(v * s[i])));
        r.v[2 * i + 1] = E::put(__builtin_fmaf(v, c[i], u * s[i]));
      }
      r.store(out + first);
    } else {
      Run<T, N> a, b;
      a.template load<ONCE>(in + first);
      b.template load<ONCE>(in + second);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const float u = E::get(a.v[i]), v = E::get(b.v[i]);
        a.v[i] = E::put(__builtin_fmaf(u, c[i], -(v * s[i])));
        b.v[i] = E::put(__builtin_fmaf(v, c[i], u * s[i]));
      }
      a.store(out + first);
      b.store(out + second);
    }
  }
}

template <class T, bool WIDE, bool ONCE>
void* kernel_of(bool interleaved, bool inverse) {
  if (interleaved)
    return inverse ? (void*)rotary_kernel<T, WIDE, true, true, ONCE>
                   : (void*)rotary_kernel<T, WIDE, true, false, ONCE>;
  return inverse ? (void*)rotary_kernel<T, WIDE, false, true, ONCE>
                 : (void*)rotary_kernel<T, WIDE, false, false, ONCE>;
}

template <class T>
void* kernel_of(bool wide, bool once, bool interleaved, bool inverse) {
  return !wide ? kernel_of<T, false, false>(interleaved, inverse)
         : once ? kernel_of<T, true, true>(interleaved, inverse)
                : kernel_of<T, true, false>(interleaved, inverse);
}

}  // namespace

hipError_t rotary_launch(const RotaryArgs& a, hipStream_t stream) {
  const int vec = a.fp32 ? 4 : 8;
  bool wide = a.head_dim % vec == 0 && a.dims % (a.interleaved ? vec : 2 * vec) == 0;
  Params p{};
  for (int i = 0; i < (a.heads[1] > 0 ? 2 : 1); ++i) {
    wide = wide && ((uintptr_t)a.in[i] | (uintptr_t)a.out[i]) % 16 == 0 &&
           a.in_stride[i] % vec == 0 && a.out_stride[i] % vec == 0;
    p.in[i] = (const char*)a.in[i];
    p.out[i] = (char*)a.out[i];
    p.in_stride[i] = a.in_stride[i];
    p.out_stride[i] = a.out_stride[i];
    p.heads[i] = (int32_t)a.heads[i];
  }
  p.positions = a.positions;
  p.frequencies = a.frequencies;
  p.head_dim = (int32_t)a.head_dim;
  p.dims = (int32_t)a.dims;
  p.amplitude = a.amplitude;
  p.pair_units = (int32_t)(a.dims / 2 / (wide ? (a.interleaved ? vec / 2 : vec) : 1));
  const int64_t units = p.pair_units + (a.head_dim - a.dims) / (wide ? vec : 1);
  const int64_t all = a.heads[0] + a.heads[1], each = a.tokens * units;
  const int64_t want = (kWanted + each - 1) / each, slots = want < all ? want : all;
  p.units = divisor_of((uint32_t)units);
  p.slots = divisor_of((uint32_t)slots);
  // Inputs that take a quarter of the last-level cache or more are read past it, so that they evict
  // nothing.  40 heads of 128, through the caches and past them: 8192 tokens 28.8 and 29.6 us where
  // nothing else runs, 33.5 and 28.9 between other work, 37.0 and 34.5 in place; 16384 tokens 65
  // and 54; 4096 tokens 16.5 and 17.1.
  const bool once = a.tokens * all * a.head_dim * (a.fp32 ? 4 : 2) >= (int64_t)64 << 20;
  void* kernel = a.fp32 ? kernel_of<float>(wide, once, a.interleaved, a.inverse)
                        : kernel_of<__bf16>(wide, once, a.interleaved, a.inverse);
  const int64_t step = (((int64_t)1 << 31) - kThreads) / (units * slots);  // tokens of a launch
  for (p.first_token = 0; p.first_token < a.tokens; p.first_token += step) {
    const int64_t tokens = a.tokens - p.first_token < step ? a.tokens - p.first_token : step;
    p.threads = (uint32_t)(tokens * units * slots);
    void* args[] = {&p};
    const hipError_t e = hipLaunchKernel(kernel, dim3((p.threads + kThreads - 1) / kThreads),
                                         dim3(kThreads), args, 0, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp4q
