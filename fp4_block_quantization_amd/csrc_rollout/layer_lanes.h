// layer_lanes.h -- reductions over the 64 lanes of a wavefront, without LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {

template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
}

// Data-parallel moves: neighbours, pairs, halves of 8 and of 16 mirrored.
constexpr int kSwap1 = 0xb1, kSwap2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;

// f (commutative, associative up to rounding) of all lanes' v, the same in every lane.
template <class T, class F>
__device__ __forceinline__ T over_lanes(T v, F f) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "one or two registers");
  constexpr int W = sizeof(T) / 4;
  auto step = [&](auto move) {
    uint32_t w[W], m[W];
    __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
    for (int i = 0; i < W; ++i) m[i] = move(w[i]);
    T o;
    __builtin_memcpy(&o, m, sizeof(T));
    v = f(v, o);
  };
  step([](uint32_t x) { return moved<kSwap1>(x); });
  step([](uint32_t x) { return moved<kSwap2>(x); });
  step([](uint32_t x) { return moved<kHalfMirror>(x); });
  step([](uint32_t x) { return moved<kMirror>(x); });
  auto halves = [&](auto swap) {
    uint32_t w[W], a[W], b[W];
    __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const auto r = swap(w[i]);
      a[i] = r[0];
      b[i] = r[1];
    }
    T x, y;
    __builtin_memcpy(&x, a, sizeof(T));
    __builtin_memcpy(&y, b, sizeof(T));
    v = f(x, y);
  };
  halves([](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false); });
  halves([](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false); });
  return v;
}

}  // namespace fp4q
