// Exchanges between the lanes of a wave on the vector units: moves within rows
// of sixteen lanes, and swaps of rows and halves. (Through the LDS, as a shuffle,
// each step of a sum takes about 100 cycles instead of 10.)
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

typedef unsigned int lanes2_t __attribute__((ext_vector_type(2)));

constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t u = __double_as_longlong(x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// x of the even rows of sixteen (or of the low half) and of the odd ones (the
// high half), each in both rows of a pair (both halves).
__device__ __forceinline__ void rows16(float x, float& even, float& odd) {
  const lanes2_t r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  even = __uint_as_float(r[0]);
  odd = __uint_as_float(r[1]);
}
__device__ __forceinline__ void halves32(float x, float& low, float& high) {
  const lanes2_t r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  low = __uint_as_float(r[0]);
  high = __uint_as_float(r[1]);
}
__device__ __forceinline__ void rows16(double x, double& even, double& odd) {
  const uint64_t u = __double_as_longlong(x);
  const lanes2_t l = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  const lanes2_t h = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  even = __longlong_as_double((long long)((uint64_t)h[0] << 32 | l[0]));
  odd = __longlong_as_double((long long)((uint64_t)h[1] << 32 | l[1]));
}
__device__ __forceinline__ void halves32(double x, double& low, double& high) {
  const uint64_t u = __double_as_longlong(x);
  const lanes2_t l = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
  const lanes2_t h = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  low = __longlong_as_double((long long)((uint64_t)h[0] << 32 | l[0]));
  high = __longlong_as_double((long long)((uint64_t)h[1] << 32 | l[1]));
}

// f over W lanes (16 or 64, neighbours from a multiple of W), the same value in all.
template <int W, typename T, typename F>
__device__ __forceinline__ T over_lanes(T x, F f) {
  static_assert(W == 16 || W == 64, "lanes");
  x = f(x, dpp<kDppXor1>(x));
  x = f(x, dpp<kDppXor2>(x));
  x = f(x, dpp<kDppHalfMirror>(x));
  x = f(x, dpp<kDppMirror>(x));
  if constexpr (W == 64) {
    T a, b;
    rows16(x, a, b);
    x = f(a, b);
    halves32(x, a, b);
    x = f(a, b);
  }
  return x;
}
template <int W, typename T>
__device__ __forceinline__ T lanes_sum(T x) {
  return over_lanes<W>(x, [](T a, T b) { return a + b; });
}

}  // namespace muon
