// Device helpers shared by the head's kernels (head_kernels.hip, head_gemm.hip).
#pragma once
#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "train.hpp"

namespace muon {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kNoExp = -256.f;    // an exponent, base 2, whose power of 2 is 0 in 32 bits

__device__ __forceinline__ float bf2f(u16 h) { return __uint_as_float((unsigned int)h << 16); }
// Two values rounded to nearest even (the hardware's packed conversion).
__device__ __forceinline__ unsigned int pack_bf16(float lo, float hi) {
  const bf16x2_t q = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(unsigned int, q);
}
__device__ __forceinline__ u16 f2bf(float f) { return (u16)pack_bf16(f, 0.f); }

// Lowest reference of a tile's logits: finite, so that a tile of logits at
// -infinity has exponentials of 0.
constexpr float kRefFloor = -FLT_MAX;

__device__ __forceinline__ int64_t target_at(const void* targets, int bytes, int64_t i) {
  return bytes == 8 ? ((const int64_t*)targets)[i] : (int64_t)((const int32_t*)targets)[i];
}
// A target as the products take it, -1 outside the vocabulary.
__device__ __forceinline__ int checked_target(const HeadArgs& a, int64_t g) { return g >= 0 && g < a.v ? (int)g : -1; }

// Valid tokens of the piece.
__device__ __forceinline__ int piece_rows(const HeadArgs& a) { return min(max(a.count[0] - a.row0, 0), a.piece); }

// What every token's gradient is multiplied by. It is applied to the 32-bit
// sums, not to the logits' gradient before its rounding: 1 / n has one and the
// same rounding error for all tokens, which no sum would average out, while
// p - 1 of a word the model did not expect is nearly exact.
__device__ __forceinline__ float common_factor(const HeadArgs& a) {
  if (a.per_token) return 1.f;
  const float g = a.grad_out ? a.grad_out[0] : 1.f;
  return a.mean ? g / (float)max(a.count[0], 1) : g;
}

// One block: the reduced loss, the tokens' losses added in a fixed order in 64
// bits. sh: one value per wave.
template <int THREADS>
__device__ __forceinline__ void total_loss(const HeadArgs& a, double* sh) {
  const int n = a.count[0];
  double x = 0;
  for (int i = threadIdx.x; i < n; i += THREADS) x += a.lossc[i];
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0;
    for (int i = 0; i < THREADS / 64; ++i) s += sh[i];
    a.loss[0] = (float)(a.mean ? (n ? s / n : 0.0) : s);
  }
}

}  // namespace muon
