// Descriptors shared by the kernels of the norms around a block
// (norm_kernels.hip) and their host code (norm_api.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libmuon.h"
#include "validate.hpp"

namespace muon {

// A parameter of the fused norms: one value, one for each channel, or (the
// gate) one for each element.
struct NormParam {
  const void* ptr;
  int64_t ld;      // NORM_FULL: row stride, elements
  int32_t kind;    // NormKind
  int32_t half;    // bf16
};
struct NormRows {  // N x D operand; ptr null: not there
  void* ptr;
  int64_t ld;
};

struct NormArgs {
  int64_t n;
  int32_t d, dp;              // channels; the same padded to whole chunks of 8
  float eps;
  int32_t post, pre;          // whether y and out are normed
  NormRows x, y, out, hidden; // forward; x and y also backward
  NormRows dout, dhidden, dx, dy, dfull;   // backward; dfull: the gate's gradient, NORM_FULL
  NormParam post_gain, pre_gain, gate, scale;
  // sums over the tokens, one partial for each block: the wanted vectors of dp
  // channels in the order of their bits, then the two single sums
  float* part;
  int64_t part_floats;        // of one block
  int32_t want;               // bits: kWant*
  int32_t blocks;             // partials
};
// What the backward pass sums over the tokens.
constexpr int kWantBlock = 1;   // dT yhat a channel: post_gain's and the gate's gradient
constexpr int kWantScale = 2;   // dT x a channel
constexpr int kWantPre = 4;     // dhidden xhat a channel
constexpr int kWantGateOne = 8, kWantScaleOne = 16;   // sums over all channels

// Where the sums go; dt as NormParam's half of the parameter itself.
struct NormSums {
  const float* part;
  int64_t part_floats;
  int32_t blocks, d, dp, want;
  NormParam post_gain, gate;  // what the shared sum is multiplied by
  int32_t post_half, gate_half, scale_half, pre_half;
  void *dpost, *dgate, *dscale, *dpre;   // or null
};

// Floats of one block's partials.
inline int64_t norm_part_floats(int want, int dp) {
  return (int64_t)dp * (((want & kWantBlock) != 0) + ((want & kWantScale) != 0) + ((want & kWantPre) != 0)) + 4;
}

// x_half, y_half: types of x (out, dout, dx) and of y (hidden, dhidden, dy, a full gate).
hipError_t launch_residual_norm(const NormArgs& a, int x_half, int y_half, hipStream_t s);
// Blocks of the backward launch (n > 0), which leaves as many partials.
constexpr int kNormMostBlocks = 1024;
int norm_grad_blocks(const NormArgs& a, int x_half, int y_half);
hipError_t launch_residual_norm_grad(const NormArgs& a, int x_half, int y_half, hipStream_t s);
hipError_t launch_norm_sums(const NormSums& a, hipStream_t s);

}  // namespace muon
