// Norms after and before a block, fused with the block's gate and the
// residual's scale, and their gradient. For a token's rows x and y:
//
//   n      = yhat post_gain, yhat = y r1, r1 = 1 / sqrt(mean y^2 + eps)   (or n = y)
//   out    = scale x + gate n
//   hidden = xhat pre_gain, xhat = out r2, r2 = 1 / sqrt(mean out^2 + eps)
//
//   dT     = dout + r2 (u - xhat mean(u xhat)),  u = dhidden pre_gain
//   dx     = scale dT,  dy = r1 (v - yhat mean(v yhat)),  v = gate dT post_gain   (or v = gate dT)
//   dpre_gain = sum dhidden xhat,  dscale = sum dT x,  S = sum dT yhat:  dpost_gain = gate S,  dgate = post_gain S
//
// Everything between the loads and the stores is 32-bit, hidden is taken from
// out before its rounding, and the backward pass makes out again from x and y,
// which it reads anyway: it saves nothing, and out's rounding is in no gradient.
// Bound by HBM: each row is read once and held in registers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "head_device.hpp"
#include "norm.hpp"
#include "wave.hpp"

namespace muon {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// Eight channels from c of a row of d as they are in memory, zero past its end;
// one or two loads where whole, aligned or not.
template <typename T>
struct Raw {
  u32x4_t q[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load_raw(const T* row, int c, int d, Raw<T>& v) {
  if (c + 8 <= d) {
    __builtin_memcpy(&v, row + c, 8 * sizeof(T));
  } else {
    T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c + e < d ? row[c + e] : T(0);
    __builtin_memcpy(&v, x, 8 * sizeof(T));
  }
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(r.q[0][e] << 16);
      v[2 * e + 1] = __uint_as_float(r.q[0][e] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r.q[e >> 2][e & 3]);
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int d, float (&v)[8]) {
  Raw<T> r;
  load_raw(row, c, d, r);
  unpack(r, v);
}
template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int d, const float (&v)[8]) {
  if (c + 8 <= d) {
    if constexpr (sizeof(T) == 2) {
      const u32x4_t q = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
      __builtin_memcpy(row + c, &q, 16);
    } else {
      __builtin_memcpy(row + c, v, 32);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < d) {
        if constexpr (sizeof(T) == 2) row[c + e] = f2bf(v[e]);
        else row[c + e] = v[e];
      }
  }
}

__device__ __forceinline__ float one_value(const NormParam& p, int64_t i) {
  return p.half ? bf2f(((const u16*)p.ptr)[i]) : ((const float*)p.ptr)[i];
}
// A parameter's eight channels (1 where it is not there; NORM_FULL is the rows').
__device__ __forceinline__ void load_param(const NormParam& p, int c, int d, float (&v)[8]) {
  if (p.kind == NORM_CHANNELS) {
    if (p.half) load8((const u16*)p.ptr, c, d, v);
    else load8((const float*)p.ptr, c, d, v);
  } else {
    const float x = p.kind == NORM_ONE ? one_value(p, 0) : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x;
  }
}

// Sums over the TPR threads of a row, the same value in all of them. Rows of
// several waves meet in LDS (sh: K places for each wave of the block); each sum of
// a row has its own place there.
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* sh) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lanes_sum<TPR < 64 ? TPR : 64>(v[k]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6, first = wave / W * W;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) sh[wave * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[k] += sh[(first + w) * K + k];
    }
  }
}

// A row's operands, loaded together and one row ahead of their use.
template <typename TX, typename TY, int NC>
struct ForwardRow {
  Raw<TX> x[NC];
  Raw<TY> y[NC], g[NC];
  template <int TPR>
  __device__ __forceinline__ void load(const NormArgs& a, int64_t r, int t) {
#pragma unroll
    for (int k = 0; k < NC; ++k) load_raw((const TX*)a.x.ptr + r * a.x.ld, 8 * (k * TPR + t), a.d, x[k]);
    if (a.y.ptr)
#pragma unroll
      for (int k = 0; k < NC; ++k) load_raw((const TY*)a.y.ptr + r * a.y.ld, 8 * (k * TPR + t), a.d, y[k]);
    if (a.gate.kind == NORM_FULL)
#pragma unroll
      for (int k = 0; k < NC; ++k) load_raw((const TY*)a.gate.ptr + r * a.gate.ld, 8 * (k * TPR + t), a.d, g[k]);
  }
};

// TPR threads to a row, NC chunks of eight channels to a thread; the threads past
// TPR of a block have other rows.
template <typename TX, typename TY, int TPR, int NC, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_residual_norm(NormArgs a) {
  constexpr int ROWS = BLOCK / TPR;
  constexpr bool AHEAD = NC == 1 || TPR <= 64;      // (the registers hold no second row otherwise)
  __shared__ float sh[2][BLOCK / 64];
  const int t = threadIdx.x % TPR, d = a.d;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  // (every thread of a block goes round as often; rows past the last one are
  // the last one again and are not stored)
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  ForwardRow<TX, TY, NC> next;
  if (AHEAD) next.template load<TPR>(a, min(row, a.n - 1), t);
  const bool there = a.y.ptr != nullptr;
  float gate[NC][8], pre[NC][8], scale[NC][8];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = 8 * (k * TPR + t);
    float post[8];
    load_param(a.scale, c, d, scale[k]);
    load_param(a.pre_gain, c, d, pre[k]);
    load_param(a.post_gain, c, d, post);
    load_param(a.gate, c, d, gate[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) gate[k][e] *= post[e];
  }
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.n; r0 += step, row += step) {
    const bool real = row < a.n;
    ForwardRow<TX, TY, NC> now;
    if (AHEAD) {
      now = next;
      if (r0 + step < a.n) next.template load<TPR>(a, min(row + step, a.n - 1), t);
    } else {
      now.template load<TPR>(a, min(row, a.n - 1), t);
    }
    float x[NC][8], s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      unpack(now.x[k], x[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] *= scale[k][e];
    }
    if (there) {
      float y[NC][8], r1 = 1.f;
#pragma unroll
      for (int k = 0; k < NC; ++k) unpack(now.y[k], y[k]);
      if (a.post) {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = fmaf(y[k][e], y[k][e], s[0]);
        row_sums<TPR>(s, sh[0]);
        r1 = 1.f / sqrtf(s[0] / d + a.eps);
      }
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        if (a.gate.kind == NORM_FULL) {
          float g[8];
          unpack(now.g[k], g);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[k][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = fmaf(y[k][e] * r1, gate[k][e], x[k][e]);
      }
    }
    if (a.out.ptr && real)
#pragma unroll
      for (int k = 0; k < NC; ++k) store8((TX*)a.out.ptr + row * a.out.ld, 8 * (k * TPR + t), d, x[k]);
    if (a.pre) {
      s[0] = 0.f;
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(x[k][e], x[k][e], s[0]);
      row_sums<TPR>(s, sh[1]);
      const float r2 = 1.f / sqrtf(s[0] / d + a.eps);
      if (real)
#pragma unroll
        for (int k = 0; k < NC; ++k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] *= r2 * pre[k][e];
          store8((TY*)a.hidden.ptr + row * a.hidden.ld, 8 * (k * TPR + t), d, x[k]);
        }
    }
    if (TPR > 64 && r0 + step < a.n) __syncthreads();   // the sums are read before the next row's are written
  }
}

template <typename TX, typename TY, int NC, bool GENERAL>
struct BackwardRow {
  Raw<TX> x[NC], dout[NC];
  Raw<TY> y[NC], g[GENERAL ? NC : 1], dhidden[NC];
  template <int TPR>
  __device__ __forceinline__ void load(const NormArgs& a, int64_t r, int t) {
#pragma unroll
    for (int k = 0; k < NC; ++k) load_raw((const TX*)a.x.ptr + r * a.x.ld, 8 * (k * TPR + t), a.d, x[k]);
    if (a.y.ptr)
#pragma unroll
      for (int k = 0; k < NC; ++k) load_raw((const TY*)a.y.ptr + r * a.y.ld, 8 * (k * TPR + t), a.d, y[k]);
    if (a.dhidden.ptr)
#pragma unroll
      for (int k = 0; k < NC; ++k) load_raw((const TY*)a.dhidden.ptr + r * a.dhidden.ld, 8 * (k * TPR + t), a.d, dhidden[k]);
    if (a.dout.ptr)
#pragma unroll
      for (int k = 0; k < NC; ++k) load_raw((const TX*)a.dout.ptr + r * a.dout.ld, 8 * (k * TPR + t), a.d, dout[k]);
    if (GENERAL && a.gate.kind == NORM_FULL)
#pragma unroll
      for (int k = 0; k < NC; ++k) load_raw((const TY*)a.gate.ptr + r * a.gate.ld, 8 * (k * TPR + t), a.d, g[k]);
  }
};

// GENERAL: with a gate for each element, or a scale for each channel.
template <typename TX, typename TY, int TPR, int NC, int BLOCK, bool GENERAL>
__global__ __launch_bounds__(BLOCK) void k_residual_norm_grad(NormArgs a) {
  constexpr int ROWS = BLOCK / TPR;
  // what the registers hold: a second row, and the parameters (read again for
  // each row otherwise)
  constexpr bool WIDE = TPR == 1024, AHEAD = !WIDE && !(GENERAL && NC > 1);
  __shared__ float sh[4][2 * (BLOCK / 64)];
  __shared__ __attribute__((aligned(16))) float joined[ROWS > 1 ? BLOCK * 8 : 8];
  const int t = threadIdx.x % TPR, d = a.d;
  const bool there = a.y.ptr != nullptr, full = GENERAL && a.gate.kind == NORM_FULL, normed = a.dhidden.ptr != nullptr;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  BackwardRow<TX, TY, NC, GENERAL> next;
  if (AHEAD) next.template load<TPR>(a, min(row, a.n - 1), t);
  // gate and post_gain multiplied (post_gain alone where the gate is full)
  auto load_gated = [&](int k, float (&v)[8]) {
    const int c = 8 * (k * TPR + t);
    float post[8];
    load_param(a.post_gain, c, d, post);
    load_param(a.gate, c, d, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= post[e];
  };
  float scale[GENERAL ? NC : 1][8], gated[WIDE ? 1 : NC][8], pre[WIDE ? 1 : NC][8];
  const float scale1 = a.scale.kind == NORM_ONE ? one_value(a.scale, 0) : 1.f;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    if (GENERAL) load_param(a.scale, 8 * (k * TPR + t), d, scale[GENERAL ? k : 0]);
    if (!WIDE) {
      load_param(a.pre_gain, 8 * (k * TPR + t), d, pre[WIDE ? 0 : k]);
      load_gated(k, gated[WIDE ? 0 : k]);
    }
  }
  // (row by row in wide rows)
  auto gated_of = [&](int k) -> float (&)[8] {
    if (WIDE) load_gated(k, gated[0]);
    return gated[WIDE ? 0 : k];
  };
  auto pre_of = [&](int k) -> float (&)[8] {
    if (WIDE) load_param(a.pre_gain, 8 * (k * TPR + t), d, pre[0]);
    return pre[WIDE ? 0 : k];
  };
  auto scale_of = [&](int k, int e) { return GENERAL ? scale[GENERAL ? k : 0][e] : scale1; };
  float sum_block[NC][8], sum_scale[GENERAL ? NC : 1][8], sum_pre[NC][8], gate_one = 0.f, scale_one = 0.f;
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum_block[k][e] = sum_scale[GENERAL ? k : 0][e] = sum_pre[k][e] = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.n; r0 += step, row += step) {
    const bool real = row < a.n;
    BackwardRow<TX, TY, NC, GENERAL> now;
    if (AHEAD) {
      now = next;
      if (r0 + step < a.n) next.template load<TPR>(a, min(row + step, a.n - 1), t);
    } else {
      now.template load<TPR>(a, min(row, a.n - 1), t);
    }
    // y becomes yhat, o the row's out
    float y[NC][8], o[NC][8], r1 = 1.f, s[2] = {0.f, 0.f};
    if (there) {
      float q[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        unpack(now.y[k], y[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[0] = fmaf(y[k][e], y[k][e], q[0]);
      }
      if (a.post) {
        row_sums<TPR>(q, sh[0]);
        r1 = 1.f / sqrtf(q[0] / d + a.eps);
      }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      unpack(now.x[k], o[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[k][e] *= scale_of(k, e);
      if (there) {
        float g[8];
        if (full) unpack(now.g[GENERAL ? k : 0], g);
        const float (&w)[8] = gated_of(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[k][e] *= r1;
          o[k][e] = fmaf(full ? w[e] * g[e] : w[e], y[k][e], o[k][e]);
        }
      }
    }
    float r2 = 0.f, m = 0.f;
    if (normed) {
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        float u[8];
        unpack(now.dhidden[k], u);
        const float (&w)[8] = pre_of(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] = fmaf(o[k][e], o[k][e], s[0]);
          s[1] = fmaf(o[k][e], u[e] * w[e], s[1]);
        }
      }
      row_sums<TPR>(s, sh[1]);
      r2 = 1.f / sqrtf(s[0] / d + a.eps);
      m = s[1] * r2 / d;
    }
    // o becomes dT, then what comes to yhat
    float v[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (k * TPR + t);
      float dt[8], x[8];
      if (a.dout.ptr) {
        unpack(now.dout[k], dt);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dt[e] = 0.f;
      }
      if (normed) {
        float u[8];
        unpack(now.dhidden[k], u);
        const float (&w)[8] = pre_of(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = o[k][e] * r2;
          dt[e] += r2 * (u[e] * w[e] - xh * m);
          if (real) sum_pre[k][e] = fmaf(u[e], xh, sum_pre[k][e]);
        }
      }
      if (a.dx.ptr && real) {
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = dt[e] * scale_of(k, e);
        store8((TX*)a.dx.ptr + row * a.dx.ld, c, d, q);
      }
      if ((a.want & (kWantScale | kWantScaleOne)) && real) {
        unpack(now.x[k], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (GENERAL && (a.want & kWantScale)) sum_scale[GENERAL ? k : 0][e] = fmaf(dt[e], x[e], sum_scale[GENERAL ? k : 0][e]);
          else scale_one = fmaf(dt[e], x[e], scale_one);
        }
      }
      if (there) {
        float g[8];
        if (full) unpack(now.g[GENERAL ? k : 0], g);
        const float (&w)[8] = gated_of(k);
        if (full && a.dfull.ptr && real) {
          float q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = dt[e] * w[e] * y[k][e];
          store8((TY*)a.dfull.ptr + row * a.dfull.ld, c, d, q);
        }
        if ((a.want & kWantBlock) && real)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum_block[k][e] = fmaf(full ? dt[e] * g[e] : dt[e], y[k][e], sum_block[k][e]);
        if ((a.want & kWantGateOne) && real) {
          float post[8];
          load_param(a.post_gain, c, d, post);
#pragma unroll
          for (int e = 0; e < 8; ++e) gate_one = fmaf(dt[e] * post[e], y[k][e], gate_one);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[k][e] = dt[e] * (full ? w[e] * g[e] : w[e]);
          v[0] = fmaf(o[k][e], y[k][e], v[0]);
        }
      }
    }
    if (there && a.dy.ptr) {
      float back = 0.f;
      if (a.post) {
        row_sums<TPR>(v, sh[2]);
        back = v[0] / d;
      }
      if (real)
#pragma unroll
        for (int k = 0; k < NC; ++k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[k][e] = r1 * (o[k][e] - y[k][e] * back);
          store8((TY*)a.dy.ptr + row * a.dy.ld, 8 * (k * TPR + t), d, o[k]);
        }
    }
    if (TPR > 64) __syncthreads();   // the sums are read before the next row's are written
  }
  // the block's partials: rows' sums joined in order
  float* part = a.part + blockIdx.x * a.part_floats;
  auto leave = [&](auto& sum) {
#pragma unroll
    for (int k = 0; k < (int)(sizeof(sum) / 32); ++k) {
      const int c = 8 * (k * TPR + t);
      if constexpr (ROWS > 1) {
        // (threads of neighbouring channels next to one another: no bank is asked twice)
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) joined[e * BLOCK + threadIdx.x] = sum[k][e];
        __syncthreads();
        for (int i = threadIdx.x; i < TPR * 8; i += BLOCK) {
          float x = 0.f;
#pragma unroll
          for (int q = 0; q < ROWS; ++q) x += joined[i / TPR * BLOCK + q * TPR + i % TPR];
          const int at = 8 * (k * TPR + i % TPR) + i / TPR;
          if (at < a.dp) part[at] = x;
        }
      } else if (c < a.dp) {
        *(f32x4_t*)(part + c) = (f32x4_t){sum[k][0], sum[k][1], sum[k][2], sum[k][3]};
        *(f32x4_t*)(part + c + 4) = (f32x4_t){sum[k][4], sum[k][5], sum[k][6], sum[k][7]};
      }
    }
    part += a.dp;
  };
  if (a.want & kWantBlock) leave(sum_block);
  if (GENERAL && (a.want & kWantScale)) leave(sum_scale);
  if (a.want & kWantPre) leave(sum_pre);
  if (a.want & (kWantGateOne | kWantScaleOne)) {
    gate_one = lanes_sum<64>(gate_one);
    scale_one = lanes_sum<64>(scale_one);
    if ((threadIdx.x & 63) == 0) {
      sh[3][(threadIdx.x >> 6) * 2] = gate_one;
      sh[3][(threadIdx.x >> 6) * 2 + 1] = scale_one;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      float x = 0.f;
      for (int w = 0; w < BLOCK / 64; ++w) x += sh[3][w * 2 + threadIdx.x];
      part[threadIdx.x] = x;
    }
  }
}

// Sums of the blocks' partials in a fixed order: 32 channels of one vector to a
// block, 32 threads to a channel; the last column of blocks has the single values.
__global__ __launch_bounds__(1024) void k_norm_sums(NormSums a) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  auto put = [&](void* p, int half, int64_t i, float x) {
    if (half) ((u16*)p)[i] = f2bf(x);
    else ((float*)p)[i] = x;
  };
  auto factor = [&](const NormParam& p) {
    return p.kind == NORM_CHANNELS ? one_value(p, c) : p.kind == NORM_ONE ? one_value(p, 0) : 1.f;
  };
  // which of the wanted vectors, in the order of their bits
  int bit = 0, left = blockIdx.y;
  for (bit = kWantBlock; bit <= kWantPre; bit *= 2)
    if ((a.want & bit) && left-- == 0) break;
  if (bit <= kWantPre) {
    float x = 0.f;
    if (c < a.d) {
      const float* p = a.part + (int64_t)blockIdx.y * a.dp + c;
#pragma unroll 8
      for (int b = share; b < a.blocks; b += 32) x += p[b * a.part_floats];
    }
    sh[share][lane] = x;
    __syncthreads();
    if (share != 0 || c >= a.d) return;
    x = 0.f;
#pragma unroll
    for (int q = 0; q < 32; ++q) x += sh[q][lane];
    if (bit == kWantBlock) {
      if (a.dpost) put(a.dpost, a.post_half, c, x * factor(a.gate));
      if (a.dgate && a.gate.kind == NORM_CHANNELS) put(a.dgate, a.gate_half, c, x * factor(a.post_gain));
    } else if (bit == kWantScale) {
      put(a.dscale, a.scale_half, c, x);
    } else {
      put(a.dpre, a.pre_half, c, x);
    }
  } else if (blockIdx.x == 0 && threadIdx.x < 64) {
    double x = 0, y = 0;
    for (int b = threadIdx.x; b < a.blocks; b += 64) {
      const float* p = a.part + b * a.part_floats + (int64_t)blockIdx.y * a.dp;
      x += p[0];
      y += p[1];
    }
    x = lanes_sum<64>(x);
    y = lanes_sum<64>(y);
    if (threadIdx.x == 0) {
      if (a.want & kWantGateOne) put(a.dgate, a.gate_half, 0, (float)x);
      if (a.want & kWantScaleOne) put(a.dscale, a.scale_half, 0, (float)y);
    }
  }
}

}  // namespace

// By the width: chunks of eight channels to a thread, sixteen threads to a row up
// to 128 channels, a wave up to 1024, then as many threads as there are chunks.
#define BY_WIDTH(d, RUN)                                  \
  do {                                                    \
    if ((d) <= 128) RUN(16, 1);                           \
    else if ((d) <= 512) RUN(64, 1);                      \
    else if ((d) <= 1024) RUN(64, 2);                     \
    else if ((d) <= 2048) RUN(256, 1);                    \
    else if ((d) <= 4096) RUN(512, 1);                    \
    else if ((d) <= 8192) RUN(512, 2);                    \
    else RUN(1024, 2);                                    \
  } while (0)
#define BY_TYPES(g, K, TPR, NC, BLOCK, ...)                                                                          \
  do {                                                                                                               \
    if (x_half) hipLaunchKernelGGL((K<u16, u16, TPR, NC, BLOCK, ##__VA_ARGS__>), g, dim3(BLOCK), 0, s, a);           \
    else if (y_half) hipLaunchKernelGGL((K<float, u16, TPR, NC, BLOCK, ##__VA_ARGS__>), g, dim3(BLOCK), 0, s, a);    \
    else hipLaunchKernelGGL((K<float, float, TPR, NC, BLOCK, ##__VA_ARGS__>), g, dim3(BLOCK), 0, s, a);              \
  } while (0)

static int threads_of(int d) {
  int tpr = 0;
#define THREADS(TPR, NC) tpr = TPR
  BY_WIDTH(d, THREADS);
#undef THREADS
  return tpr;
}
constexpr int at_least(int a, int b) { return a > b ? a : b; }
// Threads of a block: several rows where they are short.
constexpr int kForwardBlock = 256, kBackwardBlock = 512;
constexpr int kForwardMost = 2048;           // blocks of a launch

hipError_t launch_residual_norm(const NormArgs& a, int x_half, int y_half, hipStream_t s) {
  const int64_t rows = at_least(1, kForwardBlock / threads_of(a.d)), blocks = (a.n + rows - 1) / rows;
  const dim3 g((unsigned)(blocks < kForwardMost ? blocks : kForwardMost));
#define FORWARD(TPR, NC) BY_TYPES(g, k_residual_norm, TPR, NC, at_least(TPR, kForwardBlock))
  BY_WIDTH(a.d, FORWARD);
#undef FORWARD
  return hipGetLastError();
}

int norm_grad_blocks(int64_t n, int d) {
  const int64_t rows = at_least(1, kBackwardBlock / threads_of(d)), blocks = (n + rows - 1) / rows;
  const int most = d > 4096 || (d > 512 && d <= 1024) ? 256 : 512;     // what the CUs hold at once
  return (int)(blocks < most ? blocks : most);
}

hipError_t launch_residual_norm_grad(const NormArgs& a, int x_half, int y_half, hipStream_t s) {
  const dim3 g((unsigned)a.blocks);
#define BACKWARD(TPR, NC) BY_TYPES(g, k_residual_norm_grad, TPR, NC, at_least(TPR, kBackwardBlock), false)
#define BACKWARD_GENERAL(TPR, NC) BY_TYPES(g, k_residual_norm_grad, TPR, NC, at_least(TPR, kBackwardBlock), true)
  if (a.gate.kind == NORM_FULL || a.scale.kind == NORM_CHANNELS) BY_WIDTH(a.d, BACKWARD_GENERAL);
  else BY_WIDTH(a.d, BACKWARD);
#undef BACKWARD
#undef BACKWARD_GENERAL
  return hipGetLastError();
}

hipError_t launch_norm_sums(const NormSums& a, hipStream_t s) {
  int columns = 0;
  for (int bit = kWantBlock; bit <= kWantPre; bit *= 2) columns += (a.want & bit) != 0;
  columns += (a.want & (kWantGateOne | kWantScaleOne)) != 0;
  hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)((a.d + 31) / 32), (unsigned)columns), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
