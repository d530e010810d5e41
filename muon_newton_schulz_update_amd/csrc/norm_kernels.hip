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

namespace muon {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// Eight channels from c of a row of d, zero past its end; one or two loads
// where whole, aligned or not.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int d, float (&v)[8]) {
  if (c + 8 <= d) {
    if constexpr (sizeof(T) == 2) {
      u32x4_t q;
      __builtin_memcpy(&q, row + c, 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(q[e] << 16);
        v[2 * e + 1] = __uint_as_float(q[e] & 0xFFFF0000u);
      }
    } else {
      __builtin_memcpy(v, row + c, 32);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = 0.f;
      if (c + e < d) {
        if constexpr (sizeof(T) == 2) v[e] = bf2f(row[c + e]);
        else v[e] = row[c + e];
      }
    }
  }
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
// several waves meet in LDS; each sum of a row has its own place there.
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* sh) {
  constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
  for (int o = W / 2; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], o);
  if constexpr (TPR > 64) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if ((threadIdx.x & 63) == 0) sh[k * (TPR / 64) + (threadIdx.x >> 6)] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < TPR / 64; ++w) v[k] += sh[k * (TPR / 64) + w];
    }
  }
}

// TPR threads to a row, NC chunks of eight channels to a thread; threads past
// TPR of a block have other rows.
template <typename TX, typename TY, int TPR, int NC, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_residual_norm(NormArgs a) {
  constexpr int ROWS = BLOCK / TPR;
  __shared__ float sh[2 * (BLOCK / 64)];
  const int t = threadIdx.x % TPR, d = a.d;
  const bool there = a.y.ptr != nullptr;
  float post[NC][8], gate[NC][8], pre[NC][8], scale[NC][8];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = 8 * (k * TPR + t);
    load_param(a.scale, c, d, scale[k]);
    load_param(a.pre_gain, c, d, pre[k]);
    load_param(a.post_gain, c, d, post[k]);
    load_param(a.gate, c, d, gate[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) gate[k][e] *= post[k][e];
  }
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.n; r0 += (int64_t)gridDim.x * ROWS) {
    // (every thread of a block goes round as often; rows past the last one are
    // the last one again and are not stored)
    const int64_t row = r0 + threadIdx.x / TPR;
    const bool real = row < a.n;
    const int64_t r = real ? row : a.n - 1;
    float x[NC][8], y[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) load8((const TX*)a.x.ptr + r * a.x.ld, 8 * (k * TPR + t), d, x[k]);
    if (there)
#pragma unroll
      for (int k = 0; k < NC; ++k) load8((const TY*)a.y.ptr + r * a.y.ld, 8 * (k * TPR + t), d, y[k]);
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] *= scale[k][e];
    if (there) {
      float r1 = 1.f;
      if (a.post) {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = fmaf(y[k][e], y[k][e], s[0]);
        row_sums<TPR>(s, sh);
        r1 = 1.f / sqrtf(s[0] / d + a.eps);
      }
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int c = 8 * (k * TPR + t);
        if (a.gate.kind == NORM_FULL) {
          float g[8];
          load8((const TY*)a.gate.ptr + r * a.gate.ld, c, d, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[k][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = fmaf(y[k][e] * r1, gate[k][e], x[k][e]);
      }
    }
    if (a.out.ptr && real)
#pragma unroll
      for (int k = 0; k < NC; ++k) store8((TX*)a.out.ptr + r * a.out.ld, 8 * (k * TPR + t), d, x[k]);
    if (a.pre) {
      s[0] = 0.f;
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(x[k][e], x[k][e], s[0]);
      row_sums<TPR>(s, sh + BLOCK / 64);
      const float r2 = 1.f / sqrtf(s[0] / d + a.eps);
      if (real)
#pragma unroll
        for (int k = 0; k < NC; ++k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] *= r2 * pre[k][e];
          store8((TY*)a.hidden.ptr + r * a.hidden.ld, 8 * (k * TPR + t), d, x[k]);
        }
    }
    if (TPR > 64) __syncthreads();   // the sums are read before the next row's are written
  }
}

template <typename TX, typename TY, int TPR, int NC, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_residual_norm_grad(NormArgs a) {
  constexpr int ROWS = BLOCK / TPR;
  __shared__ float sh[3][2 * (BLOCK / 64)];
  __shared__ __attribute__((aligned(16))) float joined[ROWS > 1 ? ROWS * TPR * 8 : 1];
  const int t = threadIdx.x % TPR, d = a.d;
  const bool there = a.y.ptr != nullptr;
  const bool want_block = a.want & (kWantBlock | kWantGateOne), want_scale = a.want & (kWantScale | kWantScaleOne);
  const bool full = a.gate.kind == NORM_FULL;
  float sum_block[NC][8], sum_scale[NC][8], sum_pre[NC][8], gate_one = 0.f, scale_one = 0.f;
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum_block[k][e] = sum_scale[k][e] = sum_pre[k][e] = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.n; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t row = r0 + threadIdx.x / TPR;
    const bool real = row < a.n;
    const int64_t r = real ? row : a.n - 1;
    float x[NC][8], y[NC][8], o[NC][8], g[NC][8], w[8];
#pragma unroll
    for (int k = 0; k < NC; ++k) load8((const TX*)a.x.ptr + r * a.x.ld, 8 * (k * TPR + t), d, x[k]);
    float r1 = 1.f;
    if (there) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        load8((const TY*)a.y.ptr + r * a.y.ld, 8 * (k * TPR + t), d, y[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(y[k][e], y[k][e], s[0]);
      }
      if (a.post) {
        row_sums<TPR>(s, sh[0]);
        r1 = 1.f / sqrtf(s[0] / d + a.eps);
      }
    }
    // y becomes yhat, o the row's out, g the gate
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (k * TPR + t);
      load_param(a.scale, c, d, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[k][e] = x[k][e] * w[e];
      if (there) {
        if (full) load8((const TY*)a.gate.ptr + r * a.gate.ld, c, d, g[k]);
        else load_param(a.gate, c, d, g[k]);
        load_param(a.post_gain, c, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[k][e] *= r1;
          o[k][e] = fmaf(g[k][e] * w[e], y[k][e], o[k][e]);
        }
      }
    }
    float r2 = 0.f, m = 0.f;
    float u[NC][8];
    if (a.dhidden.ptr) {
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int c = 8 * (k * TPR + t);
        load8((const TY*)a.dhidden.ptr + r * a.dhidden.ld, c, d, u[k]);
        load_param(a.pre_gain, c, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] = fmaf(o[k][e], o[k][e], s[0]);
          s[1] = fmaf(o[k][e], u[k][e] * w[e], s[1]);
        }
      }
      row_sums<TPR>(s, sh[1]);
      r2 = 1.f / sqrtf(s[0] / d + a.eps);
      m = s[1] * r2 / d;
    }
    // o becomes dT
    float v[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (k * TPR + t);
      float dt[8];
      if (a.dout.ptr) {
        load8((const TX*)a.dout.ptr + r * a.dout.ld, c, d, dt);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dt[e] = 0.f;
      }
      if (a.dhidden.ptr) {
        load_param(a.pre_gain, c, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = o[k][e] * r2;
          dt[e] += r2 * (u[k][e] * w[e] - xh * m);
          if (real) sum_pre[k][e] = fmaf(u[k][e], xh, sum_pre[k][e]);
        }
      }
      load_param(a.scale, c, d, w);
      if (a.dx.ptr && real) {
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = dt[e] * w[e];
        store8((TX*)a.dx.ptr + r * a.dx.ld, c, d, q);
      }
      if (want_scale && real)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (a.want & kWantScale) sum_scale[k][e] = fmaf(dt[e], x[k][e], sum_scale[k][e]);
          else scale_one = fmaf(dt[e], x[k][e], scale_one);
        }
      if (there) {
        load_param(a.post_gain, c, d, w);
        if (full && a.dfull.ptr && real) {
          float q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = dt[e] * w[e] * y[k][e];
          store8((TY*)a.dfull.ptr + r * a.dfull.ld, c, d, q);
        }
        if (want_block && real)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float q = (full ? dt[e] * g[k][e] : dt[e]) * y[k][e];
            if (a.want & kWantBlock) sum_block[k][e] += q;
            if (a.want & kWantGateOne) gate_one = fmaf(w[e], q, gate_one);
          }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[k][e] = dt[e] * g[k][e] * (a.post ? w[e] : 1.f);
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
          store8((TY*)a.dy.ptr + r * a.dy.ld, 8 * (k * TPR + t), d, o[k]);
        }
    }
    if (TPR > 64) __syncthreads();   // the sums' buffers are read before the next row's
  }
  // the block's partials: rows' sums joined in order
  float* part = a.part + blockIdx.x * a.part_floats;
  auto leave = [&](float (&sum)[NC][8]) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (k * TPR + t);
      if constexpr (ROWS > 1) {
        float* mine = joined + threadIdx.x * 8;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[e] = sum[k][e];
        __syncthreads();
        if (threadIdx.x < TPR)
          for (int q = 1; q < ROWS; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[k][e] += joined[(q * TPR + t) * 8 + e];
      }
      if (threadIdx.x < TPR && c < a.dp) {
        *(f32x4_t*)(part + c) = (f32x4_t){sum[k][0], sum[k][1], sum[k][2], sum[k][3]};
        *(f32x4_t*)(part + c + 4) = (f32x4_t){sum[k][4], sum[k][5], sum[k][6], sum[k][7]};
      }
    }
    part += a.dp;
  };
  if (a.want & kWantBlock) leave(sum_block);
  if (a.want & kWantScale) leave(sum_scale);
  if (a.want & kWantPre) leave(sum_pre);
  if (a.want & (kWantGateOne | kWantScaleOne)) {
    float* all = &sh[0][0];
    __syncthreads();
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      gate_one += __shfl_xor(gate_one, o);
      scale_one += __shfl_xor(scale_one, o);
    }
    if ((threadIdx.x & 63) == 0) {
      all[(threadIdx.x >> 6) * 2] = gate_one;
      all[(threadIdx.x >> 6) * 2 + 1] = scale_one;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      float x = 0.f;
      for (int w = 0; w < BLOCK / 64; ++w) x += all[w * 2 + threadIdx.x];
      part[threadIdx.x] = x;
    }
  }
}

// Sums of the blocks' partials, in their order: 64 channels to a block, sixteen
// threads to a channel. The last block has the two single values.
__global__ __launch_bounds__(1024) void k_norm_sums(NormSums a) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  int vectors = 0;
  auto total = [&](int which) {
    float x = 0.f;
    if (c < a.d)
      for (int b = share; b < a.blocks; b += 16) x += a.part[b * a.part_floats + (int64_t)which * a.dp + c];
    __syncthreads();
    sh[share][lane] = x;
    __syncthreads();
    x = 0.f;
    for (int q = 0; q < 16; ++q) x += sh[q][lane];
    return x;
  };
  auto put = [&](void* p, int half, int64_t i, float x) {
    if (half) ((u16*)p)[i] = f2bf(x);
    else ((float*)p)[i] = x;
  };
  auto factor = [&](const NormParam& p) {
    return p.kind == NORM_CHANNELS ? one_value(p, c) : p.kind == NORM_ONE ? one_value(p, 0) : 1.f;
  };
  const bool mine = share == 0 && c < a.d;
  if (a.want & kWantBlock) {
    const float x = total(vectors++);
    if (mine && a.dpost) put(a.dpost, a.post_half, c, x * factor(a.gate));
    if (mine && a.dgate && a.gate.kind == NORM_CHANNELS) put(a.dgate, a.gate_half, c, x * factor(a.post_gain));
  }
  if (a.want & kWantScale) {
    const float x = total(vectors++);
    if (mine) put(a.dscale, a.scale_half, c, x);
  }
  if (a.want & kWantPre) {
    const float x = total(vectors++);
    if (mine) put(a.dpre, a.pre_half, c, x);
  }
  if (blockIdx.x == 0 && threadIdx.x < 64) {
    double x = 0, y = 0;
    if (a.want & (kWantGateOne | kWantScaleOne))
      for (int b = lane; b < a.blocks; b += 64) {
        const float* p = a.part + b * a.part_floats + (int64_t)vectors * a.dp;
        x += p[0];
        y += p[1];
      }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      x += __shfl_xor(x, o);
      y += __shfl_xor(y, o);
    }
    if (lane == 0) {
      if (a.want & kWantGateOne) put(a.dgate, a.gate_half, 0, (float)x);
      if (a.want & kWantScaleOne) put(a.dscale, a.scale_half, 0, (float)y);
    }
  }
}

constexpr int kMostBlocks = 2048;
int rows_per_block(int d) { return d <= 128 ? 16 : d <= 1024 ? 4 : 1; }

}  // namespace

// By the width: chunks of eight channels to a thread, sixteen threads to a row
// up to 128 channels, a wave up to 1024, then 256 or 1024 threads.
#define BY_WIDTH(d, RUN)                                  \
  do {                                                    \
    if ((d) <= 128) RUN(16, 1, 256);                      \
    else if ((d) <= 512) RUN(64, 1, 256);                 \
    else if ((d) <= 1024) RUN(64, 2, 256);                \
    else if ((d) <= 2048) RUN(256, 1, 256);               \
    else if ((d) <= 4096) RUN(256, 2, 256);               \
    else if ((d) <= 8192) RUN(1024, 1, 1024);             \
    else RUN(1024, 2, 1024);                              \
  } while (0)
#define BY_TYPES(K, TPR, NC, BLOCK, g)                                                                     \
  do {                                                                                                     \
    if (x_half) hipLaunchKernelGGL((K<u16, u16, TPR, NC, BLOCK>), g, dim3(BLOCK), 0, s, a);                \
    else if (y_half) hipLaunchKernelGGL((K<float, u16, TPR, NC, BLOCK>), g, dim3(BLOCK), 0, s, a);         \
    else hipLaunchKernelGGL((K<float, float, TPR, NC, BLOCK>), g, dim3(BLOCK), 0, s, a);                   \
  } while (0)

hipError_t launch_residual_norm(const NormArgs& a, int x_half, int y_half, hipStream_t s) {
  const int64_t rows = rows_per_block(a.d), blocks = (a.n + rows - 1) / rows;
  const dim3 g((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks));
#define FORWARD(TPR, NC, BLOCK) BY_TYPES(k_residual_norm, TPR, NC, BLOCK, g)
  BY_WIDTH(a.d, FORWARD);
#undef FORWARD
  return hipGetLastError();
}

int norm_grad_blocks(int64_t n, int d) {
  const int64_t rows = rows_per_block(d), blocks = (n + rows - 1) / rows;
  return (int)(blocks < 512 ? blocks : 512);
}

hipError_t launch_residual_norm_grad(const NormArgs& a, int x_half, int y_half, hipStream_t s) {
  const dim3 g((unsigned)a.blocks);
#define BACKWARD(TPR, NC, BLOCK) BY_TYPES(k_residual_norm_grad, TPR, NC, BLOCK, g)
  BY_WIDTH(a.d, BACKWARD);
#undef BACKWARD
  return hipGetLastError();
}

hipError_t launch_norm_sums(const NormSums& a, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)((a.d + 63) / 64)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
