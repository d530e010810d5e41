// Softmax cross entropy of a language-model head, z = H W^T, with its
// gradient, without the n x V logits: tokens are taken in pieces.
//
//   compact    the valid tokens (target != ignore_index) in order; ignored
//              ones are never read, so what their rows hold does not matter
//   pack       the piece's hidden rows, gathered, zero-padded, in panels
//   logits     z by tiles; per token and tile an integer reference
//              K >= log2(e) max z and the sum of 2^(log2(e) z - K) over the
//              tile without the target's term; with gradients also the
//              exponentials themselves, in 16 bits (10 bits of mantissa, 6 of
//              exponent, no sign) or 32
//   merge      per token, over tiles: K = max K_t (differences of integer
//              references scale exactly), L = sum_t 2^(K_t - K) sum_t, the
//              target's e = 2^(log2(e) z_t - K), loss = log1p(L / e); the
//              target's own gradient is -g L / (L + e), which loses nothing
//              when the model is sure of the target
//   dlogits    p - [v = t] (times the token's own factor) in the operands' type,
//              over the exponentials; a factor common to all tokens waits for
//              the 32-bit sums
//   dhidden    dz W, split over the vocabulary where tiles are few, then a
//              sum of the splits written to the tokens' rows
//   dweight    dz^T H, summed over pieces in 32 bits
//
// A 16-bit exponential carries an eighth of the rounding of the bf16 value it
// becomes, so the gradient's one rounding is the one to bf16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "train.hpp"

namespace muon {
namespace {

typedef unsigned short u16;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;
// Lowest reference: far below any finite logit's, but finite, so that a tile
// of logits at -infinity has exponentials of 0.
constexpr float kRefFloor = -3.0e38f;

__device__ __forceinline__ float bf2f(u16 h) { return __uint_as_float((unsigned int)h << 16); }
__device__ __forceinline__ u16 f2bf(float f) {
  unsigned int u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u16)((u >> 16) | 0x40);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return (u16)(u >> 16);
}
template <typename T> __device__ __forceinline__ float ld(const T* p, int64_t i);
template <> __device__ __forceinline__ float ld<float>(const float* p, int64_t i) { return p[i]; }
template <> __device__ __forceinline__ float ld<u16>(const u16* p, int64_t i) { return bf2f(p[i]); }
template <typename T> __device__ __forceinline__ T to(float x);
template <> __device__ __forceinline__ float to<float>(float x) { return x; }
template <> __device__ __forceinline__ u16 to<u16>(float x) { return f2bf(x); }

// Exponentials in (0, 1]: 6 bits of exponent (2^-63 and less become 0), 10 of
// mantissa, rounded half up; 32-bit pieces keep them as they are.
constexpr unsigned int kCodeBase = 64u << 10;
__device__ __forceinline__ u16 encode(float e) {
  const int q = (int)((__float_as_uint(e) + 0x1000u) >> 13) - (int)kCodeBase;
  return (u16)min(max(q, 0), 0xFFFF);
}
__device__ __forceinline__ float decode(u16 q) { return q ? __uint_as_float(((unsigned int)q + kCodeBase) << 13) : 0.f; }
template <typename T> __device__ __forceinline__ T keep_exp(float e);
template <> __device__ __forceinline__ u16 keep_exp<u16>(float e) { return encode(e); }
template <> __device__ __forceinline__ float keep_exp<float>(float e) { return e; }
template <typename T> __device__ __forceinline__ float kept_exp(T q);
template <> __device__ __forceinline__ float kept_exp<u16>(u16 q) { return decode(q); }
template <> __device__ __forceinline__ float kept_exp<float>(float q) { return q; }

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

// ---------------------------------------------------------------------------
// Compaction: one block; each thread takes a run of tokens, counts, and
// writes its valid ones after the threads before it. A per-token loss of an
// ignored token is 0.
// ---------------------------------------------------------------------------
template <typename I>
__global__ __launch_bounds__(1024) void k_compact(HeadArgs a, const I* __restrict__ targets, int64_t ignore) {
  __shared__ int sums[16];
  const int t = threadIdx.x;
  const int run = (a.n + 1023) / 1024;
  const int lo = (int)min((int64_t)t * run, (int64_t)a.n), hi = (int)min((int64_t)lo + run, (int64_t)a.n);
  int c = 0;
  for (int i = lo; i < hi; ++i) c += (int64_t)targets[i] != ignore;
  int x = c;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if ((t & 63) >= o) x += y;
  }
  if ((t & 63) == 63) sums[t >> 6] = x;
  __syncthreads();
  int before = x - c, all = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    if (w < (t >> 6)) before += sums[w];
    all += sums[w];
  }
  for (int i = lo; i < hi; ++i) {
    const int64_t g = (int64_t)targets[i];
    if (g == ignore) {
      if (a.per_token) a.loss[i] = 0.f;
      continue;
    }
    a.idx[before] = i;
    a.tgt[before] = g >= 0 && g < a.v ? (int)g : -1;
    ++before;
  }
  if (t == 0) a.count[0] = all;
}

// One block per row of the piece (rows past the valid ones, up to a whole
// tile, become zero).
template <typename T>
__global__ __launch_bounds__(256) void k_pack(HeadArgs a) {
  const int rows = piece_rows(a), r = blockIdx.x;
  if (r >= (rows + 255) / 256 * 256) return;
  const T* src = r < rows ? (const T*)a.h + (int64_t)a.idx[a.row0 + r] * a.ld_h : nullptr;
  T* dst = (T*)a.hp;
  for (int c = threadIdx.x; c < a.dp; c += 256) dst[panel_at<T>(r, c, a.dp)] = src && c < a.d ? src[c] : T(0);
}

template <typename T>
__global__ __launch_bounds__(256) void k_pack_weight(const T* __restrict__ src, int64_t ld, T* __restrict__ dst, int d,
                                                     int dp) {
  const int64_t r = blockIdx.x;
  for (int c = threadIdx.x; c < dp; c += 256) dst[r * dp + c] = c < d ? src[r * ld + c] : T(0);
}

// ---------------------------------------------------------------------------
// Products. One shape for the three of them: a 64 x 64 tile per block, 16 of
// K at a time in LDS, 4 x 4 sums per thread.
// ---------------------------------------------------------------------------
template <typename FA, typename FB, typename FE>
__device__ __forceinline__ void tile_product(int k0, int k1, FA fa, FB fb, FE done) {
  __shared__ float sa[16][65], sb[16][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k = k0; k < k1; k += 16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = threadIdx.x + 256 * q, m = e >> 4, kk = e & 15;
      sa[kk][m] = k + kk < k1 ? fa(m, k + kk) : 0.f;
      sb[kk][m] = k + kk < k1 ? fb(m, k + kk) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[kk][ty * 4 + i], sb[kk][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) done(ty * 4 + i, tx * 4 + j, acc[i][j]);
}

template <typename T>
__global__ __launch_bounds__(256) void k_logits(HeadArgs a, int keep) {
  __shared__ float z[64][65];   // token, vocabulary
  const int rows = piece_rows(a), r0 = blockIdx.y * 64, v0 = blockIdx.x * 64;
  if (r0 >= rows) return;
  const T* hp = (const T*)a.hp;
  const T* w = (const T*)a.w;
  tile_product(
      0, a.d, [&](int m, int k) { return ld<T>(hp, panel_at<T>(r0 + m, k, a.dp)); },
      [&](int m, int k) { return v0 + m < a.v ? ld<T>(w, (int64_t)(v0 + m) * a.ld_w + k) : 0.f; },
      [&](int i, int j, float x) { z[i][j] = a.softcap > 0.f ? a.softcap * tanhf(x / a.softcap) : x; });
  __syncthreads();
  if (threadIdx.x < 64) {
    const int i = threadIdx.x, r = r0 + i;
    const int tg = r < rows ? a.tgt[a.row0 + r] : -1, nv = min(64, a.v - v0);
    float top = kRefFloor;
    for (int j = 0; j < nv; ++j) top = fmaxf(top, z[i][j] * kLog2e);
    top = ceilf(top);
    float sum = 0.f;
    for (int j = 0; j < 64; ++j) {
      const float e = j < nv ? exp2f(fmaf(z[i][j], kLog2e, -top)) : 0.f;
      if (v0 + j == tg) a.zt[r] = z[i][j];
      else sum += e;
      if (keep) ((T*)a.e)[panel_at<T>(r, v0 + j, a.vp)] = keep_exp<T>(e);
    }
    a.tmax[(int64_t)blockIdx.x * a.piece + r] = top;
    a.tsum[(int64_t)blockIdx.x * a.piece + r] = sum;
  }
}

// One thread per token of the piece.
__global__ __launch_bounds__(256) void k_merge(HeadArgs a, int grad) {
  const int rows = piece_rows(a), r = blockIdx.x * 256 + threadIdx.x;
  if (r >= rows) return;
  const int tg = a.tgt[a.row0 + r], token = a.idx[a.row0 + r];
  float top = kRefFloor;
  for (int t = 0; t < a.n_vt; ++t) top = fmaxf(top, a.tmax[(int64_t)t * a.piece + r]);
  float others = 0.f;
  for (int t = 0; t < a.n_vt; ++t)
    others += a.tsum[(int64_t)t * a.piece + r] * exp2f(a.tmax[(int64_t)t * a.piece + r] - top);
  float loss, g = 0.f;
  float4 rs = {top, 0.f, 0.f, 0.f};
  if (tg < 0) {
    loss = __uint_as_float(0x7FC00000u);   // a target outside the vocabulary
  } else {
    const float z = a.zt[r], y = fmaf(z, kLog2e, -top), e = exp2f(y);
    loss = y > -60.f ? log1pf(others / e) : logf(others + e) - y * kLn2;
    if (grad) {
      g = a.grad_out && a.per_token ? a.grad_out[token] : 1.f;
      rs.y = g / (others + e);
      rs.z = -rs.y * others;
      if (a.softcap > 0.f) {
        const float q = z / a.softcap;
        rs.z *= 1.f - q * q;
      }
    }
  }
  a.rs[r] = rs;
  a.lossc[a.row0 + r] = loss;
  if (a.per_token) a.loss[token] = loss;
}

// The reduced loss: the tokens' losses in a fixed order, in 64 bits.
__global__ __launch_bounds__(1024) void k_total(HeadArgs a) {
  __shared__ double sh[16];
  const int n = a.count[0];
  double x = 0;
  for (int i = threadIdx.x; i < n; i += 1024) x += a.lossc[i];
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0;
    for (int i = 0; i < 16; ++i) s += sh[i];
    a.loss[0] = (float)(a.mean ? (n ? s / n : 0.0) : s);
  }
}

// Exponentials to the logits' gradient, in place; rows past the valid ones
// (up to a whole tile) and columns past the vocabulary are zero.
template <typename T>
__global__ __launch_bounds__(256) void k_dlogits(HeadArgs a) {
  const int rows = piece_rows(a), r = blockIdx.x;
  if (r >= (rows + 255) / 256 * 256) return;
  const bool real = r < rows;
  const float4 rs = real ? a.rs[r] : float4{0.f, 0.f, 0.f, 0.f};
  const int tg = real ? a.tgt[a.row0 + r] : -1;
  T* e = (T*)a.e;
  for (int c = threadIdx.x; c < a.vp; c += 256) {
    const int64_t at = panel_at<T>(r, c, a.vp);
    float x = 0.f;
    if (real && tg >= 0 && c < a.v) {
      const float k = a.tmax[(int64_t)(c / a.vtile) * a.piece + r];
      const float ex = kept_exp<T>(e[at]);
      x = ex * (rs.y * exp2f(k - rs.x));
      if (a.softcap > 0.f) {
        const float q = (__log2f(ex) + k) * (kLn2 / a.softcap);
        x = ex > 0.f ? x * (1.f - q * q) : 0.f;
      }
      if (c == tg) x = rs.z;
    }
    e[at] = to<T>(x);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_dhidden(HeadArgs a) {
  const int rows = piece_rows(a), r0 = blockIdx.y * 64, d0 = blockIdx.x * 64;
  if (r0 >= rows) return;
  const T* s = (const T*)a.e;
  const T* w = (const T*)a.w;
  tile_product(
      0, a.v, [&](int m, int k) { return ld<T>(s, panel_at<T>(r0 + m, k, a.vp)); },
      [&](int m, int k) { return d0 + m < a.d ? ld<T>(w, (int64_t)k * a.ld_w + d0 + m) : 0.f; },
      [&](int i, int j, float x) {
        if (d0 + j < a.dp) a.part[(int64_t)(r0 + i) * a.dp + d0 + j] = x;
      });
}

// Sums of the splits to the tokens' rows, and zeros to the ignored ones: one
// block per row of the piece, then one per token.
template <typename T, typename I>
__global__ __launch_bounds__(256) void k_dhidden_out(HeadArgs a, const I* __restrict__ targets, int64_t ignore) {
  T* dh = (T*)a.dh;
  if ((int)blockIdx.x >= a.piece) {   // only with the first piece
    const int64_t i = (int)blockIdx.x - a.piece;
    if ((int64_t)targets[i] != ignore) return;
    for (int c = threadIdx.x; c < a.d; c += 256) dh[i * a.ld_dh + c] = T(0);
    return;
  }
  const int rows = piece_rows(a), r = blockIdx.x;
  if (r >= rows) return;
  const int64_t token = a.idx[a.row0 + r];
  const float g = common_factor(a);
  for (int c = threadIdx.x; c < a.d; c += 256) {
    float x = 0.f;
    for (int q = 0; q < a.split; ++q) x += a.part[((int64_t)q * a.piece + r) * a.dp + c];
    dh[token * a.ld_dh + c] = to<T>(x * g);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_dweight(HeadArgs a) {
  const int rows = piece_rows(a), v0 = blockIdx.y * 64, d0 = blockIdx.x * 64;
  const T* s = (const T*)a.e;
  const T* hp = (const T*)a.hp;
  const float g = common_factor(a);
  tile_product(
      0, rows, [&](int m, int k) { return v0 + m < a.v ? ld<T>(s, panel_at<T>(k, v0 + m, a.vp)) : 0.f; },
      [&](int m, int k) { return d0 + m < a.d ? ld<T>(hp, panel_at<T>(k, d0 + m, a.dp)) : 0.f; },
      [&](int i, int j, float x) {
        const int64_t v = v0 + i, d = d0 + j;
        if (v >= a.v || d >= a.d) return;
        if (!a.first) x += a.dwacc[v * a.dp + d];
        if (a.last) ((T*)a.dw)[v * a.ld_dw + d] = to<T>(x * g);
        else a.dwacc[v * a.dp + d] = x;
      });
}

inline unsigned cdiv(int64_t a, int64_t b) { return (unsigned)((a + b - 1) / b); }

}  // namespace

#define BY_TYPE(dt, f, ...)                                                                                   \
  do {                                                                                                        \
    if ((dt) == MUON_BF16) hipLaunchKernelGGL((f<u16>), __VA_ARGS__);                                         \
    else hipLaunchKernelGGL((f<float>), __VA_ARGS__);                                                         \
    return hipGetLastError();                                                                                 \
  } while (0)

hipError_t launch_head_compact(const HeadArgs& a, const void* targets, int target_bytes, int64_t ignore,
                               hipStream_t s) {
  if (target_bytes == 8)
    hipLaunchKernelGGL((k_compact<int64_t>), dim3(1), dim3(1024), 0, s, a, (const int64_t*)targets, ignore);
  else
    hipLaunchKernelGGL((k_compact<int32_t>), dim3(1), dim3(1024), 0, s, a, (const int32_t*)targets, ignore);
  return hipGetLastError();
}
hipError_t launch_head_pack(const HeadArgs& a, int dt, hipStream_t s) {
  BY_TYPE(dt, k_pack, dim3(a.piece), dim3(256), 0, s, a);
}
hipError_t launch_head_pack_weight(const void* src, int64_t ld, void* dst, int v, int d, int dp, int dt,
                                   hipStream_t s) {
  if (dt == MUON_BF16)
    hipLaunchKernelGGL((k_pack_weight<u16>), dim3(v), dim3(256), 0, s, (const u16*)src, ld, (u16*)dst, d, dp);
  else
    hipLaunchKernelGGL((k_pack_weight<float>), dim3(v), dim3(256), 0, s, (const float*)src, ld, (float*)dst, d, dp);
  return hipGetLastError();
}
hipError_t launch_head_logits(const HeadArgs& a, int dt, int keep, hipStream_t s) {
  BY_TYPE(dt, k_logits, dim3(a.n_vt, a.piece / 64), dim3(256), 0, s, a, keep);
}
hipError_t launch_head_merge(const HeadArgs& a, int grad, hipStream_t s) {
  hipLaunchKernelGGL(k_merge, dim3(cdiv(a.piece, 256)), dim3(256), 0, s, a, grad);
  return hipGetLastError();
}
hipError_t launch_head_total(const HeadArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_total, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_head_dlogits(const HeadArgs& a, int dt, hipStream_t s) {
  BY_TYPE(dt, k_dlogits, dim3(a.piece), dim3(256), 0, s, a);
}
hipError_t launch_head_dhidden(const HeadArgs& a, int dt, hipStream_t s) {
  BY_TYPE(dt, k_dhidden, dim3(cdiv(a.d, 64), a.piece / 64), dim3(256), 0, s, a);
}
hipError_t launch_head_dhidden_out(const HeadArgs& a, int dt, const void* targets, int target_bytes, int64_t ignore,
                                   hipStream_t s) {
  const dim3 g(a.piece + (a.row0 == 0 ? a.n : 0)), b(256);
  if (dt == MUON_BF16) {
    if (target_bytes == 8) hipLaunchKernelGGL((k_dhidden_out<u16, int64_t>), g, b, 0, s, a, (const int64_t*)targets, ignore);
    else hipLaunchKernelGGL((k_dhidden_out<u16, int32_t>), g, b, 0, s, a, (const int32_t*)targets, ignore);
  } else {
    if (target_bytes == 8) hipLaunchKernelGGL((k_dhidden_out<float, int64_t>), g, b, 0, s, a, (const int64_t*)targets, ignore);
    else hipLaunchKernelGGL((k_dhidden_out<float, int32_t>), g, b, 0, s, a, (const int32_t*)targets, ignore);
  }
  return hipGetLastError();
}
hipError_t launch_head_dweight(const HeadArgs& a, int dt, hipStream_t s) {
  BY_TYPE(dt, k_dweight, dim3(cdiv(a.d, 64), cdiv(a.v, 64)), dim3(256), 0, s, a);
}

}  // namespace muon
