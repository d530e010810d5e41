// Tensor-list kernels of the training step: global gradient norm, scaling by
// a device scalar (clipping) and the AdamW update.
//
// All three are bound by HBM: each element is read (and written) once, in
// 16-byte pieces where the tensor's start is 16-byte aligned. A work item is
// kChunk (norm: kNormChunk) consecutive elements of one tensor; a tensor that is
// not one aligned contiguous run is taken element by element with its row and column from a
// 32-bit division, still coalesced within rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "train.hpp"

namespace muon {
namespace {

typedef unsigned short u16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf2f(unsigned short h) { return __uint_as_float((unsigned int)h << 16); }
// Round to nearest even; a NaN keeps its sign and becomes quiet (the rounding
// carry could otherwise turn it into an infinity).
__device__ __forceinline__ unsigned short f2bf(float f) {
  unsigned int u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (unsigned short)((u >> 16) | 0x40);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return (unsigned short)(u >> 16);
}
__device__ __forceinline__ float ld1(const void* p, int64_t i, bool bf) {
  return bf ? bf2f(((const unsigned short*)p)[i]) : ((const float*)p)[i];
}
__device__ __forceinline__ void st1(void* p, int64_t i, bool bf, float x) {
  if (bf) ((unsigned short*)p)[i] = f2bf(x);
  else ((float*)p)[i] = x;
}
__device__ __forceinline__ void ld8(const void* p, int64_t i, bool bf, float x[8]) {
  if (bf) {
    const u16x8_t q = *(const u16x8_t*)((const unsigned short*)p + i);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = bf2f(q[e]);
  } else {
    const f32x4_t a = *(const f32x4_t*)((const float*)p + i), b = *(const f32x4_t*)((const float*)p + i + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
  }
}
__device__ __forceinline__ void st8(void* p, int64_t i, bool bf, const float x[8]) {
  if (bf) {
    u16x8_t q;
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = f2bf(x[e]);
    *(u16x8_t*)((unsigned short*)p + i) = q;
  } else {
    *(f32x4_t*)((float*)p + i) = (f32x4_t){x[0], x[1], x[2], x[3]};
    *(f32x4_t*)((float*)p + i + 4) = (f32x4_t){x[4], x[5], x[6], x[7]};
  }
}

// The tensor that work item c belongs to: the last one whose first item is
// not past c (tensors without elements have no item).
template <typename L>
__device__ __forceinline__ int find_tensor(const L& list, int c) {
  int lo = 0, hi = list.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (list.chunk0[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Row and column of element i0 + k of a strided tensor (k below the item's
// length): the row division is 32-bit, since the column of i0 plus k stays
// below cols plus that length.
struct RowCol {
  int64_t r0, cols;
  uint32_t c0;
  bool wide;      // cols past 32 bits: then the item spans at most two rows
  __device__ RowCol(int64_t i0, int64_t c) : r0(i0 / c), cols(c), wide(c > 0x7FFF0000) { c0 = 0; base = i0 % c; if (!wide) c0 = (uint32_t)base; }
  int64_t base;
  __device__ void at(int k, int64_t& r, int64_t& c) const {
    if (wide) {
      c = base + k;
      r = r0;
      if (c >= cols) { c -= cols; ++r; }
    } else {
      const uint32_t x = c0 + (uint32_t)k, q = x / (uint32_t)cols;
      r = r0 + q;
      c = x - q * (uint32_t)cols;
    }
  }
};

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Global norm. Squares are summed in 64 bits from the first addition: no
// overflow or underflow for any 32-bit gradient, and the vector units have
// fp64 rate to spare under the memory bound. Each block leaves one partial;
// the block that finishes last adds the partials in index order and writes
// the norm and the clipping coefficient, so the result does not depend on
// the order in which blocks end. At most two large blocks a CU: the counts go to
// one address, about 11 ns each (48 MB: 26 us with 1462 blocks, 15 with 512).
// Bound by HBM; measured: 2 GB of bf16 335 us, 4 GB of fp32 669 (6.0 TB/s), 77
// MB x 2 31 us (5.0), 24 x 768 elements 6 us, the launch and two trips to memory.
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 1024;
__device__ __forceinline__ double block_sum(double x, double* sh) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) sh[w] = x;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int i = 0; i < kNormThreads / 64; ++i) t += sh[i];
  __syncthreads();
  return t;
}

__device__ __forceinline__ void write_norm(double sum, float max_norm, float* norm, float* coef) {
  const float n = (float)sqrt(sum);
  *norm = n;
  if (coef) {
    const float q = max_norm / (n + 1e-6f);
    *coef = q < 1.0f || q != q ? q : 1.0f;   // a NaN norm stays visible in the coefficient
  }
}

__global__ __launch_bounds__(kNormThreads) void k_norm(NormList L, int chunks, NormState* st, int part0, int total_blocks,
                                                   float max_norm, float* norm, float* coef) {
  __shared__ double sh[kNormThreads / 64];
  __shared__ int is_last;
  double acc = 0, acc2 = 0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int ti = find_tensor(L, c);
    const ListItem& t = L.t[ti];
    const int64_t i0 = (int64_t)(c - L.chunk0[ti]) * kNormChunk;
    const int len = (int)min((int64_t)kNormChunk, t.n - i0);
    const bool bf = t.dt == MUON_BF16;
    if (t.flat) {
      const int whole = len & ~7;
#pragma unroll 4
      for (int k = threadIdx.x * 8; k < whole; k += kNormThreads * 8) {
        float x[8];
        ld8(t.src, i0 + k, bf, x);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          acc = fma((double)x[e], (double)x[e], acc);
          acc2 = fma((double)x[e + 1], (double)x[e + 1], acc2);
        }
      }
      const int k = whole + threadIdx.x;
      if (k < len) {
        const double x = ld1(t.src, i0 + k, bf);
        acc = fma(x, x, acc);
      }
    } else {
      const RowCol rc(i0, t.cols);
      for (int k = threadIdx.x; k < len; k += kNormThreads) {
        int64_t r, col;
        rc.at(k, r, col);
        const double x = ld1(t.src, r * t.ld + col, bf);
        acc = fma(x, x, acc);
      }
    }
  }
  const double mine = block_sum(acc + acc2, sh);
  if (threadIdx.x == 0) {
    // The partial goes through to the memory all XCDs share (agent scope), and
    // the wait ends when it is there; only then is the block counted. Ordinary
    // release and acquire would also write back and drop every L2's contents,
    // 1462 times for 48 MB (53 us against 12).
    __hip_atomic_store(&st->part[part0 + blockIdx.x], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t done = __hip_atomic_fetch_add(&st->ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    is_last = done == (uint32_t)total_blocks - 1;
  }
  __syncthreads();
  if (!is_last) return;
  double sum = 0;
  for (int i = threadIdx.x; i < total_blocks; i += kNormThreads)
    sum += __hip_atomic_load(&st->part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) {
    write_norm(sum, max_norm, norm, coef);
    __hip_atomic_store(&st->ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

__global__ void k_norm_empty(float max_norm, float* norm, float* coef) { write_norm(0.0, max_norm, norm, coef); }
// (a kernel, not a memset: the call may be captured in a graph)
__global__ void k_norm_reset(NormState* st) { st->ticket = 0; }

// ---------------------------------------------------------------------------
// dst = coef src, coef read from the device. In place, a coefficient of 1
// leaves every element as it is, so the kernel ends after reading it.
// Bound by HBM: 268 MB read and written in 80.5 us (6.7 TB/s, the last-level
// cache helping). The list is taken from its end to its start, which leaves its
// first tensors in that cache for the next pass over it (a norm of 268 MB after
// it 76 / 68 us).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void k_scale(ScaleList L, const float* __restrict__ coef, int in_place) {
  const float f = *coef;
  if (in_place && f == 1.0f) return;
  const int c = blockIdx.x;
  const int ti = find_tensor(L, c);
  const ScaleItem& t = L.t[ti];
  const int64_t i0 = (int64_t)(L.chunk0[ti + 1] - 1 - c) * kChunk;
  const int len = (int)min((int64_t)kChunk, t.n - i0);
  const bool sb = t.dt & 1, db = t.dt & 2;
  if (t.dt & 4) {
    const int whole = len & ~7;
#pragma unroll 4
    for (int k = threadIdx.x * 8; k < whole; k += kThreads * 8) {
      float x[8];
      ld8(t.src, i0 + k, sb, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= f;
      st8(t.dst, i0 + k, db, x);
    }
    const int k = whole + threadIdx.x;
    if (k < len) st1(t.dst, i0 + k, db, ld1(t.src, i0 + k, sb) * f);
  } else {
    const RowCol rc(i0, t.cols);
    for (int k = threadIdx.x; k < len; k += kThreads) {
      int64_t r, col;
      rc.at(k, r, col);
      st1(t.dst, r * t.ld_dst + col, db, ld1(t.src, r * t.ld_src + col, sb) * f);
    }
  }
}

// ---------------------------------------------------------------------------
// AdamW with decoupled decay: g' = s g, m = b1 m + (1 - b1) g',
// v = b2 v + (1 - b2) g'^2, w = w (1 - lr wd) - lr (m / c1) / (sqrt(v / c2) +
// eps), c = 1 - beta^step; all in fp32, 16-bit weights rounded to nearest
// even once; a copy takes the same fp32 value, rounded to its own type. Bound by
// HBM: four reads and three writes of an element, 22 bytes with 16-bit gradients
// and weights, 28 with 32-bit ones. Measured: 77.3 M elements of bf16 weights
// 324 us (5.2 TB/s); 12.7 M of fp32 in odd rows with 16-bit copies 76 us (4.7)
// over two lists in turn, 55 (6.5) over one again and again, which the last-level
// cache keeps; 24 x 768 elements 4.5 us.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void adam(const AdamConst& c, float s, float g, float& m, float& v, float& w) {
  g *= s;
  m = c.beta1 * m + c.c1 * g;
  v = c.beta2 * v + c.c2 * (g * g);
  w = w * c.keep - c.lr1 * m / (__fsqrt_rn(v) * c.rs2 + c.eps);
}

// The members of AdamConst that follow from step and rate, as the host makes
// them (in 64 bits; beta^step as a power of two).
__device__ __forceinline__ void read_clock(const AdamClock& k, AdamConst& c) {
  const double n = (double)(k.step_at ? *k.step_at : k.step), lr = k.lr_at ? (double)*k.lr_at : k.lr;
  c.keep = (float)(1.0 - lr * k.weight_decay);
  c.lr1 = (float)(lr / (1.0 - exp2(n * k.log2_b1)));
  c.rs2 = (float)(1.0 / sqrt(1.0 - exp2(n * k.log2_b2)));
}

// CLOCK: step or rate come from the device; each wave works its constants out
// beside its first loads (in a graph 16 x 768 elements 3.5 -> 3.9 us, 77.3 M
// 325.0 -> 325.6; a launch of their own would take 3 or more).
template <bool CLOCK>
__global__ __launch_bounds__(kThreads) void k_adamw(AdamList L, AdamConst c, AdamClock clock,
                                                    const float* __restrict__ scale) {
  if constexpr (CLOCK) read_clock(clock, c);
  const float s = scale ? *scale : 1.0f;
  const int ci = blockIdx.x;
  const int ti = find_tensor(L, ci);
  const AdamItem& t = L.t[ti];
  const int64_t i0 = (int64_t)(ci - L.chunk0[ti]) * kChunk;
  const int len = (int)min((int64_t)kChunk, t.n - i0);
  const bool gb = t.dt & 1, wb = t.dt & 2, cb = t.dt & 4;
  if (t.dt & 8) {
    const int whole = len & ~7;
    for (int k = threadIdx.x * 8; k < whole; k += kThreads * 8) {
      const int64_t i = i0 + k;
      float g[8], m[8], v[8], w[8];
      ld8(t.g, i, gb, g);
      ld8(t.m, i, false, m);
      ld8(t.v, i, false, v);
      ld8(t.w, i, wb, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) adam(c, s, g[e], m[e], v[e], w[e]);
      st8(t.m, i, false, m);
      st8(t.v, i, false, v);
      st8(t.w, i, wb, w);
      if (t.copy) st8(t.copy, i, cb, w);
    }
    const int k = whole + threadIdx.x;
    if (k < len) {
      const int64_t i = i0 + k;
      float m = t.m[i], v = t.v[i], w = ld1(t.w, i, wb);
      adam(c, s, ld1(t.g, i, gb), m, v, w);
      t.m[i] = m;
      t.v[i] = v;
      st1(t.w, i, wb, w);
      if (t.copy) st1(t.copy, i, cb, w);
    }
  } else {
    const RowCol rc(i0, t.cols);
    for (int k = threadIdx.x; k < len; k += kThreads) {
      int64_t r, col;
      rc.at(k, r, col);
      const int64_t im = r * t.ld[1] + col, iv = r * t.ld[2] + col, iw = r * t.ld[3] + col;
      float m = t.m[im], v = t.v[iv], w = ld1(t.w, iw, wb);
      adam(c, s, ld1(t.g, r * t.ld[0] + col, gb), m, v, w);
      t.m[im] = m;
      t.v[iv] = v;
      st1(t.w, iw, wb, w);
      if (t.copy) st1(t.copy, r * t.ld[4] + col, cb, w);
    }
  }
}

}  // namespace

hipError_t launch_norm(const NormList& L, int blocks, int chunks, NormState* st, int part0, int total_blocks,
                       float max_norm, float* norm, float* coef, hipStream_t s) {
  hipLaunchKernelGGL(k_norm, dim3(blocks), dim3(kNormThreads), 0, s, L, chunks, st, part0, total_blocks, max_norm, norm,
                     coef);
  return hipGetLastError();
}
hipError_t launch_norm_empty(float max_norm, float* norm, float* coef, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_empty, dim3(1), dim3(1), 0, s, max_norm, norm, coef);
  return hipGetLastError();
}
hipError_t launch_norm_reset(NormState* st, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_reset, dim3(1), dim3(1), 0, s, st);
  return hipGetLastError();
}
hipError_t launch_scale(const ScaleList& L, int chunks, const float* coef, int in_place, hipStream_t s) {
  hipLaunchKernelGGL(k_scale, dim3(chunks), dim3(kThreads), 0, s, L, coef, in_place);
  return hipGetLastError();
}
hipError_t launch_adamw(const AdamList& L, int chunks, const AdamConst& c, const AdamClock& clock, const float* scale,
                        hipStream_t s) {
  if (clock.step_at || clock.lr_at)
    hipLaunchKernelGGL((k_adamw<true>), dim3(chunks), dim3(kThreads), 0, s, L, c, clock, scale);
  else
    hipLaunchKernelGGL((k_adamw<false>), dim3(chunks), dim3(kThreads), 0, s, L, c, clock, scale);
  return hipGetLastError();
}

}  // namespace muon
