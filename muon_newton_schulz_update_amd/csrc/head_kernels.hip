// Softmax cross entropy of a language-model head, z = H W^T, with its
// gradient. The loss alone stores no logits; with gradients a piece of tokens
// keeps one exponential a logit, in the operands' size.
//
//   compact    the valid tokens (target != ignore_index) in order; ignored
//              ones are never read, so what their rows hold does not matter
//   pack       the piece's hidden rows, gathered, zero-padded, in panels (not
//              for the loss alone of up to 64 tokens: the logits' launch lists
//              them and reads their rows itself)
//   logits     z by tiles; per token and tile the largest logit m and the sum
//              of exp(z - m) over the tile without the target's term (of
//              differences, which are as good as the logits however large these
//              are); with gradients also the exponentials themselves (times the
//              soft cap's slope at their logit, where it is still in 32 bits), in
//              16 bits (10 bits of mantissa, 6 of exponent, no sign) or 32
//   merge      per token, over tiles: t = the largest m, or the target's logit
//              if that is larger, L = sum of exp(m - t) times the tile's sum,
//              the target's e = exp(z - t), loss = log1p(L / e); the
//              target's own gradient is -g L / (L + e), which loses nothing
//              when the model is sure of the target
//   dlogits    p - [v = t] (times the token's own factor) in the operands' type,
//              over the exponentials; a factor common to all tokens waits for
//              the 32-bit sums
//   dhidden    dz W, in parts of the vocabulary where tiles are few, then a
//              sum of the parts written to the tokens' rows, with what the
//              target's own gradient lost in its rounding to 16 bits times the
//              target's row: that one term is most of a token's gradient
//   dweight    dz^T H, in parts of the tokens where tiles are few, with the same
//              remainders, summed over parts and pieces in 32 bits
//
// The products are in head_gemm.hip. A logit's gradient of 16-bit inputs is
// rounded twice: as its kept exponential (an eighth of bf16's rounding, chosen so
// that a logit takes 2 bytes) and as an operand of the 16-bit matrix cores. The
// target's loses neither: its 32-bit value is in the product's operand and the
// remainder.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "head_device.hpp"
#include "train.hpp"

namespace muon {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

template <typename T> __device__ __forceinline__ float ld(const T* p, int64_t i);
template <> __device__ __forceinline__ float ld<float>(const float* p, int64_t i) { return p[i]; }
template <> __device__ __forceinline__ float ld<u16>(const u16* p, int64_t i) { return bf2f(p[i]); }
template <typename T> __device__ __forceinline__ T to(float x);
template <> __device__ __forceinline__ float to<float>(float x) { return x; }
template <> __device__ __forceinline__ u16 to<u16>(float x) { return f2bf(x); }

// Without gradients: whether the merge kernel's only block sums a reduced
// loss; a kernel of its own does otherwise. (With gradients a block of their
// launch does. A last-block ticket in the merge kernel cost 30 us for 8192
// tokens: its release writes back every L2's share of the exponentials.)
__host__ __device__ inline bool total_in_merge(const HeadArgs& a) {
  return !a.per_token && a.last && a.n <= kPanelRows;
}
// ---------------------------------------------------------------------------
// Compaction of the valid tokens. Up to kPackScan tokens every pack block
// scans the targets itself (a kernel of its own costs about 5 us more; for
// 8192 tokens the scans would take 27 us longer than the rows, that kernel 5);
// longer lists are scanned by one block beforehand, 8192 tokens at a time (6 us,
// 16384 tokens 11, bound by latency). A per-token loss of an ignored token is 0.
// ---------------------------------------------------------------------------
constexpr int kPackScan = 2048;

// Scans tokens [i0, i0 + 8 THREADS): thread t has tokens i0 + e THREADS + t,
// their targets g[e] and, where valid, their places at[e] among the valid ones
// (-1 elsewhere); returns how many there are. Loads and, through the places,
// stores are coalesced.
template <int THREADS>
__device__ __forceinline__ int scan_targets(const void* targets, int bytes, int64_t ignore, int i0, int n,
                                            int64_t (&g)[8], int (&at)[8], int* counts) {
  constexpr int W = THREADS / 64;
  const int t = threadIdx.x, w = t >> 6, lane = t & 63;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = i0 + e * THREADS + t;
    g[e] = i < n ? target_at(targets, bytes, i) : ignore;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint64_t m = __ballot(g[e] != ignore);
    at[e] = g[e] != ignore ? __popcll(m & ((1ull << lane) - 1)) : -1;
    if (lane == 0) counts[e * W + w] = __popcll(m);
  }
  __syncthreads();
  // every wave scans the 8 W counts by itself, PER neighbours to a lane (a
  // serial sum of them took 4 us of 9.5 for 8192 tokens)
  constexpr int PER = 8 * W > 64 ? 8 * W / 64 : 1;
  int c[PER], own = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    c[j] = lane * PER + j < 8 * W ? counts[lane * PER + j] : 0;
    own += c[j];
  }
  int upto = own;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int x = __shfl_up(upto, o);
    if (lane >= o) upto += x;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = __builtin_amdgcn_readfirstlane(e * W + w), from = k / PER;
    int before = __builtin_amdgcn_readlane(upto - own, from);
#pragma unroll
    for (int j = 0; j + 1 < PER; ++j)
      if (j < k % PER) before += __builtin_amdgcn_readlane(c[j], from);
    if (at[e] >= 0) at[e] += before;
  }
  const int all = __builtin_amdgcn_readlane(upto, 63);
  __syncthreads();
  return all;
}

__global__ __launch_bounds__(1024) void k_compact(HeadArgs a) {
  __shared__ int counts[8 * 16];
  int base = 0;
  for (int i0 = 0; i0 < a.n; i0 += 8192) {
    int64_t g[8];
    int at[8];
    const int all = scan_targets<1024>(a.targets, a.target_bytes, a.ignore, i0, a.n, g, at, counts);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + e * 1024 + (int)threadIdx.x;
      if (at[e] >= 0) {
        a.idx[base + at[e]] = i;
        a.tgt[base + at[e]] = checked_target(a, g[e]);
      } else if (a.per_token && i < a.n) {
        a.loss[i] = 0.f;
      }
    }
    base += all;
  }
  if (threadIdx.x == 0) a.count[0] = base;
}

// 16 bytes of a row from column c, zero past its d columns (one load where
// whole, aligned or not).
template <typename T>
__device__ __forceinline__ u32x4_t load_chunk(const T* row, int c, int d) {
  constexpr int CH = 16 / (int)sizeof(T);
  u32x4_t q;
  if (c + CH <= d) {
    __builtin_memcpy(&q, row + c, 16);
  } else {
    T x[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) x[e] = c + e < d ? row[c + e] : T(0);
    __builtin_memcpy(&q, x, 16);
  }
  return q;
}

// Rows r0.. of a weight that the products cannot load as it is, to the padded
// copy, in the same shape of block (blocks past the rows' in the same launch).
template <typename T>
__device__ __forceinline__ void pack_weight(const HeadArgs& a, int r0) {
  constexpr int CH = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 63, c = (blockIdx.y * 8 + (lane & 7)) * CH;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = r0 + i * 32 + (threadIdx.x >> 6) * 8 + (lane >> 3);
    if (r >= a.v) continue;
    const T* src = (const T*)a.w_src + r * a.ld_src;
    *(u32x4_t*)((T*)a.w + r * a.ld_w + c) = load_chunk(src, c, a.d);
  }
}

// Gathered rows to panels: a wave takes 8 rows x 8 chunks at a time, so that
// it reads and writes whole 128-byte lines; rows past the valid ones, up to a
// whole panel (a stage of dW), become zero. One block per 64 rows and 8 chunks.
// Bound by the two trips to memory (8192 x 768: 25 MB in 8 us).
template <typename T>
__global__ __launch_bounds__(256) void k_pack(HeadArgs a, int scan, int row_blocks) {
  constexpr int CH = 16 / (int)sizeof(T);
  __shared__ int list[kPanelRows], counts[8 * 4];
  if (blockIdx.x >= row_blocks) {
    pack_weight<T>(a, ((int)blockIdx.x - row_blocks) * kPanelRows);
    return;
  }
  const int r0 = blockIdx.x * kPanelRows;
  int rows;
  if (scan) {
    const bool lists = blockIdx.y == 0 && blockIdx.x == 0;   // this block writes them
    int64_t g[8];
    int at[8];
    rows = scan_targets<256>(a.targets, a.target_bytes, a.ignore, 0, a.n, g, at, counts);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = e * 256 + (int)threadIdx.x;
      if (at[e] >= 0) {
        if (at[e] >= r0 && at[e] < r0 + kPanelRows) list[at[e] - r0] = i;
        if (lists) {
          a.idx[at[e]] = i;
          a.tgt[at[e]] = checked_target(a, g[e]);
        }
      } else if (lists && a.per_token && i < a.n) {
        a.loss[i] = 0.f;
      }
    }
    if (lists && threadIdx.x == 0) a.count[0] = rows;
  } else {
    rows = piece_rows(a);
    if (threadIdx.x < kPanelRows && r0 + (int)threadIdx.x < rows) list[threadIdx.x] = a.idx[a.row0 + r0 + threadIdx.x];
  }
  if (r0 >= rows) return;
  __syncthreads();
  const int lane = threadIdx.x & 63, ch = blockIdx.y * 8 + (lane & 7), c = ch * CH;
  uint8_t* dst = (uint8_t*)a.hp + (((int64_t)blockIdx.x * (a.dp / CH) + ch) << 10);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int rr = i * 32 + (threadIdx.x >> 6) * 8 + (lane >> 3);
    u32x4_t q = {0, 0, 0, 0};
    if (r0 + rr < rows) q = load_chunk((const T*)a.h + (int64_t)list[rr] * a.ld_h, c, a.d);
    *(u32x4_t*)(dst + rr * 16) = q;
  }
}

// exp(x - y): what an exponential of reference x counts in one of reference y.
__device__ __forceinline__ float scaled(float x, float y) { return exp2f((x - y) * kLog2e); }

// Bound by latency: 8192 tokens of 393 tiles (26 MB) 12 us.
// 64 tokens per block, 16 threads per token: each goes over every sixteenth
// tile with a running reference and sum, then the first adds the sixteen in
// order. (One thread per token, two dependent loads a tile, took 190 us for
// 393 tiles whatever the number of tokens.)
constexpr int kMergeParts = 16;
__device__ __forceinline__ void merge_tiles(const HeadArgs& a, int r, int rows, int part, int parts, float& top,
                                            float& others) {
  top = kRefFloor;
  others = 0.f;
  if (r >= rows) return;
#pragma unroll 4
  for (int t = part; t < a.n_vt; t += parts) {
    const float k = a.tmax[(int64_t)t * a.piece + r], x = a.tsum[(int64_t)t * a.piece + r], m = fmaxf(top, k);
    others = others * scaled(top, m) + x * scaled(k, m);
    top = m;
  }
}
template <int PARTS>
__device__ __forceinline__ void merge_parts(const float (*tops)[64], const float (*sums)[64], int lane, float& top,
                                            float& others) {
#pragma unroll
  for (int p = 1; p < PARTS; ++p) top = fmaxf(top, tops[p][lane]);
  others = 0.f;
#pragma unroll
  for (int p = 0; p < PARTS; ++p) others += sums[p][lane] * scaled(tops[p][lane], top);
}
__device__ __forceinline__ float4 merge_token(const HeadArgs& a, int grad, int r, float top, float others,
                                              float& loss) {
  const int tg = a.tgt[a.row0 + r];
  float4 rs = {top, 0.f, 0.f, 0.f};
  if (tg < 0) {
    loss = __uint_as_float(0x7FC00000u);   // a target outside the vocabulary
    return rs;
  }
  const float z = a.zt[r], t = fmaxf(top, z);   // no tile's reference covers the target
  others *= scaled(top, t);
  const float e = scaled(z, t);
  loss = z - t > -40.f ? log1pf(others / e) : logf(others + e) - (z - t);
  if (grad) {
    rs.x = t;
    rs.y = (a.grad_out && a.per_token ? a.grad_out[a.idx[a.row0 + r]] : 1.f) / (others + e);
    rs.z = -rs.y * others;
    if (a.softcap > 0.f) rs.z *= a.zf[r];
    if (a.half) rs.w = rs.z - bf2f(f2bf(rs.z));
  }
  return rs;
}
__device__ __forceinline__ void store_loss(const HeadArgs& a, int r, float loss) {
  if (a.per_token) a.loss[a.idx[a.row0 + r]] = loss;
  else a.lossc[a.row0 + r] = loss;
}

__global__ __launch_bounds__(256) void k_total(HeadArgs a) {
  __shared__ double sh[4];
  total_loss<256>(a, sh);
}

__global__ __launch_bounds__(1024) void k_merge(HeadArgs a, int grad) {
  __shared__ float tops[kMergeParts][64], sums[kMergeParts][64];
  __shared__ double sh[16];
  const int rows = piece_rows(a), lane = threadIdx.x & 63, part = threadIdx.x >> 6, r = blockIdx.x * 64 + lane;
  float top, others;
  if (a.rows_max <= kMergeParts) {
    // few tokens: a wave for each, its lanes over the tiles
    merge_tiles(a, part, rows, lane, 64, top, others);
    float all = top;
#pragma unroll
    for (int o = 32; o; o >>= 1) all = fmaxf(all, __shfl_xor(all, o));
    others *= scaled(top, all);
#pragma unroll
    for (int o = 32; o; o >>= 1) others += __shfl_xor(others, o);
    if (lane == 0 && part < rows) {
      float loss;
      const float4 rs = merge_token(a, grad, part, all, others, loss);
      if (grad) a.rs[part] = rs;
      store_loss(a, part, loss);
    }
  } else {
    merge_tiles(a, r, rows, part, kMergeParts, top, others);
    tops[part][lane] = top;
    sums[part][lane] = others;
    __syncthreads();
    if (part == 0 && r < rows) {
      merge_parts<kMergeParts>(tops, sums, lane, top, others);
      float loss;
      const float4 rs = merge_token(a, grad, r, top, others, loss);
      if (grad) a.rs[r] = rs;
      store_loss(a, r, loss);
    }
  }
  if (grad || !total_in_merge(a)) return;
  __syncthreads();
  total_loss<1024>(a, sh);
}

// Exponentials to the logits' gradient, in place, in panel order: a thread
// keeps its token and goes over chunks, so a wave's accesses are whole
// kilobytes. Rows past the valid ones (up to a whole panel, a stage of dW) and
// columns past the vocabulary (a stage of dH) become zero. Bound by HBM: a
// read and a write of every exponential (8192 x 50304 in 16 bits 300 us, 5.5
// TB/s). The vocabulary is taken from its end, which the logits' launch wrote
// last and the last-level cache still has, to its start, where the weight's
// gradient begins (from the start 320 us). With few tiles (merged = 0) every
// block merges its tokens' statistics itself, which costs less than a kernel.
constexpr int kFuseTiles = 64;
template <typename T>
__global__ __launch_bounds__(256) void k_dlogits(HeadArgs a, int merged, int block_chunks) {
  constexpr int CH = 16 / (int)sizeof(T);
  __shared__ float tops[4][64], sums[4][64];
  __shared__ float4 merged_rs[64];
  const int rows = piece_rows(a), r0 = blockIdx.x * kPanelRows;
  if (r0 >= rows) return;
  const int lane = threadIdx.x & 63, r = r0 + lane;
  const int tg = r < rows ? a.tgt[a.row0 + r] : -1;
  const bool real = tg >= 0;
  float4 rs = {0.f, 0.f, 0.f, 0.f};
  if (merged) {
    if (real) rs = a.rs[r];
  } else {
    const int part = threadIdx.x >> 6;
    float top, others;
    merge_tiles(a, r, rows, part, 4, top, others);
    tops[part][lane] = top;
    sums[part][lane] = others;
    __syncthreads();
    if (part == 0 && r < rows) {
      merge_parts<4>(tops, sums, lane, top, others);
      float loss;
      rs = merge_token(a, 1, r, top, others, loss);
      merged_rs[lane] = rs;
      if (blockIdx.y == 0) {
        store_loss(a, r, loss);
        a.rs[r] = rs;
      }
    }
    __syncthreads();
    if (real) rs = merged_rs[lane];
  }
  const int last = a.vp / CH, g = gridDim.y - 1 - blockIdx.y, c1 = min((g + 1) * block_chunks, last);
  uint8_t* base = (uint8_t*)a.e + ((int64_t)blockIdx.x * last << 10) + (threadIdx.x & 63) * 16;
#pragma unroll 4
  for (int c = g * block_chunks + (threadIdx.x >> 6); c < c1; c += 4) {
    uint8_t* p = base + ((int64_t)c << 10);
    const int v = c * CH;
    float x[CH];
    if (real && v < a.v) {
      const float f = rs.y * scaled(a.tmax[(int64_t)(v / a.vtile) * a.piece + r], rs.x);
      if constexpr (sizeof(T) == 2) {
        const u32x4_t q = *(const u32x4_t*)p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = __uint_as_float(((q[e] & 0xFFFFu) + kCodeBase) << 13);
          x[2 * e + 1] = __uint_as_float(((q[e] >> 16) + kCodeBase) << 13);
        }
      } else {
        const f32x4_t q = *(const f32x4_t*)p;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = q[e];
      }
#pragma unroll
      for (int e = 0; e < CH; ++e) x[e] *= f;
      if (v + CH > a.v)
#pragma unroll
        for (int e = 0; e < CH; ++e)
          if (v + e >= a.v) x[e] = 0.f;
      if (tg >= v && tg < v + CH)
#pragma unroll
        for (int e = 0; e < CH; ++e)
          if (v + e == tg) x[e] = rs.z;
    } else {
#pragma unroll
      for (int e = 0; e < CH; ++e) x[e] = 0.f;
    }
    if constexpr (sizeof(T) == 2) {
      u32x4_t q;
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
      *(u32x4_t*)p = q;
    } else {
      *(f32x4_t*)p = (f32x4_t){x[0], x[1], x[2], x[3]};
    }
  }
}

// Four results, scaled and rounded: one store, aligned or not, or the `left`
// columns of a row's end.
template <typename T>
__device__ __forceinline__ void store4(T* dst, f32x4_t x, float g, int left) {
  if (left >= 4) {
    if constexpr (sizeof(T) == 2) {
      const u32x2_t y = {pack_bf16(x[0] * g, x[1] * g), pack_bf16(x[2] * g, x[3] * g)};
      __builtin_memcpy(dst, &y, 8);
    } else {
      const f32x4_t y = x * g;
      __builtin_memcpy(dst, &y, 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) dst[e] = to<T>(x[e] * g);
  }
}
// threads that share the parts of one sum
__host__ __device__ inline int share_of(int parts) { return parts >= 32 ? 8 : parts >= 16 ? 4 : parts >= 8 ? 2 : 1; }

// One group of four columns of a sum of `parts` partial sums, `all` groups
// apart: this thread's share, then the shares of the block joined in order.
// Only the first share's threads return true.
__device__ __forceinline__ bool sum_parts(const float* part, int parts, int64_t at, int64_t all, int64_t stride, f32x4_t* sh,
                                          f32x4_t& x) {
  const int shares = share_of(parts), width = 256 / shares, share = threadIdx.x / width;
  x = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  if (at < all) {
#pragma unroll 8
    for (int q = share; q < parts; q += shares) x += *(const f32x4_t*)(part + (q * stride + at) * 4);
  }
  if (shares > 1) {
    sh[threadIdx.x] = x;
    __syncthreads();
    if (share == 0)
      for (int p = 1; p < shares; ++p) x += sh[p * width + threadIdx.x];
  }
  return share == 0 && at < all;
}

// The gradients' last steps, three kinds of blocks: sums of dH's parts to the
// tokens' rows (a thread has four columns), zeros to the ignored tokens' rows
// with the first piece (a wave has kZeroTokens tokens), sums of dW's parts and
// of the pieces before. Bound by HBM: 8192 x 768 with 50304 rows of weight 22 us.
constexpr int kZeroTokens = 16;
template <typename T>
__global__ __launch_bounds__(256) void k_gradients_out(HeadArgs a, int sums, int zeros) {
  __shared__ f32x4_t sh[256];
  const int groups = a.dp / 4, lane = threadIdx.x & 63;
  int block = blockIdx.x;
  f32x4_t x;
  if (block < sums) {
    const int width = 256 / share_of(a.split);
    const int64_t at = (int64_t)block * width + threadIdx.x % width;
    if (!sum_parts(a.part, a.split, at, (int64_t)piece_rows(a) * groups, (int64_t)a.piece * groups, sh, x)) return;
    const int r = (int)(at / groups), c = (int)(at - (int64_t)r * groups) * 4;
    if (c >= a.d) return;
    const float rest = a.rs[r].w;
    if (rest != 0.f) {
      const T* target_row = (const T*)a.w + (int64_t)a.tgt[a.row0 + r] * a.ld_w;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.d) x[e] = fmaf(rest, ld<T>(target_row, c + e), x[e]);
    }
    store4((T*)a.dh + (int64_t)a.idx[a.row0 + r] * a.ld_dh + c, x, common_factor(a), a.d - c);
    return;
  }
  block -= sums;
  if (block < zeros) {
    const int64_t t0 = ((int64_t)block * 4 + (threadIdx.x >> 6)) * kZeroTokens;
    const bool mine = lane < kZeroTokens && t0 + lane < a.n && target_at(a.targets, a.target_bytes, t0 + lane) == a.ignore;
    for (uint64_t todo = __ballot(mine); todo; todo &= todo - 1) {
      T* row = (T*)a.dh + (t0 + __builtin_ctzll(todo)) * a.ld_dh;
      for (int c = lane; c < a.d; c += 64) row[c] = T(0);
    }
    return;
  }
  block -= zeros;
  const int width = 256 / share_of(a.wsplit);
  const int64_t at = (int64_t)block * width + threadIdx.x % width, all = (int64_t)a.v * groups;
  if (!sum_parts(a.wpart, a.wsplit, at, all, all, sh, x)) return;
  const int row = (int)(at / groups), c = (int)(at - (int64_t)row * groups) * 4;
  if (c >= a.d) return;
  if (a.dwacc) {
    f32x4_t* p = (f32x4_t*)(a.dwacc + at * 4);
    if (!a.first) x += *p;
    if (!a.last) {
      *p = x;
      return;
    }
  }
  store4((T*)a.dw + (int64_t)row * a.ld_dw + c, x, common_factor(a), a.d - c);
}

inline unsigned cdiv(int64_t a, int64_t b) { return (unsigned)((a + b - 1) / b); }
// whether the rows' kernel scans the targets: few tokens, all in one piece
inline bool pack_scans(const HeadArgs& a) { return a.n <= kPackScan && a.n <= a.piece; }
inline unsigned panels(const HeadArgs& a) { return a.rows_max > 0 ? cdiv(a.rows_max, kPanelRows) : 1; }

}  // namespace

#define BY_TYPE(dt, f, ...)                                                                                   \
  do {                                                                                                        \
    if ((dt) == MUON_BF16) hipLaunchKernelGGL((f<u16>), __VA_ARGS__);                                         \
    else hipLaunchKernelGGL((f<float>), __VA_ARGS__);                                                         \
    return hipGetLastError();                                                                                 \
  } while (0)

hipError_t launch_head_compact(const HeadArgs& a, hipStream_t s) {
  if (pack_scans(a)) return hipSuccess;
  hipLaunchKernelGGL(k_compact, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_head_pack(const HeadArgs& a, int dt, hipStream_t s) {
  if (a.gather) return hipSuccess;
  const int scan = pack_scans(a), rows = (int)panels(a);
  const int weight = a.w_src && a.row0 == 0 ? (int)cdiv(a.v, kPanelRows) : 0;
  BY_TYPE(dt, k_pack, dim3(rows + weight, a.dp / (dt == MUON_BF16 ? 64 : 32)), dim3(256), 0, s, a, scan, rows);
}
hipError_t launch_head_merge(const HeadArgs& a, int grad, hipStream_t s) {
  if (grad && a.n_vt <= kFuseTiles) return hipSuccess;   // with the logits' gradient
  hipLaunchKernelGGL(k_merge, dim3(panels(a)), dim3(64 * kMergeParts), 0, s, a, grad);
  if (!grad && a.last && !a.per_token && !total_in_merge(a))
    hipLaunchKernelGGL(k_total, dim3(1), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_head_dlogits(const HeadArgs& a, int dt, hipStream_t s) {
  const int chunks = a.vp / (dt == MUON_BF16 ? 8 : 4);
  // chunks per block: 64, or 16 where that leaves CUs without four blocks
  const int per = (int64_t)cdiv(chunks, 64) * panels(a) < 1024 ? 16 : 64;
  BY_TYPE(dt, k_dlogits, dim3(panels(a), cdiv(chunks, per)), dim3(256), 0, s, a, (int)(a.n_vt > kFuseTiles), per);
}
hipError_t launch_head_gradients_out(const HeadArgs& a, int dt, hipStream_t s) {
  auto blocks = [&](int64_t rows, int parts) { return (int)cdiv(rows * (a.dp / 4), 256 / share_of(parts)); };
  const int sums = a.dh && a.split > 1 ? blocks(a.rows_max, a.split) : 0;
  const int zeros = a.dh && a.row0 == 0 ? (int)cdiv(a.n, 4 * kZeroTokens) : 0;
  const int weight = a.wsplit > 1 ? blocks(a.v, a.wsplit) : 0;
  if (sums + zeros + weight == 0) return hipSuccess;
  BY_TYPE(dt, k_gradients_out, dim3(sums + zeros + weight), dim3(256), 0, s, a, sums, zeros);
}

}  // namespace muon
