// Log probabilities of given tokens under a language-model head, the
// distribution's entropy and its likeliest tokens, from the statistics that the
// logits' launch (head_gemm.hip) leaves of each token and tile: the largest logit
// m, S = sum exp(z - m) and E = sum exp(z - m) log2 exp(z - m), both without the
// target's term, and, for the alternatives, each lane's largest raw logit with
// its place and its second largest.
//
//   statistics    over tiles, with t the largest of all: S and E joined by
//                 exp(m - t), E shifted by (m - t) S, the target's term added;
//                 log p = -log1p(others / target's), H = log S - E log(2) / S
//   alternatives  a lane's set of logits is a candidate by its largest. The
//                 top + kSpare best sets by (logit, lowest token) hold the top
//                 alternatives, each as its set's largest unless a set has two
//                 of them, which its second largest tells: then all of the set
//                 are candidates. Candidates are summed again in 64 bits (from
//                 16-bit inputs every product is exact) and sorted. What is
//                 outside the spare sets could only be in front by an error
//                 of the 32-bit sums that passes over kSpare others.
//   factors       for the gradient, dz = -p (b + g log p) with g the entropy's
//                 gradient and b = g_logprob + g H; the target's is
//                 g_logprob (1 - p) - g p (log p + H)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "head_device.hpp"
#include "train.hpp"

namespace muon {
namespace {

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kSpare = 8;          // candidates beyond the asked-for alternatives
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kNan = __builtin_nanf("");

// exp(x - y) with its exponent, base 2; no smaller than what a product with it
// still takes for nothing (an exponent of minus infinity times 0 would be NaN).
__device__ __forceinline__ float scaled_log2(float x, float y) { return __builtin_elementwise_maximum((x - y) * kLog2e, -1000.f); }

struct Stat {
  float top, sum, ent;
};
__device__ __forceinline__ Stat joined(const Stat& a, const Stat& b) {
  const float t = fmaxf(a.top, b.top), x = scaled_log2(a.top, t), y = scaled_log2(b.top, t);
  const float ex = exp2f(x), ey = exp2f(y);
  return Stat{t, a.sum * ex + b.sum * ey, ex * (a.ent + a.sum * x) + ey * (b.ent + b.sum * y)};
}
__device__ __forceinline__ Stat tiles_stat(const HeadArgs& a, int r, int part, int parts) {
  Stat s = {kRefFloor, 0.f, 0.f};
#pragma unroll 4
  for (int t = part; t < a.n_vt; t += parts) {
    const int64_t at = (int64_t)t * a.piece + r;
    s = joined(s, Stat{a.tmax[at], a.tsum[at], a.tent[at]});
  }
  return s;
}

// {reference, log of the sum over it, entropy, log probability}
__device__ __forceinline__ float4 token_stat(const HeadArgs& a, int r, Stat s) {
  const int tg = a.tgt[a.row0 + r];
  const float z = tg >= 0 ? a.zt[r] : kRefFloor;
  const float t = fmaxf(s.top, z), x = scaled_log2(s.top, t);
  const float f = exp2f(x), others = s.sum * f;
  float all = others, ent = f * (s.ent + s.sum * x), log_sum = logf(others), logp = kNan;
  if (tg >= 0) {
    const float y = scaled_log2(z, t), e = exp2f(y);
    all += e;
    ent += e * y;
    log_sum = z == t ? log1pf(others) : logf(all);
    logp = z - t > -40.f ? -log1pf(others / e) : (z - t) - logf(all);
  }
  if (!(t > kRefFloor)) log_sum = kNan;        // no logit above minus infinity, or none that is a number
  if (log_sum != log_sum) logp = kNan;
  return {t, log_sum, log_sum - kLn2 * ent / all, logp};
}
__device__ __forceinline__ void put_stat(const HeadArgs& a, int r, const float4& s) {
  const int i = a.idx[a.row0 + r];
  a.rs[r] = s;
  a.loss[i] = s.w;
  if (a.entropy) a.entropy[i] = s.z;
  if (a.stats) a.stats[i] = s;
}

// Sorting over a wave, lane 0 first: larger values, then smaller tokens.
template <typename F>
struct Ranked {
  F z;
  int token;
};
template <typename F>
__device__ __forceinline__ bool before(const Ranked<F>& a, const Ranked<F>& b) {
  return a.z > b.z || (a.z == b.z && a.token < b.token);
}
template <typename F>
__device__ __forceinline__ Ranked<F> swapped(const Ranked<F>& x, int mask) {
  return {__shfl_xor(x.z, mask), __shfl_xor(x.token, mask)};
}
template <typename F>
__device__ __forceinline__ void keep_order(Ranked<F>& x, int lane, int mask, bool falling) {
  const Ranked<F> y = swapped(x, mask);
  const bool low = (lane & mask) == 0;
  if (before(y, x) == (low == falling)) x = y;
}
template <typename F>
__device__ __forceinline__ void sort_wave(Ranked<F>& x, int lane) {
#pragma unroll 1
  for (int size = 2; size <= 64; size *= 2)
#pragma unroll 1
    for (int mask = size / 2; mask; mask /= 2) keep_order(x, lane, mask, size == 64 || (lane & size) == 0);
}
// The 64 first of two sorted waves of 64, sorted.
template <typename F>
__device__ __forceinline__ void merge_wave(Ranked<F>& x, const Ranked<F>& sorted, int lane) {
  const Ranked<F> y = {__shfl(sorted.z, 63 - lane), __shfl(sorted.token, 63 - lane)};
  if (before(y, x)) x = y;
#pragma unroll 1
  for (int mask = 32; mask; mask /= 2) keep_order(x, lane, mask, true);
}

// The logit of a token and a word in 64 bits, the wave's lanes over the width.
template <typename T>
__device__ __forceinline__ double fine_logit(const T* h, const T* w, int d, int lane) {
  constexpr int CH = 16 / (int)sizeof(T);
  double s = 0;
  for (int c = lane * CH; c < d; c += 64 * CH) {
    if (c + CH <= d) {
      T x[CH], y[CH];
      __builtin_memcpy(x, h + c, 16);
      __builtin_memcpy(y, w + c, 16);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        if constexpr (sizeof(T) == 2) s = fma((double)bf2f(x[e]), (double)bf2f(y[e]), s);
        else s = fma((double)x[e], (double)y[e], s);
      }
    } else {
      for (int e = c; e < d; ++e) {
        if constexpr (sizeof(T) == 2) s = fma((double)bf2f(h[e]), (double)bf2f(w[e]), s);
        else s = fma((double)h[e], (double)w[e], s);
      }
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  return s;
}

constexpr int kNoToken = 0x7FFFFFFF;
// A set's second largest logit, or a little more (its last bits are a place).
__device__ __forceinline__ float second_of(uint2 b) {
  const uint32_t up = b.y >> 31 ? b.y & ~63u : b.y | 63u;
  return __uint_as_float(up > 0x7F800000u && up < 0x80000000u ? 0x7F800000u : up);
}

// One token's alternatives, by one wave.
template <typename T>
__device__ __forceinline__ void alternatives(const HeadArgs& a, int r, const float4& stat, int lane) {
  const int i = a.idx[a.row0 + r], target = a.tgt[a.row0 + r], top = a.top;
  float* logps = a.top_logprobs + (int64_t)i * top;
  int64_t* tokens = a.top_tokens + (int64_t)i * top;
  if (stat.y != stat.y) {
    if (lane < top) {
      logps[lane] = kNan;
      tokens[lane] = -1;
    }
    return;
  }
  const int per = a.vtile / a.sets, all = a.n_vt * a.sets;
  const float none = -__builtin_inff();
  auto entry = [&](int s, Ranked<float>& x, float& bound) {
    // (sets past the last, and of no logit, rank behind every other)
    x = {none, kNoToken};
    bound = none;
    if (s >= all) return;
    const int tile = s / a.sets, set = s % a.sets;
    const uint2 b = a.best[((int64_t)tile * a.piece + r) * a.sets + set];
    const float z = __uint_as_float(b.x);
    if (!(z > none)) return;
    x = {z, tile * a.vtile + set_column(set, a.sets, b.y & 63)};
    bound = second_of(b);
  };
  // the 64 best sets
  Ranked<float> best = {none, kNoToken};
  float bounds_of = none;
  for (int s0 = 0; s0 < all; s0 += 64) {
    Ranked<float> x;
    float bound;
    entry(s0 + lane, x, bound);
    sort_wave(x, lane);
    if (s0 == 0) best = x;
    else merge_wave(best, x, lane);
  }
  // the second largest of each, and which sets have two among the best
  const float kth = __shfl(best.z, top - 1);
  if (best.token != kNoToken) {
    const int tile = best.token / a.vtile, col = best.token % a.vtile;
    const int set = (a.sets == 4 ? (col >> 5) * 2 : 0) + ((col >> 2) & 1);
    const uint2 b = a.best[((int64_t)tile * a.piece + r) * a.sets + set];
    bounds_of = second_of(b);
  }
  const int count = top + kSpare;
  const uint64_t whole = __ballot(lane < count && bounds_of > none && bounds_of >= kth - fabsf(kth) * 0x1p-18f);
  if (lane >= count) best.token = kNoToken;
  if (lane == 63 && target >= 0 && a.zt[r] > none) best.token = target;       // (its set leaves it out)
  const T* h = (const T*)a.h + (int64_t)i * a.ld_h;
  const T* w = (const T*)(a.w_src ? a.w_src : a.w);
  const int64_t ld = a.w_src ? a.ld_src : a.ld_w;
  auto fine = [&](int token) {
    Ranked<double> x = {-__builtin_inf(), kNoToken};
    for (uint64_t todo = __ballot(token != kNoToken); todo; todo &= todo - 1) {
      const int from = __builtin_ctzll(todo), word = __shfl(token, from);
      const double z = fine_logit(h, w + (int64_t)word * ld, a.d, lane);
      if (lane == from) x = {z, word};
    }
    sort_wave(x, lane);
    return x;
  };
  const int firsts = best.token;
  Ranked<double> found = fine(firsts);
  for (uint64_t todo = whole; todo; todo &= todo - 1) {
    const int word = __shfl(firsts, __builtin_ctzll(todo));
    const int tile = word / a.vtile, col = word % a.vtile;
    const int set = (a.sets == 4 ? (col >> 5) * 2 : 0) + ((col >> 2) & 1);
    int token = kNoToken;
    if (lane < per) token = tile * a.vtile + set_column(set, a.sets, lane);
    if (token >= a.v || token == word || token == target) token = kNoToken;
    merge_wave(found, fine(token), lane);
  }
  if (lane >= top) return;
  const bool there = found.token != kNoToken && found.z > -__builtin_inf();
  double logp = (found.z - stat.x) - stat.y;
  if (a.softcap > 0.f) {
    const double c = a.softcap, x = tanh(found.z / c) * c;
    logp = (x - stat.x) - stat.y;
  }
  logps[lane] = !there ? none : found.token == target ? stat.w : (float)logp;
  tokens[lane] = there ? found.token : -1;
}

// Blocks past the tokens': zeros for the ignored ones, with the first piece.
__device__ __forceinline__ void clear_ignored(const HeadArgs& a, int64_t from) {
  for (int64_t i = from + threadIdx.x; i < from + 1024 && i < a.n; i += blockDim.x) {
    if (target_at(a.targets, a.target_bytes, i) != a.ignore) continue;
    if (a.entropy) a.entropy[i] = 0.f;
    if (a.stats) a.stats[i] = float4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < a.top; ++k) {
      a.top_logprobs[i * a.top + k] = 0.f;
      a.top_tokens[i * a.top + k] = -1;
    }
  }
}

// 64 tokens a block, a token's tiles over 16 threads.
constexpr int kParts = 16;
__global__ __launch_bounds__(1024) void k_logprob_stats(HeadArgs a, int blocks) {
  __shared__ Stat sh[kParts][64];
  if ((int)blockIdx.x >= blocks) {
    clear_ignored(a, ((int64_t)blockIdx.x - blocks) * 1024);
    return;
  }
  const int rows = piece_rows(a), lane = threadIdx.x & 63, part = threadIdx.x >> 6, r = blockIdx.x * 64 + lane;
  if (r < rows) sh[part][lane] = tiles_stat(a, r, part, kParts);
  __syncthreads();
  if (part != 0 || r >= rows) return;
  Stat s = sh[0][lane];
#pragma unroll
  for (int p = 1; p < kParts; ++p) s = joined(s, sh[p][lane]);
  put_stat(a, r, token_stat(a, r, s));
}

// A wave a token; neighbouring tokens, whose statistics share lines, on one XCD.
template <typename T>
__global__ __launch_bounds__(256) void k_alternatives(HeadArgs a) {
  const int rows = piece_rows(a), per = (gridDim.x + 7) / 8;
  const int block = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  const int r = block * 4 + (threadIdx.x >> 6);
  if (r < rows) alternatives<T>(a, r, a.rs[r], threadIdx.x & 63);
}

__global__ __launch_bounds__(256) void k_logprob_factors(HeadArgs a) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= piece_rows(a)) return;
  const int i = a.idx[a.row0 + r], tg = a.tgt[a.row0 + r];
  const float4 s = a.stats_in[i];
  const float gp = tg >= 0 && a.grad_logprobs ? a.grad_logprobs[i] : 0.f, ge = a.grad_entropy ? a.grad_entropy[i] : 0.f;
  a.ts[r] = float4{s.x, s.y, fmaf(ge, s.z, gp), ge};
  // (1 - p from log p, which keeps what a token that is nearly sure still has to learn)
  const float lp = __builtin_elementwise_maximum(s.w, -126.f / kLog2e);   // (as the other words': no infinity times 0)
  a.rs[r] = float4{0.f, 0.f, tg >= 0 ? -gp * expm1f(lp) - ge * expf(lp) * (lp + s.z) : 0.f, 0.f};
}

inline unsigned cdiv(int64_t a, int64_t b) { return (unsigned)((a + b - 1) / b); }

}  // namespace

hipError_t launch_logprobs(const HeadArgs& a, int dt, hipStream_t s) {
  const int blocks = (int)cdiv(a.rows_max, 64), clear = a.row0 == 0 ? (int)cdiv(a.n, 1024) : 0;
  hipLaunchKernelGGL(k_logprob_stats, dim3(blocks + clear), dim3(1024), 0, s, a, blocks);
  if (a.top == 0) return hipGetLastError();
  const dim3 g(cdiv(cdiv(a.rows_max, 4), 8) * 8);
  if (dt == MUON_BF16) hipLaunchKernelGGL(k_alternatives<u16>, g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_alternatives<float>, g, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_logprob_factors(const HeadArgs& a, hipStream_t s) {
  if (a.rows_max == 0) return hipSuccess;
  hipLaunchKernelGGL(k_logprob_factors, dim3(cdiv(a.rows_max, 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
