// Log probabilities of given tokens under a language-model head, the
// distribution's entropy and its likeliest tokens, from the statistics that the
// logits' launch (head_gemm.hip) leaves of each token and tile: the largest logit
// m, S = sum exp(z - m) without one of the largest and E = sum exp(z - m) log2 exp(z -
// m), both without the target's term, and, for the alternatives, each lane's largest
// raw logit with its place and its second largest.
//
//   statistics    over tiles, with t the largest of all: S and E joined by
//                 exp(m - t), E shifted by (m - t) S; then over the leading
//                 word, the target or the largest other one, whose term of 1
//                 is in no sum: log p of it = -log1p(S), H = log1p(S) - E
//                 log(2) / (1 + S), so a word that is nearly sure keeps all
//                 bits of what it is not. Its logit is summed again in 64
//                 bits, if it is the target or alternatives are asked for
//   alternatives  a lane's set of logits is a candidate by its largest. The
//                 top + kSpare best sets by (logit, lowest token) hold the top
//                 alternatives, each as its set's largest unless a set has two
//                 words as large as the (top + kSpare)-th, which its second
//                 largest tells: then all of the set are candidates. Candidates
//                 are summed again in 64 bits (from 16-bit inputs every product
//                 is exact) and sorted. What is outside could only be in front
//                 by an error of the 32-bit sums that passes over kSpare others.
//
// A block of four waves takes a token: its first reads (statistics, sets, target)
// are asked for together, the sets stay in registers, and what bounds it is that
// chain of dependent steps, most of all the candidates' rows of the weight (from
// the caches: 3000 tokens x 29 of 4 KB are 356 MB). 50304 words: one token top 8
// 14 us, 1536 tokens top 5 x 768 40, 3000 top 20 x 2048 125 (before sets had spare
// places and the leading word 64 bits 13, 37, 114; then a wave a token 16, 42, 149, and
// sorting every set instead of a threshold 88, 166, 596); statistics alone, 8192
// tokens, 17 us, of which 52 MB and the targets' 25 are a read of 12.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "head_device.hpp"
#include "train.hpp"
#include "wave.hpp"

namespace muon {
namespace {

constexpr int kSpare = 8;          // candidates beyond the asked-for alternatives
constexpr float kNan = __builtin_nanf("");

// exp(x - y) with its exponent, base 2; no smaller than what a product with it
// still takes for nothing (an exponent of minus infinity times 0 would be NaN).
__device__ __forceinline__ float scaled_log2(float x, float y) { return __builtin_elementwise_maximum((x - y) * kLog2e, -1000.f); }

// Sums over a reference, a logit of which one word is left out of `sum` (one: 1; its
// exponential is 1 and its logarithm 0): beside it nothing of the others is lost.
struct Stat {
  float top, sum, ent, one;
};
// The same over another reference t, no smaller (or next to it). The exponential of a
// difference of 16 is off by 2^-20 from the rounding of its exponent alone (one word
// or one tile may be all that others there are): what the difference, the product
// and log2(e) lose is multiplied to it.
__device__ __forceinline__ Stat over(const Stat& s, float t) {
  const float x = scaled_log2(s.top, t);
  float f = __builtin_amdgcn_exp2f(x);
  if (x > -200.f) {
    const float d = s.top - t, b = d - s.top, rest = (s.top - (d - b)) - (t + b);
    const float lost = fmaf(d, kLog2e, -x) + fmaf(rest, kLog2e, d * 1.92596299e-8f);
    f = fmaf(f, lost * kLn2, f);
  }
  const bool same = s.top == t;
  const float sum = same ? s.sum : s.sum + s.one;
  return {t, sum * f, f * (s.ent + sum * x), same ? s.one : 0.f};
}
// Sums added up over one reference, `ones` of which have a word left out.
__device__ __forceinline__ Stat settled(float t, float sum, float ent, float ones) {
  return {t, sum + fmaxf(ones - 1.f, 0.f), ent, fminf(ones, 1.f)};
}
__device__ __forceinline__ Stat joined(const Stat& a, const Stat& b) {
  const float t = fmaxf(a.top, b.top);
  const Stat x = over(a, t), y = over(b, t);
  return settled(t, x.sum + y.sum, x.ent + y.ent, x.one + y.one);
}
// Every parts-th tile's, eight at a time over their common reference.
__device__ __forceinline__ Stat tiles_stat(const HeadArgs& a, int r, int part, int parts) {
  Stat s = {kRefFloor, 0.f, 0.f, 0.f};
  for (int t0 = part; t0 < a.n_vt; t0 += 8 * parts) {
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = float4{kRefFloor, 0.f, 0.f, 0.f};
      if (t0 + k * parts < a.n_vt) x[k] = a.tstat[(int64_t)r * a.n_vt + t0 + k * parts];
    }
    float top = s.top;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, x[k].x);
    s = over(s, top);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const Stat y = over(Stat{x[k].x, x[k].y, x[k].z, x[k].w}, top);
      s.sum += y.sum;
      s.ent += y.ent;
      s.one += y.one;
    }
    s = settled(top, s.sum, s.ent, s.one);
  }
  return s;
}

// A token's place in the call and its target (-1 outside the vocabulary).
struct Token {
  int at, target;
};
__device__ __forceinline__ Token token_of(const HeadArgs& a, int r) { return {a.idx[a.row0 + r], a.tgt[a.row0 + r]}; }

// A word's logit, from its raw one in 64 bits: a 32-bit value and what its rounding
// lost. A word that the model is sure of has the largest logit by far, and a 32-bit
// sum's error of it (2^-20 and more at 16) would be all of its log probability and much
// of the entropy; the other words' average out. So the target's is taken in 64 bits,
// and the largest of the alternatives', where these are asked for.
struct Logit {
  float z, lost;
  double exact;
};
__device__ __forceinline__ Logit fine_logit(const HeadArgs& a, double raw) {
  const double c = a.softcap, y = c > 0 ? tanh(raw / c) * c : raw;
  const float z = (float)y;
  // (past 2^24 it would be more than 1, and 32-bit sums of the others as far off)
  return {z, fabsf(z) < 0x1p24f ? (float)(y - (double)z) : 0.f, y};
}
__device__ __forceinline__ Logit rough_logit(float z) { return {z, 0.f, z}; }

struct TokenStat {
  float4 of;        // {reference, log of the sum over it, entropy, log probability}
  float others;     // all but the leading word's exponentials, over that word's
  double lead;      // its logit
  bool given;       // it is the target
};
// own: the target's logit; s: the others', of which the largest one has the logit alt.
__device__ __forceinline__ TokenStat token_stat(int tg, const Logit& own, const Stat& s, const Logit& alt) {
  const bool given = tg >= 0 && own.z >= alt.z;
  const Logit& lead = given ? own : alt;
  Stat rest = over(Stat{s.top, s.sum, s.ent, 0.f}, alt.z);
  float target = 0.f, y = 0.f;
  if (given) {
    const float x = alt.lost * kLog2e, e = s.one * exp2f(x);
    rest = over(Stat{alt.z, rest.sum + e, fmaf(e, x, rest.ent), 0.f}, own.z);
  } else if (tg >= 0) {
    y = fmaf(own.lost, kLog2e, scaled_log2(own.z, alt.z));
    target = exp2f(y);
  }
  // over the leading word's logit to the last bit
  const float f = expf(-lead.lost);
  target *= f;
  const float words = rest.sum * f, others = words + target;
  const float ent = f * rest.ent + target * y - others * (lead.lost * kLog2e), sum = log1pf(others);
  float log_sum = lead.lost + sum, logp = kNan;
  if (given) logp = -sum;
  else if (tg >= 0) logp = own.z - alt.z > -40.f ? -log1pf((1.f + words) / target) : (own.z - alt.z) - log_sum;
  float entropy = sum - kLn2 * ent / (1.f + others);
  if (!(lead.z > kRefFloor)) log_sum = kNan;   // no logit above minus infinity, or none that is a number
  // (an infinite target leaves the alternatives their order)
  if (log_sum != log_sum || lead.z == __builtin_inff()) logp = entropy = kNan;
  return {{lead.z, log_sum, entropy, logp}, others, lead.exact, given};
}
// stats: what the gradient takes, whose logits are 32-bit sums all of them
__device__ __forceinline__ void put_stat(const HeadArgs& a, int i, const float4& s, const float4& stats) {
  a.loss[i] = s.w;
  if (a.entropy) a.entropy[i] = s.z;
  if (a.stats) a.stats[i] = float4{stats.x, stats.y, stats.z, s.w};
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

// Logits of a token and kGroup words in 64 bits, the wave's lanes over the width.
// (Groups of 8 hold twice as many loads in flight, but fewer tokens fit a CU:
// 3000 x top 20 x 2048 114 us, with 4 111; 1536 x top 5 38, 35.)
constexpr int kGroup = 4;
template <typename T, int G>
__device__ __forceinline__ void fine_logits(const T* h, const T* w, int64_t ld, int d, const int (&words)[G], int lane,
                                            double (&z)[G]) {
  constexpr int CH = 16 / (int)sizeof(T);
  auto value = [](T x) -> double {
    if constexpr (sizeof(T) == 2) return (double)bf2f(x);
    else return (double)x;
  };
#pragma unroll
  for (int g = 0; g < G; ++g) z[g] = 0;
  for (int c = lane * CH; c < d; c += 64 * CH) {
    T x[CH], y[G][CH];
    if (c + CH <= d) {
      __builtin_memcpy(x, h + c, 16);
#pragma unroll
      for (int g = 0; g < G; ++g) __builtin_memcpy(y[g], w + words[g] * ld + c, 16);
    } else {
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        x[e] = c + e < d ? h[c + e] : T(0);
#pragma unroll
        for (int g = 0; g < G; ++g) y[g][e] = c + e < d ? w[words[g] * ld + c + e] : T(0);
      }
    }
#pragma unroll
    for (int e = 0; e < CH; ++e) {
      const double v = value(x[e]);
#pragma unroll
      for (int g = 0; g < G; ++g) z[g] = fma(v, value(y[g][e]), z[g]);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) z[g] = lanes_sum<64>(z[g]);
}

// The caller's rows, whatever the products read.
template <typename T>
struct Operands {
  const T *h, *w;
  int64_t ld;
  __device__ __forceinline__ Operands(const HeadArgs& a, int token)
      : h((const T*)a.h + (int64_t)token * a.ld_h), w((const T*)(a.w_src ? a.w_src : a.w)), ld(a.w_src ? a.ld_src : a.ld_w) {}
};
// A token's raw target logit in 64 bits, by a wave.
template <typename T>
__device__ __forceinline__ double fine_target(const HeadArgs& a, const Token& token, int lane) {
  if (token.target < 0) return 0;
  const Operands<T> o(a, token.at);
  const int words[1] = {token.target};
  double z[1];
  fine_logits(o.h, o.w, o.ld, a.d, words, lane, z);
  return z[0];
}

constexpr int kNoToken = 0x7FFFFFFF;
constexpr float kNone = -__builtin_inff();
// A set's second largest logit, or a little more (its last bits are a place).
__device__ __forceinline__ float second_of(uint2 b) {
  const uint32_t up = b.y >> 31 ? b.y & ~63u : b.y | 63u;
  return __uint_as_float(up > 0x7F800000u && up < 0x80000000u ? 0x7F800000u : up);
}
// Whole numbers in the order of their floats (which are no NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}
// The largest number, to 20 bits (a float's 11 of mantissa), that at least `count`
// of the lanes' keys reach; 0 if there are not as many keys.
template <int K>
__device__ __forceinline__ uint32_t reached_by(const uint32_t (&key)[K], int count) {
  uint32_t least = 0;
#pragma unroll 4
  for (int bit = 31; bit >= 12; --bit) {
    const uint32_t trial = least | 1u << bit;
    int found = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) found += __popcll(__ballot(key[k] >= trial));
    if (found >= count) least = trial;
  }
  return least;
}

// Four waves work on a token.
constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kMostSets = 63;      // with the target one for each lane
struct Found {
  float z, bound;                  // a set's largest logit, and what its others do not pass
  int word;
};
struct TokenShare {
  Stat stat[kWaves];
  Found of[kWaves][64];            // each wave's sets
  int count[kWaves], total;
  double target;                   // the target's raw logit
  Found sets[64];
  double z[64];
  int word[64];
};

// A thread's statistics of a token's sets, 1024 at a time: they stay in registers
// where these are all (131072 words; fp32 and few tokens 65536).
template <int SETS>
struct Sets {
  static constexpr int kTiles = 4, kSpan = kThreads * kTiles;
  uint2 of[kTiles][SETS];
  __device__ __forceinline__ static int tile(int t0, int j) { return t0 + j * kThreads + (int)threadIdx.x; }
  __device__ __forceinline__ void load(const uint2* best, int n_vt, int t0) {
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
#pragma unroll
      for (int k = 0; k < SETS; ++k) of[j][k] = make_uint2(0xFF800000u, 0u);
      if (tile(t0, j) < n_vt) __builtin_memcpy(of[j], best + tile(t0, j) * SETS, sizeof(of[j]));
    }
  }
};

// The sets that the alternatives are in, in no order, to sh.sets, at most
// kMostSets; returns how many (the same in all threads). e: the first statistics.
template <typename T, int SETS>
__device__ __forceinline__ int candidate_sets(const HeadArgs& a, const uint2* best, Sets<SETS>& e, int wave, int lane, TokenShare& sh) {
  const int count = a.top + kSpare;
  const uint64_t below = (1ull << lane) - 1;
  constexpr int TILES = Sets<SETS>::kTiles, SPAN = Sets<SETS>::kSpan;
  // each lane's largest logit of two halves of its sets: what `count` of a wave's
  // reach is reached by as many of its sets, and by few more
  float most[2] = {kNone, kNone};
  for (int t0 = 0; t0 < a.n_vt; t0 += SPAN) {
    if (t0) e.load(best, a.n_vt, t0);
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int k = 0; k < SETS; ++k) most[k & 1] = fmaxf(most[k & 1], __uint_as_float(e.of[j][k].x));
  }
  const uint32_t halves[2] = {most[0] > kNone ? ordered(most[0]) : 0u, most[1] > kNone ? ordered(most[1]) : 0u};
  const uint32_t least = reached_by(halves, count);
  int found = 0;
  for (int t0 = 0; t0 < a.n_vt; t0 += SPAN) {
    if (a.n_vt > SPAN) e.load(best, a.n_vt, t0);
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int k = 0; k < SETS; ++k) {
        const float z = __uint_as_float(e.of[j][k].x);
        const bool in = z > kNone && ordered(z) >= least;
        const uint64_t mask = __ballot(in);
        if (mask == 0) continue;
        const int at = found + __popcll(mask & below);
        if (in && at < 64) sh.of[wave][at] = Found{z, second_of(e.of[j][k]), e.tile(t0, j) * a.vtile + set_column<T, SETS>(k, e.of[j][k].y & 63)};
        found += __popcll(mask);
      }
  }
  if (lane == 0) sh.count[wave] = found;
  __syncthreads();
  // of all waves' sets, those that `count` reach
  if (wave == 0) {
    uint32_t keys[kWaves];
    bool over = false;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      over |= sh.count[w] > 64;
      keys[w] = lane < sh.count[w] ? ordered(sh.of[w][lane].z) : 0u;
    }
    const uint32_t all_least = reached_by(keys, count);
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const bool in = keys[w] != 0 && keys[w] >= all_least;
      const uint64_t mask = __ballot(in);
      const int at = total + __popcll(mask & below);
      if (in && at < 64) sh.sets[at] = sh.of[w][lane];
      total += __popcll(mask);
    }
    if (over || total > kMostSets) {
      // more of them (equal logits, or neighbours in one lane's sets): the first
      // `count` by (logit, word), by sorting all sets 64 at a time
      auto word_of = [&](int s, uint2 b) { return s / SETS * a.vtile + set_column<T, SETS>(s % SETS, b.y & 63); };
      Ranked<float> list = {kNone, kNoToken};
      for (int s0 = 0; s0 < a.n_vt * SETS; s0 += 64) {
        Ranked<float> x = {kNone, kNoToken};
        if (s0 + lane < a.n_vt * SETS) {
          const uint2 b = best[s0 + lane];
          if (__uint_as_float(b.x) > kNone) x = {__uint_as_float(b.x), word_of(s0 + lane, b)};
        }
        // (most have nothing for a list that is full)
        if (s0 && !__any(before(x, Ranked<float>{__shfl(list.z, 63), __shfl(list.token, 63)}))) continue;
        sort_wave(x, lane);
        if (s0 == 0) list = x;
        else merge_wave(list, x, lane);
      }
      total = count;         // (there are 64 and more)
      if (lane < count)
        sh.sets[lane] = Found{list.z, second_of(best[list.token / a.vtile * SETS + column_set<T, SETS>(list.token % a.vtile)]), list.token};
    }
    if (lane == 0) sh.total = total;
  }
  __syncthreads();
  return sh.total;
}

// One token's alternatives, and its values: its target's logit is summed beside theirs.
template <typename T, int SETS>
__device__ __forceinline__ void alternatives(const HeadArgs& a, const Token& token, const uint2* best, Sets<SETS>& e,
                                             const Stat& others, int wave, int lane, TokenShare& sh) {
  const int i = token.at, target = token.target, top = a.top;
  float* logps = a.top_logprobs + (int64_t)i * top;
  int64_t* tokens = a.top_tokens + (int64_t)i * top;
  int count = candidate_sets<T, SETS>(a, best, e, wave, lane, sh);
  // (no other of a set passes its second largest, nor its largest)
  const float bound = lane < count ? fminf(sh.sets[lane].bound, sh.sets[lane].z) : kNone;
  int word = lane < count ? sh.sets[lane].word : kNoToken;
  // the one that the statistics have as their largest
  const float z32 = lane < count ? sh.sets[lane].z : kNone;
  const float most = over_lanes<64>(z32, [](float x, float y) { return fmaxf(x, y); });      // (every lane takes part)
  const uint64_t largest = __ballot(z32 > kNone && z32 == most);
  const int first_lane = largest ? __builtin_ctzll(largest) : -1;
  const int first = largest ? __builtin_amdgcn_readlane(word, __builtin_ctzll(largest)) : kNoToken;
  if (target >= 0) {          // (its set leaves it out)
    if (lane == count) word = target;
    ++count;
  }
  const Operands<T> o(a, i);
  // the first n lanes' words with their 64-bit logits, to which every wave sums a
  // group at a time
  auto fine = [&](int words, int n) {
    for (int g0 = wave * kGroup; g0 < n; g0 += kWaves * kGroup) {
      int of[kGroup];
      double z[kGroup];
#pragma unroll
      for (int g = 0; g < kGroup; ++g) of[g] = __builtin_amdgcn_readlane(words, min(g0 + g, n - 1));
      fine_logits(o.h, o.w, o.ld, a.d, of, lane, z);
#pragma unroll
      for (int g = 0; g < kGroup; ++g)
        if (lane == g && g0 + g < n) sh.z[g0 + g] = z[g];
    }
    __syncthreads();
    return Ranked<double>{lane < n ? sh.z[lane] : -__builtin_inf(), lane < n ? words : kNoToken};
  };
  Ranked<double> found = fine(word, count);
  const Logit own = fine_logit(a, target >= 0 ? sh.z[count - 1] : 0.);
  Logit alt = first_lane < 0 ? rough_logit(kRefFloor) : fine_logit(a, sh.z[first_lane]);
  // (a sum further off than that has lost all that these are for)
  if (!(fabsf(alt.z - others.top) < 64.f)) alt = rough_logit(others.top);
  const TokenStat stat = token_stat(target, own, others, alt);
  if (threadIdx.x == 0) put_stat(a, i, stat.of, token_stat(target, own, others, rough_logit(others.top)).of);
  if (stat.of.y != stat.of.y) {
    if (wave == 0 && lane < top) {
      logps[lane] = kNan;
      tokens[lane] = -1;
    }
    return;
  }
  // ranks by counting who is in front
  int rank = 0;
  for (int k = 0; k < count; ++k)
    rank += before(Ranked<double>{sh.z[k], __builtin_amdgcn_readlane(word, k)}, found) ? 1 : 0;
  __syncthreads();
  if (wave == 0 && lane < count) {
    sh.z[rank] = found.z;
    sh.word[rank] = found.token;
  }
  __syncthreads();
  found = {lane < count ? sh.z[lane] : -__builtin_inf(), lane < count ? sh.word[lane] : kNoToken};
  // sets that may have two of the alternatives: all of them. A set's other words are
  // out only behind top + kSpare that are found, as its largest is behind those of as
  // many sets: by the set's second sum in 32 bits, or as large (no logit of a zero row
  // or weight has an error) but of later words. Its error goes with its products,
  // however small the sum, so nothing short of other words' places makes up for it.
  // The largest second goes first: more sets are out as the words fill (3000 tokens x
  // 1000 words, top 20, in any order / so: 425 / 314 us).
  const double reach = (double)bound + fabs((double)bound) * 0x1p-18;
  uint64_t left = ~0ull;
  auto next_set = [&]() {
    const double last = __shfl(found.z, top + kSpare - 1);              // (every lane takes part)
    const int last_word = __shfl(found.token, top + kSpare - 1);
    const bool in = bound > kNone && !(reach < last || (reach == last && word > last_word)) && (left >> lane & 1);
    if (!__any(in)) return -1;
    const float of = in ? bound : kNone, most = over_lanes<64>(of, [](float x, float y) { return fmaxf(x, y); });
    return __builtin_ctzll(__ballot(of == most));
  };
  for (int at = next_set(); at >= 0; at = next_set()) {
    left &= ~(1ull << at);
    const int known = __builtin_amdgcn_readlane(word, at);
    const int member = known / a.vtile * a.vtile + set_column<T, SETS>(column_set<T, SETS>(known % a.vtile), lane);
    const bool in = lane < kSetRows<T> / 2 && member < a.v && member != known && member != target;
    // the members side by side in the first lanes
    const uint64_t mask = __ballot(in);
    __syncthreads();
    if (wave == 0 && in) sh.word[__popcll(mask & ((1ull << lane) - 1))] = member;
    __syncthreads();
    const int n = __popcll(mask);
    Ranked<double> x = fine(lane < n ? sh.word[lane] : kNoToken, n);
    sort_wave(x, lane);
    merge_wave(found, x, lane);
  }
  if (wave != 0 || lane >= top) return;
  const bool there = found.token != kNoToken && found.z > -__builtin_inf();
  const double c = a.softcap, z = c > 0 ? tanh(found.z / c) * c : found.z;
  // (the leading word's difference is 0 in every bit)
  const double less = (!stat.given && found.token == first ? 0. : z - stat.lead) - log1p((double)stat.others);
  // (above 0 where the sums have another word, whose products cancel, for far too little)
  logps[lane] = !there ? kNone : found.token == target ? stat.of.w : less > 0. ? 0.f : (float)less;
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

// All of a wave's statistics joined, the same in every lane.
__device__ __forceinline__ Stat wave_stat(Stat s) {
  s = over(s, over_lanes<64>(s.top, [](float x, float y) { return fmaxf(x, y); }));
  return settled(s.top, lanes_sum<64>(s.sum), lanes_sum<64>(s.ent), lanes_sum<64>(s.one));
}

// Many tokens without alternatives: a wave a token.
template <typename T>
__global__ __launch_bounds__(256) void k_logprob_stats(HeadArgs a, int blocks) {
  if ((int)blockIdx.x >= blocks) {
    clear_ignored(a, ((int64_t)blockIdx.x - blocks) * 1024);
    return;
  }
  const int lane = threadIdx.x & 63, r = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= piece_rows(a)) return;
  const Token token = token_of(a, r);
  const double target = fine_target<T>(a, token, lane);
  const Stat s = wave_stat(tiles_stat(a, r, lane, 64));
  const float4 stat = token_stat(token.target, fine_logit(a, target), s, rough_logit(s.top)).of;
  if (lane == 0) put_stat(a, token.at, stat, stat);
}

// A block a token.
template <typename T, int SETS>
__global__ __launch_bounds__(kThreads) void k_logprobs(HeadArgs a, int blocks) {
  __shared__ TokenShare sh;
  if ((int)blockIdx.x >= blocks) {
    clear_ignored(a, ((int64_t)blockIdx.x - blocks) * 1024);
    return;
  }
  const int rows = piece_rows(a), lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = blockIdx.x;
  if (r >= rows) return;
  // (all that the token's first steps read is asked for together)
  const Token token = token_of(a, r);
  const uint2* best = a.best + (int64_t)r * a.n_vt * SETS;
  Sets<SETS> e;
  if (a.top) e.load(best, a.n_vt, 0);
  Stat s = wave_stat(tiles_stat(a, r, threadIdx.x, kThreads));
  if (lane == 0) sh.stat[wave] = s;
  if (a.top == 0 && wave == 0) {
    const double target = fine_target<T>(a, token, lane);
    if (lane == 0) sh.target = target;
  }
  __syncthreads();
  s = sh.stat[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s = joined(s, sh.stat[w]);
  if (a.top) alternatives<T, SETS>(a, token, best, e, s, wave, lane, sh);
  else if (threadIdx.x == 0) {
    const float4 stat = token_stat(token.target, fine_logit(a, sh.target), s, rough_logit(s.top)).of;
    put_stat(a, token.at, stat, stat);
  }
}

// Statistics alone: tokens of which a block each goes faster than a wave each, where
// the vocabulary is large (whole calls, a block / a wave each: 1 and 64 tokens x 50304
// x 768 21.5 / 21.9 and 22.7 / 23.4 us, x 128000 x 768 40.4 / 41.0 and 41.5 / 42.2, x
// 8000 x 768 12.2 / 11.6 and 13.2 / 12.7; 256 tokens 38.7 / 38.3, 66.1 / 66.5 and 18.7
// / 18.2; 2048 x 8000 x 768 49 / 45).
constexpr int kFewTokens = 64;
inline unsigned cdiv(int64_t a, int64_t b) { return (unsigned)((a + b - 1) / b); }

}  // namespace

hipError_t launch_logprobs(const HeadArgs& a, int dt, hipStream_t s) {
  const int clear = a.row0 == 0 ? (int)cdiv(a.n, 1024) : 0;
  if (a.top == 0 && a.rows_max > kFewTokens) {
    const int blocks = (int)cdiv(a.rows_max, 4);
    if (dt != MUON_BF16) hipLaunchKernelGGL(k_logprob_stats<float>, dim3(blocks + clear), dim3(256), 0, s, a, blocks);
    else hipLaunchKernelGGL(k_logprob_stats<u16>, dim3(blocks + clear), dim3(256), 0, s, a, blocks);
    return hipGetLastError();
  }
  const int blocks = a.rows_max;
  const dim3 g(blocks + clear), b(kThreads);
  // (head_plan: fp32 has 64-tiles alone)
  if (dt != MUON_BF16) hipLaunchKernelGGL((k_logprobs<float, 4>), g, b, 0, s, a, blocks);
  else if (a.sets == 4) hipLaunchKernelGGL((k_logprobs<u16, 4>), g, b, 0, s, a, blocks);
  else hipLaunchKernelGGL((k_logprobs<u16, 2>), g, b, 0, s, a, blocks);
  return hipGetLastError();
}

}  // namespace muon
