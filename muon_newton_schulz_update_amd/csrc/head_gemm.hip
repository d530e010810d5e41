// Matrix-core products of the head's cross entropy and log probabilities.
//
//   logits    z^T = W H^T       vocabulary x tokens, K = width
//   dhidden   dH  = dz W        tokens x width,      K = vocabulary (in parts)
//   dweight   dW  = dz^T H      vocabulary x width,  K = tokens (in parts)
//
// One kernel shape for the three: a 256 x 256 tile per workgroup of 8 waves, or
// 128 x 128 of 4 and 64 x 64 of 2, two and four workgroups to a CU, where tiles
// are few (fp32: 64 x 64 of 4); K in stages of 128 bytes (64 bf16, 32 fp32),
// both operands of a stage brought to LDS by direct buffer loads into a ring of
// five slots (nine in small launches of 64-tiles), so that while one stage feeds
// the matrix cores the next and half of the one after (three and a half) are on
// their way. bf16 runs v_mfma_f32_32x32x16_bf16, fp32 v_mfma_f32_32x32x2f32.
//
// Neither the weight nor the per-piece matrices are ever transposed in
// memory: an operand whose tile rows are the contraction index is read from
// LDS with the transposing 64-bit read (bf16: four rows of sixteen columns
// per sixteen lanes, so two reads make one operand) or with 32-bit reads
// (fp32). LDS layouts, in 16-byte chunks, and their bank swizzles:
//   OP_ROW_K    row-major matrix, K along the row: [256 rows][8 chunks],
//               chunk ^ (row / 2) % 8
//   OP_GATHER_K the same of rows in any order
//   OP_ROW_T    row-major matrix, K down the rows: [K rows][columns],
//               bf16: chunk ^ (row % 4) 4 (64-tiles: chunk ^ (row / 2 % 2) 4)
//   OP_PANEL_K  panels (train.hpp), K along the chunks: [4 token blocks]
//               [8 chunks][64 tokens], no conflicts as it is
//   OP_PANEL_T  panels, K down the tokens: [chunks][K tokens], token ^ (chunk
//               % 4) 4 (bf16) or chunk % 8 (fp32)
// Every address is clamped into its matrix: rows and columns past the edge
// repeat the last ones and their results are not stored (K itself is padded
// with zeros: in the panels, and past the end of the weight's rows by the
// buffer's range check).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "head_device.hpp"
#include "train.hpp"

namespace muon {
namespace {

typedef __bf16 bf16x8_t __attribute__((__vector_size__(8 * sizeof(__bf16))));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

#define LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

enum OpLayout { OP_ROW_K, OP_GATHER_K, OP_ROW_T, OP_PANEL_K, OP_PANEL_T };

template <int n>
__device__ __forceinline__ void wait_vm() {
  static_assert(n >= 0 && n < 64, "vmcnt immediate");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | 0x0F70);
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }
// A barrier the compiler does not drain the direct loads for; every wait it
// needs is written before it.
__device__ __forceinline__ void ring_barrier() { asm volatile("s_barrier" ::: "memory"); }

// Hand-off through LDS between the lanes of one wave: the LDS executes a
// wave's accesses in order, so only the compiler has to keep them so.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Transposing LDS read: sixteen lanes give the addresses of four rows, four
// 16-bit columns each (lanes 0-3 the first row, ...), and lane l gets column l
// of the four rows. The pointer is restrict so that the read carries alias
// information: without any, the compiler waits for every direct load in flight
// before each such read (plain reads carry a type's; the waits that are needed
// are in the K loop).
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
__device__ __forceinline__ s16x4_t read_tr16(lds_s16x4_t* __restrict p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// The soft cap z = c tanh(y / c) of a raw logit y, to within a dozen roundings of
// itself whatever the cap, and its slope 1 - tanh^2, to the same of itself. With
// x = |y / c|: below kCapPoly z = y (1 + q r(q)), q = x^2, where r interpolates
// (tanh(x) / x - 1) / q at the five Chebyshev nodes of [0, kCapPoly^2] (2 units of
// 2^-24 at most; exact where q vanishes); from there on tanh is (1 - e) / (1 + e)
// and the slope 4 e / (1 + e)^2 with e = exp(-2 x). (A small logit taken from the
// difference of two numbers near c would be off by c 2^-23, and a slope near 0
// from 1 - tanh^2 by as much as itself: at x = 5 by 7 % from z of 11 bits.)
constexpr float kCapPoly = 0.625f;
__device__ __forceinline__ float cap_low(float y, float inv, float& slope) {
  const float x = y * inv, q = x * x;
  float p = fmaf(q, -6.09671418e-3f, 2.09971797e-2f);
  p = fmaf(q, p, -5.38509078e-2f);
  p = fmaf(q, p, 1.33327693e-1f);
  p = fmaf(q, p, -3.33333284e-1f);
  p = fmaf(q, p, 1.f);
  slope = fmaf(-q * p, p, 1.f);
  return y * p;
}
__device__ __forceinline__ float cap_any(float y, float c, float inv, float& slope) {
  const float x = fabsf(y * inv), low = cap_low(y, inv, slope);
  if (x < kCapPoly) return low;                              // (a NaN goes on to the end)
  const float e = __builtin_amdgcn_exp2f(x * (-2.f * kLog2e)), r = __builtin_amdgcn_rcpf(1.f + e);
  slope = 4.f * e * r * r;
  return copysignf(c * ((1.f - e) * r), y);
}
// Sixteen of them. Where no lane of the wave has one past kCapPoly, the usual
// case (18.75 of a cap of 30), there are no exponentials to take: 4096 x 50304 x
// 768, the loss alone, 373 us, with logits of a few times the cap 448.
__device__ __forceinline__ void cap16(f32x16_t& y, float c, float inv, float (&slope)[16]) {
  float most = 0.f;
#pragma unroll
  for (int q = 0; q < 16; ++q) most = fmaxf(most, fabsf(y[q]));
  if (__any(most * inv >= kCapPoly)) {
#pragma unroll
    for (int q = 0; q < 16; ++q) y[q] = cap_any(y[q], c, inv, slope[q]);
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q) y[q] = cap_low(y[q], inv, slope[q]);
  }
}

// One operand of a tile's product.
struct Operand {
  const uint8_t* base;   // tile start at the first stage
  uint32_t pitch;        // bytes: row pitch (row layouts), token-block pitch (panels)
  int lim;               // last valid row (row layouts), last valid chunk (OP_PANEL_T)
  int row_bytes;         // OP_ROW_K: bytes of a row; what a stage has past them is zero
  uint32_t lane;         // this lane's byte offset, the same in every stage
  uint32_t row[4];       // OP_GATHER_K: the offset of this lane's row in each of its loads
};

// Tile edges: 256 (8 waves, one workgroup per CU), 128 (4 waves, two) and 64
// (2 waves, or 4 for fp32, whose products take sixteen times as long; four
// workgroups, or two with the long ring). A stage of an operand is
// TILE x 128 bytes, TILE / 8 loads of 1 KB shared by the NW waves.
template <typename T, int TILE>
constexpr int waves_of() {
  return sizeof(T) == 4 ? 4 : TILE / 32;
}
template <typename T, int L, int TILE, int NW = waves_of<T, TILE>()>
struct Op {
  static constexpr int KE = 128 / (int)sizeof(T);
  static constexpr int kRowT = TILE * (int)sizeof(T);         // LDS row of OP_ROW_T, bytes
  static constexpr int kRowsPerLoad = 1024 / kRowT;           // its rows per load
  // bank swizzle of an OP_ROW_T row (16-bit): a read takes four chunks of four
  // rows at once, which the pitch puts on the same banks (or every second row)
  __device__ static int row_t_swizzle(int row) { return kRowT == 128 ? (row & 2) << 1 : (row & 3) << 2; }
  // the lane's part of a load's address (row layouts: the column part)
  __device__ static uint32_t lane_part(int lane, int wave, int last_chunk) {
    if constexpr (L == OP_ROW_K || L == OP_GATHER_K) {
      const int row = 8 * wave + (lane >> 3);
      return ((lane & 7) ^ ((row >> 1) & 7)) * 16;
    } else if constexpr (L == OP_ROW_T) {
      const int per = 64 / kRowsPerLoad, row = kRowsPerLoad * wave + lane / per, c = lane % per;
      return min(sizeof(T) == 2 ? c ^ row_t_swizzle(row) : c, last_chunk) * 16;
    } else if constexpr (L == OP_PANEL_K) {
      return lane * 16;
    } else {
      if constexpr (sizeof(T) == 2) return (lane ^ ((wave & 3) << 2)) * 16;
      else return (lane >> 5) * 1024 + ((lane & 31) ^ ((2 * wave + (lane >> 5)) & 7)) * 16;
    }
  }
  // direct load i of this wave for stage ks (of the whole K), into slot memory sm
  __device__ static __forceinline__ void load(const Operand& o, uint8_t* sm, int lane, int wave, int ks, int i) {
    const uint8_t* p = o.base;
    uint32_t voff = o.lane, soff = 0;
    const int g = NW * i + wave;
    if constexpr (L == OP_ROW_K || L == OP_GATHER_K) {
      p += (int64_t)ks * 128;
      // past the row's end the offset is out of the buffer's range, and such
      // lanes load zeros
      const bool past = (int)o.lane >= o.row_bytes - ks * 128;
      voff += L == OP_ROW_K ? __umul24(min(8 * g + (lane >> 3), o.lim), o.pitch) : o.row[i];
      voff = past ? 0x80000000u : voff;
    } else if constexpr (L == OP_ROW_T) {
      p += (int64_t)ks * KE * o.pitch;
      voff += __umul24(min(kRowsPerLoad * g + lane / (64 / kRowsPerLoad), o.lim - ks * KE), o.pitch);
    } else if constexpr (L == OP_PANEL_K) {
      p += (int64_t)ks * 8192;
      soff = (g >> 3) * o.pitch + (g & 7) * 1024;
    } else {
      // (two waves: a wave's loads alternate between two values of the swizzle)
      if constexpr (NW == 2) voff ^= (i & 1) * (sizeof(T) == 2 ? 128 : 64);
      if constexpr (sizeof(T) == 2) {
        p += (int64_t)ks * o.pitch;
        soff = min(g, o.lim) * 1024;
      } else {
        p += (int64_t)(ks >> 1) * o.pitch + (ks & 1) * 512;
        soff = min(2 * g, o.lim - 1) * 1024;
      }
    }
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, L == OP_ROW_K || L == OP_GATHER_K ? 0x7FFFFFF0 : -1, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(sm + g * 1024), 16, voff, soff, 0, 0);
  }
  static constexpr int kReads = L == OP_ROW_K || L == OP_GATHER_K || L == OP_PANEL_K ? 1 : sizeof(T) == 2 ? 2 : 4;   // LDS reads a fragment
  // fragment of rows (columns) at..at+31 for k-step s: lane l holds index
  // at + l % 32 and the k of chunk 2 s + l / 32
  template <typename F>
  __device__ static __forceinline__ F frag(const uint8_t* sm, int lane, int at, int s) {
    const int lr = lane & 31, hf = lane >> 5;
    if constexpr (L == OP_ROW_K || L == OP_GATHER_K) {
      return *(const F*)(sm + (at + lr) * 128 + (((2 * s + hf) ^ ((lr >> 1) & 7)) * 16));
    } else if constexpr (L == OP_PANEL_K) {
      return *(const F*)(sm + ((at >> 6) * 8 + 2 * s + hf) * 1024 + ((at & 63) + lr) * 16);
    } else if constexpr (sizeof(T) == 2) {
      // sixteen lanes give the addresses of four rows of K, sixteen columns
      // each, and get a column's four rows back
      const int i = lane & 15, k = 16 * s + 8 * hf + (i >> 2);
      const int c = (at >> 3) + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
      s16x4_t q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int kk = k + 4 * j;
        const uint8_t* p = L == OP_ROW_T ? sm + kk * kRowT + (c ^ row_t_swizzle(kk)) * 16 + (i & 1) * 8
                                         : sm + c * 1024 + (kk ^ ((c & 3) << 2)) * 16 + (i & 1) * 8;
        q[j] = read_tr16((lds_s16x4_t*)p);
      }
      const s16x8_t v = __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(F, v);
    } else {
      F v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 4 * (2 * s + hf) + e, m = at + lr, c = m >> 2;
        v[e] = L == OP_ROW_T ? *(const float*)(sm + k * kRowT + m * 4)
                             : *(const float*)(sm + c * 512 + (k ^ (c & 7)) * 16 + (m & 3) * 4);
      }
      return v;
    }
  }
};

template <typename T> struct FragOf { typedef bf16x8_t type; };
template <> struct FragOf<float> { typedef f32x4_t type; };

// The K loop: acc += A B over stages [k0, k1).
template <typename T, int LA, int LB, int TILE, int NW, int S, int MI, int NI>
__device__ __forceinline__ void k_loop(f32x16_t (&acc)[MI][NI], uint8_t* smem, const Operand& oa, const Operand& ob,
                                       int lane, int wave, int am, int bn, int k0, int k1) {
  typedef typename FragOf<T>::type Frag;
  typedef Op<T, LA, TILE, NW> A;
  typedef Op<T, LB, TILE, NW> B;
  constexpr int kSlot = TILE * 128;                        // one operand of one stage
  constexpr int LPO = TILE / 8 / NW;                       // loads per wave per operand and stage
  constexpr int kReadStep = MI * A::kReads + NI * B::kReads;
  static_assert(S >= 5 && S % 2 == 1 && (S - 4) * LPO < 64, "slots");
  Frag fa[2][MI], fb[2][NI];
  // operand stage o: A (o even) or B (o odd) of stage k0 + o / 2, slot o % S
  auto issue = [&](int slot, int o, int i0, int i1) {
    const int ks = min(k0 + (o >> 1), k1 - 1);
#pragma unroll
    for (int i = i0; i < i1; ++i) {
      if (o & 1) B::load(ob, smem + slot * kSlot, lane, wave, ks, i);
      else A::load(oa, smem + slot * kSlot, lane, wave, ks, i);
    }
  };
  auto read = [&](int sa, int sb, int s, int buf) {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) fa[buf][mi] = A::template frag<Frag>(smem + sa * kSlot, lane, am + mi * 32, s);
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) fb[buf][ni] = B::template frag<Frag>(smem + sb * kSlot, lane, bn + ni * 32, s);
  };
  auto mfmas = [&](int buf) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[buf][mi], fb[buf][ni], acc[mi][ni], 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[buf][mi][e], fb[buf][ni][e], acc[mi][ni], 0, 0, 0);
    }
  };
  auto spread = [&](int loads) {
    constexpr int nmf = MI * NI * (sizeof(T) == 4 ? 4 : 1);
    const int nmem = kReadStep + loads;
#pragma unroll
    for (int q = 0; q < nmf; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
      for (int t = q * nmem / nmf; t < (q + 1) * nmem / nmf; ++t) {
        if (t < loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
    }
  };
  const int nk = k1 - k0;
  issue(0, 0, 0, LPO);
  issue(1, 1, 0, LPO);
  wait_vm<0>();
#pragma unroll
  for (int o = 2; o < S - 2; ++o) issue(o, o, 0, LPO);
  issue(S - 2, S - 2, 0, LPO / 2);
  ring_barrier();
  read(0, 1, 0, 0);
  int sa = 0, sb = 1, na = 2, nb = 3;   // slots of this stage and the next
  int ha = S - 2, ds = S - 1;           // of the operand stages 2 k + S - 2 and 2 k + S - 1
  for (int k = 0; k < nk - 1; ++k) {
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      if (s == 0) {
        __builtin_amdgcn_s_setprio(1);
        __builtin_amdgcn_sched_barrier(0);
        issue(ha, 2 * k + S - 2, LPO / 2, LPO);
      } else {
        issue(ds, 2 * k + S - 1, (s - 1) * LPO / 2, s * LPO / 2);
      }
      read(sa, sb, s + 1, (s + 1) & 1);
      mfmas(s & 1);
      spread(LPO / 2);
      if (s == 0) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // the next stage has landed (only the S - 4 operand stages after it may be
    // on their way); this stage's fragments have been read by every wave
    wait_lgkm0();
    wait_vm<(S - 4) * LPO>();
    ring_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(2);
    __builtin_amdgcn_sched_barrier(0);
    issue(sa, 2 * k + S, 0, LPO / 2);
    read(na, nb, 0, 0);
    mfmas(1);
    spread(LPO / 2);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    // operand stage 2 k + S went to this stage's first slot, 2 k + S + 1 goes to
    // its second
    ha = sa;
    ds = sb;
    sa = na;
    sb = nb;
    na = na + 2 >= S ? na + 2 - S : na + 2;
    nb = nb + 2 >= S ? nb + 2 - S : nb + 2;
  }
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    read(sa, sb, s + 1, (s + 1) & 1);
    mfmas(s & 1);
  }
  mfmas(1);
  wait_vm<0>();
}

// Tile order: blocks b, b + 8, ... run on one XCD; each XCD takes runs of at
// most 32 consecutive tiles, and tiles go down strips of SM rows, so a run
// shares SM row panels and about 32 / SM column panels in that XCD's L2. The
// runs are as long as gives every XCD as many where there are few: in runs of
// 32, 300 tiles would be 64 for one XCD and 32 for another (one token x 50304 x
// 768 27.9 / 25.7 us; fp32 777 x 8191 x 331 with gradients 161 / 155).
constexpr int kEvenRounds = 6;
__host__ __device__ inline int rounds_of(int n) { return n > 256 ? (n + 255) / 256 : 1; }
__host__ __device__ inline int run_of(int n, int rounds) {
  return rounds > kEvenRounds ? 32 : n > 0 ? (n + 8 * rounds - 1) / (8 * rounds) : 1;
}
__device__ __forceinline__ int xcd_index(int b, int n) {
  const int run = run_of(n, rounds_of(n)), j = b >> 3;
  return (j / run * 8 + (b & 7)) * run + j % run;
}
template <int SM>
__device__ __forceinline__ bool strip_tile(int idx, int rows, int cols, int& r, int& c) {
  if (idx >= rows * cols) return false;
  const int strip = idx / (SM * cols), h = min(SM, rows - strip * SM), pos = idx - strip * SM * cols;
  c = pos / h;
  r = strip * SM + pos % h;
  return true;
}

// The sets of a lane's MI x 16 raw logits of one token (z[mi * step]), to `to`: the
// largest, its first place (6 bits) and the second largest, whose last 6 bits the
// place takes: only that a set holds another candidate, and no larger a one, is
// read from the second. Returns the largest of all.
template <typename T, int MI>
__device__ __forceinline__ float store_best(const f32x16_t* z, int step, uint2* to) {
  constexpr int EACH = kSetRows<T> / 32 < MI ? kSetRows<T> / 32 : MI;
  float top = -__builtin_inff();
  uint2 b[MI / EACH];
#pragma unroll
  for (int m0 = 0; m0 < MI; m0 += EACH) {
    float first = -__builtin_inff(), second = first;
#pragma unroll
    for (int mi = m0; mi < m0 + EACH; ++mi)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        second = __builtin_amdgcn_fmed3f(first, second, z[mi * step][q]);
        first = fmaxf(first, z[mi * step][q]);
      }
    uint32_t place = 0;
#pragma unroll
    for (int i = EACH * 16 - 1; i >= 0; --i) place = z[(m0 + i / 16) * step][i % 16] == first ? i : place;
    b[m0 / EACH] = make_uint2(__float_as_uint(first), (__float_as_uint(second) & ~63u) | place);
    top = fmaxf(top, first);
  }
  __builtin_memcpy(to, b, sizeof(b));
  return top;
}

// The logits' gradient dz = p (b + g log2 p) and the target's (train.hpp: ts), to
// the panels in the operands' type; z are a lane's raw logits of token r. Rows past
// the piece's and columns past the vocabulary become zero (stages of dW and dH).
template <typename T, int MI>
__device__ __forceinline__ void store_logits_grad(const HeadArgs& a, f32x16_t (&z)[MI], int r, int rows, int vw, int hf,
                                                  int tg, bool any_mine, bool edge) {
  const bool real = r < rows, cap = a.softcap > 0.f, some_past = !__all(real);
  float4 ts = {0.f, 0.f, 0.f, 0.f};
  if (real) ts = a.ts[r];
  float own = 0.f;
  if (tg >= 0) own = a.rs[r].z;
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    float e[16], slope[16];
    if (cap) cap16(z[mi], a.softcap, a.cap_inv, slope);
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      // log p, base 2, from a difference, which is as good as the logits however large
      // these are (p is 0 past kNoExp, and what it is multiplied by no infinity: a word
      // that the head masks may have a row as large as its type goes)
      const float y = __builtin_elementwise_maximum(fmaf(z[mi][q] - ts.x, kLog2e, ts.y), kNoExp);
      e[q] = __builtin_amdgcn_exp2f(y) * fmaf(ts.w, y, ts.z);
    }
    if (cap) {
#pragma unroll
      for (int q = 0; q < 16; ++q) e[q] *= slope[q];
    }
    if (some_past) {
#pragma unroll
      for (int q = 0; q < 16; ++q) e[q] = real ? e[q] : 0.f;
    }
    if (any_mine) {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (mi * 32 + 8 * (q >> 2) + (q & 3) == tg) {
          // most of a token's gradient: what its rounding loses is added to both products
          const float x = cap ? own * slope[q] : own;
          float4 rs = {0.f, 0.f, x, 0.f};
          if (sizeof(T) == 2) rs.w = x - bf2f(f2bf(x));
          a.rs[r] = rs;
          e[q] = x;
        }
    }
    if (edge) {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (vw + mi * 32 + 8 * (q >> 2) + 4 * hf + (q & 3) >= a.v) e[q] = 0.f;
    }
    const int64_t col = vw + mi * 32;
    if constexpr (sizeof(T) == 2) {
      unsigned int c[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) c[q] = pack_bf16(e[2 * q], e[2 * q + 1]);
      uint8_t* dst = (uint8_t*)a.e + (((int64_t)(r >> 6) * (a.vp >> 3) + (col >> 3)) << 10) + (r & 63) * 16;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        // (as the exponentials below: whole chunks after a half-wave swap)
        const u32x2_t x = __builtin_amdgcn_permlane32_swap(c[4 * g], c[4 * g + 2], false, false);
        const u32x2_t y = __builtin_amdgcn_permlane32_swap(c[4 * g + 1], c[4 * g + 3], false, false);
        *(u32x4_t*)(dst + ((2 * g + hf) << 10)) = (u32x4_t){x[0], y[0], x[1], y[1]};
      }
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(f32x4_t*)((float*)a.e + panel_at<float>(r, col + 8 * g + 4 * hf, a.vp)) =
            (f32x4_t){e[4 * g], e[4 * g + 1], e[4 * g + 2], e[4 * g + 3]};
    }
  }
}

// ---------------------------------------------------------------------------
// Logits. The vocabulary is on the accumulators' rows and the tokens on their
// columns, so a lane holds 64 logits of each of its two tokens (32 or 16 of one
// in the smallest tiles): maximum and sum need one exchange with the other
// half-wave. The statistics are per wave's vocabulary rows, so bf16's waves
// never wait for one another. The exponentials go to the panels as whole chunks
// after a half-wave swap.
//
// In large calls the matrix cores are busy 56 % of the time (at 1.3 to 1.45 GHz;
// 62 % at 1.8 in a launch of 130 us), the rest is the epilogue: as many
// exponentials as results, and 2 bytes of each kept; few tokens are bound by the
// weight's one read. Measured: 8192 x 50304 x 768 with the exponentials kept
// 672 us (940 TFLOP/s and 1.2 TB/s), 6963 x 50304 x 2048 with a soft cap 1259
// (1140), 1536 x 50304 x 768 without 131 (905); one token x 50304 x 768 16.6
// (4.7 TB/s); fp32 1987 x 30961 x 704 680 (127).
// Two workgroups of 256 x 128 to a CU, so that one's epilogue runs beside the
// other's products, took 13 % longer (more operand traffic from LDS).
//
// LOGITS_STATS adds each tile's entropy to the statistics, leaves one of the largest
// out of the sum (two operations a logit: 3 % of the launch) and, where alternatives
// are asked for, each set's largest logits; LOGITS_GRAD, with a token's statistics
// from an earlier call, leaves the gradient itself (8192 x 50304 x 768, bf16:
// statistics 590 us, 1.07 PFLOP/s with the matrix cores 59 % busy; gradient 690,
// 824 MB written under the products: kept exponentials and their own pass take 672
// + 300).
// ---------------------------------------------------------------------------
template <typename T, int TILE, int S, bool FEW, bool GATHER, LogitsMode MODE = LOGITS_LOSS>
__global__ __launch_bounds__((FEW ? 2 : waves_of<T, TILE>()) * 64, S > 5 ? 1 : 2) void k_logits_mfma(HeadArgs a, int keep, int vt, int tt) {
  // a wave: 128 vocabulary rows x 64 tokens (256-tiles) or 32, 64 x 32 of a
  // 64-tile. PAIR: 32 x 32 of one, and two waves put their statistics together:
  // fp32, four waves, or (FEW: at most 32 tokens) two on the first 32 tokens
  constexpr int NW = FEW ? 2 : waves_of<T, TILE>();
  constexpr bool PAIR = sizeof(T) == 4;
  constexpr int MI = PAIR ? 1 : TILE == 64 ? 2 : 4, NI = TILE == 256 ? 2 : 1;
  constexpr int WM = TILE / (MI * 32), WN = NW / WM;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * TILE * 128];
  int vi, ti;
  const int lane = threadIdx.x & 63;
  int rows, token = 0, target = 0;
  if constexpr (GATHER) {
    // at most 64 tokens: every wave lists the valid ones itself, lane r the
    // r-th; the first block writes the list for the statistics' merge (with
    // rows packed by a launch before this one: one token x 50304 x 768 24.9 us
    // a call instead of 21.2, 16 x 3200 x 256 14.2 instead of 10.4)
    const int64_t g = lane < a.n ? target_at(a.targets, a.target_bytes, lane) : a.ignore;
    const bool valid = g != a.ignore;
    const uint64_t mask = __ballot(valid), below = (1ull << lane) - 1;
    rows = __popcll(mask);
    const int to = 4 * (valid ? __popcll(mask & below) : rows + __popcll(~mask & below));
    token = __builtin_amdgcn_ds_permute(to, lane);
    target = __builtin_amdgcn_ds_permute(to, checked_target(a, g));
    if (blockIdx.x == 0 && threadIdx.x < 64) {
      if (lane < rows) {
        a.idx[lane] = token;
        a.tgt[lane] = target;
      }
      if (a.per_token && !valid && lane < a.n) a.loss[lane] = 0.f;
      if (lane == 0) a.count[0] = rows;
    }
  } else {
    rows = piece_rows(a);
  }
  const int nt = min(tt, (rows + TILE - 1) / TILE);
  if (!strip_tile<4>(xcd_index(blockIdx.x, vt * nt), vt, nt, vi, ti)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  const int v0 = vi * TILE, r0 = ti * TILE;
  typedef Op<T, OP_ROW_K, TILE, NW> A;
  constexpr int LB = GATHER ? OP_GATHER_K : OP_PANEL_K;
  typedef Op<T, LB, TILE, NW> B;
  const Operand oa = {(const uint8_t*)a.w + (int64_t)v0 * a.ld_w * sizeof(T), (uint32_t)(a.ld_w * sizeof(T)),
                      a.v - 1 - v0, a.w_cols * (int)sizeof(T), A::lane_part(lane, wave, 0)};
  const uint32_t blk = (uint32_t)a.dp * sizeof(T) * kPanelRows;
  Operand ob = {(const uint8_t*)a.hp + (int64_t)ti * (TILE / 64) * blk, blk, 0, 0, B::lane_part(lane, wave, 0)};
  if constexpr (GATHER) {
    ob.base = (const uint8_t*)a.h;
    ob.row_bytes = a.d * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < TILE / 8 / NW; ++i) {
      const int r = min(8 * (NW * i + wave) + (lane >> 3), rows - 1);   // (r0 is 0)
      ob.row[i] = (uint32_t)__shfl(token, r) * (uint32_t)(a.ld_h * sizeof(T));
    }
  }
  f32x16_t acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = (f32x16_t){};
  k_loop<T, OP_ROW_K, LB, TILE, NW, S, MI, NI>(acc, smem, oa, ob, lane, wave, wm * MI * 32, wn * NI * 32, 0, a.dp / A::KE);

  const int lr = lane & 31, hf = lane >> 5;
  const int vw = v0 + wm * MI * 32;                  // the wave's first vocabulary row
  if (!PAIR && vw >= a.v) return;                    // (the exponentials' padding is cleared with the gradient)
  const int tile = PAIR ? vi : vi * WM + wm;
  const float none = -__builtin_inff();
  // what takes no part in a token's sum: rows past the vocabulary, its target.
  // (With a soft cap these are raw logits, capped below, where the slopes are
  // needed; the cap rises with its logit, so the largest stays the largest.)
  const bool cap = a.softcap > 0.f, edge = vw + MI * 32 > a.v;
  auto drop_past = [&](f32x16_t& z, int mi) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (vw + mi * 32 + 8 * (r >> 2) + 4 * hf + (r & 3) >= a.v) z[r] = none;
  };
  if (edge) {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) drop_past(acc[mi][ni], mi);
  }
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int r = r0 + (wn * NI + ni) * 32 + lr;       // the lane's token in the piece
    const int listed = GATHER ? __shfl(target, r & 63) : 0;
    // the target's logit leaves the tile: it has its own place in the sums
    const int tg = (r >= rows ? -1 : GATHER ? listed : a.tgt[a.row0 + r]) - vw - 4 * hf;
    const bool mine = tg >= 0 && tg < MI * 32 && (tg & 4) == 0;
    const bool any_mine = __any(mine);
    if constexpr (MODE == LOGITS_GRAD) {
      f32x16_t z[MI];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) z[mi] = acc[mi][ni];
      store_logits_grad<T, MI>(a, z, r, rows, vw, hf, mine ? tg : -1, any_mine, edge);
      continue;
    }
    if (any_mine) {
      float z = 0.f, slope = 1.f;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (mi * 32 + 8 * (q >> 2) + (q & 3) == tg) {
            z = acc[mi][ni][q];
            acc[mi][ni][q] = none;
          }
      if constexpr (MODE == LOGITS_LOSS) {       // (head_logprobs.hip takes the target's in 64 bits)
        if (cap) z = cap_any(z, a.softcap, a.cap_inv, slope);
        if (mine) a.zt[r] = z;
        if (mine && cap) a.zf[r] = slope;
      }
    }
    float top = kRefFloor;
    if constexpr (MODE == LOGITS_STATS) {
      if (a.top) {
        // (a token's statistics lie side by side: the four vocabulary tiles that run
        // next to one another fill its lines)
        constexpr int LANE_SETS = MI * 32 / kSetRows<T> > 0 ? MI * 32 / kSetRows<T> : 1;
        uint2* to = a.best + ((int64_t)r * a.n_vt + tile) * a.sets + (PAIR ? 2 * wm + hf : hf * LANE_SETS);
        top = fmaxf(top, store_best<T, MI>(&acc[0][ni], NI, to));
      }
      if (cap) {
        // (capped before their largest is taken: it is one of them to the last bit)
        top = kRefFloor;
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          float slope[16];
          cap16(acc[mi][ni], a.softcap, a.cap_inv, slope);
          if (edge) drop_past(acc[mi][ni], mi);
          if (any_mine) {
#pragma unroll
            for (int q = 0; q < 16; ++q)
              if (mi * 32 + 8 * (q >> 2) + (q & 3) == tg) acc[mi][ni][q] = none;
          }
        }
      }
    }
    if (MODE != LOGITS_STATS || cap || !a.top) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int q = 0; q < 16; ++q) top = fmaxf(top, acc[mi][ni][q]);
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    if (MODE != LOGITS_STATS && cap) {
      float slope;
      top = cap_any(top, a.softcap, a.cap_inv, slope);
    }
    // PAIR: the two waves' rows have one reference and one sum
    float* stat = (float*)smem + wn * 32 + lr;       // [wave row][token], then the second row's sums
    if constexpr (PAIR) {
      ring_barrier();                                // every wave is done with the slots
      if (hf == 0) stat[wm * 64] = top;
      wait_lgkm0();
      ring_barrier();
      top = fmaxf(stat[0], stat[64]);
    }
    float sum = 0.f, ent = 0.f, rest = 0.f;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      float e[16], slope[16];
      f32x16_t z = acc[mi][ni];
      if (MODE != LOGITS_STATS && cap) {
        cap16(z, a.softcap, a.cap_inv, slope);
        // (a few roundings can put one above the largest's, which for logits of
        // 10^8 and more is past what an exponential may say)
#pragma unroll
        for (int q = 0; q < 16; ++q) z[q] = __builtin_elementwise_minimum(z[q], top);
        if (edge) drop_past(z, mi);
        if (any_mine) {
#pragma unroll
          for (int q = 0; q < 16; ++q)
            if (mi * 32 + 8 * (q >> 2) + (q & 3) == tg) z[q] = none;
        }
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        // from the difference, which is exact near the largest however large
        // both are (z log2(e) less its rounded maximum, one instruction fewer,
        // is off by more than 1 past 2^24); no smaller than a kept exponential
        // can say (kCodeBase); a maximum that keeps NaN, so that one bad logit
        // reaches the token's loss
        const float y = __builtin_elementwise_maximum((z[q] - top) * kLog2e, MODE == LOGITS_STATS ? kNoExp : -63.f);
        e[q] = __builtin_amdgcn_exp2f(y);
        sum += e[q];
        if constexpr (MODE == LOGITS_STATS) {
          ent = fmaf(e[q], y, ent);
          rest += __builtin_amdgcn_fractf(e[q]);       // (all below 1)
        }
      }
      if (MODE == LOGITS_STATS || !keep) continue;
      if (cap) {
        // what the gradient takes of the logit: its exponential times the slope
#pragma unroll
        for (int q = 0; q < 16; ++q)
          e[q] = sizeof(T) == 2 ? __builtin_elementwise_maximum(e[q] * slope[q], 0x1p-63f) : e[q] * slope[q];
      }
      const int64_t col = vw + mi * 32;
      if constexpr (sizeof(T) == 2) {
        // in [2^-63, 1] the pattern's upper two exponent bits say nothing:
        // shifted out, the code is the upper half, rounded half up
        unsigned int c[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          c[q] = __builtin_amdgcn_perm((__float_as_uint(e[2 * q + 1]) << 3) + 0x8000u,
                                       (__float_as_uint(e[2 * q]) << 3) + 0x8000u, 0x07060302u);
        uint8_t* dst = (uint8_t*)a.e + (((int64_t)(r >> 6) * (a.vp >> 3) + (col >> 3)) << 10) + (r & 63) * 16;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          // groups 2 g and 2 g + 1 of four rows: the low half-wave ends up
          // with the even group's eight rows, the high one with the odd's
          const u32x2_t x = __builtin_amdgcn_permlane32_swap(c[4 * g], c[4 * g + 2], false, false);
          const u32x2_t y = __builtin_amdgcn_permlane32_swap(c[4 * g + 1], c[4 * g + 3], false, false);
          *(u32x4_t*)(dst + ((2 * g + hf) << 10)) = (u32x4_t){x[0], y[0], x[1], y[1]};
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(f32x4_t*)((float*)a.e + panel_at<float>(r, col + 8 * g + 4 * hf, a.vp)) =
              (f32x4_t){e[4 * g], e[4 * g + 1], e[4 * g + 2], e[4 * g + 3]};
      }
    }
    sum += __shfl_xor(sum, 32);
    if constexpr (MODE == LOGITS_STATS) {
      ent += __shfl_xor(ent, 32);
      rest += __shfl_xor(rest, 32);
    }
    if constexpr (PAIR) {
      if (wm == 1 && hf == 0) {
        stat[128] = sum;
        if constexpr (MODE == LOGITS_STATS) {
          stat[192] = ent;
          stat[256] = rest;
        }
      }
      wait_lgkm0();
      ring_barrier();
      if (wm == 1) return;
      sum += stat[128];
      if constexpr (MODE == LOGITS_STATS) {
        ent += stat[192];
        rest += stat[256];
      }
    }
    if (hf == 0) {
      if constexpr (MODE == LOGITS_STATS) {
        // the sum without one of the largest: how many of these there are is a whole number
        const float ones = rintf(sum - rest), one = ones > 0.f ? 1.f : 0.f;
        a.tstat[(int64_t)r * a.n_vt + tile] = float4{top, rest + (ones - one), ent, one};
      } else {
        a.tmax[(int64_t)tile * a.piece + r] = top;
        a.tsum[(int64_t)tile * a.piece + r] = sum;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// dH: partial sums over a range of the vocabulary, 32-bit, row-major; one
// range alone writes the tokens' rows itself.
// ---------------------------------------------------------------------------
template <typename T, int TILE, int S>
__device__ __forceinline__ void dhidden_tile(const HeadArgs& a, uint8_t* smem, int ti, int di, int q, int rows) {
  constexpr int NW = waves_of<T, TILE>(), MI = NW * 32 > TILE ? 1 : 2, NI = TILE == 64 ? 1 : TILE / 64;   // waves: NW / 2 x 2
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
  const int r0 = ti * TILE, d0 = di * TILE;
  typedef Op<T, OP_PANEL_K, TILE, NW> A;
  typedef Op<T, OP_ROW_T, TILE, NW> B;
  const uint32_t blk = (uint32_t)a.vp * sizeof(T) * kPanelRows;
  const Operand oa = {(const uint8_t*)a.e + (int64_t)ti * (TILE / 64) * blk, blk, 0, 0, A::lane_part(lane, wave, 0)};
  const int chunks = (a.w_cols - d0) * (int)sizeof(T) / 16;
  const Operand ob = {(const uint8_t*)a.w + (int64_t)d0 * sizeof(T), (uint32_t)(a.ld_w * sizeof(T)), a.v - 1, 0,
                      B::lane_part(lane, wave, chunks - 1)};
  const int nk = (a.v + A::KE - 1) / A::KE;
  const int k0 = (int)((int64_t)nk * q / a.split), k1 = (int)((int64_t)nk * (q + 1) / a.split);
  f32x16_t acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = (f32x16_t){};
  if (k1 > k0)
    k_loop<T, OP_PANEL_K, OP_ROW_T, TILE, NW, S, MI, NI>(acc, smem, oa, ob, lane, wave, wm * MI * 32, wn * NI * 32, k0, k1);
  const int lr = lane & 31, hf = lane >> 5;
  if (a.split > 1) {
    float* out = a.part + (int64_t)q * a.piece * a.dp;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const int d = d0 + (wn * NI + ni) * 32 + lr;
      if (d >= a.dp) continue;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = r0 + (wm * MI + mi) * 32 + 8 * (r >> 2) + 4 * hf + (r & 3);
          out[(int64_t)row * a.dp + d] = acc[mi][ni][r];
        }
    }
    return;
  }
  // one split: the tokens' rows themselves, put together in the idle LDS as
  // 32-bit sums, so that what the target's gradient lost in its rounding is
  // added, and the weight's row read, by whole chunks
  const float g = common_factor(a);
  const int rw = r0 + wm * MI * 32, dw = d0 + wn * NI * 32;      // the wave's part
  constexpr int CH = 16 / (int)sizeof(T), NF = NI * 8, NC = NI * 32 / CH;   // 16-byte chunks of its row: sums, results
  ring_barrier();                                           // every wave is done with the slots
  uint8_t* slab = smem + wave * (32 * NF * 16);
  auto chunk_at = [&](int row, int c) { return slab + row * NF * 16 + ((c ^ (row & (NF - 1))) * 16); };
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        ((float*)chunk_at(8 * (r >> 2) + 4 * hf + (r & 3), ni * 8 + (lr >> 2)))[lr & 3] = acc[mi][ni][r];
    wave_lds_sync();
#pragma unroll 2
    for (int i = 0; i < NC / 2; ++i) {
      const int row = i * (64 / NC) + lane / NC, c = lane % NC;
      const int t = rw + mi * 32 + row, d = dw + c * CH;
      if (t >= rows || d >= a.d) continue;
      T y[CH];
      f32x4_t x[CH / 4];
#pragma unroll
      for (int j = 0; j < CH / 4; ++j) x[j] = *(const f32x4_t*)chunk_at(row, c * (CH / 4) + j);
      if constexpr (sizeof(T) == 2) {
        const float rest = a.rs[t].w;
        if (rest != 0.f) {
          const u32x4_t w = *(const u32x4_t*)((const u16*)a.w + (int64_t)a.tgt[a.row0 + t] * a.ld_w + d);
#pragma unroll
          for (int e = 0; e < CH; ++e) x[e >> 2][e & 3] = fmaf(rest, bf2f((u16)(w[e >> 1] >> (16 * (e & 1)))), x[e >> 2][e & 3]);
        }
        const u32x4_t q = {pack_bf16(x[0][0] * g, x[0][1] * g), pack_bf16(x[0][2] * g, x[0][3] * g),
                           pack_bf16(x[1][0] * g, x[1][1] * g), pack_bf16(x[1][2] * g, x[1][3] * g)};
        __builtin_memcpy(y, &q, 16);
      } else {
        const f32x4_t q = x[0] * g;
        __builtin_memcpy(y, &q, 16);
      }
      T* p = (T*)a.dh + (int64_t)a.idx[a.row0 + t] * a.ld_dh + d;
      if (d + CH <= a.d) {
        __builtin_memcpy(p, y, 16);       // (one store, aligned or not)
      } else {
#pragma unroll
        for (int e = 0; e < CH; ++e)
          if (d + e < a.d) p[e] = y[e];
      }
    }
    wave_lds_sync();
  }
}

// ---------------------------------------------------------------------------
// What the targets' own gradients lost in their rounding to 16 bits, times the
// tokens' rows, to dW's accumulators. That one term is most of a word's gradient
// where few tokens have it as their target: without it dW of 65 x 8000 x 256 is
// 1.99e-3 off and of 8192 x 50304 x 768 1.90e-3, with it 1.66e-3, which is the
// output's own rounding. (The other words' terms are small, and their roundings
// add nothing that shows.)
// A tile lists the tokens t0 to t1 of the piece whose target is among its rows
// and takes them 64 at a time through one more stage of its product: their
// hidden rows gathered to LDS (from the caller's matrix, a row's chunks side by
// side, where these are whole 16-byte pieces; from the panels otherwise), and
// beside them a matrix that holds each remainder (in 16 bits again: sixteen of
// the target's gradient in all) in its token's and word's place and is zero
// elsewhere. The lists keep the tokens' order, so the sums repeat.
// Measured, without / with: 8192 x 50304 x 768 1999 / 2016 us, 1000 x 8000 x 256
// 55.5 / 58.5, 300 x 50304 x 2048 365 / 382; most where many tokens share few
// words, whose tiles have the longest lists: 8192 x 2000 x 512 111 / 134.
// ---------------------------------------------------------------------------
// A wave's targets of a window of tokens, as they are in memory.
template <int TILE, int NW>
struct TargetWindow {
  static constexpr int kTokens = 16 * TILE;                     // (their lists fit the ring)
  static constexpr int kShare = kTokens / NW, kLoads = kShare / 256;
  i32x4_t at[kLoads];
  __device__ __forceinline__ static int token(int w0, int wave, int lane, int l) {
    return w0 + wave * kShare + (l * 64 + lane) * 4;
  }
  // whole pieces of four (the list of targets is padded), the last one again past the end
  __device__ __forceinline__ void load(const HeadArgs& a, int lane, int wave, int w0, int t1) {
#pragma unroll
    for (int l = 0; l < kLoads; ++l)
      at[l] = *(const i32x4_t*)(a.tgt + a.row0 + min(token(w0, wave, lane, l), (t1 - 1) & ~3));
  }
};
template <int TILE, int NW, int MI, int NI>
__device__ __forceinline__ void add_target_rests(f32x16_t (&acc)[MI][NI], const HeadArgs& a, uint8_t* smem,
                                                 const Operand& rows, TargetWindow<TILE, NW>& window, int lane, int wave,
                                                 int am, int bn, int v0, int d0, int t0, int t1) {
  typedef Op<u16, OP_ROW_T, TILE, NW> R;                        // the gathered rows
  typedef Op<u16, OP_PANEL_T, TILE, NW> O;                      // the remainders
  typedef TargetWindow<TILE, NW> Window;
  constexpr int kShare = Window::kShare, LPO = TILE / 8 / NW;
  uint8_t* sb = smem + 2 * TILE * 128;                          // after two slots for the gathered rows
  uint32_t* list = (uint32_t*)(sb + TILE * 128);                // token | word << 16, each wave's share
  uint2* places = (uint2*)(list + Window::kTokens);             // row's offset, remainder | word << 16
  int* counts = (int*)(places + Window::kTokens);
  const uint64_t below = (1ull << lane) - 1;
  const uint8_t* base = a.rows_direct ? (const uint8_t*)a.h + d0 * 2 : rows.base;
  // last chunk of the tile's columns: the caller's rows end with their width,
  // the panels are padded
  const int last_chunk = a.rows_direct ? (a.d - d0) / 8 - 1 : rows.lim;
  auto all_waves = [&]() {
    wait_lgkm0();
    ring_barrier();
  };
  bool cleared = false;
  for (int w0 = t0; w0 < t1; w0 += Window::kTokens) {
    if (w0 != t0) window.load(a, lane, wave, w0, t1);           // (the first one's came beside the product)
    all_waves();                                                // the slots, and the list before, have been read
    int found = 0;
#pragma unroll
    for (int l = 0; l < Window::kLoads; ++l) {
      const int token = Window::token(w0, wave, lane, l);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int word = window.at[l][c] - v0;
        const bool hit = token + c < t1 && word >= 0 && word < TILE;
        const uint64_t m = __ballot(hit);
        if (hit) list[wave * kShare + found + __popcll(m & below)] = (uint32_t)(token + c) | (uint32_t)word << 16;
        found += __popcll(m);
      }
    }
    if (lane == 0) counts[wave] = found;
    all_waves();
    int upto[NW], all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) upto[w] = all += counts[w];
    all = __builtin_amdgcn_readfirstlane(all);
    if (all == 0) continue;
    // the shares put together, and what the stages need of each token
    for (int h = wave * 64 + lane; h < all; h += NW * 64) {
      int at = h;
#pragma unroll
      for (int w = 0; w < NW - 1; ++w)
        if (h >= upto[w]) at = (w + 1) * kShare + h - upto[w];
      const uint32_t entry = list[at], token = entry & 0xFFFF;
      const uint32_t off = a.rows_direct ? (uint32_t)a.idx[a.row0 + token] * (uint32_t)(a.ld_h * 2)
                                         : (token >> 6) * rows.pitch + (token & 63) * 16;
      places[h] = make_uint2(off, pack_bf16(a.rs[token].w, 0.f) | (entry & 0xFFFF0000u));
    }
    if (!cleared)
      for (int b = (wave * 64 + lane) * 16; b < TILE * 128; b += NW * 1024) *(u32x4_t*)(sb + b) = (u32x4_t){0, 0, 0, 0};
    cleared = true;
    all_waves();
    // tokens h0.. h0 + 63 of the list, one to a lane (past the last, that one
    // again: its second place in the sum is 0): their rows on their way to a slot
    auto fetch = [&](int h0, int slot) {
      const uint2 p = places[min(h0 + lane, all - 1)];
      const int step = a.rows_direct ? 16 : 1024;               // from chunk to chunk of a token's row
#pragma unroll
      for (int i = 0; i < LPO; ++i) {
        const int g = NW * i + wave, row = R::kRowsPerLoad * g + lane / (64 / R::kRowsPerLoad);
        const int c = min((lane % (64 / R::kRowsPerLoad)) ^ R::row_t_swizzle(row), last_chunk);
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, -1, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(smem + slot * TILE * 128 + g * 1024), 16,
                                                 __shfl(p.x, row) + c * step, 0, 0, 0);
      }
      return p.y;
    };
    uint32_t mark = fetch(0, 0), next_mark = 0;
    for (int h0 = 0, slot = 0; h0 < all; h0 += 64, slot ^= 1) {
      const int word = mark >> 16;
      u16* place = (u16*)(sb + (word >> 3) * 1024 + ((lane ^ ((word >> 3 & 3) << 2)) * 16) + (word & 7) * 2);
      const bool mine = wave == 0 && h0 + lane < all;
      if (mine) *place = (u16)mark;
      if (h0 + 64 < all) {
        next_mark = fetch(h0 + 64, slot ^ 1);
        wait_vm<LPO>();                                         // no more than the next ones' rows on their way
      } else {
        wait_vm<0>();
      }
      all_waves();
      const uint8_t* sa = smem + slot * TILE * 128;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8_t fa[MI], fb[NI];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) fa[mi] = R::template frag<bf16x8_t>(sa, lane, am + mi * 32, s);
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) fb[ni] = O::template frag<bf16x8_t>(sb, lane, bn + ni * 32, s);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[mi], fb[ni], acc[mi][ni], 0, 0, 0);
      }
      all_waves();                                              // the slot and the places have been read
      if (mine) *place = 0;
      mark = next_mark;
    }
  }
  if (cleared) wait_lgkm0();                                    // (the last places, before others write the slots)
}

// ---------------------------------------------------------------------------
// dW: the piece's sum, or a part of its tokens', added to the pieces before
// it; the last one is scaled and rounded to the weight's type. The width is on the accumulators' rows, so
// a lane has four neighbouring columns of one weight row; the results are put
// together to whole rows of the wave's part in the idle LDS (chunks swizzled by
// row) and leave as 16-byte stores.
// ---------------------------------------------------------------------------
template <typename T, int TILE, int S>
__device__ __forceinline__ void dweight_tile(const HeadArgs& a, uint8_t* smem, int vi, int di, int part, int rows) {
  constexpr int NW = waves_of<T, TILE>(), MI = TILE / 64, NI = NW * 32 > TILE ? 1 : 2, WN = NW / 2;   // waves: 2 x WN
  const int lane = threadIdx.x & 63, lr = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int v0 = vi * TILE, d0 = di * TILE;
  typedef Op<T, OP_PANEL_T, TILE, NW> O;
  constexpr int CH = 16 / (int)sizeof(T);
  const uint32_t be = (uint32_t)a.vp * sizeof(T) * kPanelRows, bh = (uint32_t)a.dp * sizeof(T) * kPanelRows;
  const Operand oa = {(const uint8_t*)a.hp + (int64_t)(d0 / CH) * 1024, bh, (a.dp - d0) / CH - 1, 0,
                      O::lane_part(lane, wave, 0)};
  const Operand ob = {(const uint8_t*)a.e + (int64_t)(v0 / CH) * 1024, be, TILE / CH - 1, 0,
                      O::lane_part(lane, wave, 0)};
  f32x16_t acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = (f32x16_t){};
  const int nk = (rows + O::KE - 1) / O::KE;
  const int k0 = (int)((int64_t)nk * part / a.wsplit), k1 = (int)((int64_t)nk * (part + 1) / a.wsplit);
  TargetWindow<TILE, NW> window;
  if constexpr (sizeof(T) == 2)
    if (k1 > k0) window.load(a, lane, wave, k0 * O::KE, min(k1 * O::KE, rows));
  if (k1 > k0)
    k_loop<T, OP_PANEL_T, OP_PANEL_T, TILE, NW, S, MI, NI>(acc, smem, oa, ob, lane, wave, wm * MI * 32, wn * NI * 32, k0, k1);
  if constexpr (sizeof(T) == 2)
    add_target_rests<TILE, NW, MI, NI>(acc, a, smem, oa, window, lane, wave, wm * MI * 32, wn * NI * 32, v0, d0, k0 * O::KE,
                                       min(k1 * O::KE, rows));
  const float g = common_factor(a);
  const int vw = v0 + wn * NI * 32, dw = d0 + wm * MI * 32;      // the wave's part
  const bool split = a.wsplit > 1;
  if (split || a.dwacc) {
    // sums over parts or pieces: padded rows, whole 16-byte groups
    float* acc_at = (split ? a.wpart + (int64_t)part * a.v * a.dp : a.dwacc) + (int64_t)(vw + lr) * a.dp + dw + 4 * hf;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      if (vw + ni * 32 + lr >= a.v) continue;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        if (dw + mi * 32 >= a.dp) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4_t* p = (f32x4_t*)(acc_at + (int64_t)ni * 32 * a.dp + mi * 32 + 8 * q);
          f32x4_t x = {acc[mi][ni][4 * q], acc[mi][ni][4 * q + 1], acc[mi][ni][4 * q + 2], acc[mi][ni][4 * q + 3]};
          if (!split && !a.first) x += *p;
          if (split || !a.last) *p = x;
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mi][ni][4 * q + e] = x[e];
        }
      }
    }
    if (split || !a.last) return;
  }
  constexpr int NC = MI * 2 * (int)sizeof(T);               // chunks of the wave's row
  if (nk > 0) ring_barrier();                               // every wave is done with the slots
  uint8_t* slab = smem + wave * (NI * 32 * NC * 16);
#pragma unroll
  for (int ni = 0; ni < NI; ++ni)
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = ni * 32 + lr;
        const f32x4_t x = {acc[mi][ni][4 * q] * g, acc[mi][ni][4 * q + 1] * g, acc[mi][ni][4 * q + 2] * g,
                           acc[mi][ni][4 * q + 3] * g};
        if constexpr (sizeof(T) == 2)
          *(u32x2_t*)(slab + row * NC * 16 + (((mi * 4 + q) ^ (row & (NC - 1))) * 16) + hf * 8) =
              (u32x2_t){pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        else
          *(f32x4_t*)(slab + row * NC * 16 + (((mi * 8 + 2 * q + hf) ^ (row & (NC - 1))) * 16)) = x;
      }
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < NI * NC / 2; ++i) {
    const int row = i * (64 / NC) + lane / NC, c = lane % NC;
    const u32x4_t x = *(const u32x4_t*)(slab + row * NC * 16 + ((c ^ (row & (NC - 1))) * 16));
    const int v = vw + row, d = dw + c * CH;
    if (v >= a.v || d >= a.d) continue;
    T* p = (T*)a.dw + (int64_t)v * a.ld_dw + d;
    if (d + CH <= a.d) {
      __builtin_memcpy(p, &x, 16);        // (one store, aligned or not)
    } else {
      T y[CH];
      __builtin_memcpy(y, &x, 16);
#pragma unroll
      for (int e = 0; e < CH; ++e)
        if (d + e < a.d) p[e] = y[e];
    }
  }
}

// Both gradients in one launch: they need only dz, and the tiles of one fill
// the CUs that the last round of the other's leaves idle (the 50304 x 768
// weight's 591 tiles are 2.3 rounds of the 256 CUs). The kind with the longer
// tiles comes first. In few rounds each kind is dealt to the XCDs by itself,
// the first to the blocks below `first`; in many (first = 0) one follows the
// other, which leaves the runs whole (8192 x 50304 x 2048: 3.73 / 3.82 ms).
// Bound by the matrix cores at their clock under this load (busy 86 % of the time
// at 1.6 GHz; memory kernels run at 2.2). Measured: 8192 x 50304 x 768 1003 us
// (1260 TFLOP/s of both products), 6963 x 50304 x 2048 2256 (1270), 16 x 3200 x
// 256 6; fp32 777 x 8191 x 331 91 (83).
template <typename T, int TILE, int S>
__global__ __launch_bounds__((waves_of<T, TILE>() * 64), S > 5 ? 1 : 2) void k_gradients_mfma(HeadArgs a, int vt, int tt, int nd,
                                                                                  int weight_first, int first) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * TILE * 128];
  const int rows = piece_rows(a);
  const int nt = min(tt, (rows + TILE - 1) / TILE), n_h = nt * nd * a.split, n_w = vt * nd * a.wsplit;
  const int n_first = weight_first ? n_w : n_h, n_second = n_h + n_w - n_first;
  int idx;
  bool in_first = (int)blockIdx.x < first;
  if (in_first) {
    idx = xcd_index(blockIdx.x, n_first);
    if (idx >= n_first) return;
  } else {
    const int before = first ? 0 : n_first, n = before + n_second;
    idx = xcd_index(blockIdx.x - first, n + 1);     // (the last item is the sum of the losses)
    if (idx == n && a.last && !a.per_token) total_loss<waves_of<T, TILE>() * 64>(a, (double*)smem);
    if (idx >= n) return;
    in_first = idx < before;
    if (!in_first) idx -= before;
  }
  const bool weight = in_first == (weight_first != 0);
  if (weight) {
    const int q = idx / (vt * nd);
    int vi, di;
    if (strip_tile<8>(idx - q * vt * nd, vt, nd, vi, di)) dweight_tile<T, TILE, S>(a, smem, vi, di, q, rows);
  } else {
    const int q = idx / (nt * nd), t = idx - q * nt * nd;
    dhidden_tile<T, TILE, S>(a, smem, t / nd, t % nd, q, rows);
  }
}

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
// blocks for up to n tiles dealt to the XCDs (xcd_index; a launch with fewer
// tiles never needs more)
inline int xcd_grid(int n) { return 8 * rounds_of(n) * run_of(n, rounds_of(n)); }

// Tile edge of a launch, from its number of 256-tiles: with few of them
// 128-tiles, four times as many and two to a CU, cover the CUs better, and
// 64-tiles where those are few in turn. Measured:
//   128 / 256, bf16, loss alone: 384 tiles 62.7 / 67.6 us, 591 170.5 / 174.4,
//   768 113.6 / 103.6, 1182 142.8 / 136.8; whole calls with gradients: 708
//   249 / 253, 825 470 / 459, 1760 916 / 764
//   64 / 128, bf16, loss alone: 64 tiles 22.1 / 25.9 us, 200 18.0 / 18.7, 393
//   39.2 / 34.0, 471 23.6 / 21.5; gradients without the loss: 350 32.7 / 33.7,
//   410 60.5 / 57.8, 2358 65 / 55
// fp32's matrix instructions are slow enough to hide the operand traffic of
// 64-tiles, which it always takes (loss alone, 64 / 128: 777 x 8191 x 331 64 /
// 66 us, 300 x 50304 x 768 211 / 247, 1987 x 30961 x 704 686 / 685, 4000 x 3000
// x 1024 215 / 211; 256-tiles would not fit the registers).
constexpr int kFewTiles = 768, kFewSmallTiles = 384;
// Tokens that fill at most half of a 256-tile: 128-tiles however large the
// vocabulary (128 / 256, 200000 x 768: 1 token 78.9 / 103.4 us, 64 96.1 / 118.1,
// 128 108.1 / 126.0, 129 139.3 / 129.1; 262144 x 2048: 128 279.8 / 307.4, 129
// 350.4 / 310.4).
constexpr int kHalfTile = 128;
// 64-tiles that all fit the chip two to a CU: a ring of nine slots, whose loads
// are asked for three and a half stages ahead. Such a launch reads its operands
// for the first time, and a stage waits for memory rather than for its products.
constexpr int kDeepTiles = 512;
int tile_of(int dt, int rows, int64_t tiles256, int64_t tiles128) {
  if (dt != MUON_BF16) return 64;
  if (tiles256 >= kFewTiles && rows > kHalfTile) return 256;
  return tiles128 >= kFewSmallTiles ? 128 : 64;
}
// Statistics with entropy of one row of tokens: 64-tiles that all run at once, four
// to a CU, which is worth a little for the narrower heads (one token x 50304 x 768:
// 64 / 128 16.6 / 18.1 us; whole calls, weights in turn: one token x 50304 x 768 24.3 /
// 25.2, x 65536 x 768 28.5 / 29.2, x 65536 x 2048 72.4 / 74.1, x 32000 x 768 to 4096
// within 2 %, x 50304 x 2048 60.1 / 57.5, 64 tokens there 64.6 / 59.2; more tiles than
// that: 128000 x 2048 134.7 / 126.0). The loss alone keeps the order of its sums.
constexpr int kAllSmallTiles = 1024;
// The gradients' tiles also go by their own shape (whole calls):
//   few tokens: dW's K is short, its tiles all start-up and epilogue, which two
//   workgroups to a CU overlap (128 / 256: 300 tokens x 50304 x 2048 338 / 384
//   us, 700 tokens 587 / 556); from there on 128 also pays with fewer tiles
//   (64 / 128, 1000 x 8000: width 256, 158 tiles, 55.0 / 52.0 us)
//   narrow: a 256-tile would be mostly padding (4000 x 44000, 128 / 256: width
//   64 430 / 457 us, 128 458 / 488, 192 528 / 506)
constexpr int kShortK = 512, kNarrow = 128;
int grad_tile_of(int dt, int rows, int dp, int64_t tiles256, int64_t tiles128) {
  if (dt != MUON_BF16) return 64;
  if (rows >= kShortK && dp > kNarrow && tiles256 >= kFewTiles) return 256;
  return tiles128 >= (rows >= kShortK ? 128 : kFewSmallTiles) ? 128 : 64;
}

}  // namespace

template <LogitsMode MODE>
static hipError_t launch_logits(const HeadArgs& a, int dt, int keep, hipStream_t s) {
  const int tile = a.logit_tile, vt = cdiv(a.v, tile), tt = cdiv(a.rows_max, tile);
  const bool deep = tile == 64 && (int64_t)vt * tt <= kDeepTiles, few = a.n <= 32;
  const dim3 g(xcd_grid(vt * tt)), b(dt != MUON_BF16 && !few ? 256 : tile * 2);
#define LOGITS_OF(T, TILE, S, FEW, GATHER) \
  hipLaunchKernelGGL((k_logits_mfma<T, TILE, S, FEW, GATHER, MODE>), g, b, 0, s, a, keep, vt, tt)
  // (the gradient reads its rows from panels, which dW needs)
#define LOGITS(T, TILE, S, FEW)                                                      \
  do {                                                                               \
    if (MODE != LOGITS_GRAD && a.gather) LOGITS_OF(T, TILE, S, FEW, MODE != LOGITS_GRAD); \
    else LOGITS_OF(T, TILE, S, FEW, false);                                          \
  } while (0)
  if (dt == MUON_BF16) {
    if (tile == 256) LOGITS_OF(u16, 256, 5, false, false);
    else if (tile == 128) LOGITS(u16, 128, 5, false);
    else if (deep) LOGITS(u16, 64, 9, false);
    else LOGITS(u16, 64, 5, false);
  } else {
    if (deep && few) LOGITS(float, 64, 9, true);
    else if (deep) LOGITS(float, 64, 9, false);
    else if (few) LOGITS(float, 64, 5, true);
    else LOGITS(float, 64, 5, false);
  }
#undef LOGITS
#undef LOGITS_OF
  return hipGetLastError();
}
hipError_t launch_head_logits(const HeadArgs& a, int dt, int keep, LogitsMode mode, hipStream_t s) {
  if (mode == LOGITS_STATS) return launch_logits<LOGITS_STATS>(a, dt, 0, s);
  if (mode == LOGITS_GRAD) return launch_logits<LOGITS_GRAD>(a, dt, 0, s);
  return launch_logits<LOGITS_LOSS>(a, dt, keep, s);
}

hipError_t launch_head_gradients(const HeadArgs& a, int dt, hipStream_t s) {
  const int rows = a.rows_max, unit = dt == MUON_BF16 ? 64 : 32, tile = a.grad_tile;
  const int tt = a.dh ? cdiv(rows, tile) : 0, vt = a.dw ? cdiv(a.v, tile) : 0, nd = cdiv(a.dp, tile);
  // the longer tiles go first
  const int wf = cdiv(rows, unit) / a.wsplit > cdiv(a.v, unit) / a.split;
  const int n_h = tt * nd * a.split, n_w = vt * nd * a.wsplit, tiles = n_h + n_w, n_first = wf ? n_w : n_h;
  const int first = rounds_of(tiles) > kEvenRounds || n_first == 0 ? 0 : xcd_grid(n_first);
  const dim3 g(first + xcd_grid(tiles + 1 - (first ? n_first : 0))), b(dt == MUON_BF16 ? tile * 2 : 256);
  const bool deep = tile == 64 && tiles <= kDeepTiles;
#define GRADIENTS(T, ...) hipLaunchKernelGGL((k_gradients_mfma<T, __VA_ARGS__>), g, b, 0, s, a, vt, tt, nd, wf, first)
  if (dt == MUON_BF16) {
    if (tile == 256) GRADIENTS(u16, 256, 5);
    else if (tile == 128) GRADIENTS(u16, 128, 5);
    else if (deep) GRADIENTS(u16, 64, 9);
    else GRADIENTS(u16, 64, 5);
  } else {
    if (deep) GRADIENTS(float, 64, 9);
    else GRADIENTS(float, 64, 5);
  }
#undef GRADIENTS
  return hipGetLastError();
}

// Tile edges of the products, columns per statistic, and the parts in which dH
// goes over the vocabulary and dW over the piece's tokens: the tiles alone
// (tokens x width, vocabulary x width) can be fewer than the CUs. The
// gradients' launch lasts its stages over the CUs, each tile with the ring's
// start-up, half of its shorter kind at the end, and no less than its longest
// tile; then the partial sums' traffic and the launch that adds them. Counted
// in stages, whose length, as start-up and traffic, follows from the tile and
// type (a least-squares choice over 300 shapes of 64 to 16384 tokens: calls
// within 0.3 % (256), 1.1 % (128), 0.6 % (64) and 1.7 % (fp32) of the best
// parts). dW's parts measured (1 / chosen): 16384 x 6000 x 256 350 / 324 us,
// 65536 x 256 x 512 646 / 250, fp32 2000 x 300 x 128 78 / 37.
void head_plan(HeadArgs& a, int dt, LogitsMode mode) {
  const int rows = a.n < a.piece ? a.n : a.piece, unit = dt == MUON_BF16 ? 64 : 32;
  a.logit_tile = tile_of(dt, rows, (int64_t)cdiv(a.v, 256) * cdiv(rows, 256), (int64_t)cdiv(a.v, 128) * cdiv(rows, 128));
  if (mode == LOGITS_STATS && rows <= 64 && cdiv(a.v, 64) <= kAllSmallTiles) a.logit_tile = 64;
  a.vtile = a.logit_tile == 64 ? 64 : 128;
  a.n_vt = cdiv(a.v, a.vtile);
  a.sets = a.vtile / (dt == MUON_BF16 ? kSetRows<u16> : kSetRows<float>) * 2;
  a.split = a.wsplit = 1;
  if (!a.dh && !a.dw) return;
  const int64_t stages = cdiv(a.v, unit), wstages = cdiv(rows, unit);
  auto tiles_of = [&](int edge) {
    return (a.dw ? (int64_t)cdiv(a.v, edge) * cdiv(a.dp, edge) : 0) +
           (a.dh ? (int64_t)cdiv(rows, edge) * cdiv(a.dp, edge) * (stages / 64 + 1) : 0);
  };
  a.grad_tile = grad_tile_of(dt, rows, a.dp, tiles_of(256), tiles_of(128));
  const int tile = a.grad_tile, slots = 256 * (256 / tile);
  const int64_t h_tiles = a.dh ? (int64_t)cdiv(rows, tile) * cdiv(a.dp, tile) : 0;
  const int64_t w_tiles = a.dw ? (int64_t)cdiv(a.v, tile) * cdiv(a.dp, tile) : 0;
  // start-up, the sums' launch, and bytes of traffic in a stage's time (2 us of
  // a 256-tile, 0.7, 1, and 1.8 of fp32)
  const bool half = dt == MUON_BF16;
  const double start = half && tile == 64 ? 10 : 6, launch = half ? (tile == 256 ? 3 : 4) : 2;
  const double bytes = !half ? 8e6 : tile == 256 ? 9e6 : tile == 128 ? 1.6e6 : 4.5e6;
  const double h_sum = (double)rows * a.dp * 8 / bytes, w_sum = (double)a.v * a.dp * 8 / bytes;
  // (partial sums stay within 256 MB, and a part has four stages or more)
  const int h_most = a.dh ? (int)std::min<double>(std::min<int64_t>(256, stages / 4), 256e6 / ((double)a.piece * a.dp * 4)) : 1;
  const int w_most = a.dw ? (int)std::min<double>(std::min<int64_t>(256, wstages / 4), 256e6 / ((double)a.v * a.dp * 4)) : 1;
  double least = 0;
  for (int m = 1; m == 1 || m <= w_most; m *= 2) {
    for (int n = 1; n == 1 || n <= h_most; n += (n + 7) / 8) {
      const double h_each = a.dh ? cdiv(stages, n) + start : 0, w_each = a.dw ? cdiv(wstages, m) + start : 0;
      const double shorter = !a.dh ? w_each : !a.dw ? h_each : std::min(h_each, w_each);
      double t = std::max((h_tiles * n * h_each + w_tiles * m * w_each) / slots + shorter / 2, std::max(h_each, w_each));
      t += (n > 1 ? n * h_sum : 0) + (m > 1 ? m * w_sum : 0) + (n > 1 || m > 1 ? launch : 0);
      // (more parts of dW for a gain that the model can tell)
      if ((n == 1 && m == 1) || t < (m > a.wsplit ? 0.95 : 1.0) * least) {
        least = t;
        a.split = n;
        a.wsplit = m;
      }
    }
    if (2.0 * (cdiv(wstages, m) + start) < least) break;     // dW's tiles are not what it waits for
  }
}

}  // namespace muon
