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
// Bound by HBM: each row is read once and held in registers, the next one is on
// its way meanwhile. 8192 rows with all their gradients, forward / backward (and
// the sums of its partials): 768 channels bf16 10.5 us (4.8 TB/s) / 17 (4.4; 4),
// 2048 of fp32 beside bf16 37.5 (5.4) / 55 (5.5; 5).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "head_device.hpp"
#include "norm.hpp"
#include "wave.hpp"

namespace muon {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// A thread's chunk of CH (4 or 8) channels from c of a row of d, as in memory: one
// or two loads where whole, aligned or not. TAIL: whether a row can end inside a
// chunk. Such a chunk and those past it are the row's last CH channels, until
// `ended` moves them to their places and zeros behind: no load waits for a branch
// (8192 x 1023 bf16, channel by channel / so: forward 18.7 / 14.7 us, backward 49 /
// 29). SHORT rows, which can have fewer channels than a chunk and end in every wave,
// take theirs channel by channel, the last one past the end (16384 x 100: 7.1, moved 9.3).
template <typename T, int CH>
struct Raw {
  uint32_t w[CH * sizeof(T) / 4];
};
template <bool TAIL, bool SHORT, typename T, int CH>
__device__ __forceinline__ void load_raw(const T* row, int c, int d, Raw<T, CH>& v) {
  if constexpr (TAIL && !SHORT) {
    __builtin_memcpy(&v, row + min(c, d - CH), sizeof(v));
  } else if (c + CH <= d) {
    __builtin_memcpy(&v, row + c, sizeof(v));
  } else if (!TAIL) {
    v = {};
  } else {
    T x[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) x[e] = row[min(c + e, d - 1)];
#pragma unroll
    for (int e = 0; e < CH; ++e) x[e] = c + e < d ? x[e] : T(0);
    __builtin_memcpy(&v, x, sizeof(v));
  }
}
// Channels from k on to the front, zeros behind.
template <typename T, int CH>
__device__ __forceinline__ void move_down(Raw<T, CH>& v, int k) {
  constexpr int N = CH * sizeof(T) / 4;
  const int words = k * (int)sizeof(T) / 4;
#pragma unroll
  for (int step = N / 2; step; step /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) v.w[i] = words & step ? (i + step < N ? v.w[i + step] : 0u) : v.w[i];
  if (sizeof(T) == 2 && (k & 1))
#pragma unroll
    for (int i = 0; i < N; ++i) v.w[i] = v.w[i] >> 16 | (i + 1 < N ? v.w[i + 1] << 16 : 0u);
#pragma unroll
  for (int i = 0; i < N; ++i) v.w[i] = words < N ? v.w[i] : 0u;
}
template <bool TAIL, bool SHORT, typename T, int CH>
__device__ __forceinline__ void ended(Raw<T, CH>& v, int c, int d) {
  if (TAIL && !SHORT && c + CH > d) move_down(v, c + CH - d);
}
template <typename T, int CH>
__device__ __forceinline__ void unpack(const Raw<T, CH>& r, float (&v)[CH]) {
#pragma unroll
  for (int e = 0; e < CH; ++e) {
    if constexpr (sizeof(T) == 2) v[e] = __uint_as_float(e & 1 ? r.w[e / 2] & 0xFFFF0000u : r.w[e / 2] << 16);
    else v[e] = __uint_as_float(r.w[e]);
  }
}
template <bool TAIL, bool SHORT, int CH, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int c, int d, float (&v)[CH]) {
  Raw<T, CH> r;
  load_raw<TAIL, SHORT>(row, c, d, r);
  ended<TAIL, SHORT>(r, c, d);
  unpack(r, v);
}
template <bool TAIL, int CH, typename T>
__device__ __forceinline__ void store_chunk(T* row, int c, int d, const float (&v)[CH]) {
  if (c + CH <= d) {
    Raw<T, CH> r;
#pragma unroll
    for (int e = 0; e < CH; ++e) {
      if constexpr (sizeof(T) == 2) r.w[e / 2] = e & 1 ? pack_bf16(v[e & ~1], v[e]) : 0u;
      else r.w[e] = __float_as_uint(v[e]);
    }
    __builtin_memcpy(row + c, &r, sizeof(r));
  } else if (TAIL) {
#pragma unroll
    for (int e = 0; e < CH; ++e)
      if (c + e < d) {
        if constexpr (sizeof(T) == 2) row[c + e] = f2bf(v[e]);
        else row[c + e] = v[e];
      }
  }
}

__device__ __forceinline__ float one_value(const NormParam& p, int64_t i) {
  return p.half ? bf2f(((const u16*)p.ptr)[i]) : ((const float*)p.ptr)[i];
}
// A parameter's chunk (1 where it is not there; NORM_FULL is the rows').
template <bool TAIL, bool SHORT, int CH>
__device__ __forceinline__ void load_param(const NormParam& p, int c, int d, float (&v)[CH]) {
  if (p.kind == NORM_CHANNELS) {
    if (p.half) load_chunk<TAIL, SHORT>((const u16*)p.ptr, c, d, v);
    else load_chunk<TAIL, SHORT>((const float*)p.ptr, c, d, v);
  } else {
    const float x = p.kind == NORM_ONE ? one_value(p, 0) : 1.f;
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] = x;
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

// A row's operands, loaded together and, where the registers hold two, one row
// ahead of their use. Three forms, kept apart for the registers that they take:
// rows of whole chunks, rows that can end inside one (TAIL), and with a gate for
// each element or a scale for each channel (MORE, which has TAIL).
enum NormForm { FORM_WHOLE, FORM_TAIL, FORM_MORE };
template <typename TX, typename TY, int TPR, int NC, int CH, int FORM, bool BACKWARD>
struct Row {
  static constexpr bool TAIL = FORM != FORM_WHOLE, MORE = FORM == FORM_MORE;
  static constexpr bool SHORT = TPR == 16, LATER = TPR == 1024;   // (LATER: loaded where needed)
  Raw<TX, CH> x[NC], dout[BACKWARD ? NC : 1];
  Raw<TY, CH> y[NC], g[MORE ? NC : 1], dhidden[BACKWARD ? NC : 1];
  __device__ __forceinline__ void load(const NormArgs& a, int64_t r, int t) {
    auto rows = [&](auto& to, const void* p, int64_t ld, auto type) {
      typedef decltype(type) T;
#pragma unroll
      for (int k = 0; k < NC; ++k) load_raw<TAIL, SHORT>((const T*)p + r * ld, CH * (k * TPR + t), a.d, to[k]);
    };
    rows(x, a.x.ptr, a.x.ld, TX());
    if (a.y.ptr) rows(y, a.y.ptr, a.y.ld, TY());
    if constexpr (BACKWARD && !LATER) {
      if (a.dhidden.ptr) rows(dhidden, a.dhidden.ptr, a.dhidden.ld, TY());
      if (a.dout.ptr) rows(dout, a.dout.ptr, a.dout.ld, TX());
    }
    if constexpr (MORE)
      if (a.gate.kind == NORM_FULL) rows(g, a.gate.ptr, a.gate.ld, TY());
  }
  // (before the first use)
  __device__ __forceinline__ void arrived(int d, int t) {
    if constexpr (TAIL && !SHORT) {
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int c = CH * (k * TPR + t);
        if (c + CH <= d) continue;
        ended<TAIL, SHORT>(x[k], c, d);
        ended<TAIL, SHORT>(y[k], c, d);
        ended<TAIL, SHORT>(g[MORE ? k : 0], c, d);
        if constexpr (BACKWARD && !LATER) {
          ended<TAIL, SHORT>(dhidden[k], c, d);
          ended<TAIL, SHORT>(dout[k], c, d);
        }
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ static void load_late(const NormRows& m, int64_t r, int c, int d, Raw<T, CH>& v) {
    load_raw<TAIL, SHORT>((const T*)m.ptr + r * m.ld, c, d, v);
    ended<TAIL, SHORT>(v, c, d);
  }
};

// TPR threads to a row, NC chunks of CH channels to a thread; the threads past TPR
// of a block have other rows.
template <typename TX, typename TY, int TPR, int NC, int CH, int BLOCK, int FORM>
__global__ __launch_bounds__(BLOCK) void k_residual_norm(NormArgs a) {
  constexpr int ROWS = BLOCK / TPR;
  constexpr bool TAIL = FORM != FORM_WHOLE, MORE = FORM == FORM_MORE;
  constexpr bool AHEAD = NC * CH <= 12 || TPR <= 64;
  __shared__ float sh[2][BLOCK / 64];
  const int t = threadIdx.x % TPR, d = a.d;
  const float inv_d = 1.f / d;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  // (every thread of a block goes round as often; rows past the last one are
  // the last one again and are not stored)
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  Row<TX, TY, TPR, NC, CH, FORM, false> now, next;
  if (AHEAD) next.load(a, min(row, a.n - 1), t);
  const bool there = a.y.ptr != nullptr;
  float gate[NC][CH], pre[NC][CH], scale[MORE ? NC : 1][CH];
  const float scale1 = a.scale.kind == NORM_ONE ? one_value(a.scale, 0) : 1.f;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = CH * (k * TPR + t);
    float post[CH];
    if (MORE) load_param<TAIL, TPR == 16>(a.scale, c, d, scale[MORE ? k : 0]);
    load_param<TAIL, TPR == 16>(a.pre_gain, c, d, pre[k]);
    load_param<TAIL, TPR == 16>(a.post_gain, c, d, post);
    load_param<TAIL, TPR == 16>(a.gate, c, d, gate[k]);
#pragma unroll
    for (int e = 0; e < CH; ++e) gate[k][e] *= post[e];
  }
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.n; r0 += step, row += step) {
    const bool real = row < a.n;
    if (AHEAD) {
      now = next;
      if (r0 + step < a.n) next.load(a, min(row + step, a.n - 1), t);
    } else {
      now.load(a, min(row, a.n - 1), t);
    }
    now.arrived(d, t);
    float x[NC][CH], s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      unpack(now.x[k], x[k]);
      if (a.scale.ptr)
#pragma unroll
        for (int e = 0; e < CH; ++e) x[k][e] *= MORE ? scale[MORE ? k : 0][e] : scale1;
    }
    if (there) {
      float y[NC][CH], r1 = 1.f;
#pragma unroll
      for (int k = 0; k < NC; ++k) unpack(now.y[k], y[k]);
      if (a.post) {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < CH; ++e) s[0] = fmaf(y[k][e], y[k][e], s[0]);
        row_sums<TPR>(s, sh[0]);
        r1 = rsqrtf(fmaf(s[0], inv_d, a.eps));
      }
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        if (MORE && a.gate.kind == NORM_FULL) {
          float g[CH];
          unpack(now.g[MORE ? k : 0], g);
#pragma unroll
          for (int e = 0; e < CH; ++e) y[k][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < CH; ++e) x[k][e] = fmaf(y[k][e] * r1, gate[k][e], x[k][e]);
      }
    }
    if (a.out.ptr && real)
#pragma unroll
      for (int k = 0; k < NC; ++k) store_chunk<TAIL>((TX*)a.out.ptr + row * a.out.ld, CH * (k * TPR + t), d, x[k]);
    if (a.pre) {
      s[0] = 0.f;
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int e = 0; e < CH; ++e) s[0] = fmaf(x[k][e], x[k][e], s[0]);
      row_sums<TPR>(s, sh[1]);
      const float r2 = rsqrtf(fmaf(s[0], inv_d, a.eps));
      if (real)
#pragma unroll
        for (int k = 0; k < NC; ++k) {
#pragma unroll
          for (int e = 0; e < CH; ++e) x[k][e] *= r2 * pre[k][e];
          store_chunk<TAIL>((TY*)a.hidden.ptr + row * a.hidden.ld, CH * (k * TPR + t), d, x[k]);
        }
    }
    if (TPR > 64 && r0 + step < a.n) __syncthreads();   // the sums are read before the next row's are written
  }
}

template <int CH>
__device__ __forceinline__ void add_products(const float (&a)[CH], const float (&b)[CH], double& sum) {
#pragma unroll
  for (int e = 0; e < CH; e += 4)
    sum += (double)(fmaf(a[e], b[e], a[e + 1] * b[e + 1]) + fmaf(a[e + 2], b[e + 2], a[e + 3] * b[e + 3]));
}

// Waves to a SIMD that the backward pass is compiled for, where rows have several
// waves: as many as the registers hold (a second raw row of 32-bit operands takes
// twice as many), and four where a block alone has eight.
constexpr int waves_wanted(int tpr, int nc, bool more, int bytes) {
  return tpr <= 64 || nc > 1 || more ? 1 : bytes == 2 || tpr > 256 ? 4 : 3;
}
template <typename TX, typename TY, int TPR, int NC, int CH, int BLOCK, int FORM>
__global__ __launch_bounds__(BLOCK, waves_wanted(TPR, NC, FORM == FORM_MORE, sizeof(TX))) void k_residual_norm_grad(NormArgs a) {
  constexpr int ROWS = BLOCK / TPR;
  constexpr bool TAIL = FORM != FORM_WHOLE, MORE = FORM == FORM_MORE;
  // what the registers hold: the parameters (wide rows read these and the results'
  // gradients again where they are needed), and a second row (4096 x 4096 of 32
  // bits, with / without 117 / 88 us: it does not fit beside eight waves)
  constexpr bool WIDE = TPR == 1024, AHEAD = !WIDE && !(TPR >= 512 && sizeof(TX) == 4);
  __shared__ float sh[3][2 * (BLOCK / 64)];
  __shared__ double ones[BLOCK / 64][2];
  __shared__ float joined[ROWS > 1 ? BLOCK * CH : 1];
  const int t = threadIdx.x % TPR, d = a.d;
  const float inv_d = 1.f / d;
  const bool there = a.y.ptr != nullptr, full = MORE && a.gate.kind == NORM_FULL, normed = a.dhidden.ptr != nullptr;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  Row<TX, TY, TPR, NC, CH, FORM, true> now, next;
  if (AHEAD) next.load(a, min(row, a.n - 1), t);
  // gate and post_gain multiplied (post_gain alone where the gate is full or single:
  // a single one's gradient takes what comes to yhat without it)
  const float gate1 = a.gate.kind == NORM_ONE ? one_value(a.gate, 0) : 1.f;
  auto load_gated = [&](int k, float (&v)[CH]) {
    const int c = CH * (k * TPR + t);
    load_param<TAIL, TPR == 16>(a.post_gain, c, d, v);
    if (a.gate.kind == NORM_CHANNELS) {
      float gate[CH];
      load_param<TAIL, TPR == 16>(a.gate, c, d, gate);
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] *= gate[e];
    }
  };
  float scale[MORE ? NC : 1][CH], gated[WIDE ? 1 : NC][CH], pre[WIDE ? 1 : NC][CH];
  const float scale1 = a.scale.kind == NORM_ONE ? one_value(a.scale, 0) : 1.f;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    if (MORE) load_param<TAIL, TPR == 16>(a.scale, CH * (k * TPR + t), d, scale[MORE ? k : 0]);
    if (!WIDE) {
      load_param<TAIL, TPR == 16>(a.pre_gain, CH * (k * TPR + t), d, pre[WIDE ? 0 : k]);
      load_gated(k, gated[WIDE ? 0 : k]);
    }
  }
  auto gated_of = [&](int k) -> float (&)[CH] {
    if (WIDE) load_gated(k, gated[0]);
    return gated[WIDE ? 0 : k];
  };
  auto pre_of = [&](int k) -> float (&)[CH] {
    if (WIDE) load_param<TAIL, TPR == 16>(a.pre_gain, CH * (k * TPR + t), d, pre[0]);
    return pre[WIDE ? 0 : k];
  };
  auto scale_of = [&](int k, int e) { return MORE ? scale[MORE ? k : 0][e] : scale1; };
  // the channels' sums over the rows: of wide rows in LDS, a thread's own (1024 x
  // 16384 bf16, in registers / so: 112 / 76 us)
  constexpr int KEPT = WIDE ? NC * CH / 4 * BLOCK : 1;
  __shared__ f32x4_t kept[2][KEPT];
  auto fetch = [&](float (&sum)[CH], int which, int k) {
    if (WIDE)
#pragma unroll
      for (int e = 0; e < CH; e += 4) {
        const f32x4_t v = kept[which][(k * (CH / 4) + e / 4) * BLOCK + threadIdx.x];
        sum[e] = v[0], sum[e + 1] = v[1], sum[e + 2] = v[2], sum[e + 3] = v[3];
      }
  };
  auto keep = [&](const float (&sum)[CH], int which, int k) {
    if (WIDE)
#pragma unroll
      for (int e = 0; e < CH; e += 4)
        kept[which][(k * (CH / 4) + e / 4) * BLOCK + threadIdx.x] = (f32x4_t){sum[e], sum[e + 1], sum[e + 2], sum[e + 3]};
  };
  const bool vector = a.want & kWantBlock, gate_sum = (a.want & kWantGateOne) && a.post_gain.ptr;
  float sum_block[WIDE ? 1 : NC][CH], sum_scale[MORE ? NC : 1][CH], sum_pre[WIDE ? 1 : NC][CH];
  // (single values are sums over all elements, which may cancel: 64 bits past four, or
  // beside a post_gain past a thread's part of a row, which the way back has anyway)
  double gate_one = 0, scale_one = 0;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
#pragma unroll
    for (int e = 0; e < CH; ++e) sum_block[WIDE ? 0 : k][e] = sum_scale[MORE ? k : 0][e] = sum_pre[WIDE ? 0 : k][e] = 0.f;
    keep(sum_block[0], 0, k);
    keep(sum_pre[0], 1, k);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.n; r0 += step, row += step) {
    const bool real = row < a.n;
    if (AHEAD) {
      now = next;
      if (r0 + step < a.n) next.load(a, min(row + step, a.n - 1), t);
    } else {
      now.load(a, min(row, a.n - 1), t);
    }
    now.arrived(d, t);
    const int64_t at = min(row, a.n - 1);
    // y becomes yhat, o the row's out
    float y[NC][CH], o[NC][CH], r1 = 1.f;
    if (there) {
#pragma unroll
      for (int k = 0; k < NC; ++k) unpack(now.y[k], y[k]);
      if (a.post) {
        float q[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < CH; ++e) q[0] = fmaf(y[k][e], y[k][e], q[0]);
        row_sums<TPR>(q, sh[0]);
        r1 = rsqrtf(fmaf(q[0], inv_d, a.eps));
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < CH; ++e) y[k][e] *= r1;
      }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      unpack(now.x[k], o[k]);
      if (a.scale.ptr)
#pragma unroll
        for (int e = 0; e < CH; ++e) o[k][e] *= scale_of(k, e);
      if (there) {
        float g[CH];
        if (full) unpack(now.g[MORE ? k : 0], g);
        const float (&w)[CH] = gated_of(k);
#pragma unroll
        for (int e = 0; e < CH; ++e) o[k][e] = fmaf(full ? w[e] * g[e] : w[e] * gate1, y[k][e], o[k][e]);
      }
    }
    float r2 = 0.f, m = 0.f;
    if (normed) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        float u[CH];
        if (WIDE) now.load_late(a.dhidden, at, CH * (k * TPR + t), d, now.dhidden[0]);
        unpack(now.dhidden[WIDE ? 0 : k], u);
        const float (&w)[CH] = pre_of(k);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          s[0] = fmaf(o[k][e], o[k][e], s[0]);
          s[1] = fmaf(o[k][e], u[e] * w[e], s[1]);
        }
      }
      row_sums<TPR>(s, sh[1]);
      r2 = rsqrtf(fmaf(s[0], inv_d, a.eps));
      m = s[1] * r2 * inv_d;
    }
    // o becomes dT, then what comes to yhat
    float v[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = CH * (k * TPR + t);
      float dt[CH], x[CH];
      if (a.dout.ptr) {
        if (WIDE) now.load_late(a.dout, at, c, d, now.dout[0]);
        unpack(now.dout[WIDE ? 0 : k], dt);
      } else {
#pragma unroll
        for (int e = 0; e < CH; ++e) dt[e] = 0.f;
      }
      if (normed) {
        float u[CH];
        if (WIDE) now.load_late(a.dhidden, at, CH * (k * TPR + t), d, now.dhidden[0]);
        unpack(now.dhidden[WIDE ? 0 : k], u);
        const float (&w)[CH] = pre_of(k);
        float (&sum)[CH] = sum_pre[WIDE ? 0 : k];
        fetch(sum, 1, k);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          const float xh = o[k][e] * r2;
          dt[e] += r2 * (u[e] * w[e] - xh * m);
          if (real) sum[e] = fmaf(u[e], xh, sum[e]);
        }
        keep(sum, 1, k);
      }
      if (a.dx.ptr && real) {
        float q[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e) q[e] = a.scale.ptr ? dt[e] * scale_of(k, e) : dt[e];
        store_chunk<TAIL>((TX*)a.dx.ptr + row * a.dx.ld, c, d, q);
      }
      if ((a.want & (kWantScale | kWantScaleOne)) && real) {
        unpack(now.x[k], x);
#pragma unroll
        for (int e = 0; e < CH; ++e)
          if (MORE && (a.want & kWantScale)) sum_scale[MORE ? k : 0][e] = fmaf(dt[e], x[e], sum_scale[MORE ? k : 0][e]);
        if (a.want & kWantScaleOne) add_products(dt, x, scale_one);
      }
      if (there) {
        float g[CH];
        if (full) unpack(now.g[MORE ? k : 0], g);
        const float (&w)[CH] = gated_of(k);
        if (full && a.dfull.ptr && real) {
          float q[CH];
#pragma unroll
          for (int e = 0; e < CH; ++e) q[e] = dt[e] * w[e] * y[k][e];
          store_chunk<TAIL>((TY*)a.dfull.ptr + row * a.dfull.ld, c, d, q);
        }
        if (vector && real) {
          float (&sum)[CH] = sum_block[WIDE ? 0 : k];
          fetch(sum, 0, k);
#pragma unroll
          for (int e = 0; e < CH; ++e) sum[e] = fmaf(full ? dt[e] * g[e] : dt[e], y[k][e], sum[e]);
          keep(sum, 0, k);
        }
        if ((a.want & kWantGateOne) && !a.post_gain.ptr && real) add_products(dt, y[k], gate_one);
#pragma unroll
        for (int e = 0; e < CH; ++e) o[k][e] = dt[e] * (full ? w[e] * g[e] : w[e]);
      }
    }
    if (there && (a.dy.ptr || gate_sum)) {
      if (a.post) {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < CH; ++e) v[0] = fmaf(o[k][e], y[k][e], v[0]);
        if (gate_sum && real) gate_one += (double)v[0];
        row_sums<TPR>(v, sh[2]);
        const float back = v[0] * inv_d, by = r1 * gate1;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < CH; ++e) o[k][e] = by * (o[k][e] - y[k][e] * back);
      } else {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < CH; ++e) o[k][e] *= gate1;
      }
      if (a.dy.ptr && real)
#pragma unroll
        for (int k = 0; k < NC; ++k) store_chunk<TAIL>((TY*)a.dy.ptr + row * a.dy.ld, CH * (k * TPR + t), d, o[k]);
    }
    if (TPR > 64) __syncthreads();   // the sums are read before the next row's are written
  }
  // the block's partials: rows' sums joined in order
  float* part = a.part + blockIdx.x * a.part_floats;
  auto leave = [&](auto& sums, int which) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const bool from_lds = WIDE && which < 2;
      float (&sum)[CH] = sums[from_lds ? 0 : k];
      if (from_lds) fetch(sum, which, k);
      if constexpr (ROWS > 1) {
        // (threads of neighbouring chunks next to one another: no bank is asked twice)
        __syncthreads();
#pragma unroll
        for (int e = 0; e < CH; ++e) joined[e * BLOCK + threadIdx.x] = sum[e];
        __syncthreads();
        for (int i = threadIdx.x; i < TPR * CH; i += BLOCK) {
          // (neighbouring threads write neighbouring channels)
          const int of = i / CH, e = i % CH, at = CH * (k * TPR) + i;
          float x = 0.f;
#pragma unroll
          for (int q = 0; q < ROWS; ++q) x += joined[e * BLOCK + q * TPR + of];
          if (at < a.dp) part[at] = x;
        }
      } else {
        const int c = CH * (k * TPR + t);
#pragma unroll
        for (int e = 0; e < CH; e += 4)
          if (c + e < a.dp) *(f32x4_t*)(part + c + e) = (f32x4_t){sum[e], sum[e + 1], sum[e + 2], sum[e + 3]};
      }
    }
    part += a.dp;
  };
  if (a.want & kWantBlock) leave(sum_block, 0);
  if constexpr (MORE)
    if (a.want & kWantScale) leave(sum_scale, 2);
  if (a.want & kWantPre) leave(sum_pre, 1);
  if (a.want & (kWantGateOne | kWantScaleOne)) {
    gate_one = lanes_sum<64>(gate_one);
    scale_one = lanes_sum<64>(scale_one);
    if ((threadIdx.x & 63) == 0) {
      ones[threadIdx.x >> 6][0] = gate_one;
      ones[threadIdx.x >> 6][1] = scale_one;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      double x = 0;
      for (int w = 0; w < BLOCK / 64; ++w) x += ones[w][threadIdx.x];
      const float high = (float)x;
      part[threadIdx.x] = high;
      part[2 + threadIdx.x] = fabsf(high) < __builtin_inff() ? (float)(x - (double)high) : 0.f;
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
      // (loads past the last partial left out one by one: a loop for the rest would wait for each)
      const float* p = a.part + (int64_t)blockIdx.y * a.dp + c;
      for (int b0 = share; b0 < a.blocks; b0 += 32 * 12) {
        float v[12];
#pragma unroll
        for (int k = 0; k < 12; ++k) v[k] = b0 + 32 * k < a.blocks ? p[(b0 + 32 * k) * a.part_floats] : 0.f;
#pragma unroll
        for (int k = 0; k < 12; ++k) x += v[k];
      }
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
      x += (double)p[0] + (double)p[2];
      y += (double)p[1] + (double)p[3];
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

// By the width, RUN(threads to a row, chunks to a thread, channels of a chunk):
// sixteen threads up to 128 channels, a wave up to 512, then as many threads as
// there are chunks. Up to 768 a wave takes three chunks of 4 (two of 8 would leave
// a quarter of its lanes nothing), but for the forward pass of 16-bit rows two
// waves are faster where there are few (two waves / one: one row of 768 3.2 / 4.0 us,
// 8192 9.9 / 9.9, of 32 bits 16.5 / 15.1). Between the two widths, 8192 rows:
// forward, 16 bits, 520 8.7 / 8.4, 640 9.2 / 9.0, 700 11.1 / 9.9, 32 bits beside 16
// 10.1 / 10.3, 11.5 / 11.3, 13.5 / 12.7, 32 bits 13.0 / 11.3, 14.2 / 12.8, 17.1 / 14.5;
// backward 19.7 / 18.9, 20.5 / 20.1, 24.8 / 20.5 and of 32 bits 25.7 / 24.0, 27.0 / 26.6,
// 32.5 / 28.3. Up to 8192 the backward pass has the registers of eight waves for two
// chunks a thread, the forward one of sixteen for one (2048 x 8192: backward 43 / 56
// us, forward 23.5 / 22.5).
#define BY_WIDTH(d, RUN, RUN_768, RUN_8192)               \
  do {                                                    \
    if ((d) <= 128) RUN(16, 1, 8);                        \
    else if ((d) <= 512) RUN(64, 1, 8);                   \
    else if ((d) <= 768) RUN_768;                         \
    else if ((d) <= 1024) RUN(128, 1, 8);                 \
    else if ((d) <= 1536) RUN(192, 1, 8);                 \
    else if ((d) <= 2048) RUN(256, 1, 8);                 \
    else if ((d) <= 4096) RUN(512, 1, 8);                 \
    else if ((d) <= 8192) RUN_8192;                       \
    else RUN(1024, 2, 8);                                 \
  } while (0)

namespace {

// A block of whole rows, of about so many threads.
constexpr int whole_rows(int threads, int about) { return about > threads ? about / threads * threads : threads; }
// Threads of a block: one row where that has a wave or more; several rows in the
// backward pass, whose blocks leave a partial each.
constexpr int kForwardBlock = 64, kBackwardBlock = 512;

// Blocks of a kernel that the device holds at once.
template <typename K>
int resident(K kernel, int block) {
  int device = 0, cus = 256, each = 1;
  if (hipGetDevice(&device) != hipSuccess || hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess ||
      hipOccupancyMaxActiveBlocksPerMultiprocessor(&each, kernel, block, 0) != hipSuccess)
    (void)hipGetLastError();
  return cus * (each > 0 ? each : 1);
}
// As many blocks as go through the rows in the fewest rounds of resident ones,
// all of them as often: a block keeps its parameters and loads a row ahead.
int blocks_of(int64_t n, int rows, int resident) {
  const int64_t blocks = (n + rows - 1) / rows, rounds = (blocks + resident - 1) / resident;
  return (int)((blocks + rounds - 1) / rounds);
}
int form_of(const NormArgs& a, int chunk) {
  if (a.gate.kind == NORM_FULL || a.scale.kind == NORM_CHANNELS) return FORM_MORE;
  return a.d % chunk != 0 ? FORM_TAIL : FORM_WHOLE;
}

template <typename TX, typename TY, int TPR, int NC, int CH, int FORM>
void forward(const NormArgs& a, hipStream_t s) {
  constexpr int BLOCK = whole_rows(TPR, kForwardBlock);
  static const int most = resident(k_residual_norm<TX, TY, TPR, NC, CH, BLOCK, FORM>, BLOCK);
  const dim3 g((unsigned)blocks_of(a.n, BLOCK / TPR, most));
  hipLaunchKernelGGL((k_residual_norm<TX, TY, TPR, NC, CH, BLOCK, FORM>), g, dim3(BLOCK), 0, s, a);
}
// blocks alone, or the launch
template <typename TX, typename TY, int TPR, int NC, int CH, int FORM>
int backward(const NormArgs& a, bool launch, hipStream_t s) {
  constexpr int BLOCK = whole_rows(TPR, kBackwardBlock);
  static const int most = resident(k_residual_norm_grad<TX, TY, TPR, NC, CH, BLOCK, FORM>, BLOCK);
  const int blocks = blocks_of(a.n, BLOCK / TPR, most < kNormMostBlocks ? most : kNormMostBlocks);
  if (launch) hipLaunchKernelGGL((k_residual_norm_grad<TX, TY, TPR, NC, CH, BLOCK, FORM>), dim3(blocks), dim3(BLOCK), 0, s, a);
  return blocks;
}

#define BY_TYPES(f, TPR, NC, CH, ...)                                                    \
  do {                                                                                   \
    const int form = form_of(a, CH);                                                     \
    if (x_half) f##_of<u16, u16, TPR, NC, CH>(form, a, ##__VA_ARGS__, s);                    \
    else if (y_half) f##_of<float, u16, TPR, NC, CH>(form, a, ##__VA_ARGS__, s);             \
    else f##_of<float, float, TPR, NC, CH>(form, a, ##__VA_ARGS__, s);                       \
  } while (0)

template <typename TX, typename TY, int TPR, int NC, int CH>
void forward_of(int form, const NormArgs& a, hipStream_t s) {
  if (form == FORM_WHOLE) forward<TX, TY, TPR, NC, CH, FORM_WHOLE>(a, s);
  else if (form == FORM_TAIL) forward<TX, TY, TPR, NC, CH, FORM_TAIL>(a, s);
  else forward<TX, TY, TPR, NC, CH, FORM_MORE>(a, s);
}
template <typename TX, typename TY, int TPR, int NC, int CH>
void backward_of(int form, const NormArgs& a, int* blocks, hipStream_t s) {
  if (form == FORM_WHOLE) *blocks = backward<TX, TY, TPR, NC, CH, FORM_WHOLE>(a, !blocks[1], s);
  else if (form == FORM_TAIL) *blocks = backward<TX, TY, TPR, NC, CH, FORM_TAIL>(a, !blocks[1], s);
  else *blocks = backward<TX, TY, TPR, NC, CH, FORM_MORE>(a, !blocks[1], s);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, int x_half, int y_half, hipStream_t s) {
#define FORWARD(TPR, NC, CH) BY_TYPES(forward, TPR, NC, CH)
#define FORWARD_768                   \
  do {                                \
    if (x_half) FORWARD(128, 1, 8);   \
    else FORWARD(64, 3, 4);           \
  } while (0)
  BY_WIDTH(a.d, FORWARD, FORWARD_768, FORWARD(1024, 1, 8));
#undef FORWARD_768
#undef FORWARD
  return hipGetLastError();
}

int norm_grad_blocks(const NormArgs& a, int x_half, int y_half) {
  int blocks[2] = {0, 1};      // (1: no launch)
  hipStream_t s = nullptr;
#define BLOCKS(TPR, NC, CH) BY_TYPES(backward, TPR, NC, CH, blocks)
  BY_WIDTH(a.d, BLOCKS, BLOCKS(64, 3, 4), BLOCKS(512, 2, 8));
#undef BLOCKS
  return blocks[0];
}

hipError_t launch_residual_norm_grad(const NormArgs& a, int x_half, int y_half, hipStream_t s) {
  int blocks[2] = {0, 0};
#define BACKWARD(TPR, NC, CH) BY_TYPES(backward, TPR, NC, CH, blocks)
  BY_WIDTH(a.d, BACKWARD, BACKWARD(64, 3, 4), BACKWARD(512, 2, 8));
#undef BACKWARD
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
