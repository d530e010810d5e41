// C entry points of the training step around the Muon update: the global
// gradient norm and clipping, AdamW for the parameters Muon does not take,
// and the head's softmax cross entropy with its gradient. Arguments are
// validated on the host (validate.cpp) before anything is enqueued; the
// kernels are in train_kernels.hip and head_kernels.hip.
#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <string>

#include "../../include/libmuon.h"
#include "handle.hpp"
#include "train.hpp"
#include "validate.hpp"

namespace muon {
namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }
inline int esz(int dt) { return dt == MUON_BF16 ? 2 : 4; }
inline bool empty(const muon_matrix& m) { return m.rows == 0 || m.cols == 0; }

// One contiguous run of rows x cols elements starting on 16 bytes.
bool is_flat(const muon_matrix& m) { return (m.rows == 1 || m.ld == m.cols) && (uintptr_t)m.ptr % 16 == 0; }

// Work items of a launch fit its grid (and the 32-bit item index).
constexpr int64_t kMaxChunks = int64_t(1) << 30;

muon_status norm_run(muon_handle* h, int n, const muon_matrix* g, float max_norm, float* norm, float* coef) {
  TrainState& ts = train_state(h);
  const hipStream_t s = handle_stream(h);
  int64_t live = 0;
  for (int i = 0; i < n; ++i) live += !empty(g[i]);
  if (live == 0) {
    HIP_DO(h, launch_norm_empty(max_norm, norm, coef, s));
    return MUON_OK;
  }
  // blocks of every launch, before the first: the last one to finish sums them all
  auto fill = [&](NormList& L, int& i, int& chunks) {
    int64_t c = 0;
    L.n = 0;
    for (; i < n && L.n < kNormMax; ++i) {
      if (empty(g[i])) continue;
      const int64_t e = g[i].rows * g[i].cols, k = cdiv(e, kNormChunk);
      if (c + k > kMaxChunks && L.n) break;
      L.chunk0[L.n] = (int32_t)c;
      L.t[L.n++] = ListItem{g[i].ptr, g[i].ld, g[i].cols, e, g[i].dtype, is_flat(g[i]) ? 1 : 0};
      c += k;
    }
    L.chunk0[L.n] = (int32_t)c;
    chunks = (int)c;
  };
  NormList L;
  int total = 0, chunks = 0;
  for (int i = 0; i < n;) {
    fill(L, i, chunks);
    total += std::min(chunks, kNormBlocks);
  }
  const size_t need = sizeof(NormState) + (size_t)total * sizeof(double);
  const size_t before = ts.norm.bytes;    // (a larger buffer can have the freed one's address)
  if (muon_status e = grow(h, ts.norm, std::max(need, size_t(64) << 10), "gradient norm")) return e;
  const bool clean = ts.norm_clean && ts.norm.bytes == before;
  if (!clean) {
    // a new buffer, or a call that ended between its launches
    HIP_DO(h, launch_norm_reset((NormState*)ts.norm.ptr, s));
  }
  ts.norm_clean = false;
  int part0 = 0;
  for (int i = 0; i < n;) {
    fill(L, i, chunks);
    if (L.n == 0) break;
    const int blocks = std::min(chunks, kNormBlocks);
    HIP_DO(h, launch_norm(L, blocks, chunks, (NormState*)ts.norm.ptr, part0, total, max_norm, norm, coef, s));
    part0 += blocks;
  }
  ts.norm_clean = clean || !handle_capturing(h);   // (a captured reset has not run yet)
  return MUON_OK;
}

muon_status scale_run(muon_handle* h, int n, const muon_matrix* src, const muon_matrix* dst, const float* coef) {
  const hipStream_t s = handle_stream(h);
  // from the last tensor's end to the first's start (k_scale says why)
  for (int i = n - 1; i >= 0;) {
    ScaleList L;
    L.n = 0;
    int64_t c = 0;
    for (; i >= 0 && L.n < kScaleMax; --i) {
      if (empty(src[i])) continue;
      const muon_matrix& d = dst ? dst[i] : src[i];
      const int64_t e = src[i].rows * src[i].cols, k = cdiv(e, kChunk);
      if (c + k > kMaxChunks && L.n) break;
      L.chunk0[L.n] = (int32_t)c;
      const bool flat = is_flat(src[i]) && is_flat(d);
      L.t[L.n++] = ScaleItem{src[i].ptr, d.ptr, src[i].ld, d.ld, src[i].cols, e,
                             (src[i].dtype == MUON_BF16 ? 1 : 0) | (d.dtype == MUON_BF16 ? 2 : 0) | (flat ? 4 : 0)};
      c += k;
    }
    L.chunk0[L.n] = (int32_t)c;
    if (L.n) HIP_DO(h, launch_scale(L, (int)c, coef, dst ? 0 : 1, s));
  }
  return MUON_OK;
}

// ---------------------------------------------------------------------------
// Head cross entropy
// ---------------------------------------------------------------------------
// Bytes of a call's per-piece buffers at most (a piece has at least
// kPieceRows tokens, whatever the vocabulary).
constexpr size_t kHeadBytes = size_t(1) << 30;
constexpr int kPieceRows = 256;
constexpr int kGatherTokens = 64;       // tokens that one wave can list
constexpr int64_t kPieceMost = 65536;   // keeps a launch's tiles far from 2^31

// A call on a head: the loss or log probabilities, alone or with gradients.
struct HeadCall {
  const muon_matrix *hidden, *weight;
  const void* targets;
  int target_bytes;
  int64_t ignore;
  float softcap;
  const muon_matrix *dh = nullptr, *dw = nullptr;
  LogitsMode mode = LOGITS_LOSS;
  // the loss
  int reduction = MUON_REDUCE_NONE;
  const float* grad_out = nullptr;
  float* loss = nullptr;                     // log probabilities: the values
  // log probabilities, and what their gradient takes
  int top = 0;
  float *entropy = nullptr, *stats = nullptr, *top_logprobs = nullptr;
  int64_t* top_tokens = nullptr;
  const float *stats_in = nullptr, *grad_logprobs = nullptr, *grad_entropy = nullptr;
};

muon_status head_run(muon_handle* h, const HeadCall& c) {
  TrainState& ts = train_state(h);
  const hipStream_t s = handle_stream(h);
  const muon_matrix &hid = *c.hidden, &wgt = *c.weight;
  const int dt = wgt.dtype, e = esz(dt);
  HeadArgs a{};
  a.n = (int)hid.rows;
  a.v = (int)wgt.rows;
  a.d = (int)wgt.cols;
  const int unit = 128 / e;                       // a stage of a product: 128 bytes of the contraction
  a.dp = (int)(cdiv(a.d, unit) * unit);
  a.vp = (int)(cdiv(a.v, 256) * 256);
  a.per_token = c.reduction == MUON_REDUCE_NONE;
  a.mean = c.reduction == MUON_REDUCE_MEAN;
  a.half = dt == MUON_BF16;
  a.softcap = c.softcap;
  a.cap_inv = c.softcap > 0.f ? std::min(1.f / c.softcap, FLT_MAX) : 0.f;   // (of a denormal cap: 0 times it stays 0)
  a.targets = c.targets;
  a.target_bytes = c.target_bytes;
  a.ignore = c.ignore;
  a.h = hid.ptr;
  a.ld_h = hid.ld;
  a.loss = c.loss;
  a.grad_out = c.grad_out;
  a.top = c.top;
  a.entropy = c.entropy;
  a.stats = (float4*)c.stats;
  a.top_logprobs = c.top_logprobs;
  a.top_tokens = c.top_tokens;
  a.stats_in = (const float4*)c.stats_in;
  a.grad_logprobs = c.grad_logprobs;
  a.grad_entropy = c.grad_entropy;
  // (a gradient without elements is none: with no tokens and no dweight only
  // the loss is left)
  if (c.dh && !empty(*c.dh)) {
    a.dh = c.dh->ptr;
    a.ld_dh = c.dh->ld;
  }
  if (c.dw && !empty(*c.dw)) {
    a.dw = c.dw->ptr;
    a.ld_dw = c.dw->ld;
  }
  const bool grad = a.dh || a.dw;
  if (c.mode == LOGITS_GRAD && !grad) return MUON_OK;
  // the weight as it is, where its rows are whole 16-byte pieces on 16 bytes;
  // otherwise a padded copy (the pitch also fits the products' 24-bit multiply)
  const bool direct = a.d * e % 16 == 0 && (uintptr_t)wgt.ptr % 16 == 0 &&
                      (wgt.rows == 1 || (wgt.ld * e % 16 == 0 && wgt.ld * e < (1 << 23)));
  a.w_cols = direct ? a.d : a.dp;
  // pieces
  // (a row's statistics: at most 8 bytes for 64 words of the vocabulary, with entropy
  // 16, and 8 more for each lane that shares them with the candidates)
  const size_t each = c.mode == LOGITS_STATS ? 16 + (c.top ? (a.half ? 16 : 32) : 0) : 8;   // (sets of 32 and 16)
  const size_t row = (size_t)a.dp * e + (size_t)cdiv(a.v, 64) * each + 24 + (grad ? (size_t)a.vp * e : 0);
  const int64_t most =
      std::min(kPieceMost, std::max<int64_t>(kPieceRows, (int64_t)(kHeadBytes / row) / kPieceRows * kPieceRows));
  const int64_t pieces = std::max<int64_t>(1, cdiv(a.n, most));
  a.piece = (int)(std::max<int64_t>(1, cdiv(cdiv(a.n, pieces), kPieceRows)) * kPieceRows);
  head_plan(a, dt, c.mode);
  // few tokens without gradients, whose rows the products can load as they are:
  // no panels
  a.gather = !grad && direct && a.n > 0 && a.n <= kGatherTokens && a.logit_tile < 256 && (uintptr_t)hid.ptr % 16 == 0 &&
             (a.n == 1 || (hid.ld * e % 16 == 0 && hid.ld * e < (1 << 23)));
  a.rows_direct = a.d * e % 16 == 0 && (uintptr_t)hid.ptr % 16 == 0 &&
                  (a.n == 1 || (hid.ld * e % 16 == 0 && hid.ld < (int64_t(1) << 31) / e / std::max(a.n, 1)));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align_up(bytes);
    return o;
  };
  const size_t n = (size_t)a.n, p = (size_t)a.piece;
  const size_t o_count = take(16), o_idx = take(n * 4), o_tgt = take(n * 4), o_lossc = take(n * 4);
  const bool stats = c.mode == LOGITS_STATS, loss = c.mode == LOGITS_LOSS;
  const size_t o_hp = take(p * a.dp * e), o_tmax = take(loss ? p * a.n_vt * 4 : 0), o_tsum = take(loss ? p * a.n_vt * 4 : 0);
  const size_t o_zt = take(loss ? p * 4 : 0), o_zf = take(loss && c.softcap > 0.f ? p * 4 : 0), o_rs = take(p * 16);
  const size_t o_tstat = take(stats ? p * a.n_vt * 16 : 0), o_best = take(stats && c.top ? p * a.n_vt * a.sets * 8 : 0);
  const size_t o_ts = take(c.mode == LOGITS_GRAD ? p * 16 : 0);
  const size_t o_w = direct ? 0 : take((size_t)a.v * a.dp * e);
  const size_t o_e = grad ? take(p * a.vp * e) : 0, o_part = a.split > 1 ? take(p * a.dp * 4 * a.split) : 0;
  const size_t o_wpart = a.wsplit > 1 ? take((size_t)a.v * a.dp * 4 * a.wsplit) : 0;
  const bool acc = a.dw && pieces > 1;
  const size_t o_acc = acc ? take((size_t)a.v * a.dp * 4) : 0;
  if (muon_status st = grow(h, ts.head, at, "cross entropy")) return st;
  uint8_t* b = (uint8_t*)ts.head.ptr;
  a.count = (int32_t*)(b + o_count);
  a.idx = (int32_t*)(b + o_idx);
  a.tgt = (int32_t*)(b + o_tgt);
  a.lossc = (float*)(b + o_lossc);
  a.hp = b + o_hp;
  a.tmax = (float*)(b + o_tmax);
  a.tsum = (float*)(b + o_tsum);
  a.zt = (float*)(b + o_zt);
  a.zf = (float*)(b + o_zf);
  a.rs = (float4*)(b + o_rs);
  a.tstat = (float4*)(b + o_tstat);
  a.best = (uint2*)(b + o_best);
  a.ts = c.mode == LOGITS_GRAD ? (float4*)(b + o_ts) : nullptr;
  if (c.mode == LOGITS_GRAD) a.loss = a.lossc;    // (zeros of the ignored tokens go there)
  a.e = b + o_e;
  a.part = (float*)(b + o_part);
  a.wpart = (float*)(b + o_wpart);
  a.dwacc = acc ? (float*)(b + o_acc) : nullptr;
  a.w = wgt.ptr;
  a.ld_w = wgt.rows == 1 ? a.d : wgt.ld;
  HIP_DO(h, launch_head_compact(a, s));
  if (!direct) {
    a.w_src = wgt.ptr;
    a.ld_src = wgt.ld;
    a.w = b + o_w;
    a.ld_w = a.dp;
  }
  for (int64_t k = 0; k < pieces; ++k) {
    a.row0 = (int)(k * a.piece);
    a.rows_max = std::max(0, std::min(a.piece, a.n - a.row0));
    a.first = k == 0;
    a.last = k + 1 == pieces;
    HIP_DO(h, launch_head_pack(a, dt, s));
    HIP_DO(h, launch_head_logits(a, dt, grad ? 1 : 0, c.mode, s));
    if (c.mode == LOGITS_STATS) {
      HIP_DO(h, launch_logprobs(a, dt, s));
      continue;
    }
    if (c.mode == LOGITS_LOSS) {
      HIP_DO(h, launch_head_merge(a, grad ? 1 : 0, s));
      if (!grad) continue;
      HIP_DO(h, launch_head_dlogits(a, dt, s));
    }
    HIP_DO(h, launch_head_gradients(a, dt, s));
    HIP_DO(h, launch_head_gradients_out(a, dt, s));
  }
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" muon_status muon_grad_norm(muon_handle* h, int n, const muon_matrix* grad, float max_norm, float* norm,
                                      float* coef) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  const int rc = check_norm(n, grad, nullptr, max_norm, norm, coef, 0, msg, sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  return norm_run(h, n, grad, max_norm, norm, coef);
  });
}

extern "C" muon_status muon_clip_grad_norm(muon_handle* h, int n, const muon_matrix* grad, const muon_matrix* out,
                                           float max_norm, float* norm, float* coef) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  int rc = check_norm(n, grad, out, max_norm, norm, coef, 1, msg, sizeof(msg));
  if (!rc && !coef) {
    snprintf(msg, sizeof(msg), "coef is NULL");
    rc = MUON_ERR_INVALID_ARG;
  }
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  if (muon_status e = norm_run(h, n, grad, max_norm, norm, coef)) return e;
  return scale_run(h, n, grad, out, coef);
  });
}

extern "C" muon_status muon_scale(muon_handle* h, int n, const muon_matrix* in, const muon_matrix* out,
                                  const float* coef) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  const int rc = check_scale(n, in, out, coef, msg, sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  return scale_run(h, n, in, out, coef);
  });
}

extern "C" muon_status adamw_update(muon_handle* h, int n, const muon_matrix* grad, const muon_matrix* exp_avg,
                                    const muon_matrix* exp_avg_sq, const muon_matrix* weight, const muon_matrix* copy,
                                    const muon_adamw_config* cfg, const float* grad_scale) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  const int rc = check_adamw(n, grad, exp_avg, exp_avg_sq, weight, copy, cfg, grad_scale, msg, sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  AdamConst c;
  const double b1 = cfg->beta1, b2 = cfg->beta2;
  c.beta1 = cfg->beta1;
  c.c1 = (float)(1.0 - b1);
  c.beta2 = cfg->beta2;
  c.c2 = (float)(1.0 - b2);
  c.keep = (float)(1.0 - (double)cfg->lr * (double)cfg->weight_decay);
  c.lr1 = (float)((double)cfg->lr / (1.0 - pow(b1, (double)cfg->step)));
  c.rs2 = (float)(1.0 / sqrt(1.0 - pow(b2, (double)cfg->step)));
  c.eps = cfg->eps;
  const AdamClock clock{cfg->step_at, cfg->lr_at, cfg->step, cfg->lr, cfg->weight_decay, log2(b1), log2(b2)};
  const hipStream_t s = handle_stream(h);
  for (int i = 0; i < n;) {
    AdamList L;
    L.n = 0;
    int64_t k0 = 0;
    for (; i < n && L.n < kAdamMax; ++i) {
      if (empty(weight[i])) continue;
      const int64_t e = weight[i].rows * weight[i].cols, k = cdiv(e, kChunk);
      if (k0 + k > kMaxChunks && L.n) break;
      const bool cp = copy && !empty(copy[i]);
      const bool flat = is_flat(grad[i]) && is_flat(exp_avg[i]) && is_flat(exp_avg_sq[i]) && is_flat(weight[i]) &&
                        (!cp || is_flat(copy[i]));
      AdamItem& t = L.t[L.n];
      L.chunk0[L.n++] = (int32_t)k0;
      t.g = grad[i].ptr;
      t.m = (float*)exp_avg[i].ptr;
      t.v = (float*)exp_avg_sq[i].ptr;
      t.w = weight[i].ptr;
      t.copy = cp ? copy[i].ptr : nullptr;
      t.ld[0] = grad[i].ld;
      t.ld[1] = exp_avg[i].ld;
      t.ld[2] = exp_avg_sq[i].ld;
      t.ld[3] = weight[i].ld;
      t.ld[4] = cp ? copy[i].ld : 0;
      t.cols = weight[i].cols;
      t.n = e;
      t.dt = (grad[i].dtype == MUON_BF16 ? 1 : 0) | (weight[i].dtype == MUON_BF16 ? 2 : 0) |
             (cp && copy[i].dtype == MUON_BF16 ? 4 : 0) | (flat ? 8 : 0);
      k0 += k;
    }
    L.chunk0[L.n] = (int32_t)k0;
    if (L.n) HIP_DO(h, launch_adamw(L, (int)k0, c, clock, grad_scale, s));
  }
  return MUON_OK;
  });
}

extern "C" muon_status linear_cross_entropy(muon_handle* h, const muon_matrix* hidden, const muon_matrix* weight,
                                            const void* targets, int target_bytes, const muon_loss_config* cfg,
                                            float* loss) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  muon_loss_config c;
  muon_loss_config_default(&c);
  if (cfg) c = *cfg;
  const int rc = check_loss(hidden, weight, targets, target_bytes, &c, nullptr, loss, nullptr, nullptr, 0, msg,
                            sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  HeadCall call{hidden, weight, targets, target_bytes, c.ignore_index, c.softcap};
  call.reduction = c.reduction;
  call.loss = loss;
  return head_run(h, call);
  });
}

extern "C" muon_status linear_cross_entropy_grad(muon_handle* h, const muon_matrix* hidden, const muon_matrix* weight,
                                                 const void* targets, int target_bytes, const muon_loss_config* cfg,
                                                 const float* grad_out, float* loss, const muon_matrix* dhidden,
                                                 const muon_matrix* dweight) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  muon_loss_config c;
  muon_loss_config_default(&c);
  if (cfg) c = *cfg;
  const int rc = check_loss(hidden, weight, targets, target_bytes, &c, grad_out, loss, dhidden, dweight, 1, msg,
                            sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  HeadCall call{hidden, weight, targets, target_bytes, c.ignore_index, c.softcap, dhidden, dweight};
  call.reduction = c.reduction;
  call.grad_out = grad_out;
  call.loss = loss;
  return head_run(h, call);
  });
}

extern "C" muon_status linear_logprobs(muon_handle* h, const muon_matrix* hidden, const muon_matrix* weight,
                                       const void* targets, int target_bytes, const muon_logprob_config* cfg,
                                       float* logprobs, float* entropy, float* stats, float* top_logprobs,
                                       int64_t* top_tokens) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  muon_logprob_config c;
  muon_logprob_config_default(&c);
  if (cfg) c = *cfg;
  const int rc = check_logprobs(hidden, weight, targets, target_bytes, &c, logprobs, entropy, stats, top_logprobs,
                                top_tokens, msg, sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  if (hidden->rows == 0) return MUON_OK;
  HeadCall call{hidden, weight, targets, target_bytes, c.ignore_index, c.softcap};
  call.mode = LOGITS_STATS;
  call.loss = logprobs;
  call.top = c.top;
  call.entropy = entropy;
  call.stats = stats;
  call.top_logprobs = top_logprobs;
  call.top_tokens = top_tokens;
  return head_run(h, call);
  });
}

extern "C" muon_status linear_logprobs_grad(muon_handle* h, const muon_matrix* hidden, const muon_matrix* weight,
                                            const void* targets, int target_bytes, const muon_logprob_config* cfg,
                                            const float* stats, const float* grad_logprobs, const float* grad_entropy,
                                            const muon_matrix* dhidden, const muon_matrix* dweight) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  muon_logprob_config c;
  muon_logprob_config_default(&c);
  if (cfg) c = *cfg;
  const int rc = check_logprobs_grad(hidden, weight, targets, target_bytes, &c, stats, grad_logprobs, grad_entropy,
                                     dhidden, dweight, msg, sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  HeadCall call{hidden, weight, targets, target_bytes, c.ignore_index, c.softcap, dhidden, dweight};
  call.mode = LOGITS_GRAD;
  call.stats_in = stats;
  call.grad_logprobs = grad_logprobs;
  call.grad_entropy = grad_entropy;
  return head_run(h, call);
  });
}
