// Host fuzz driver for the validation of the norms around a block and of the
// head's log probabilities, built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_norms_abi.py (CPU only). Random and
// edge descriptors go to the four checkers; every call must return a declared
// status and a terminated message. Accepted small calls are then checked byte by
// byte: no byte that the call writes belongs to two of its buffers.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <limits>
#include <random>
#include <vector>

#include "libmuon.h"

namespace {

std::mt19937_64 rng(20261209);

int64_t pick_dim(bool small) {
  static const int64_t edge[] = {0, 1, 2, 63, 64, 16384, 16385, 65536, 65537, int64_t(1) << 22, (int64_t(1) << 22) + 1,
                                 int64_t(1) << 31, int64_t(1) << 42, -1, std::numeric_limits<int64_t>::max(),
                                 std::numeric_limits<int64_t>::min()};
  if (small) return (int64_t)(rng() % 5);
  if (rng() % 3 == 0) return edge[rng() % (sizeof(edge) / sizeof(edge[0]))];
  return (int64_t)(rng() % 1000);
}
uintptr_t pick_address(bool small, int unit) {
  return small ? 4096 + (uintptr_t)unit * (rng() % (1600 / unit)) : rng() % 6 == 0 ? 0 : unit * (rng() % (uint64_t(1) << 40));
}
muon_matrix pick(bool small) {
  muon_matrix m;
  m.rows = pick_dim(small);
  m.cols = pick_dim(small);
  m.ld = small ? m.cols + (int64_t)(rng() % 3) : rng() % 2 ? m.cols : pick_dim(false);
  m.dtype = (int32_t)(rng() % (small ? 2 : 3));
  m.ptr = (void*)pick_address(small, 4);
  return m;
}
muon_matrix like(const muon_matrix& m, bool small, int dtype) {
  muon_matrix x = pick(small);
  if (small || rng() % 5) x.rows = m.rows, x.cols = m.cols;
  if (small) x.ld = x.cols + (int64_t)(rng() % 3);
  if (small || rng() % 5) x.dtype = dtype;
  return x;
}

bool fine(int rc, const char* msg, int len) {
  if (rc != MUON_OK && rc != MUON_ERR_INVALID_ARG && rc != MUON_ERR_UNSUPPORTED_DTYPE && rc != MUON_ERR_SHAPE_MISMATCH)
    return false;
  return memchr(msg, 0, (size_t)len) != nullptr && (rc == MUON_OK) == (msg[0] == 0);
}

struct Bytes {
  std::vector<uint8_t> read = std::vector<uint8_t>(16384), written = std::vector<uint8_t>(16384);
  bool ok = true;
  void mark(const muon_matrix* m, bool writes) {
    if (!m) return;
    const int e = m->dtype == MUON_BF16 ? 2 : 4;
    std::vector<size_t> mine;
    for (int64_t r = 0; r < m->rows; ++r)
      for (int64_t b = 0; b < m->cols * e; ++b) mine.push_back((uintptr_t)m->ptr - 4096 + (size_t)(r * m->ld * e + b));
    take(mine, writes);
  }
  void mark(const void* p, int64_t bytes, bool writes) {
    if (!p) return;
    std::vector<size_t> mine;
    for (int64_t b = 0; b < bytes; ++b) mine.push_back((uintptr_t)p - 4096 + (size_t)b);
    take(mine, writes);
  }
  void take(const std::vector<size_t>& mine, bool writes) {
    for (size_t i : mine) ok = ok && !written[i] && !(writes && read[i]);
    for (size_t i : mine) (writes ? written : read)[i] = 1;
  }
};

}  // namespace

int main() {
  long accepted = 0, checked = 0;
  for (int it = 0; it < 120000; ++it) {
    const bool small = it % 3 != 0;
    const int len = 1 + (int)(rng() % 200);
    std::vector<char> msg((size_t)len, 'x');
    auto maybe = [&](const muon_matrix& m) { return rng() % 4 ? &m : nullptr; };

    // norms
    muon_matrix x = pick(small);
    const int ty = small && x.dtype == MUON_BF16 ? MUON_BF16 : (int)(rng() % 2);
    const muon_matrix y = like(x, small, ty);
    const muon_matrix row{nullptr, 1, x.cols, x.cols, 0};
    auto param = [&](bool full) {
      muon_matrix p = full && rng() % 3 == 0 ? like(x, small, ty) : like(row, small, (int)(rng() % 2));
      if (rng() % 4 == 0 && full) p.rows = p.cols = 1;
      return p;
    };
    const muon_matrix post = param(false), pre = param(false), gate = param(true), scale = param(true);
    muon_norm_params p{maybe(post), maybe(pre), maybe(gate), maybe(scale), (int32_t)(rng() % 5 != 0), (int32_t)(rng() % 5 != 0),
                       rng() % 9 ? 1e-6f : (float)(rng() % 2) - 1.f};
    const muon_matrix* yp = maybe(y);
    const muon_matrix out = like(x, small, x.dtype), hidden = like(x, small, yp ? ty : x.dtype);
    const muon_matrix* outp = maybe(out);
    const muon_matrix* hidp = p.pre_norm || rng() % 4 == 0 ? &hidden : nullptr;
    int rc = muon_check_residual_norm_args(&x, yp, rng() % 9 ? &p : nullptr, outp, hidp, msg.data(), len);
    if (!fine(rc, msg.data(), len) && len > 1) return printf("norm %d: %d %s\n", it, rc, msg.data()), 1;
    rc = muon_check_residual_norm_args(&x, yp, &p, outp, hidp, msg.data(), len);
    accepted += rc == MUON_OK;
    if (rc == MUON_OK && small) {
      Bytes b;
      for (const muon_matrix* m : {(const muon_matrix*)&x, yp, p.post_gain, p.pre_gain, p.gate, p.scale}) b.mark(m, false);
      b.mark(outp, true);
      b.mark(hidp, true);
      ++checked;
      if (!b.ok) return printf("norm %d accepted shared memory\n", it), 1;
    }
    const muon_matrix dx = like(x, small, x.dtype), dy = like(y, small, ty), dpost = like(post, small, post.dtype);
    const muon_matrix dpre = like(pre, small, pre.dtype), dgate = like(gate, small, gate.dtype);
    const muon_matrix dscale = like(scale, small, scale.dtype);
    auto gradient = [&](const muon_matrix& m, const void* of) { return of && rng() % 3 ? &m : nullptr; };
    muon_norm_grads g{gradient(dx, &x),           gradient(dy, yp),         gradient(dpost, p.post_gain),
                      gradient(dgate, p.gate),    gradient(dscale, p.scale), gradient(dpre, p.pre_gain)};
    rc = muon_check_residual_norm_grad_args(&x, yp, &p, outp, hidp, rng() % 20 ? &g : nullptr, msg.data(), len);
    if (!fine(rc, msg.data(), len) && len > 1) return printf("norm gradient %d: %d %s\n", it, rc, msg.data()), 1;
    accepted += rc == MUON_OK;
    if (rc == MUON_OK && small) {
      Bytes b;
      for (const muon_matrix* m : {(const muon_matrix*)&x, yp, p.post_gain, p.pre_gain, p.gate, p.scale, outp, hidp}) b.mark(m, false);
      for (const muon_matrix* m : {g.x, g.y, g.post_gain, g.gate, g.scale, g.pre_gain}) b.mark(m, true);
      ++checked;
      if (!b.ok) return printf("norm gradient %d accepted shared memory\n", it), 1;
    }

    // log probabilities
    muon_matrix h = pick(small), w = pick(small);
    if (small || rng() % 4) w.cols = h.cols, w.dtype = h.dtype;
    if (small) w.ld = w.cols + (int64_t)(rng() % 2);
    const int bytes = small || rng() % 5 ? (rng() % 2 ? 8 : 4) : 2;
    muon_logprob_config c;
    muon_logprob_config_default(&c);
    c.top = (int32_t)(rng() % (small ? 4 : 36)) - (int32_t)(rng() % 9 == 0);
    const void* targets = (const void*)pick_address(small, 8);
    float* out1 = (float*)pick_address(small, 4);
    float* out2 = rng() % 2 ? (float*)pick_address(small, 4) : nullptr;
    float* stats = rng() % 2 ? (float*)pick_address(small, 16) : nullptr;
    float* top1 = (float*)pick_address(small, 4);
    int64_t* top2 = (int64_t*)pick_address(small, 8);
    rc = muon_check_logprob_args(&h, &w, targets, bytes, &c, out1, out2, stats, top1, top2, msg.data(), len);
    if (!fine(rc, msg.data(), len) && len > 1) return printf("logprobs %d: %d %s\n", it, rc, msg.data()), 1;
    accepted += rc == MUON_OK;
    if (rc == MUON_OK && small && h.rows > 0) {
      Bytes b;
      b.mark(&h, false);
      b.mark(&w, false);
      b.mark(targets, h.rows * bytes, false);
      b.mark(out1, h.rows * 4, true);
      b.mark(out2, h.rows * 4, true);
      b.mark(stats, h.rows * 16, true);
      if (c.top) b.mark(top1, h.rows * c.top * 4, true), b.mark(top2, h.rows * c.top * 8, true);
      ++checked;
      if (!b.ok) return printf("logprobs %d accepted shared memory\n", it), 1;
    }
    const muon_matrix dh = like(h, small, h.dtype), dw = like(w, small, w.dtype);
    const muon_matrix *dhp = maybe(dh), *dwp = maybe(dw);
    rc = muon_check_logprob_grad_args(&h, &w, targets, bytes, rng() % 9 ? &c : nullptr, stats, out1, out2, dhp, dwp, msg.data(), len);
    if (!fine(rc, msg.data(), len) && len > 1) return printf("logprobs gradient %d: %d %s\n", it, rc, msg.data()), 1;
    accepted += rc == MUON_OK;
    if (rc == MUON_OK && small) {
      Bytes b;
      if (h.rows > 0) {
        b.mark(&h, false);
        b.mark(targets, h.rows * bytes, false);
        b.mark(stats, h.rows * 16, false);
        b.mark(out1, h.rows * 4, false);
        b.mark(out2, h.rows * 4, false);
      }
      b.mark(&w, false);
      b.mark(dhp, true);
      b.mark(dwp, true);
      ++checked;
      if (!b.ok) return printf("logprobs gradient %d accepted shared memory\n", it), 1;
    }
  }
  printf("ok %ld accepted, %ld checked byte by byte\n", accepted, checked);
  return accepted > 1000 && checked > 500 ? 0 : 1;
}
