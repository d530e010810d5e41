// Host fuzz driver for the validation of the training-step entry points, built
// with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_training_abi.py (CPU only). Random and edge descriptors go to the
// three checkers; every call must return a declared status and a terminated
// message. Accepted lists of small tensors in a few hundred bytes are then
// checked byte by byte: no byte that the call writes belongs to two buffers.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <limits>
#include <random>
#include <vector>

#include "libmuon.h"

namespace {

std::mt19937_64 rng(20261206);

int64_t pick_dim(bool small) {
  static const int64_t edge[] = {0, 1, 2, 63, 64, 65, 50304, 65536, 65537, int64_t(1) << 22, (int64_t(1) << 22) + 1,
                                 int64_t(1) << 42, -1, std::numeric_limits<int64_t>::max(),
                                 std::numeric_limits<int64_t>::min()};
  if (small) return (int64_t)(rng() % 6);
  if (rng() % 3 == 0) return edge[rng() % (sizeof(edge) / sizeof(edge[0]))];
  return (int64_t)(rng() % 1000);
}

muon_matrix pick(bool small) {
  muon_matrix m;
  m.rows = pick_dim(small);
  m.cols = pick_dim(small);
  m.ld = small ? m.cols + (int64_t)(rng() % 3) : rng() % 2 ? m.cols : pick_dim(false);
  m.dtype = (int32_t)(rng() % (small ? 2 : 3));
  m.ptr = (void*)(uintptr_t)(small ? 4096 + 4 * (rng() % 60) : rng() % 5 == 0 ? 0 : 4 * (rng() % (uint64_t(1) << 40)));
  return m;
}

bool fine(int rc, const char* msg, int len) {
  if (rc != MUON_OK && rc != MUON_ERR_INVALID_ARG && rc != MUON_ERR_UNSUPPORTED_DTYPE && rc != MUON_ERR_SHAPE_MISMATCH)
    return false;
  return memchr(msg, 0, (size_t)len) != nullptr && (rc == MUON_OK) == (msg[0] == 0);
}

// Marks a tensor's bytes; false when one is already taken by another buffer
// and either writes it.
struct Bytes {
  std::vector<uint8_t> read = std::vector<uint8_t>(8192), written = std::vector<uint8_t>(8192);
  bool mark(const muon_matrix& m, bool writes) {
    const int e = m.dtype == MUON_BF16 ? 2 : 4;
    bool ok = true;
    std::vector<size_t> mine;
    for (int64_t r = 0; r < m.rows; ++r)
      for (int64_t b = 0; b < m.cols * e; ++b) mine.push_back((uintptr_t)m.ptr - 4096 + (size_t)(r * m.ld * e + b));
    for (size_t i : mine) ok = ok && !written[i] && !(writes && read[i]);
    for (size_t i : mine) (writes ? written : read)[i] = 1;
    return ok;
  }
};

}  // namespace

int main() {
  long accepted = 0, checked = 0;
  for (int it = 0; it < 60000; ++it) {
    const bool small = it % 2;
    const int n = (int)(rng() % 4);
    const int len = 1 + (int)(rng() % 200);
    std::vector<char> msg((size_t)len, 'x');
    std::vector<muon_matrix> a, b, c, d, e;
    for (int i = 0; i < n; ++i) {
      const muon_matrix m = pick(small);
      for (auto* v : {&a, &b, &c, &d, &e}) {
        muon_matrix x = pick(small);
        if (small || rng() % 4) x.rows = m.rows, x.cols = m.cols;
        if (small) x.ld = x.cols + (int64_t)(rng() % 3);
        if ((v == &b || v == &c) && small) x.dtype = MUON_F32;
        v->push_back(x);
      }
    }
    muon_adamw_config cfg;
    muon_adamw_config_default(&cfg);
    if (rng() % 8 == 0) cfg.step = (int64_t)(rng() % 2) - 1;
    const float* far = (const float*)(uintptr_t)(uint64_t(1) << 50);
    int rc = muon_check_adamw_args(n, a.data(), b.data(), c.data(), d.data(), it % 3 ? e.data() : nullptr, &cfg,
                                   it % 5 ? far : nullptr, msg.data(), len);
    if (!fine(rc, msg.data(), len) && len > 1) return printf("adamw %d: %d %s\n", it, rc, msg.data()), 1;
    if (rc == MUON_OK && small) {
      Bytes bytes;
      for (int i = 0; i < n; ++i) {
        ++checked;
        if (!bytes.mark(a[i], false) || !bytes.mark(b[i], true) || !bytes.mark(c[i], true) || !bytes.mark(d[i], true) ||
            (it % 3 && !bytes.mark(e[i], true)))
          return printf("adamw %d accepted shared memory\n", it), 1;
      }
    }
    accepted += rc == MUON_OK;
    const bool out = it % 3 == 0;
    rc = muon_check_norm_args(n, a.data(), out ? d.data() : nullptr, 1.0f, far, it % 2 ? far + 1 : nullptr, msg.data(), len);
    if (!fine(rc, msg.data(), len) && len > 1) return printf("norm %d: %d %s\n", it, rc, msg.data()), 1;
    accepted += rc == MUON_OK;
    if (n < 2) continue;
    muon_loss_config lc;
    muon_loss_config_default(&lc);
    lc.reduction = (int32_t)(rng() % 4);
    muon_matrix h = a[0], w = d[0], dh = b[0], dw = c[0];
    if (small) {
      w.cols = h.cols, w.dtype = h.dtype, w.ld = w.cols + (int64_t)(rng() % 3);
      w.rows = 1 + (int64_t)(rng() % 4);
      dh.rows = h.rows, dh.cols = h.cols, dh.dtype = h.dtype, dh.ld = dh.cols + 1;
      dw.rows = w.rows, dw.cols = w.cols, dw.dtype = h.dtype, dw.ld = dw.cols + 1;
    }
    rc = muon_check_loss_args(&h, &w, (const void*)(uintptr_t)(uint64_t(1) << 51), rng() % 2 ? 8 : 4, &lc,
                              rng() % 2 ? far : nullptr, far + 4096, &dh, rng() % 2 ? &dw : nullptr, msg.data(), len);
    if (!fine(rc, msg.data(), len) && len > 1) return printf("loss %d: %d %s\n", it, rc, msg.data()), 1;
    accepted += rc == MUON_OK;
  }
  printf("ok %ld accepted, %ld lists checked byte by byte\n", accepted, checked);
  return accepted > 1000 && checked > 100 ? 0 : 1;
}
