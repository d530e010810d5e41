// The host-only validation when memory runs out, built by
// tests/test_training_abi.py (CPU only): each allocation of each call fails in
// turn, and every call returns MUON_ERR_ALLOC with a terminated message; no
// exception leaves a C entry point.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <new>

#include "libmuon.h"

static long left = -1;   // allocations until one fails; negative: none does

void* operator new(size_t n) {
  if (left == 0) throw std::bad_alloc();
  if (left > 0) --left;
  void* p = malloc(n ? n : 1);
  if (!p) abort();
  return p;
}
void operator delete(void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }

static muon_matrix at(uint64_t place, int dtype = MUON_F32) {
  muon_matrix m;
  m.ptr = (void*)(uintptr_t)(place << 32);
  m.rows = 4, m.cols = 8, m.ld = 16, m.dtype = dtype;
  return m;
}

int main() {
  muon_matrix g[] = {at(1), at(2)}, a[] = {at(3), at(4)}, b[] = {at(5), at(6)}, w[] = {at(7), at(8)};
  // columns of one buffer: the rules for interleaved rows allocate too
  muon_matrix left_half[] = {at(9), at(9)}, right_half[] = {at(10), at(11)};
  left_half[1].ptr = (char*)left_half[1].ptr + 32;
  const float *norm = (const float*)(uintptr_t)(20ull << 32), *coef = norm + 4;
  muon_adamw_config adam;
  muon_adamw_config_default(&adam);
  char msg[64];
  for (int call = 0; call < 6; ++call) {
    for (long k = 0;; ++k) {
      memset(msg, 'x', sizeof(msg));
      left = k;
      int rc = -100;
      switch (call) {
        case 0: rc = muon_check_norm_args(2, g, a, 1.0f, norm, coef, msg, sizeof(msg)); break;
        case 1: rc = muon_check_norm_args(2, left_half, right_half, 1.0f, norm, coef, msg, sizeof(msg)); break;
        case 2: rc = muon_check_adamw_args(2, g, a, b, w, nullptr, &adam, coef, msg, sizeof(msg)); break;
        case 3:
          rc = muon_check_loss_args(&g[0], &w[0], norm, 8, nullptr, coef, coef + 64, &a[0], &b[0], msg, sizeof(msg));
          break;
        case 4: rc = muon_check_update_args(2, g, a, w, b, nullptr, msg, sizeof(msg)); break;
        default: rc = muon_check_polar_args(2, g, w, nullptr, msg, sizeof(msg));
      }
      left = -1;
      if (!memchr(msg, 0, sizeof(msg))) return printf("call %d: message not terminated\n", call), 1;
      if (rc == MUON_OK && k > 0) break;   // it needed k allocations
      if (rc != MUON_ERR_ALLOC) return printf("call %d, allocation %ld: %d %s\n", call, k, rc, msg), 1;
    }
  }
  printf("ok\n");
  return 0;
}
