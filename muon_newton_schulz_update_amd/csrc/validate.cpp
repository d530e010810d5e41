// Host-only argument validation for the libmuon entry points. Pure C++ (no
// HIP): it runs before anything is enqueued, so an invalid call touches no
// device memory. Rules are the ones stated in include/libmuon.h.
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "../../include/libmuon.h"
#include "validate.hpp"

namespace muon {

namespace {

int fail(char* msg, int len, int code, const char* fmt, ...) {
  if (msg && len > 0) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, (size_t)len, fmt, ap);
    va_end(ap);
  }
  return code;
}

bool finitef(float x) { return isfinite(x) != 0; }

int elem_size(int32_t dt) { return dt == MUON_BF16 ? 2 : 4; }

// One descriptor. `need_ptr`: a non-empty matrix must have a pointer.
int check_matrix(const muon_matrix& m, const char* what, int i, char* msg, int len) {
  if (m.dtype != MUON_F32 && m.dtype != MUON_BF16)
    return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "%s[%d]: dtype %d is not MUON_F32 or MUON_BF16", what, i,
                (int)m.dtype);
  if (m.rows < 0 || m.cols < 0)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: negative shape %lld x %lld", what, i,
                (long long)m.rows, (long long)m.cols);
  if (m.rows == 0 || m.cols == 0) return MUON_OK;
  if (!m.ptr) return fail(msg, len, MUON_ERR_INVALID_ARG, "%s[%d]: NULL pointer for a non-empty matrix", what, i);
  if (m.ld < m.cols)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: ld %lld < cols %lld", what, i, (long long)m.ld,
                (long long)m.cols);
  if (m.ld > kMaxLd)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: ld %lld exceeds 2^40", what, i, (long long)m.ld);
  if (m.rows > kMaxDim || m.cols > kMaxDim)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: %lld x %lld exceeds the %d per-dimension limit", what, i,
                (long long)m.rows, (long long)m.cols, kMaxDim);
  const int64_t s = m.rows < m.cols ? m.rows : m.cols;
  if (s > kMaxShort)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: short side %lld exceeds %d", what, i, (long long)s,
                kMaxShort);
  if (m.rows * m.cols >= kMaxElems)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: %lld elements exceed the 2^31 limit", what, i,
                (long long)(m.rows * m.cols));
  if (((uintptr_t)m.ptr) % (uintptr_t)elem_size(m.dtype) != 0)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "%s[%d]: pointer not aligned to its element size", what, i);
  return MUON_OK;
}

// Buffers of one call that share memory. A matrix occupies the byte
// intervals [ptr + r ld e, ptr + r ld e + cols e) for r < rows (e = element
// size): disjoint and in address order, since ld >= cols. Two matrices
// overlap when one of these intervals meets one of the other's, so column
// slices of one parent buffer (same ld, disjoint columns) do not overlap.
// Offsets are 128-bit: rows x ld x e reaches 2^58 and the pointer adds to it.
typedef unsigned __int128 u128;
struct Span {
  u128 lo, hi;     // first byte; one past the last row's last byte
  u128 ldb, rowb;  // row stride and row length, in bytes
  int64_t rows;
  const char* what;
  int idx;
  bool writes;     // the call writes this buffer
};

Span make_span(const muon_matrix& m, const char* what, int idx, bool writes) {
  const u128 e = (u128)elem_size(m.dtype);
  Span s;
  s.lo = (u128)(uintptr_t)m.ptr;
  s.ldb = (u128)m.ld * e;
  s.rowb = (u128)m.cols * e;
  s.rows = m.rows;
  s.hi = s.lo + (u128)(m.rows - 1) * s.ldb + s.rowb;
  s.what = what;
  s.idx = idx;
  s.writes = writes;
  return s;
}

bool spans_meet(const Span& a, const Span& b) {
  if (a.hi <= b.lo || b.hi <= a.lo) return false;
  const Span& p = a.lo <= b.lo ? a : b;   // starts first
  const Span& q = a.lo <= b.lo ? b : a;
  if (p.ldb == q.ldb) {
    // q's row s starts at byte `rem` of p's row k + s and, when it runs past
    // that row's stride, ends in row k + s + 1 (never further: rowb <= ldb)
    const u128 d = q.lo - p.lo, k = d / p.ldb, rem = d % p.ldb, prow = (u128)p.rows;
    if (k < prow && rem < p.rowb) return true;
    return rem + q.rowb > p.ldb && k + 1 < prow;
  }
  // different strides: for each row of the matrix with fewer rows, the other
  // matrix's last row starting before that row's end is the only one that
  // can reach into it
  const Span& x = a.rows <= b.rows ? a : b;
  const Span& y = a.rows <= b.rows ? b : a;
  for (int64_t r = 0; r < x.rows; ++r) {
    const u128 x0 = x.lo + (u128)r * x.ldb, x1 = x0 + x.rowb;
    if (x1 <= y.lo) continue;
    if (x0 >= y.hi) break;
    u128 t = (x1 - 1 - y.lo) / y.ldb;
    if (t >= (u128)y.rows) t = (u128)y.rows - 1;
    if (y.lo + t * y.ldb + y.rowb > x0) return true;
  }
  return false;
}

// Sweep in address order; `outputs_may_overlap_inputs`: a pair of one
// written and one read-only buffer is allowed (the polar entry points read
// every input before they write the first output).
int check_overlaps(std::vector<Span>& v, bool outputs_may_overlap_inputs, char* msg, int len) {
  std::stable_sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  std::vector<int> live;   // earlier spans that may still reach the current one
  for (int i = 0; i < (int)v.size(); ++i) {
    size_t k = 0;
    for (int j : live)
      if (v[j].hi > v[i].lo) live[k++] = j;
    live.resize(k);
    for (int j : live) {
      const Span& a = v[j];
      const Span& b = v[i];
      if (!a.writes && !b.writes) continue;
      if (outputs_may_overlap_inputs && a.writes != b.writes) continue;
      if (spans_meet(a, b))
        return fail(msg, len, MUON_ERR_INVALID_ARG, "%s[%d] and %s[%d] share memory", a.what, a.idx, b.what,
                    b.idx);
    }
    live.push_back(i);
  }
  return MUON_OK;
}

bool nonempty(const muon_matrix& m) { return m.rows > 0 && m.cols > 0; }

int same_shape(const muon_matrix& a, const muon_matrix& b, const char* wa, const char* wb, int i, char* msg,
               int len) {
  if (a.rows != b.rows || a.cols != b.cols)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d] is %lld x %lld but %s[%d] is %lld x %lld", wb, i,
                (long long)b.rows, (long long)b.cols, wa, i, (long long)a.rows, (long long)a.cols);
  return MUON_OK;
}

}  // namespace

int check_config(const muon_config* c, char* msg, int len) {
  if (!c) return MUON_OK;
  if (c->ns_steps < 1 || c->ns_steps > 64)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "ns_steps %d outside [1, 64]", (int)c->ns_steps);
  if (!finitef(c->ns_a) || !finitef(c->ns_b) || !finitef(c->ns_c))
    return fail(msg, len, MUON_ERR_INVALID_ARG, "ns coefficients must be finite");
  if (!finitef(c->ns_eps) || c->ns_eps < 0.f) return fail(msg, len, MUON_ERR_INVALID_ARG, "ns_eps must be >= 0");
  if (c->pp_iterations < 0 || c->pp_iterations > 8)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "pp_iterations %d outside [0, 8]", (int)c->pp_iterations);
  if (!finitef(c->pp_beta)) return fail(msg, len, MUON_ERR_INVALID_ARG, "pp_beta must be finite");
  if (!finitef(c->pp_eps) || !(c->pp_eps > 0.f)) return fail(msg, len, MUON_ERR_INVALID_ARG, "pp_eps must be > 0");
  if (!finitef(c->mu) || c->mu < 0.f || c->mu > 1.f)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "mu must lie in [0, 1]");
  if (c->nesterov != 0 && c->nesterov != 1) return fail(msg, len, MUON_ERR_INVALID_ARG, "nesterov must be 0 or 1");
  if (c->power_steps < 1 || c->power_steps > 64)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "power_steps %d outside [1, 64]", (int)c->power_steps);
  if (!finitef(c->contra)) return fail(msg, len, MUON_ERR_INVALID_ARG, "contra must be finite");
  if (!finitef(c->target_uw) || c->target_uw < 0.f)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "target_uw must be >= 0");
  if (!finitef(c->lr)) return fail(msg, len, MUON_ERR_INVALID_ARG, "lr must be finite");
  if (c->flags & ~MUON_FLAG_ALL)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "flags 0x%x has unknown bits", (unsigned)c->flags);
  return MUON_OK;
}

int check_polar(int n, const muon_matrix* in, const muon_matrix* out, const muon_config* cfg, char* msg, int len) {
  if (msg && len > 0) msg[0] = 0;
  if (n < 0 || n > kMaxBatch) return fail(msg, len, MUON_ERR_INVALID_ARG, "batch size %d outside [0, %d]", n, kMaxBatch);
  if (n > 0 && (!in || !out)) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL descriptor array");
  int rc = check_config(cfg, msg, len);
  if (rc) return rc;
  for (int i = 0; i < n; ++i) {
    if ((rc = check_matrix(in[i], "in", i, msg, len))) return rc;
    if ((rc = check_matrix(out[i], "out", i, msg, len))) return rc;
    if ((rc = same_shape(in[i], out[i], "in", "out", i, msg, len))) return rc;
  }
  std::vector<Span> v;
  for (int i = 0; i < n; ++i) {
    if (nonempty(in[i])) v.push_back(make_span(in[i], "in", i, false));
    if (nonempty(out[i])) v.push_back(make_span(out[i], "out", i, true));
  }
  return check_overlaps(v, true, msg, len);
}

int check_update(int n, const muon_matrix* g, const muon_matrix* m, const muon_matrix* w, const muon_matrix* uo,
                 const muon_config* cfg, char* msg, int len) {
  if (msg && len > 0) msg[0] = 0;
  if (n < 0 || n > kMaxBatch) return fail(msg, len, MUON_ERR_INVALID_ARG, "batch size %d outside [0, %d]", n, kMaxBatch);
  if (n > 0 && (!g || !m)) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL grad or momentum array");
  int rc = check_config(cfg, msg, len);
  if (rc) return rc;
  for (int i = 0; i < n; ++i) {
    if ((rc = check_matrix(g[i], "grad", i, msg, len))) return rc;
    if ((rc = check_matrix(m[i], "momentum", i, msg, len))) return rc;
    if (m[i].dtype != MUON_F32)
      return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "momentum[%d] must be MUON_F32", i);
    if ((rc = same_shape(g[i], m[i], "grad", "momentum", i, msg, len))) return rc;
    if (w && w[i].ptr) {
      if ((rc = check_matrix(w[i], "weight", i, msg, len))) return rc;
      if ((rc = same_shape(g[i], w[i], "grad", "weight", i, msg, len))) return rc;
    }
    if (uo && uo[i].ptr) {
      if ((rc = check_matrix(uo[i], "update_out", i, msg, len))) return rc;
      if ((rc = same_shape(g[i], uo[i], "grad", "update_out", i, msg, len))) return rc;
    }
  }
  std::vector<Span> v;
  for (int i = 0; i < n; ++i) {
    if (nonempty(g[i])) v.push_back(make_span(g[i], "grad", i, false));
    if (nonempty(m[i])) v.push_back(make_span(m[i], "momentum", i, true));
    if (w && w[i].ptr && nonempty(w[i])) v.push_back(make_span(w[i], "weight", i, true));
    if (uo && uo[i].ptr && nonempty(uo[i])) v.push_back(make_span(uo[i], "update_out", i, true));
  }
  return check_overlaps(v, false, msg, len);
}

// ---------------------------------------------------------------------------
// Training-step entry points. Their tensors are not tied to the matrix limits
// of the Newton-Schulz engine: vectors of any length and tall embeddings.
// ---------------------------------------------------------------------------
namespace {

int check_tensor(const muon_matrix& m, const char* what, int i, char* msg, int len) {
  if (m.dtype != MUON_F32 && m.dtype != MUON_BF16)
    return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "%s[%d]: dtype %d is not MUON_F32 or MUON_BF16", what, i,
                (int)m.dtype);
  if (m.rows < 0 || m.cols < 0)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: negative shape %lld x %lld", what, i,
                (long long)m.rows, (long long)m.cols);
  if (m.rows == 0 || m.cols == 0) return MUON_OK;
  if (!m.ptr) return fail(msg, len, MUON_ERR_INVALID_ARG, "%s[%d]: NULL pointer for a non-empty tensor", what, i);
  if ((u128)m.rows * (u128)m.cols > (u128)kMaxListElems)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: %lld x %lld exceeds 2^42 elements", what, i,
                (long long)m.rows, (long long)m.cols);
  if (m.rows > 1 && m.ld < m.cols)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: ld %lld < cols %lld", what, i, (long long)m.ld,
                (long long)m.cols);
  if (m.rows > 1 && m.ld > kMaxLd)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s[%d]: ld %lld exceeds 2^40", what, i, (long long)m.ld);
  if (((uintptr_t)m.ptr) % (uintptr_t)elem_size(m.dtype) != 0)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "%s[%d]: pointer not aligned to its element size", what, i);
  return MUON_OK;
}

// A single row has no stride of its own: the span takes its length.
Span tensor_span(muon_matrix m, const char* what, int idx, bool writes) {
  if (m.rows == 1) m.ld = m.cols;
  return make_span(m, what, idx, writes);
}

bool same_buffer(const muon_matrix& a, const muon_matrix& b) {
  return a.ptr == b.ptr && a.dtype == b.dtype && a.rows == b.rows && a.cols == b.cols &&
         (a.rows <= 1 || a.ld == b.ld);
}

// check_overlaps behind a quick look: buffers whose extents are all apart, the
// ordinary case, need neither the spans' sort nor the rules for interleaved
// rows (most of a short list's validation time otherwise).
int check_apart(std::vector<Span>& v, char* msg, int len) {
  struct Extent {
    uint64_t lo, hi;
  };
  std::vector<Extent> e;
  e.reserve(v.size());
  bool apart = true;
  for (const Span& s : v) {
    apart = apart && s.hi <= (u128)UINT64_MAX;
    e.push_back(Extent{(uint64_t)s.lo, (uint64_t)s.hi});
  }
  if (apart) {
    std::sort(e.begin(), e.end(), [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
    for (size_t i = 1; i < e.size(); ++i) apart = apart && e[i - 1].hi <= e[i].lo;
  }
  return apart ? (int)MUON_OK : check_overlaps(v, false, msg, len);
}

// Device scalars and vectors as one-row spans.
Span flat_span(const void* p, int64_t bytes, const char* what, bool writes) {
  Span s;
  s.lo = (u128)(uintptr_t)p;
  s.ldb = s.rowb = (u128)bytes;
  s.hi = s.lo + (u128)bytes;
  s.rows = 1;
  s.what = what;
  s.idx = 0;
  s.writes = writes;
  return s;
}

}  // namespace

namespace {

// A list with its outputs and device scalars: writes tells whether tensors
// without an output of their own are written, `scalars` whether norm and coef are.
int check_list(int n, const muon_matrix* g, const muon_matrix* out, float max_norm, const float* norm,
               const float* coef, bool writes, bool scalars, char* msg, int len) {
  if (msg && len > 0) msg[0] = 0;
  if (n < 0 || n > kMaxBatch) return fail(msg, len, MUON_ERR_INVALID_ARG, "list length %d outside [0, %d]", n, kMaxBatch);
  if (n > 0 && !g) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL grad array");
  if (((uintptr_t)norm | (uintptr_t)coef) % 4 != 0)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "norm or coefficient not aligned to 4 bytes");
  if (coef && !(max_norm > 0.0f)) return fail(msg, len, MUON_ERR_INVALID_ARG, "max_norm must be positive");
  int rc;
  for (int i = 0; i < n; ++i) {
    if ((rc = check_tensor(g[i], "grad", i, msg, len))) return rc;
    if (!out) continue;
    if ((rc = check_tensor(out[i], "out", i, msg, len))) return rc;
    if ((rc = same_shape(g[i], out[i], "grad", "out", i, msg, len))) return rc;
  }
  // the kernels read a tensor again after they wrote others: an output shares
  // memory with nothing but the input it replaces, element for element
  std::vector<Span> v;
  v.reserve((size_t)n * 2 + 2);
  for (int i = 0; i < n; ++i) {
    if (!nonempty(g[i])) continue;
    const bool own = !out || same_buffer(g[i], out[i]);
    v.push_back(tensor_span(g[i], "grad", i, own && writes));
    if (!own) v.push_back(tensor_span(out[i], "out", i, true));
  }
  if (norm) v.push_back(flat_span(norm, 4, "norm", scalars));
  if (coef) v.push_back(flat_span(coef, 4, "coefficient", scalars));
  return check_apart(v, msg, len);
}

}  // namespace

int check_norm(int n, const muon_matrix* g, const muon_matrix* out, float max_norm, const float* norm,
               const float* coef, int writes, char* msg, int len) {
  if (!norm) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL norm");
  return check_list(n, g, out, max_norm, norm, coef, writes != 0, true, msg, len);
}

int check_scale(int n, const muon_matrix* in, const muon_matrix* out, const float* coef, char* msg, int len) {
  if (!coef) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL coefficient");
  return check_list(n, in, out, 1.0f, nullptr, coef, true, false, msg, len);
}

int check_adamw(int n, const muon_matrix* g, const muon_matrix* m, const muon_matrix* v, const muon_matrix* w,
                const muon_matrix* copy, const muon_adamw_config* c, const float* scale, char* msg, int len) {
  if (msg && len > 0) msg[0] = 0;
  if (n < 0 || n > kMaxBatch) return fail(msg, len, MUON_ERR_INVALID_ARG, "list length %d outside [0, %d]", n, kMaxBatch);
  if (n > 0 && (!g || !m || !v || !w)) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL tensor array");
  if (!c) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL configuration");
  if (!c->lr_at && !finitef(c->lr)) return fail(msg, len, MUON_ERR_INVALID_ARG, "lr must be finite");
  if (!(c->beta1 >= 0.0f && c->beta1 < 1.0f) || !(c->beta2 >= 0.0f && c->beta2 < 1.0f))
    return fail(msg, len, MUON_ERR_INVALID_ARG, "betas %g, %g outside [0, 1)", c->beta1, c->beta2);
  if (!(c->eps >= 0.0f) || !finitef(c->eps)) return fail(msg, len, MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!(c->weight_decay >= 0.0f) || !finitef(c->weight_decay))
    return fail(msg, len, MUON_ERR_INVALID_ARG, "weight_decay must be finite and >= 0");
  if (!c->step_at && c->step < 1) return fail(msg, len, MUON_ERR_INVALID_ARG, "step %lld: the first step is 1", (long long)c->step);
  if ((uintptr_t)scale % 4 != 0) return fail(msg, len, MUON_ERR_INVALID_ARG, "grad_scale not aligned to 4 bytes");
  if ((uintptr_t)c->step_at % 8 != 0 || (uintptr_t)c->lr_at % 4 != 0)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "step_at or lr_at not aligned to its value's size");
  int rc;
  std::vector<Span> spans;
  spans.reserve((size_t)n * 5 + 3);
  for (int i = 0; i < n; ++i) {
    if ((rc = check_tensor(w[i], "weight", i, msg, len))) return rc;
    const muon_matrix* xs[] = {&g[i], &m[i], &v[i]};
    const char* names[] = {"grad", "exp_avg", "exp_avg_sq"};
    for (int k = 0; k < 3; ++k) {
      if ((rc = check_tensor(*xs[k], names[k], i, msg, len))) return rc;
      if ((rc = same_shape(w[i], *xs[k], "weight", names[k], i, msg, len))) return rc;
      if (k && xs[k]->dtype != MUON_F32)
        return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "%s[%d] must be MUON_F32", names[k], i);
    }
    const bool cp = copy && nonempty(copy[i]);
    if (cp) {
      if ((rc = check_tensor(copy[i], "copy", i, msg, len))) return rc;
      if ((rc = same_shape(w[i], copy[i], "weight", "copy", i, msg, len))) return rc;
    }
    if (!nonempty(w[i])) continue;
    spans.push_back(tensor_span(g[i], "grad", i, false));
    spans.push_back(tensor_span(m[i], "exp_avg", i, true));
    spans.push_back(tensor_span(v[i], "exp_avg_sq", i, true));
    spans.push_back(tensor_span(w[i], "weight", i, true));
    if (cp) spans.push_back(tensor_span(copy[i], "copy", i, true));
  }
  if (scale) spans.push_back(flat_span(scale, 4, "grad_scale", false));
  if (c->step_at) spans.push_back(flat_span(c->step_at, 8, "step_at", false));
  if (c->lr_at) spans.push_back(flat_span(c->lr_at, 4, "lr_at", false));
  return check_apart(spans, msg, len);
}

namespace {

// A head's hidden states, weight, targets and soft cap, with the spans of what is read.
int check_head(const muon_matrix* hidden, const muon_matrix* weight, const void* targets, int target_bytes, float softcap,
               std::vector<Span>& v, char* msg, int len) {
  if (!hidden || !weight) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL hidden or weight");
  if (target_bytes != 4 && target_bytes != 8)
    return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "targets of %d bytes: 4 or 8 are supported", target_bytes);
  if (!(softcap >= 0.0f) || !finitef(softcap))
    return fail(msg, len, MUON_ERR_INVALID_ARG, "softcap must be finite and >= 0");
  int rc;
  if ((rc = check_tensor(*hidden, "hidden", 0, msg, len))) return rc;
  if ((rc = check_tensor(*weight, "weight", 0, msg, len))) return rc;
  if (weight->rows < 1 || weight->cols < 1)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "weight is %lld x %lld: at least one row and column are needed",
                (long long)weight->rows, (long long)weight->cols);
  if (hidden->cols != weight->cols)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "hidden has %lld columns, weight %lld", (long long)hidden->cols,
                (long long)weight->cols);
  if (hidden->dtype != weight->dtype)
    return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "hidden and weight have different types");
  if (hidden->rows > (1 << 24) || weight->rows > kMaxVocab || weight->cols > kMaxDim)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%lld tokens, %lld x %lld weight: past 2^24, 2^22, %d",
                (long long)hidden->rows, (long long)weight->rows, (long long)weight->cols, kMaxDim);
  const int64_t n = hidden->rows;
  if (n > 0 && !targets) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL targets");
  if ((uintptr_t)targets % (uintptr_t)target_bytes != 0)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "targets not aligned to their element size");
  if (n > 0) v.push_back(tensor_span(*hidden, "hidden", 0, false));
  v.push_back(tensor_span(*weight, "weight", 0, false));
  if (n > 0) v.push_back(flat_span(targets, n * target_bytes, "targets", false));
  return MUON_OK;
}
int check_head_gradients(const muon_matrix* hidden, const muon_matrix* weight, const muon_matrix* dh,
                         const muon_matrix* dw, std::vector<Span>& v, char* msg, int len) {
  const muon_matrix* in[] = {hidden, weight};
  const muon_matrix* out[] = {dh, dw};
  const char* from[] = {"hidden", "weight"};
  const char* to[] = {"dhidden", "dweight"};
  int rc;
  for (int k = 0; k < 2; ++k) {
    if (!out[k]) continue;
    if ((rc = check_tensor(*out[k], to[k], 0, msg, len))) return rc;
    if ((rc = same_shape(*in[k], *out[k], from[k], to[k], 0, msg, len))) return rc;
    if (out[k]->dtype != in[k]->dtype)
      return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "%s has not the type of %s", to[k], from[k]);
    if (nonempty(*out[k])) v.push_back(tensor_span(*out[k], to[k], 0, true));
  }
  return MUON_OK;
}

}  // namespace

int check_loss(const muon_matrix* hidden, const muon_matrix* weight, const void* targets, int target_bytes,
               const muon_loss_config* c, const float* grad_out, const float* loss, const muon_matrix* dh,
               const muon_matrix* dw, int grad, char* msg, int len) {
  if (msg && len > 0) msg[0] = 0;
  std::vector<Span> v;
  int rc;
  if ((rc = check_head(hidden, weight, targets, target_bytes, c->softcap, v, msg, len))) return rc;
  if (grad && !dh && !dw) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL dhidden and dweight");
  if (c->reduction != MUON_REDUCE_NONE && c->reduction != MUON_REDUCE_SUM && c->reduction != MUON_REDUCE_MEAN)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "unknown reduction %d", (int)c->reduction);
  if (((uintptr_t)loss | (uintptr_t)grad_out) % 4 != 0)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "loss or grad_out not aligned to its element size");
  const int64_t each = c->reduction == MUON_REDUCE_NONE ? hidden->rows : 1;
  if (each > 0 && !loss) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL loss");
  if (each > 0) v.push_back(flat_span(loss, each * 4, "loss", true));
  if (grad && (rc = check_head_gradients(hidden, weight, dh, dw, v, msg, len))) return rc;
  if (grad && grad_out && each > 0) v.push_back(flat_span(grad_out, each * 4, "grad_out", false));
  return check_apart(v, msg, len);
}

int check_logprobs(const muon_matrix* hidden, const muon_matrix* weight, const void* targets, int target_bytes,
                   const muon_logprob_config* c, const float* logprobs, const float* entropy, const float* stats,
                   const float* top_logprobs, const int64_t* top_tokens, char* msg, int len) {
  if (msg && len > 0) msg[0] = 0;
  std::vector<Span> v;
  int rc;
  if ((rc = check_head(hidden, weight, targets, target_bytes, c->softcap, v, msg, len))) return rc;
  if (c->top < 0 || c->top > MUON_TOP_MOST || c->top > weight->rows)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "%d alternatives: 0 to %d, and no more than the vocabulary's %lld, are supported",
                (int)c->top, MUON_TOP_MOST, (long long)weight->rows);
  const int64_t n = hidden->rows;
  if (n == 0) return MUON_OK;
  if (!logprobs) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL logprobs");
  if (c->top && (!top_logprobs || !top_tokens))
    return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL top_logprobs or top_tokens");
  if (((uintptr_t)logprobs | (uintptr_t)entropy) % 4 != 0 || (uintptr_t)stats % 16 != 0 ||
      (c->top && ((uintptr_t)top_logprobs % 4 != 0 || (uintptr_t)top_tokens % 8 != 0)))
    return fail(msg, len, MUON_ERR_INVALID_ARG, "an output is not aligned to its element size (stats: 16 bytes)");
  v.push_back(flat_span(logprobs, n * 4, "logprobs", true));
  if (entropy) v.push_back(flat_span(entropy, n * 4, "entropy", true));
  if (stats) v.push_back(flat_span(stats, n * 16, "stats", true));
  if (c->top) {
    v.push_back(flat_span(top_logprobs, n * c->top * 4, "top_logprobs", true));
    v.push_back(flat_span(top_tokens, n * c->top * 8, "top_tokens", true));
  }
  return check_apart(v, msg, len);
}

int check_logprobs_grad(const muon_matrix* hidden, const muon_matrix* weight, const void* targets, int target_bytes,
                        const muon_logprob_config* c, const float* stats, const float* grad_logprobs,
                        const float* grad_entropy, const muon_matrix* dh, const muon_matrix* dw, char* msg, int len) {
  if (msg && len > 0) msg[0] = 0;
  std::vector<Span> v;
  int rc;
  if ((rc = check_head(hidden, weight, targets, target_bytes, c->softcap, v, msg, len))) return rc;
  if (!dh && !dw) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL dhidden and dweight");
  const int64_t n = hidden->rows;
  if (n > 0 && !stats) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL stats");
  if (n > 0 && !grad_logprobs && !grad_entropy)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL grad_logprobs and grad_entropy");
  if ((uintptr_t)stats % 16 != 0 || ((uintptr_t)grad_logprobs | (uintptr_t)grad_entropy) % 4 != 0)
    return fail(msg, len, MUON_ERR_INVALID_ARG, "stats or a gradient is not aligned to its element size (stats: 16 bytes)");
  if (n > 0) {
    v.push_back(flat_span(stats, n * 16, "stats", false));
    if (grad_logprobs) v.push_back(flat_span(grad_logprobs, n * 4, "grad_logprobs", false));
    if (grad_entropy) v.push_back(flat_span(grad_entropy, n * 4, "grad_entropy", false));
  }
  if ((rc = check_head_gradients(hidden, weight, dh, dw, v, msg, len))) return rc;
  return check_apart(v, msg, len);
}


namespace {

// x, y and the parameters, with the spans of what is read.
int check_norm_inputs(const muon_matrix* x, const muon_matrix* y, const muon_norm_params* p, std::vector<Span>& v,
                      char* msg, int len) {
  if (!x) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL x");
  if (!(p->eps > 0.0f) || !finitef(p->eps)) return fail(msg, len, MUON_ERR_INVALID_ARG, "eps must be finite and > 0");
  int rc;
  if ((rc = check_tensor(*x, "x", 0, msg, len))) return rc;
  if (x->cols < 1 || x->cols > kNormMostD || x->rows >= kNormMostRows)
    return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "x is %lld x %lld: 1 to %d columns and fewer than 2^31 rows are supported",
                (long long)x->rows, (long long)x->cols, kNormMostD);
  if (y) {
    if ((rc = check_tensor(*y, "y", 0, msg, len))) return rc;
    if ((rc = same_shape(*x, *y, "x", "y", 0, msg, len))) return rc;
    if (y->dtype == MUON_F32 && x->dtype != MUON_F32)
      return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "y is MUON_F32 beside a MUON_BF16 x");
  }
  if (p->post_gain && (!y || !p->post_norm)) return fail(msg, len, MUON_ERR_INVALID_ARG, "post_gain without a norm of y");
  if (p->gate && !y) return fail(msg, len, MUON_ERR_INVALID_ARG, "gate without y");
  if (p->pre_gain && !p->pre_norm) return fail(msg, len, MUON_ERR_INVALID_ARG, "pre_gain without a norm of out");
  if (nonempty(*x)) v.push_back(tensor_span(*x, "x", 0, false));
  if (y && nonempty(*y)) v.push_back(tensor_span(*y, "y", 0, false));
  const muon_matrix* params[] = {p->post_gain, p->pre_gain, p->gate, p->scale};
  const char* names[] = {"post_gain", "pre_gain", "gate", "scale"};
  for (int k = 0; k < 4; ++k) {
    if (!params[k]) continue;
    const muon_matrix& m = *params[k];
    if ((rc = check_tensor(m, names[k], 0, msg, len))) return rc;
    const int kind = norm_kind(m, x->rows, x->cols);
    // (one channel: its one value is the vector)
    const bool fits = k < 2 ? m.rows == 1 && m.cols == x->cols
                            : kind == NORM_ONE || kind == NORM_CHANNELS || (kind == NORM_FULL && k == 2);
    if (!fits)
      return fail(msg, len, MUON_ERR_SHAPE_MISMATCH, "%s is %lld x %lld for %lld x %lld", names[k], (long long)m.rows,
                  (long long)m.cols, (long long)x->rows, (long long)x->cols);
    if (kind == NORM_FULL && k == 2 && m.dtype != y->dtype)
      return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "a gate of y's shape has not y's type");
    if (nonempty(m)) v.push_back(tensor_span(m, names[k], 0, false));
  }
  return MUON_OK;
}

// A tensor with the shape of another and a given type, or null.
int check_like(const muon_matrix* m, const char* what, const muon_matrix& like, const char* like_what, int dtype,
               bool writes, std::vector<Span>& v, char* msg, int len) {
  if (!m) return MUON_OK;
  int rc;
  if ((rc = check_tensor(*m, what, 0, msg, len))) return rc;
  if ((rc = same_shape(like, *m, like_what, what, 0, msg, len))) return rc;
  if (m->dtype != dtype) return fail(msg, len, MUON_ERR_UNSUPPORTED_DTYPE, "%s has not the type of %s", what, like_what);
  if (nonempty(*m)) v.push_back(tensor_span(*m, what, 0, writes));
  return MUON_OK;
}

// The type of hidden and its gradient: y's, or without y x's or a 16-bit one.
int hidden_dtype(const muon_matrix& x, const muon_matrix* y, const muon_matrix* hidden) {
  if (y) return y->dtype;
  return hidden && hidden->dtype == MUON_BF16 ? (int)MUON_BF16 : x.dtype;
}

}  // namespace

int check_residual_norm(const muon_matrix* x, const muon_matrix* y, const muon_norm_params* p, const muon_matrix* out,
                        const muon_matrix* hidden, char* msg, int len) {
  if (msg && len > 0) msg[0] = 0;
  std::vector<Span> v;
  int rc;
  if ((rc = check_norm_inputs(x, y, p, v, msg, len))) return rc;
  if (y && !out) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL out beside y");
  if (!out && !hidden) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL out and hidden");
  if ((hidden != nullptr) != (p->pre_norm != 0))
    return fail(msg, len, MUON_ERR_INVALID_ARG, hidden ? "hidden without a norm of out" : "NULL hidden");
  if ((rc = check_like(out, "out", *x, "x", x->dtype, true, v, msg, len))) return rc;
  if ((rc = check_like(hidden, "hidden", *x, y ? "y" : "x", hidden_dtype(*x, y, hidden), true, v, msg, len))) return rc;
  return check_apart(v, msg, len);
}

int check_residual_norm_grad(const muon_matrix* x, const muon_matrix* y, const muon_norm_params* p,
                             const muon_matrix* dout, const muon_matrix* dhidden, const muon_norm_grads* g, char* msg,
                             int len) {
  if (msg && len > 0) msg[0] = 0;
  std::vector<Span> v;
  int rc;
  if ((rc = check_norm_inputs(x, y, p, v, msg, len))) return rc;
  if (!dout && !dhidden) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL dout and dhidden");
  if (dhidden && !p->pre_norm) return fail(msg, len, MUON_ERR_INVALID_ARG, "dhidden without a norm of out");
  if ((rc = check_like(dout, "dout", *x, "x", x->dtype, false, v, msg, len))) return rc;
  if ((rc = check_like(dhidden, "dhidden", *x, y ? "y" : "x", hidden_dtype(*x, y, dhidden), false, v, msg, len))) return rc;
  if (!g) return fail(msg, len, MUON_ERR_INVALID_ARG, "NULL gradients");
  const muon_matrix* of[] = {x, y, p->post_gain, p->gate, p->scale, p->pre_gain};
  const muon_matrix* to[] = {g->x, g->y, g->post_gain, g->gate, g->scale, g->pre_gain};
  const char* names[] = {"x", "y", "post_gain", "gate", "scale", "pre_gain"};
  const char* grads[] = {"dx", "dy", "dpost_gain", "dgate", "dscale", "dpre_gain"};
  bool any = false;
  for (int k = 0; k < 6; ++k) {
    if (!to[k]) continue;
    any = true;
    if (!of[k]) return fail(msg, len, MUON_ERR_INVALID_ARG, "%s without %s", grads[k], names[k]);
    if ((rc = check_like(to[k], grads[k], *of[k], names[k], of[k]->dtype, true, v, msg, len))) return rc;
  }
  if (!any) return fail(msg, len, MUON_ERR_INVALID_ARG, "no gradient is asked for");
  return check_apart(v, msg, len);
}

}  // namespace muon

namespace {

// A validation's body behind a C entry point: no exception (the lists' spans are
// on the heap) leaves it.
template <typename F>
muon_status checked(char* msg, int len, F body) noexcept {
  try {
    return body();
  } catch (...) {
    return muon::fail(msg, len, MUON_ERR_ALLOC, "out of host memory");
  }
}

}  // namespace

extern "C" muon_status muon_check_norm_args(int n, const muon_matrix* grad, const muon_matrix* out, float max_norm,
                                            const float* norm, const float* coef, char* msg, int msg_len) {
  return checked(msg, msg_len, [&] {
    return muon::check_norm(n, grad, out, max_norm, norm, coef, out != nullptr, msg, msg_len);
  });
}
extern "C" muon_status muon_check_adamw_args(int n, const muon_matrix* grad, const muon_matrix* exp_avg,
                                             const muon_matrix* exp_avg_sq, const muon_matrix* weight,
                                             const muon_matrix* copy, const muon_adamw_config* cfg,
                                             const float* grad_scale, char* msg, int msg_len) {
  return checked(msg, msg_len, [&] {
    return muon::check_adamw(n, grad, exp_avg, exp_avg_sq, weight, copy, cfg, grad_scale, msg, msg_len);
  });
}
extern "C" muon_status muon_check_loss_args(const muon_matrix* hidden, const muon_matrix* weight, const void* targets,
                                            int target_bytes, const muon_loss_config* cfg, const float* grad_out,
                                            const float* loss, const muon_matrix* dhidden, const muon_matrix* dweight,
                                            char* msg, int msg_len) {
  muon_loss_config c;
  muon_loss_config_default(&c);
  if (cfg) c = *cfg;
  return checked(msg, msg_len, [&] {
    return muon::check_loss(hidden, weight, targets, target_bytes, &c, grad_out, loss, dhidden, dweight,
                            dhidden || dweight ? 1 : 0, msg, msg_len);
  });
}

extern "C" muon_status muon_check_logprob_args(const muon_matrix* hidden, const muon_matrix* weight,
                                               const void* targets, int target_bytes, const muon_logprob_config* cfg,
                                               const float* logprobs, const float* entropy, const float* stats,
                                               const float* top_logprobs, const int64_t* top_tokens, char* msg,
                                               int msg_len) {
  muon_logprob_config c;
  muon_logprob_config_default(&c);
  if (cfg) c = *cfg;
  return checked(msg, msg_len, [&] {
    return muon::check_logprobs(hidden, weight, targets, target_bytes, &c, logprobs, entropy, stats, top_logprobs,
                                top_tokens, msg, msg_len);
  });
}
extern "C" muon_status muon_check_logprob_grad_args(const muon_matrix* hidden, const muon_matrix* weight,
                                                    const void* targets, int target_bytes,
                                                    const muon_logprob_config* cfg, const float* stats,
                                                    const float* grad_logprobs, const float* grad_entropy,
                                                    const muon_matrix* dhidden, const muon_matrix* dweight, char* msg,
                                                    int msg_len) {
  muon_logprob_config c;
  muon_logprob_config_default(&c);
  if (cfg) c = *cfg;
  return checked(msg, msg_len, [&] {
    return muon::check_logprobs_grad(hidden, weight, targets, target_bytes, &c, stats, grad_logprobs, grad_entropy,
                                     dhidden, dweight, msg, msg_len);
  });
}

extern "C" void muon_logprob_config_default(muon_logprob_config* c) {
  if (!c) return;
  *c = muon_logprob_config{0, 0.0f, -100};
}

namespace {

muon_norm_params params_or_default(const muon_norm_params* p) {
  muon_norm_params q;
  muon_norm_params_default(&q);
  return p ? *p : q;
}

}  // namespace

extern "C" muon_status muon_check_residual_norm_args(const muon_matrix* x, const muon_matrix* y,
                                                     const muon_norm_params* params, const muon_matrix* out,
                                                     const muon_matrix* hidden, char* msg, int msg_len) {
  const muon_norm_params p = params_or_default(params);
  return checked(msg, msg_len, [&] { return muon::check_residual_norm(x, y, &p, out, hidden, msg, msg_len); });
}
extern "C" muon_status muon_check_residual_norm_grad_args(const muon_matrix* x, const muon_matrix* y,
                                                          const muon_norm_params* params, const muon_matrix* dout,
                                                          const muon_matrix* dhidden, const muon_norm_grads* grads,
                                                          char* msg, int msg_len) {
  const muon_norm_params p = params_or_default(params);
  return checked(msg, msg_len,
                 [&] { return muon::check_residual_norm_grad(x, y, &p, dout, dhidden, grads, msg, msg_len); });
}

extern "C" void muon_norm_params_default(muon_norm_params* p) {
  if (!p) return;
  *p = muon_norm_params{nullptr, nullptr, nullptr, nullptr, 1, 1, 1e-6f};
}

extern "C" void muon_loss_config_default(muon_loss_config* c) {
  if (!c) return;
  c->reduction = MUON_REDUCE_MEAN;
  c->softcap = 0.0f;
  c->ignore_index = -100;
}

extern "C" void muon_adamw_config_default(muon_adamw_config* c) {
  if (!c) return;
  c->lr = 0.01f;
  c->beta1 = 0.8f;
  c->beta2 = 0.95f;
  c->eps = 1e-10f;
  c->weight_decay = 0.0f;
  c->step = 1;
  c->step_at = nullptr;
  c->lr_at = nullptr;
}

extern "C" muon_status muon_check_update_args(int n, const muon_matrix* grad, const muon_matrix* momentum,
                                              const muon_matrix* weight, const muon_matrix* update_out,
                                              const muon_config* cfg, char* msg, int msg_len) {
  return checked(msg, msg_len,
                 [&] { return muon::check_update(n, grad, momentum, weight, update_out, cfg, msg, msg_len); });
}

extern "C" muon_status muon_check_polar_args(int n, const muon_matrix* in, const muon_matrix* out,
                                             const muon_config* cfg, char* msg, int msg_len) {
  return checked(msg, msg_len, [&] { return muon::check_polar(n, in, out, cfg, msg, msg_len); });
}

extern "C" void muon_config_default(muon_config* c) {
  if (!c) return;
  c->ns_steps = 12;
  c->ns_a = 2.0f;
  c->ns_b = -1.5f;
  c->ns_c = 0.5f;
  c->ns_eps = 1e-7f;
  c->pp_iterations = 2;
  c->pp_beta = 0.5f;
  c->pp_eps = 1e-7f;
  c->mu = 0.95f;
  c->nesterov = 1;
  c->power_steps = 5;
  c->contra = 0.4f;
  c->target_uw = 0.35f;
  c->lr = 0.0375f;
  c->flags = 0;
}

// Classic recipe of the Track-1 record page, §"训练管线与系统实现".
extern "C" void muon_config_classic(muon_config* c) {
  if (!c) return;
  muon_config_default(c);
  c->ns_steps = 5;
  c->ns_a = 3.4445f;
  c->ns_b = -4.7750f;
  c->ns_c = 2.0315f;
  c->pp_iterations = 0;
  c->contra = 0.0f;
  c->target_uw = 0.0f;
  c->mu = 0.95f;
  c->nesterov = 1;
  c->lr = 0.04f;
  c->flags = MUON_FLAG_SGD_MOMENTUM;
}

// Linear momentum warm-up of the same page: frac = min(step / n, 1).
extern "C" float muon_momentum_warmup(int64_t step, float mu_start, float mu_end, int64_t warmup_steps) {
  if (warmup_steps <= 0) return mu_end;
  const double s = step < 0 ? 0.0 : (double)step;
  const double frac = s >= (double)warmup_steps ? 1.0 : s / (double)warmup_steps;
  return (float)((1.0 - frac) * (double)mu_start + frac * (double)mu_end);
}

extern "C" const char* muon_status_string(muon_status s) {
  switch (s) {
    case MUON_OK: return "MUON_OK";
    case MUON_ERR_INVALID_ARG: return "MUON_ERR_INVALID_ARG";
    case MUON_ERR_UNSUPPORTED_DTYPE: return "MUON_ERR_UNSUPPORTED_DTYPE";
    case MUON_ERR_SHAPE_MISMATCH: return "MUON_ERR_SHAPE_MISMATCH";
    case MUON_ERR_ALLOC: return "MUON_ERR_ALLOC";
    case MUON_ERR_HIP: return "MUON_ERR_HIP";
    case MUON_ERR_NO_DEVICE: return "MUON_ERR_NO_DEVICE";
    case MUON_ERR_TOO_LARGE: return "MUON_ERR_TOO_LARGE";
    case MUON_ERR_NONFINITE: return "MUON_ERR_NONFINITE";
    default: return "MUON_ERR_UNKNOWN";
  }
}

extern "C" const char* muon_version(void) { return "0.1.0"; }
