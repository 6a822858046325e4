// args.h -- argument checks shared by the C entry points (api.cu and
// block/api_block.cu), and what api.cu keeps for all of them: the device
// facts, the status word and the test hooks.
#pragma once

#include <cmath>

#include "../launch.h"

namespace gb300norm {

// The current device's facts (with the test hooks filled in) and its status
// word.  Defined in api.cu.
int get_device(DevInfo* out, int** status);

// Test hook: 1 = the kernels whose rows come by bulk copies withhold each row
// group's last one.
int hold_last_hook();

inline int elem_size(int dt) {
  switch (dt) {
    case NORM_F32: return 4;
    case NORM_F16: return 2;
    case NORM_BF16: return 2;
    default: return 0;
  }
}

inline bool types_ok(int dt, int wdt) {
  return (dt == NORM_F32 && wdt == NORM_F32) || (dt == NORM_F16 && wdt == NORM_F16) ||
         (dt == NORM_BF16 && wdt == NORM_BF16) || (dt == NORM_BF16 && wdt == NORM_F32) ||
         (dt == NORM_F16 && wdt == NORM_F32);
}

// ---------------------------------------------------------------------------
// Argument checks
// ---------------------------------------------------------------------------
inline bool finite(float v) { return std::isfinite(v); }

// A 2-D row tensor argument.
struct Mat {
  const void* p;
  int64_t stride;
};

inline int check_mat(const Mat& m, int64_t M, int64_t N, int es, bool required) {
  if (M == 0) return NORM_OK;
  if (!m.p) return required ? NORM_ERR_NULL : NORM_OK;
  if (m.stride < N) return NORM_ERR_STRIDE;
  // the byte extent ((M - 1) * stride + N) * es must fit in 63 bits (it is
  // formed on the host for the overlap checks and in the kernels' row offsets)
  if (M - 1 > (INT64_MAX / es - N) / m.stride) return NORM_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(m.p) % (uintptr_t)es) return NORM_ERR_ALIGN;
  return NORM_OK;
}

inline bool row16(const Mat& m, int64_t M, int es) {
  if (!m.p) return true;
  if (reinterpret_cast<uintptr_t>(m.p) % 16) return false;
  return M <= 1 || (m.stride * es) % 16 == 0;
}

// A byte range touched by a call, for overlap checks.
struct Span {
  uintptr_t lo = 0, hi = 0;   // [lo, hi)
  const void* p = nullptr;
  int64_t stride = 0;
  bool out = false;
  unsigned tag = 0;            // outputs may coincide exactly with inputs sharing a tag bit
};

inline Span mat_span(const Mat& m, int64_t M, int64_t N, int es, bool out, unsigned tag) {
  Span s;
  if (!m.p || M == 0) return s;
  s.p = m.p;
  s.stride = m.stride;
  s.lo = reinterpret_cast<uintptr_t>(m.p);
  s.hi = s.lo + (uintptr_t)(((M - 1) * m.stride + N) * es);
  s.out = out;
  s.tag = tag;
  return s;
}

inline Span vec_span(const void* p, int64_t n, int es, bool out) {
  Span s;
  if (!p || n == 0) return s;
  s.p = p;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.hi = s.lo + (uintptr_t)(n * es);
  s.out = out;
  return s;
}

inline int check_overlaps(const Span* s, int n) {
  for (int i = 0; i < n; ++i) {
    if (!s[i].out || s[i].lo == s[i].hi) continue;
    for (int j = 0; j < n; ++j) {
      if (i == j || s[j].lo == s[j].hi) continue;
      if (s[i].lo >= s[j].hi || s[j].lo >= s[i].hi) continue;
      const bool exact = !s[j].out && (s[i].tag & s[j].tag) && s[i].p == s[j].p && s[i].stride == s[j].stride;
      if (!exact) return NORM_ERR_ALIAS;
    }
  }
  return NORM_OK;
}

inline int check_common(int64_t M, int64_t N, float offset, float eps, int dtype, int w_dtype, const void* w) {
  if (M < 0 || N <= 0 || N > INT32_MAX) return NORM_ERR_SHAPE;
  if (!types_ok(dtype, w_dtype)) return NORM_ERR_DTYPE;
  if (!finite(offset) || !finite(eps) || eps < 0.f) return NORM_ERR_VALUE;
  if (!w) return NORM_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(w) % (uintptr_t)elem_size(w_dtype)) return NORM_ERR_ALIGN;
  return NORM_OK;
}

inline int check_vec_f32(const void* p) {
  return (p && reinterpret_cast<uintptr_t>(p) % 4) ? NORM_ERR_ALIGN : NORM_OK;
}

inline int64_t ws_bytes_needed(int64_t M, int64_t N, int sms, int nbuf) {
  return partial_rows(M, N, sms) * N * 4 * nbuf;
}

// The workspace pointer is checked before the device is queried for its size.
inline int check_workspace_ptr(const void* ws) {
  return (!ws || reinterpret_cast<uintptr_t>(ws) % 16) ? NORM_ERR_WORKSPACE : NORM_OK;
}

inline int check_workspace(const void* ws, size_t ws_bytes, int64_t need) {
  if (need == 0) return NORM_OK;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 16 || ws_bytes < (size_t)need) return NORM_ERR_WORKSPACE;
  return NORM_OK;
}

#define RETURN_IF(x)            \
  do {                          \
    int rc_ = (x);              \
    if (rc_ != NORM_OK) return rc_; \
  } while (0)

}  // namespace gb300norm
