// ssd_args.h -- argument checks of the calls that take views and a workspace of
// the caller's (the recurrence, the norm with rotation, the cache and the
// attention over it).  Host only; not installed, not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_check.h"

namespace ssd {

constexpr int64_t kMaxOuter = (int64_t)1 << 36; // strides, where nothing narrower is said

inline const char *dtype_name(int d) {
  switch (d) {
  case SSD_F32: return "f32";
  case SSD_BF16: return "bf16";
  case SSD_U8: return "u8";
  case SSD_I32: return "i32";
  case SSD_I64: return "i64";
  }
  return "unknown";
}

// Memory from the first element's first byte to the last one's last.
inline Range span_of(const ssd_tensor *t) {
  Range r;
  if (!t || !t->data) return r;
  int64_t last = 0;
  for (int i = 0; i < t->ndim; ++i) last += (t->shape[i] - 1) * t->strides[i];
  r.lo = (uintptr_t)t->data;
  r.hi = r.lo + (uintptr_t)((last + 1) * elem_size(t->dtype));
  return r;
}

// Presence, dtype, rank, shape, and the alignment of one element; dense
// row-major, or (view) a contiguous last dimension with other strides >= 0,
// those behind the batch at most max_stride.
inline int check_arg(const ssd_tensor *t, const char *name, int dtype, int ndim, const int64_t *shape, bool view = false,
              int64_t max_stride = kMaxOuter) {
  if (!t) return fail(SSD_ERR_NULL, "%s: descriptor is NULL", name);
  if (!t->data) return fail(SSD_ERR_NULL, "%s: data pointer is NULL", name);
  if (t->dtype != dtype)
    return fail(SSD_ERR_DTYPE, "%s: dtype %s, expected %s", name, dtype_name(t->dtype), dtype_name(dtype));
  if (t->ndim != ndim) return fail(SSD_ERR_SHAPE, "%s: rank %d, expected %d", name, t->ndim, ndim);
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] != shape[i])
      return fail(SSD_ERR_SHAPE, "%s: dim %d is %lld, expected %lld", name, i, (long long)t->shape[i],
                  (long long)shape[i]);
  int64_t dense = 1;
  for (int i = ndim - 1; i >= 0; --i) {
    const int64_t st = t->strides[i];
    if (t->shape[i] != 1) {
      if ((!view || i == ndim - 1) && st != dense)
        return fail(SSD_ERR_LAYOUT, "%s: stride of dim %d is %lld, expected %lld", name, i, (long long)st,
                    (long long)dense);
      if (view && (st < 0 || st > (i == 0 ? kMaxOuter : max_stride)))
        return fail(st < 0 ? SSD_ERR_LAYOUT : SSD_ERR_UNSUPPORTED, "%s: stride of dim %d is %lld", name, i,
                    (long long)st);
    }
    dense *= t->shape[i];
  }
  if ((uintptr_t)t->data % (uintptr_t)elem_size(dtype) != 0)
    return fail(SSD_ERR_LAYOUT, "%s: data pointer is not aligned to its element", name);
  return SSD_OK;
}

inline int act_dtype(const ssd_tensor *t, const char *name) {
  if (t->dtype != SSD_F32 && t->dtype != SSD_BF16)
    return fail(SSD_ERR_DTYPE, "%s: dtype %s, expected f32 or bf16", name, dtype_name(t->dtype));
  return SSD_OK;
}

// The type asked of an output's gradient: f32 or that of x.
inline int grad_dtype(const ssd_tensor *t, const ssd_tensor *x) { return t && t->dtype == SSD_F32 ? SSD_F32 : x->dtype; }

// A call's tensors, for the checks over all of them.
struct Args {
  static constexpr int kMax = 24;
  const ssd_tensor *t[kMax];
  const char *name[kMax];
  bool out[kMax];
  int n = 0;
  const ssd_tensor *apart[2] = {nullptr, nullptr}; // two that share a span, but no element
  void add(const ssd_tensor *q, const char *nm, bool is_out) {
    if (!q) return;
    t[n] = q;
    name[n] = nm;
    out[n] = is_out;
    ++n;
  }
  // No output overlaps another argument; `same_out` may be exactly `same_in`.
  int overlaps(const ssd_tensor *same_out, const ssd_tensor *same_in) const {
    for (int i = 0; i < n; ++i) {
      if (!out[i]) continue;
      const Range ri = span_of(t[i]);
      for (int j = 0; j < n; ++j) {
        if (j == i || (out[j] && j < i)) continue;
        if (t[i] == same_out && t[j] == same_in && t[i]->data == t[j]->data) continue;
        if (t[i] == apart[0] && t[j] == apart[1]) continue;
        if (overlap(ri, span_of(t[j]))) return fail(SSD_ERR_ALIAS, "%s overlaps %s", name[i], name[j]);
      }
    }
    return SSD_OK;
  }
  int workspace(const void *ws, int64_t have, int64_t need) const {
    if (need == 0) return SSD_OK;
    if (!ws) return fail(SSD_ERR_NULL, "workspace: NULL, %lld bytes needed", (long long)need);
    if (have < need)
      return fail(SSD_ERR_NOMEM, "workspace: %lld bytes, %lld needed", (long long)have, (long long)need);
    if ((uintptr_t)ws % 16 != 0) return fail(SSD_ERR_LAYOUT, "workspace: not 16-byte aligned");
    Range w;
    w.lo = (uintptr_t)ws;
    w.hi = w.lo + (uintptr_t)need;
    for (int i = 0; i < n; ++i)
      if (overlap(w, span_of(t[i]))) return fail(SSD_ERR_ALIAS, "workspace overlaps %s", name[i]);
    return SSD_OK;
  }
  int addressable(const void *ws) const {
    SSD_CHECK(check_addressable(t, name, n));
    if (!ws) return SSD_OK;
    ssd_tensor w{};
    w.data = const_cast<void *>(ws);
    const ssd_tensor *wt[1] = {&w};
    const char *wn[1] = {"workspace"};
    return check_addressable(wt, wn, 1);
  }
};

inline const float *fptr(const ssd_tensor *t) { return t ? (const float *)t->data : nullptr; }
inline float *fptr_out(ssd_tensor *t) { return t ? (float *)t->data : nullptr; }

// Rows in pieces of `bytes`: the width, the strides that are used and the
// pointers are multiples of them.
inline bool rows_of(const ssd_tensor *t, int bytes) {
  const int V = bytes / elem_size(t->dtype), n = t->ndim;
  if ((uintptr_t)t->data % (uintptr_t)bytes != 0 || t->shape[n - 1] % V != 0) return false;
  for (int i = 0; i < n - 1; ++i)
    if (t->shape[i] != 1 && t->strides[i] % V != 0) return false;
  return true;
}

// Element groups of four at 8 (bf16) or 16 bytes (f32).
inline bool rows4(const ssd_tensor *t) {
  if (!t) return true;
  if ((uintptr_t)t->data % (uintptr_t)(4 * elem_size(t->dtype)) != 0) return false;
  for (int i = 0; i < t->ndim - 1; ++i)
    if (t->shape[i] != 1 && t->strides[i] % 4 != 0) return false;
  return true;
}

} // namespace ssd
