// ssd_check.h -- argument checks and error text shared by the files that
// implement the C ABI.  Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd.h"

#define SSD_CHECK(expr)                                                                   \
  do {                                                                                    \
    int _s = (expr);                                                                      \
    if (_s != SSD_OK) return _s;                                                          \
  } while (0)

namespace ssd {

// The calling thread's error text (ssd_last_error): fail() sets it and
// returns the status.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char *what);
void clear_error();

inline int elem_size(int dtype) {
  return dtype == SSD_BF16 ? 2 : dtype == SSD_U8 ? 1 : dtype == SSD_I64 ? 8 : 4;
}

inline int64_t numel(const ssd_tensor *t) {
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
  return n;
}

struct Range {
  uintptr_t lo = 0, hi = 0; // [lo, hi)
  bool empty() const { return hi <= lo; }
};

inline bool overlap(const Range &a, const Range &b) {
  return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi;
}

// Every tensor (null entries are skipped) must be memory the current device
// can address.
int check_addressable(const ssd_tensor *const *ts, const char *const *names, int n);

} // namespace ssd
