// What the host sides of the operators beside kda_prefill share: the error text, bounds on
// sizes, and the overlap of address ranges.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kda.h"
#include "kda_ops_internal.h"

namespace {

__attribute__((format(printf, 2, 3))) inline kda_status fail(kda_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return kda::set_error(s, buf);
}

inline kda_status clear() { return kda::set_error(KDA_OK, ""); }

constexpr int64_t kBig = int64_t(1) << 40;  // bound on sizes, strides and pitches
constexpr int64_t kMaxThreads = 0xffffffffLL;  // of one launch: HIP refuses more

inline bool known_dtype(int32_t d) { return d == KDA_BF16 || d == KDA_FP32; }
inline int64_t elem_size(int32_t d) { return d == KDA_BF16 ? 2 : 4; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

typedef __int128 Wide;

struct Range {
  Wide lo, hi;
  const char* name;
};
inline Range range_of(const void* p, Wide bytes, const char* name) {
  const Wide lo = static_cast<Wide>(reinterpret_cast<uintptr_t>(p));
  return Range{lo, p ? lo + bytes : lo, name};
}
inline bool overlap(const Range& a, const Range& b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline kda_status done(hipError_t e) {
  return e == hipSuccess ? KDA_OK : fail(KDA_ERR_HIP, "%s", hipGetErrorString(e));
}

}  // namespace
