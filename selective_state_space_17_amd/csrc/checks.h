// Host-side argument checks shared by the C-ABI front ends.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <limits>

namespace mssm {

// keeps the HIP error's text for mssm_last_error_detail (per thread)
void set_err(hipError_t e);

namespace checks {

// *r = a * b; false on a negative factor or overflow
inline bool mul_ok(int64_t a, int64_t b, int64_t* r) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > std::numeric_limits<int64_t>::max() / a) return false;
  *r = a * b;
  return true;
}

inline bool aligned(const void* p, size_t a) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
  uintptr_t lo, hi;
};
inline Range rng(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(const void* p, int64_t pb, const void* q, int64_t qb) {
  if (p == nullptr || q == nullptr || pb <= 0 || qb <= 0) return false;
  const Range a = rng(p, pb), b = rng(q, qb);
  return a.lo < b.hi && b.lo < a.hi;
}

}  // namespace checks
}  // namespace mssm
