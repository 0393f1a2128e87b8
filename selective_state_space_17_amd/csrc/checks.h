// Host-side argument checks shared by the C-ABI front ends.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <limits>

#include "../../include/mssm.h"

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

inline bool io_ok(int32_t t) { return t == MSSM_F32 || t == MSSM_BF16; }
inline int64_t size_of(int32_t t) { return t == MSSM_BF16 ? 2 : 4; }

inline int done(hipError_t e) {
  if (e == hipSuccess) return MSSM_OK;
  set_err(e);
  return MSSM_ERR_HIP;
}

struct Buf {
  const void* p;
  int64_t bytes;
};
// no output may overlap an input or another output
template <int NI, int NO> bool disjoint(const Buf (&in)[NI], const Buf (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (overlap(out[o].p, out[o].bytes, in[i].p, in[i].bytes)) return false;
    for (int k = 0; k < o; ++k)
      if (overlap(out[o].p, out[o].bytes, out[k].p, out[k].bytes)) return false;
  }
  return true;
}

inline int workspace_status(const void* ws, size_t have, size_t need) {
  if (need == 0) return MSSM_OK;
  if (ws == nullptr || have < need) return MSSM_ERR_WORKSPACE;
  return aligned(ws, 256) ? MSSM_OK : MSSM_ERR_MISALIGNED;
}

}  // namespace checks
}  // namespace mssm
