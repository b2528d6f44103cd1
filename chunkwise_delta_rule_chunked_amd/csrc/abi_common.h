// Host-side helpers shared by the C ABI's translation units: pointer and shape checks, the
// environment switches, error mapping.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "../../include/delta.h"

namespace delta {
namespace abi {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned(const void* p, unsigned a) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Range range(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

inline size_t esize(int dtype) { return dtype == DELTA_BF16 ? 2 : 4; }

// Shape checks common to all entry points.
inline int check_shape(const delta_shape* s) {
  if (!s) return DELTA_ERR_NULL_ARG;
  if (s->B < 0 || s->L < 0 || s->H < 0 || s->n_h < 1) return DELTA_ERR_BAD_SHAPE;
  if (s->dtype != DELTA_F32 && s->dtype != DELTA_BF16) return DELTA_ERR_UNSUPPORTED_DIM;
  if (s->dk != 16 && s->dk != 32 && s->dk != 64 && s->dk != 128) return DELTA_ERR_UNSUPPORTED_DIM;
  if (s->dv < 16 || s->dv > 256 || s->dv % 16 != 0) return DELTA_ERR_UNSUPPORTED_DIM;
  // grid sizes and 64-bit element counts stay well inside what the kernels index
  const long long Lx = (long long)s->L * s->n_h;
  if (Lx > (1LL << 31) || (long long)s->B * s->H > (1LL << 24)) return DELTA_ERR_BAD_SHAPE;
  return DELTA_OK;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? DELTA_OK : DELTA_ERR_HIP; }

// Opt-in switches, read from the environment at every call:
//   DELTA_VALIDATE=1    check beta and the log gates before enqueuing work (validate.hip); a
//                       value outside the contract returns DELTA_ERR_BAD_VALUE with nothing
//                       written.  The check waits for the stream, so the call is synchronous.
//   DELTA_FAULT=launch  every entry point that has work to enqueue fails as if its first launch
//                       had failed: DELTA_ERR_HIP, nothing enqueued (for testing error paths).
inline bool env_is(const char* name, const char* value) {
  const char* e = getenv(name);
  return e && strcmp(e, value) == 0;
}
inline bool validate_on() { return env_is("DELTA_VALIDATE", "1"); }
inline int launch_guard() { return env_is("DELTA_FAULT", "launch") ? DELTA_ERR_HIP : DELTA_OK; }

// True if an output overlaps an input or another output.
template <int NI, int NO>
bool any_overlap(const Range (&in)[NI], const Range (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return true;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

// DELTA_VALIDATE: log gates finite or -inf, read back in pieces (no allocation).
inline int validate_gates(const float* g, size_t n, hipStream_t st) {
  constexpr size_t PIECE = 8192;
  float buf[PIECE];
  for (size_t i = 0; i < n; i += PIECE) {
    const size_t m = std::min(PIECE, n - i);
    if (hipMemcpyAsync(buf, g + i, m * 4, hipMemcpyDeviceToHost, st) != hipSuccess) return DELTA_ERR_HIP;
    if (hipStreamSynchronize(st) != hipSuccess) return DELTA_ERR_HIP;
    for (size_t k = 0; k < m; ++k)
      if (buf[k] != buf[k] || buf[k] == __builtin_inff()) return DELTA_ERR_BAD_VALUE;
  }
  return DELTA_OK;
}

}  // namespace abi
}  // namespace delta
