// Argument checks shared by the files that implement the C ABI (host code only).
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "../../include/kda.h"

#include <hip/hip_runtime_api.h>

namespace kda {

// Records the hipError_t that kda_last_hip_error returns on this thread.
void set_last_hip_error(int e);

namespace check {

inline bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// A C caller may pass any int where the header says kda_dtype or kda_status;
// reading such a value as the C++ enum type is undefined, so it is read as the
// integer it is.
// (Taken by reference: passing it by value would already read it as the enum.)
template <typename E>
inline int raw_enum(const E& e) {
  static_assert(sizeof(E) == sizeof(int), "enum size");
  int v;
  memcpy(&v, &e, sizeof v);
  return v;
}
inline bool dtype_ok(int d) { return d == KDA_F32 || d == KDA_BF16; }
inline int io_of(int d) { return d == KDA_BF16 ? 1 : 0; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Span span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + bytes};
}
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

template <size_t N>
inline bool any_overlap(Span out, const Span (&ins)[N]) {
  for (const Span& s : ins)
    if (overlap(out, s)) return true;
  return false;
}

inline Span opt_span(const void* p, size_t bytes) { return p ? span(p, bytes) : Span{0, 0}; }

// n rows of `len` bytes, `stride` bytes apart.
struct Rows {
  uintptr_t at;
  unsigned long long n, len, stride;
  Span all() const { return n ? Span{at, at + (n - 1) * stride + len} : Span{0, 0}; }
};

// Whether two sets of rows share a byte.  Rows of one stride that lie side by
// side (slices of one wider row) do not; for different strides, sets whose
// ranges meet are taken to.
inline bool rows_overlap(const Rows& a, const Rows& b) {
  if (!overlap(a.all(), b.all())) return false;
  if (a.n <= 1 && b.n <= 1) return true;
  const unsigned long long st = a.n > 1 ? a.stride : b.stride;
  if ((a.n > 1 && b.n > 1 && a.stride != b.stride) || a.len > st || b.len > st) return true;
  // offset of b's rows in a's raster
  const unsigned long long d = b.at >= a.at ? (b.at - a.at) % st : (st - (a.at - b.at) % st) % st;
  return d < a.len || st - d < b.len;
}

// Element counts fit in size_t and every row index used by the kernels fits in
// an int64; the kernels index tokens with 64-bit arithmetic.
inline bool sizes_ok(long long B, long long T, long long H, long long dk, long long dv) {
  const long long lim = (1LL << 40);
  if (B * H > (1LL << 26)) return false;
  if (B * T * H > lim / 128) return false;
  (void)dk;
  (void)dv;
  return true;
}

inline kda_status launched(hipError_t e) {
  if (e == hipSuccess) return KDA_OK;
  set_last_hip_error((int)e);
  return KDA_ERR_HIP;
}

}  // namespace check
}  // namespace kda
