// Pages of keys and values: where a token lies, and the e4m3 format's conversions.
//
// A page holds page_tokens tokens of one layer:
//   keys   [H][page_tokens][d_k], values [H][page_tokens][d_v], in bf16 or e4m3,
//   e4m3:  scales [2][H] fp32 (of each head's keys, then values), padded to 16 bytes.
// A head's keys on a page are one dense block, which is what attention streams.
#pragma once

#include "kda_device.h"
#include "kda_launch.h"

namespace kda {

constexpr int kLeastScale = -100;  // exponent of the smallest e4m3 scale

// The page that holds the idx-th block of tokens of sequence b, or -1.
__device__ __forceinline__ int kv_page(const KvCache& c, int b, long long idx) {
  const int row = c.rows ? c.rows[b] : b;
  if (row < 0 || row >= c.n_rows || idx < 0 || idx >= c.width) return -1;
  const int page = c.table[(size_t)row * c.width + idx];
  return page >= 0 && page < c.n_pages ? page : -1;
}

__device__ __forceinline__ size_t kv_elem(const KvCache& c) { return c.e4m3 ? 1 : 2; }
// Offsets within a page: head h's keys, values, and the scales.
__device__ __forceinline__ size_t kv_keys(const KvCache& c, int h) {
  return (size_t)h * c.page_tokens * c.dk * kv_elem(c);
}
__device__ __forceinline__ size_t kv_values(const KvCache& c, int h) {
  return ((size_t)c.H * c.dk + (size_t)h * c.dv) * c.page_tokens * kv_elem(c);
}
__device__ __forceinline__ size_t kv_scales(const KvCache& c) {
  return (size_t)c.H * (c.dk + c.dv) * c.page_tokens * kv_elem(c);
}

// The smallest power of two >= 2^kLeastScale that brings amax (finite, >= 0) to 448 or below.
__device__ __forceinline__ float e4m3_scale(float amax) {
  // amax = m 2^x with 1 <= m < 2, 448 = 1.75 2^8: x - 8, one more where m > 1.75.  (Subnormal amax: x = -127, below the least.)
  const uint32_t u = __builtin_bit_cast(uint32_t, amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  return __builtin_bit_cast(float, (uint32_t)(max(e, kLeastScale) + 127) << 23);
}

// Four values to e4m3, nearest even.  Values are within 448 or not finite; those become NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  auto fix = [](float x) { return __builtin_fabsf(x) <= 448.0f ? x : __builtin_nanf(""); };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(fix(a), fix(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(fix(c), fix(d), w, true);
  return (uint32_t)w;
}
__device__ __forceinline__ f32x4 from_e4m3x4(uint32_t w) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return f32x4{lo[0], lo[1], hi[0], hi[1]};
}

// The last index b in [0, n) with at(b) <= x, for at that does not fall; 0 where there is none.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, long long x, F at) {
  int lo = 0, hi = n;  // at(lo) <= x (or lo = 0) and at(hi) > x (or hi = n)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (at(mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same, by all 64 lanes of a wave together: 64 places at a time, so that up to 64 take one load.
template <typename F>
__device__ __forceinline__ int last_at_most_wave(int n, long long x, F at) {
  int lo = 0, hi = n;
  const int lane = threadIdx.x % 64;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64;
    const long long i = lo + (long long)lane * step;
    const int below = __popcll(__ballot(lane == 0 || (i < hi && at((int)i) <= x)));
    lo = min(lo + (below - 1) * step, hi - 1);  // (in range whatever the list holds)
    hi = min(lo + step, hi);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

__device__ __forceinline__ int clamp_to(int x, int hi) { return min(max(x, 0), hi); }

}  // namespace kda
