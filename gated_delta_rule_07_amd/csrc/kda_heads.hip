// Norms of queries and keys for each head, with the rotation by position, for gfx950.
//
//   y = w . x / sqrt(sum_i x_i^2 + eps)      (or the mean of the squares)
//   (a, b) -> (a cos f - b sin f, b cos f + a sin f),   f = pos * inv_freq[i]
//
// Every value is read once and written once, so the pass is bound by those bytes.
// A group of G lanes (a power of two) holds one head of one token, 8 values a
// lane: 16 bytes of bf16, one wave instruction covering 1 KB of dense rows.  The
// sum of squares is a butterfly over the group's lanes; the partner of a value in
// the other half of the rotated part sits in a lane a fixed distance away, one
// shuffle per value.  A workgroup takes all heads of a few tokens, so that the
// cosines and sines, which the heads of a token share, are formed once: in LDS,
// from an angle reduced in fp64 to a fraction of a turn.  That fraction is rounded to fp32
// before its sine, and the norm's reciprocal before it multiplies the head: at most 2 pi 2^-25
// of |a| + |b| and half a step of fp32, below the rounding of any bf16 output; fp32 outputs end
// 7.0e-8 from the formula where dividing and 64-bit sines end 5.9e-8 from it.
//
// Measured: 65,536 tokens of 32 + 32 heads of 128 in bf16 (2.15 GB) 370 us, 5.8 TB/s;
// 4,099 tokens of 32 + 4 heads of 64 in fp32 with half of each head rotated (76 MB)
// 17.0 us, 4.5 TB/s; one token of 8 + 8 heads 2.0 us.  Twice as many heads for each group
// took 385 us on the first, four heads loaded ahead of their sums 403 us (80 registers,
// half the waves), non-temporal loads and stores 353 us: not used, since what reads the
// outputs next finds those of all but the longest calls in the caches.
#include <algorithm>

#include "kda_device.h"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRot = 256;
constexpr int kMaxTokens = 16;  // tokens of one workgroup

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 load8(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x8 load8(const __bf16* p) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
  f32x8 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r[2 * e] = __builtin_bit_cast(float, w[e] << 16);
    r[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ void store8(float* p, f32x8 x) {
  *reinterpret_cast<f32x4*>(p) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
  *reinterpret_cast<f32x4*>(p + 4) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
}
__device__ __forceinline__ void store8(__bf16* p, f32x8 x) {
  bf16x8 h;
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = (__bf16)x[e];  // round to nearest even
  *reinterpret_cast<bf16x8*>(p) = h;
}

template <typename IO, typename OUT, int G>
__global__ __launch_bounds__(kThreads) void kda_heads_kernel(HeadsParams p, int tokens) {
  extern __shared__ float2 turn[];  // [tokens][rot / 2]: cosine and sine
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * tokens, nt = min(tokens, p.n - t0);
  const int half = p.rot / 2;
  if (p.rot) {
    for (int e = tid; e < nt * half; e += kThreads) {
      const int t = e / half, i = e % half;
      const double turns = (double)p.positions[t0 + t] * (double)p.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
      float s, c;
      sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
      turn[e] = float2{c, s};
    }
    __syncthreads();
  }
  const int heads = p.Hq + p.Hk;
  const int gl = tid % G, i0 = 8 * gl;
  const bool live = i0 < p.d;
  for (int r = tid / G; r < nt * heads; r += kThreads / G) {
    const int t = r / heads, hh = r % heads;
    const bool isq = hh < p.Hq;
    const int h = isq ? hh : hh - p.Hq;
    const size_t tok = (size_t)(t0 + t);
    const IO* x = isq ? static_cast<const IO*>(p.q) + tok * p.q_stride : static_cast<const IO*>(p.k) + tok * p.k_stride;
    f32x8 y = (f32x8)0.0f;
    if (live) y = load8(x + (size_t)h * p.d + i0);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += y[e] * y[e];
#pragma unroll
    for (int m = 1; m < G; m *= 2) ss += __shfl_xor(ss, m);
    if (p.rms) ss /= (float)p.d;
    const float inv = 1.0f / sqrtf(ss + p.eps);
    y *= inv;
    const float* w = isq ? p.q_weight : p.k_weight;
    if (w && live) y *= load8(w + i0);
    if (p.rot) {
      const float2* ft = turn + t * half;
      if (p.adjacent) {
        if (i0 < p.rot) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 f = ft[(i0 + e) / 2];
            const float a = y[e], b = y[e + 1];
            y[e] = a * f.x - b * f.y;
            y[e + 1] = b * f.x + a * f.y;
          }
        }
      } else {
        const int m = half / 8;  // lanes of each half
        const int partner = gl < m ? gl + m : gl < 2 * m ? gl - m : gl;
        f32x8 other;
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] = __shfl(y[e], partner, G);
        if (gl < 2 * m) {
          const float sign = gl < m ? -1.0f : 1.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = ft[(gl < m ? i0 : i0 - half) + e];
            y[e] = y[e] * f.x + sign * other[e] * f.y;
          }
        }
      }
    }
    if (isq) y *= p.q_scale;
    if (live) {
      OUT* o = isq ? static_cast<OUT*>(p.q_out) + tok * p.q_out_stride : static_cast<OUT*>(p.k_out) + tok * p.k_out_stride;
      store8(o + (size_t)h * p.d + i0, y);
    }
  }
}

template <typename IO, typename OUT, int G>
hipError_t launch_one(const HeadsParams& p, hipStream_t s) {
  // as many tokens a workgroup as give each lane about four heads, fewer where
  // the launch would not fill the compute units
  const int heads = p.Hq + p.Hk;
  int tokens = std::max(1, std::min(kMaxTokens, 4 * (kThreads / G) / heads));
  while (tokens > 1 && (long long)p.n < 1024LL * tokens) tokens /= 2;
  const size_t lds = (size_t)tokens * (p.rot / 2) * sizeof(float2);
  // (a launch has fewer than 2^32 threads: longer calls in slices)
  const long long slice = (1LL << 23) * tokens;
  for (long long t = 0; t < p.n; t += slice) {
    HeadsParams c = p;
    c.n = (int)std::min(slice, (long long)p.n - t);
    c.q = static_cast<const IO*>(p.q) + t * p.q_stride;
    c.q_out = static_cast<OUT*>(p.q_out) + t * p.q_out_stride;
    if (p.Hk) {
      c.k = static_cast<const IO*>(p.k) + t * p.k_stride;
      c.k_out = static_cast<OUT*>(p.k_out) + t * p.k_out_stride;
    }
    if (p.rot) c.positions = p.positions + t;
    hipLaunchKernelGGL((kda_heads_kernel<IO, OUT, G>), dim3((unsigned)((c.n + tokens - 1) / tokens)), dim3(kThreads), lds,
                       s, c, tokens);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename IO, typename OUT>
hipError_t pick_group(const HeadsParams& p, hipStream_t s) {
  if (p.d <= 8) return launch_one<IO, OUT, 1>(p, s);
  if (p.d <= 16) return launch_one<IO, OUT, 2>(p, s);
  if (p.d <= 32) return launch_one<IO, OUT, 4>(p, s);
  if (p.d <= 64) return launch_one<IO, OUT, 8>(p, s);
  if (p.d <= 128) return launch_one<IO, OUT, 16>(p, s);
  return launch_one<IO, OUT, 32>(p, s);
}

}  // namespace

hipError_t launch_heads(const HeadsParams& p, int io_dtype, int out_dtype, hipStream_t s) {
  if (p.d < 8 || p.d > 256 || p.d % 8 || p.rot < 0 || p.rot > p.d || p.rot > kMaxRot || p.rot % 16 || p.n < 1)
    return hipErrorInvalidValue;
  if (io_dtype == 1) return out_dtype == 1 ? pick_group<__bf16, __bf16>(p, s) : pick_group<__bf16, float>(p, s);
  return out_dtype == 1 ? pick_group<float, __bf16>(p, s) : pick_group<float, float>(p, s);
}

}  // namespace kda
