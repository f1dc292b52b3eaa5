// Keys and values onto the pages of a cache, turned by position, and back, for gfx950.
//
//   (a, b) -> (a cos f - b sin f, b cos f + a sin f),  f = pos * inv_freq[i]
//   bf16 pages: the value rounded once.  e4m3 pages: codes of y / s, where a head's scale s on a
//   page is the smallest power of two that brings its largest finite value to 448 or below; it only
//   grows while a page fills, and the codes that are there are then rounded to the new one (exactly,
//   but for those that fall below the format's normal range).
//
// Append: a workgroup takes one page of one sequence, so that the tokens of a page share the scale's
// maximum and the cosines and sines (in LDS) serve all heads; a wave takes one head's keys or values.
// Lanes hold 8 values of a row.  Workgroups behind the pages turn the queries.
#include <algorithm>

#include "kda_kv_device.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

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

// Cosine and sine of pos * freq: the angle's reduction to a fraction of a turn in fp64.
__device__ __forceinline__ float2 turn_of(long long pos, float freq) {
  const double turns = (double)pos * (double)freq * 0.15915494309189535;  // 1 / (2 pi)
  float s, c;
  sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
  return float2{c, s};
}

// y, 8 values from i0 = 8 gl on of a head that `lanes` lanes hold, with the first rot of them turned by ft.
__device__ __forceinline__ f32x8 rotate8(f32x8 y, const float2* ft, int rot, int adjacent, int gl, int lanes) {
  if (!rot) return y;
  const int i0 = 8 * gl, half = rot / 2;
  if (adjacent) {
    if (i0 < rot) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 f = ft[(i0 + e) / 2];
        const float a = y[e], b = y[e + 1];
        y[e] = a * f.x - b * f.y;
        y[e + 1] = b * f.x + a * f.y;
      }
    }
    return y;
  }
  const int m = half / 8;  // lanes of each half
  const int partner = gl < m ? gl + m : gl < 2 * m ? gl - m : gl;
  f32x8 other;
#pragma unroll
  for (int e = 0; e < 8; ++e) other[e] = __shfl(y[e], partner, lanes);
  if (gl < 2 * m) {
    const float sign = gl < m ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = ft[(gl < m ? i0 : i0 - half) + e];
      y[e] = y[e] * f.x + sign * other[e] * f.y;
    }
  }
  return y;
}

// Tokens [t0, t0 + n) of the call are sequence b's, behind the `before` it has.
struct Span {
  int t0, n;
  long long before;
};
__device__ __forceinline__ Span span_of(const AppendParams& p, int b) {
  Span s;
  s.t0 = p.cu ? clamp_to(p.cu[b], p.total) : b;
  s.n = p.cu ? clamp_to(p.cu[b + 1], p.total) - s.t0 : 1;
  s.before = max(p.lens[b], 0);
  return s;
}
// Pages that n > 0 tokens behind `before` others touch.
__device__ __forceinline__ long long touched(const Span& s, int pt) {
  return s.n > 0 ? (s.before + s.n - 1) / pt - s.before / pt + 1 : 0;
}

// Whether another page of the call than the j-th of sequence b is `page` too (seen by any thread of the workgroup).
__device__ bool shared_page(const AppendParams& p, int page, int b, long long j, int tid) {
  const int lane = tid % 64, wave = tid / 64;
  bool hit = false;
  for (int c0 = 64 * wave; c0 < p.N; c0 += 64 * kWaves) {
    // a lane looks after one sequence; where one has many pages, the wave takes sequence after sequence
    const int c = c0 + lane;
    long long first = 0, n = 0;
    if (c < p.N) {
      const Span s = span_of(p, c);
      first = s.before / p.c.page_tokens;
      n = min(touched(s, p.c.page_tokens), max(0LL, p.c.width - first));
    }
    if (!__any(n > 8)) {
      for (long long i = 0; i < n; ++i) hit |= !(c == b && i == j) && kv_page(p.c, c, first + i) == page;
    } else {
      for (int l = 0; l < 64 && c0 + l < p.N; ++l) {
        const long long f = __shfl(first, l), m = __shfl(n, l);
        for (long long i = lane; i < m; i += 64) hit |= !(c0 + l == b && i == j) && kv_page(p.c, c0 + l, f + i) == page;
      }
    }
  }
  return hit;
}

template <typename IO>
__device__ void append_queries(const AppendParams& p, int block, int tokens, float2* turn, int tid) {
  const int t0 = block * tokens, nt = min(tokens, p.total - t0), half = p.rot / 2;
  for (int e = tid; e < nt * half; e += kThreads) {
    const int t = t0 + e / half;
    long long pos = 0;
    if (p.positions) {
      pos = p.positions[t];
    } else {
      const int b = p.cu ? last_at_most(p.N, t, [&](int i) { return (long long)p.cu[i]; }) : t;
      const Span s = span_of(p, b);
      pos = s.before + t - s.t0;
    }
    turn[e] = turn_of(pos, p.inv_freq[e % half]);
  }
  __syncthreads();
  const int lanes = p.c.dk / 8, gl = tid % lanes;
  // tokens behind the last sequence's are left as they were
  const int end = p.cu ? clamp_to(p.cu[p.N], p.total) : p.total;
  for (int r = tid / lanes; r < nt * p.Hq; r += kThreads / lanes) {
    const int t = r / p.Hq, h = r % p.Hq;
    const size_t tok = (size_t)(t0 + t);
    if ((int)tok >= end || (p.cu && (int)tok < p.cu[0])) continue;
    const f32x8 x = load8(static_cast<const IO*>(p.q) + tok * p.q_stride + (size_t)h * p.c.dk + 8 * gl);
    store8(static_cast<IO*>(p.q_out) + tok * p.q_out_stride + (size_t)h * p.c.dk + 8 * gl,
           rotate8(x, turn + t * half, p.rot, p.adjacent, gl, lanes));
  }
}

template <typename IO, bool E4>
__global__ __launch_bounds__(kThreads) void kda_kv_append_kernel(AppendParams p, int page_blocks, int q_tokens) {
  extern __shared__ float2 turn[];  // [tokens][rot / 2]: cosine and sine
  __shared__ int flag[kWaves];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  if ((int)blockIdx.x >= page_blocks) {
    if (blockIdx.y == 0) append_queries<IO>(p, blockIdx.x - page_blocks, q_tokens, turn, tid);
    return;
  }
  const KvCache& c = p.c;
  const int pt = c.page_tokens;
  // sequence b has room for cu[b + 1] / pt - cu[b] / pt + 2 workgroups, as many as its tokens touch pages at most
  int b = blockIdx.x;
  long long j = 0;
  if (p.cu) {
    auto first = [&](int i) { return (long long)(clamp_to(p.cu[i], p.total) / pt) + 2LL * i; };
    b = last_at_most(p.N, blockIdx.x, first);
    j = blockIdx.x - first(b);
  }
  const Span s = span_of(p, b);
  if (j < 0 || j >= touched(s, pt)) return;  // (the same for the whole workgroup)
  const long long at = s.before / pt + j;  // the page's place in the row
  const int slot0 = j == 0 ? (int)(s.before % pt) : 0;
  const int first = j == 0 ? 0 : (int)(at * pt - s.before);  // its first token among the sequence's new ones
  const int nt = min(pt - slot0, s.n - first);
  const int t0 = s.t0 + first, half = p.rot / 2;
  const int page = kv_page(c, b, at);
  const bool any = __any(page >= 0 && shared_page(p, page, b, j, tid));
  if (lane == 0) flag[wave] = any;
  for (int e = tid; e < nt * half; e += kThreads) {
    const int t = e / half;
    turn[e] = turn_of(p.positions ? (long long)p.positions[t0 + t] : s.before + first + t, p.inv_freq[e % half]);
  }
  __syncthreads();
  bool store = page >= 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) store = store && !flag[w];

  for (int pair = blockIdx.y * kWaves + wave; pair < 2 * c.H; pair += gridDim.y * kWaves) {
    const bool is_v = pair >= c.H;
    const int h = is_v ? pair - c.H : pair, d = is_v ? c.dv : c.dk;
    const int lanes = d / 8, gl = lane % lanes, rows = 64 / lanes;
    const long long stride = is_v ? p.v_stride : p.k_stride;
    const IO* x = static_cast<const IO*>(is_v ? p.v : p.k) + (size_t)t0 * stride + (size_t)h * d + 8 * gl;
    char* block = c.pool + (size_t)max(page, 0) * c.page_bytes + (is_v ? kv_values(c, h) : kv_keys(c, h));
    auto row = [&](int t) {
      f32x8 y = (f32x8)0.0f;
      if (t < nt) y = load8(x + (size_t)t * stride);
      return is_v ? y : rotate8(y, turn + min(t, nt - 1) * half, p.rot, p.adjacent, gl, lanes);
    };
    float inv = 1.0f;
    if (E4 && store) {
      float amax = 0.0f;
      for (int t = lane / lanes; t < nt + lane / lanes; t += rows) {  // (all lanes take part in every turn: rotations exchange values)
        const f32x8 y = row(t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = __builtin_fabsf(y[e]);
          amax = a < __builtin_inff() ? fmaxf(amax, a) : amax;
        }
      }
#pragma unroll
      for (int m = 1; m < 64; m *= 2) amax = fmaxf(amax, __shfl_xor(amax, m));
      float* scale = reinterpret_cast<float*>(c.pool + (size_t)page * c.page_bytes + kv_scales(c)) + (is_v ? c.H : 0) + h;
      float now = e4m3_scale(amax);
      if (slot0 > 0) {
        const float was = *scale;
        now = fmaxf(was, now);
        if (now != was) {  // the codes that are there, rounded to the new scale
          const float ratio = was / now;
          for (int i = lane; i < slot0 * d / 8; i += 64) {
            u32x2* w = reinterpret_cast<u32x2*>(block) + i;
            const f32x4 lo = from_e4m3x4((*w)[0]) * ratio, hi = from_e4m3x4((*w)[1]) * ratio;
            *w = u32x2{to_e4m3x4(lo[0], lo[1], lo[2], lo[3]), to_e4m3x4(hi[0], hi[1], hi[2], hi[3])};
          }
        }
      }
      if (lane == 0) *scale = now;
      inv = 1.0f / now;  // (a power of two: exact)
    }
    for (int t = lane / lanes; t < nt + lane / lanes; t += rows) {
      const f32x8 y = row(t);
      if (t >= nt) continue;
      if (store) {
        if constexpr (E4) {
          const f32x8 z = y * inv;
          *reinterpret_cast<u32x2*>(block + ((size_t)(slot0 + t) * d + 8 * gl)) =
              u32x2{to_e4m3x4(z[0], z[1], z[2], z[3]), to_e4m3x4(z[4], z[5], z[6], z[7])};
        } else {
          store8(reinterpret_cast<__bf16*>(block) + (size_t)(slot0 + t) * d + 8 * gl, y);
        }
      }
      if (!is_v && p.k_out)
        store8(static_cast<IO*>(p.k_out) + (size_t)(t0 + t) * p.k_out_stride + (size_t)h * d + 8 * gl, y);
    }
  }
}

template <typename IO, bool E4>
hipError_t append_one(const AppendParams& p, hipStream_t s) {
  const long long pages = p.cu ? (long long)p.total / p.c.page_tokens + 2LL * p.N : p.N;
  const int q_tokens = p.q ? std::max(1, std::min(16, 4 * kThreads / (p.Hq * (p.c.dk / 8)))) : 1;
  const long long q_blocks = p.q ? (p.total + q_tokens - 1) / q_tokens : 0;
  // a wave a head where the pages alone would not fill the compute units
  const int most = (2 * p.c.H + kWaves - 1) / kWaves;
  const int split = (int)std::max(1LL, std::min((long long)most, 2048 / std::max(pages, 1LL)));
  const size_t lds = (size_t)std::max(p.cu ? p.c.page_tokens : 1, q_tokens) * (p.rot / 2) * sizeof(float2);
  if (lds > 65000) {  // more than the default has to be asked for
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&kda_kv_append_kernel<IO, E4>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((kda_kv_append_kernel<IO, E4>), dim3((unsigned)(pages + q_blocks), split), dim3(kThreads), lds, s, p,
                     (int)pages, q_tokens);
  return hipGetLastError();
}

// ---- back ---------------------------------------------------------------------------------

constexpr int kReadTokens = 32;

// A lane moves V values (16 bytes of the page) of a token's head.
template <typename OUT, bool E4>
__global__ __launch_bounds__(kThreads) void kda_kv_read_kernel(ReadParams p) {
  __shared__ int page[kReadTokens], slot[kReadTokens];
  constexpr int V = E4 ? 16 : 8;
  const KvCache& c = p.c;
  const int tid = threadIdx.x, t0 = blockIdx.x * kReadTokens, nt = min(kReadTokens, p.total - t0);
  if (tid < nt) {
    const int t = t0 + tid;
    const int b = last_at_most(p.N, t, [&](int i) { return (long long)p.cu[i]; });
    const int begin = clamp_to(p.cu[b], p.total), end = clamp_to(p.cu[b + 1], p.total);
    const long long pos = (p.starts ? max(p.starts[b], 0) : 0) + (long long)(t - begin);
    page[tid] = t >= begin && t < end ? kv_page(c, b, pos / c.page_tokens) : -1;
    slot[tid] = (int)(pos % c.page_tokens);
  }
  __syncthreads();
  const int nk = c.H * c.dk / V, nv = c.H * c.dv / V;  // lanes of a token's keys, values
  for (int i = tid; i < nt * (nk + nv); i += kThreads) {
    const int t = i / (nk + nv), r = i % (nk + nv);
    if (page[t] < 0) continue;
    const bool is_v = r >= nk;
    const int d = is_v ? c.dv : c.dk, j = (is_v ? r - nk : r) * V, h = j / d;
    const char* base = c.pool + (size_t)page[t] * c.page_bytes;
    const char* from = base + (is_v ? kv_values(c, h) : kv_keys(c, h)) + ((size_t)slot[t] * d + j % d) * (E4 ? 1 : 2);
    OUT* to = static_cast<OUT*>(is_v ? p.v_out : p.k_out) + (size_t)(t0 + t) * c.H * d + j;
    if constexpr (E4) {
      const float s = reinterpret_cast<const float*>(base + kv_scales(c))[(is_v ? c.H : 0) + h];
      const u32x4 w = *reinterpret_cast<const u32x4*>(from);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const f32x4 lo = from_e4m3x4(w[e]) * s, hi = from_e4m3x4(w[e + 1]) * s;
        store8(to + 4 * e, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    } else {
      store8(to, load8(reinterpret_cast<const __bf16*>(from)));
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendParams& p, int io_dtype, hipStream_t s) {
  if (p.total < 1 || p.N < 1 || p.c.dk % 64 || p.c.dv % 64 || p.c.dk > 128 || p.c.dv > 128 || p.rot > p.c.dk || p.rot % 16)
    return hipErrorInvalidValue;
  if (io_dtype == 1) return p.c.e4m3 ? append_one<__bf16, true>(p, s) : append_one<__bf16, false>(p, s);
  return p.c.e4m3 ? append_one<float, true>(p, s) : append_one<float, false>(p, s);
}

hipError_t launch_kv_read(const ReadParams& p, int out_dtype, hipStream_t s) {
  if (p.total < 1 || p.N < 1 || p.c.dk % 64 || p.c.dv % 64) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((p.total + kReadTokens - 1) / kReadTokens)), threads(kThreads);
  if (out_dtype == 1) {
    if (p.c.e4m3) hipLaunchKernelGGL((kda_kv_read_kernel<__bf16, true>), grid, threads, 0, s, p);
    else hipLaunchKernelGGL((kda_kv_read_kernel<__bf16, false>), grid, threads, 0, s, p);
  } else {
    if (p.c.e4m3) hipLaunchKernelGGL((kda_kv_read_kernel<float, true>), grid, threads, 0, s, p);
    else hipLaunchKernelGGL((kda_kv_read_kernel<float, false>), grid, threads, 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace kda
