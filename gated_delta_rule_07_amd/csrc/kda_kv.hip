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
// Workgroups behind the pages turn the queries.  A lane holds two pieces of 8 values of a row, those
// that turn together, so that a rotation exchanges nothing between lanes.
// Cosines and sines are formed in fp64, the rest is fp32; values are rounded once, to the page's or the output's type.
// Measured: 65,536 tokens of 32 + 8 heads of 128 in 16 sequences onto e4m3 pages 290 us, 5.1 TB/s of the bytes that it cannot do
// without and 5.9 of those it moves (rows of a page beyond the first 32 are fetched again for the codes, when the scale
// is known; sharing a head among waves, so that all rows stay in registers, gains 2% there and costs 8% with few heads).  256
// sequences of one token 10 us, one 3.3: the latency of lengths, table and page, and of the look for pages that others write.
#include <algorithm>

#include "kda_kv_device.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

typedef float f32x8 __attribute__((ext_vector_type(8)));

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

// Eight values in bf16, rounded to nearest even.
__device__ __forceinline__ u32x4 bits_of(const f32x4& lo, const f32x4& hi) {
  bf16x8 h;
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = (__bf16)lo[e], h[4 + e] = (__bf16)hi[e];
  return __builtin_bit_cast(u32x4, h);
}

// Cosine and sine of pos times a frequency in turns, in fp64 and then rounded: the angle's distance x from the nearest quarter
// turn, and the series about 0 (|x| <= pi / 4: what is left out is below 1.2e-10).  From an angle rounded to fp32 they would be more than a
// step off, and with them more codes on the other side of a border. (The time is the same.)
__device__ __forceinline__ float2 turn_of(double pos, double freq) {
  const double turns = pos * freq, t = turns - rint(turns), quarter = rint(4.0 * t);
  const double x = (t - 0.25 * quarter) * 6.283185307179586, y = x * x;
  const double c = 1.0 + y * (-1.0 / 2 + y * (1.0 / 24 + y * (-1.0 / 720 + y * (1.0 / 40320 + y * (-1.0 / 3628800)))));
  const double s = x * (1.0 + y * (-1.0 / 6 + y * (1.0 / 120 + y * (-1.0 / 5040 + y * (1.0 / 362880 + y * (-1.0 / 39916800))))));
  const int q = (int)quarter;  // -2 .. 2
  const float cf = (float)(q & 1 ? s : c), sf = (float)(q & 1 ? c : s);
  return float2{q + 1 & 2 ? -cf : cf, q & 2 ? -sf : sf};
}

// The turns of nt tokens at positions pos(t) to turn[t][half]: a thread keeps to one frequency.
template <typename F>
__device__ __forceinline__ void turns_of(float2* turn, const float* inv_freq, int half, int nt, int tid, F pos) {
  if (!half) return;
  const int step = kThreads / half, i = tid % half;
  if (tid >= step * half) return;
  const double freq = (double)inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
  for (int t = tid / half; t < nt; t += step) turn[t * half + i] = turn_of(pos(t), freq);
}

// The two pieces of 8 values that a lane of a row's d / 16 holds.
struct Pieces {
  int c0, c1;
  bool turned;
};
__device__ __forceinline__ Pieces pieces_of(int lane, int lanes, int rot) {
  const int m = rot / 16;  // the first m lanes hold what turns: pieces j and j + m; the others halves of the rest
  return lane < m ? Pieces{lane, lane + m, true} : Pieces{m + lane, lanes + lane, false};
}

// A lane's cosines and sines: of its 8 pairs (i, i + rot/2), or of the 4 + 4 neighbours in its pieces.
struct Turns {
  float2 f[8];
};
__device__ __forceinline__ Turns turns_at(const float2* ft, const Pieces& c, int adjacent) {
  Turns t;
#pragma unroll
  for (int e = 0; e < 8; ++e) t.f[e] = float2{1.0f, 0.0f};
  if (c.turned) {
    const float2* lo = ft + (adjacent ? 4 : 8) * c.c0;
    const float2* hi = adjacent ? ft + 4 * c.c1 : lo + 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) t.f[e] = lo[e], t.f[4 + e] = hi[e];
  }
  return t;
}
__device__ __forceinline__ void rotate(f32x8& a, f32x8& b, const Turns& t, int adjacent) {
  if (adjacent) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = t.f[e], g = t.f[4 + e];
      const float x = a[2 * e], y = a[2 * e + 1], z = b[2 * e], w = b[2 * e + 1];
      a[2 * e] = x * f.x - y * f.y;
      a[2 * e + 1] = y * f.x + x * f.y;
      b[2 * e] = z * g.x - w * g.y;
      b[2 * e + 1] = w * g.x + z * g.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = a[e], y = b[e];
      a[e] = x * t.f[e].x - y * t.f[e].y;
      b[e] = y * t.f[e].x + x * t.f[e].y;
    }
  }
}

// 8 values as they lie in memory, so that many rows can be in flight.
template <typename IO>
struct Raw {
  u32x4 w[sizeof(IO) / 2];
  __device__ __forceinline__ void load(const IO* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(IO) / 2; ++i) w[i] = reinterpret_cast<const u32x4*>(p)[i];
  }
  __device__ __forceinline__ f32x8 values() const {
    f32x8 r;
    if constexpr (sizeof(IO) == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r[2 * e] = __builtin_bit_cast(float, w[0][e] << 16);
        r[2 * e + 1] = __builtin_bit_cast(float, w[0][e] & 0xffff0000u);
      }
    } else {
      const f32x4 lo = __builtin_bit_cast(f32x4, w[0]), hi = __builtin_bit_cast(f32x4, w[1]);
      r = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
  }
};

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
// The loads of a turn do not wait for one another: indexes are brought into range instead of being tested first.
__device__ bool shared_page(const AppendParams& p, int page, int b, long long j, int tid) {
  const int lane = tid % 64, wave = tid / 64, pt = p.c.page_tokens;
  auto names = [&](int row, long long at) {
    const int e = p.c.table[(size_t)clamp_to(row, p.c.n_rows - 1) * p.c.width + min(max(at, 0LL), p.c.width - 1LL)];
    return row >= 0 && row < p.c.n_rows && at >= 0 && at < p.c.width && e == page;
  };
  bool hit = false;
  if (!p.cu) {  // one page a sequence
    for (int c = tid; c < p.N; c += kThreads) hit |= c != b && names(p.c.rows ? p.c.rows[c] : c, max(p.lens[c], 0) / pt);
    return hit;
  }
  for (int c0 = 0; c0 < p.N; c0 += 64) {
    // a lane looks after one sequence: four of its first 16 pages in each wave
    const int c = min(c0 + lane, p.N - 1);
    const Span s = span_of(p, c);
    const int row = p.c.rows ? p.c.rows[c] : c;
    const long long first = s.before / pt;
    const int n = c0 + lane < p.N ? (int)min(touched(s, pt), max(0LL, p.c.width - first)) : 0;
#pragma unroll
    for (int i = wave; i < 4 * kWaves; i += kWaves) hit |= i < n && !(c == b && i == j) && names(row, first + i);
    // the others of the sequences that have more: the waves take these sequences in turn, or all of them the few there are
    unsigned long long more = __ballot(n > 4 * kWaves);
    const bool few = __popcll(more) < kWaves;
    for (int k = 0; more; ++k, more &= more - 1) {
      if (!few && k % kWaves != wave) continue;
      const int l = __builtin_ctzll(more), m = __shfl(n, l), r = __shfl(row, l), q = c0 + l;
      const long long f = __shfl(first, l);
#pragma unroll 4
      for (int i = 4 * kWaves + (few ? tid : lane); i < m; i += few ? kThreads : 64) hit |= !(q == b && i == j) && names(r, f + i);
    }
  }
  return hit;
}

constexpr int kMostQueryTokens = 8;

template <typename IO>
__device__ void append_queries(const AppendParams& p, int block, int tokens, float2* turn, int tid) {
  const int t0 = block * tokens, nt = min(tokens, p.total - t0), half = p.rot / 2;
  const int b0 = p.cu && !p.positions && half ? last_at_most_wave(p.N, t0, [&](int i) { return (long long)p.cu[i]; }) : 0;
  turns_of(turn, p.inv_freq, half, nt, tid, [&](int i) {
    const int t = t0 + i;
    if (p.positions) return (double)p.positions[t];
    int b = p.cu ? b0 : t;
    if (p.cu)
      while (b + 1 < p.N && p.cu[b + 1] <= t) ++b;
    const Span s = span_of(p, b);
    return (double)(s.before + t - s.t0);
  });
  __syncthreads();
  // a group of lanes takes one token, and some of its heads: its cosines and sines stay in registers
  const int lanes = p.c.dk / 16, groups = kThreads / lanes, gr = tid / lanes, d = p.c.dk;
  const int t = gr % tokens, tok = t0 + t;
  // tokens behind the last sequence's are left as they were
  if (t >= nt || (p.cu && (tok < p.cu[0] || tok >= clamp_to(p.cu[p.N], p.total)))) return;
  const Pieces c = pieces_of(tid % lanes, lanes, p.rot);
  const Turns f = turns_at(turn + t * half, c, p.adjacent);
  const IO* x = static_cast<const IO*>(p.q) + (size_t)tok * p.q_stride;
  IO* y = static_cast<IO*>(p.q_out) + (size_t)tok * p.q_out_stride;
  constexpr int NB = 4;  // heads in flight
  const int step = groups / tokens;
  for (int h0 = gr / tokens; h0 < p.Hq; h0 += NB * step) {
    Raw<IO> a[NB], b[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int h = h0 + i * step;
      if (h < p.Hq) a[i].load(x + (size_t)h * d + 8 * c.c0), b[i].load(x + (size_t)h * d + 8 * c.c1);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int h = h0 + i * step;
      if (h >= p.Hq) break;
      f32x8 u = a[i].values(), v = b[i].values();
      if (c.turned) rotate(u, v, f, p.adjacent);
      store8(y + (size_t)h * d + 8 * c.c0, u);
      store8(y + (size_t)h * d + 8 * c.c1, v);
    }
  }
}

template <typename IO, bool E4, int NB>
__global__ __launch_bounds__(kThreads) void kda_kv_append_kernel(AppendParams p, int page_blocks, int q_tokens) {
  extern __shared__ __attribute__((aligned(16))) float2 turn[];  // [tokens][rot / 2]: cosine and sine
  __shared__ int flag[kWaves];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  if ((int)blockIdx.x >= page_blocks) {
    append_queries<IO>(p, (blockIdx.x - page_blocks) * gridDim.y + blockIdx.y, q_tokens, turn, tid);
    return;
  }
  const KvCache& c = p.c;
  const int pt = c.page_tokens;
  // sequence b has room for cu[b + 1] / pt - cu[b] / pt + 2 workgroups, as many as its tokens touch pages at most
  int b = blockIdx.x;
  long long j = 0;
  if (p.cu) {
    auto first = [&](int i) { return (long long)(clamp_to(p.cu[i], p.total) / pt) + 2LL * i; };
    b = last_at_most_wave(p.N, blockIdx.x, first);
    j = blockIdx.x - first(b);
  }
  const Span s = span_of(p, b);
  if (j < 0 || j >= touched(s, pt)) return;  // (the same for the whole workgroup)
  const long long at = s.before / pt + j;  // the page's place in the row
  const int slot0 = j == 0 ? (int)(s.before % pt) : 0;
  const int first = j == 0 ? 0 : (int)(at * pt - s.before);  // its first token among the sequence's new ones
  const int nt = min(pt - slot0, s.n - first);
  const int t0 = s.t0 + first, half = p.rot / 2;
  // a wave's head: of the keys, then of the values
  int pair = blockIdx.y * kWaves + wave, h = 0, d = 0, rows = 0, r0 = 0;
  bool is_v = false;
  Pieces pc{0, 0, false};
  long long stride = 0;
  const IO* x = nullptr;
  Raw<IO> ra[NB], rb[NB];
  auto fetch = [&](int t1) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int t = t1 + i * rows + r0;
      if (t < nt) {
        const IO* y = x + (size_t)t * stride;
        ra[i].load(y + 8 * pc.c0), rb[i].load(y + 8 * pc.c1);
      }
    }
  };
  auto begin = [&] {  // its first rows in flight
    is_v = pair >= c.H;
    h = is_v ? pair - c.H : pair, d = is_v ? c.dv : c.dk;
    const int lanes = d / 16;
    rows = 64 / lanes, r0 = lane / lanes;
    pc = pieces_of(lane % lanes, lanes, is_v ? 0 : p.rot);
    stride = is_v ? p.v_stride : p.k_stride;
    x = static_cast<const IO*>(is_v ? p.v : p.k) + (size_t)t0 * stride + (size_t)h * d;
    fetch(0);
  };
  if (pair < 2 * c.H) begin();
  const int page = kv_page(c, b, at);
  const bool any = __any(page >= 0 && shared_page(p, page, b, j, tid));
  if (lane == 0) flag[wave] = any;
  const double place = (double)(s.before + first);
  turns_of(turn, p.inv_freq, half, nt, tid, [&](int t) { return p.positions ? (double)p.positions[t0 + t] : place + (double)t; });
  __syncthreads();
  bool store = page >= 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) store = store && !flag[w];

  for (; pair < 2 * c.H;) {
    char* block = c.pool + (size_t)max(page, 0) * c.page_bytes + (is_v ? kv_values(c, h) : kv_keys(c, h));
    auto value = [&](int i, int t, f32x8& a, f32x8& b8) {
      a = ra[i].values(), b8 = rb[i].values();
      if (pc.turned) rotate(a, b8, turns_at(turn + t * half, pc, p.adjacent), p.adjacent);
    };
    float inv = 1.0f;
    if (E4 && store) {
      float amax = 0.0f;
      for (int t1 = 0; t1 < nt; t1 += NB * rows) {
        if (t1) fetch(t1);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int t = t1 + i * rows + r0;
          if (t >= nt) break;
          f32x8 a, b8;
          value(i, t, a, b8);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = __builtin_fabsf(a[e]), v = __builtin_fabsf(b8[e]);
            amax = u < __builtin_inff() ? fmaxf(amax, u) : amax;
            amax = v < __builtin_inff() ? fmaxf(amax, v) : amax;
          }
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
      if (nt > NB * rows) fetch(0);
    }
    for (int t1 = 0; t1 < nt; t1 += NB * rows) {
      if (t1) fetch(t1);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int t = t1 + i * rows + r0;
        if (t >= nt) break;
        f32x8 a, b8;
        value(i, t, a, b8);
        if (store) {
          const size_t to = (size_t)(slot0 + t) * d;
          if constexpr (E4) {
            const f32x8 u = a * inv, v = b8 * inv;
            *reinterpret_cast<u32x2*>(block + to + 8 * pc.c0) = u32x2{to_e4m3x4(u[0], u[1], u[2], u[3]), to_e4m3x4(u[4], u[5], u[6], u[7])};
            *reinterpret_cast<u32x2*>(block + to + 8 * pc.c1) = u32x2{to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7])};
          } else {
            store8(reinterpret_cast<__bf16*>(block) + to + 8 * pc.c0, a);
            store8(reinterpret_cast<__bf16*>(block) + to + 8 * pc.c1, b8);
          }
        }
        if (!is_v && p.k_out) {
          IO* y = static_cast<IO*>(p.k_out) + (size_t)(t0 + t) * p.k_out_stride + (size_t)h * d;
          store8(y + 8 * pc.c0, a);
          store8(y + 8 * pc.c1, b8);
        }
      }
    }
    pair += gridDim.y * kWaves;
    if (pair < 2 * c.H) begin();
  }
}

template <typename IO, bool E4, int NB>
hipError_t append_nb(const AppendParams& p, hipStream_t s) {
  const long long pages = p.cu ? (long long)p.total / p.c.page_tokens + 2LL * p.N : p.N;
  // more tokens a workgroup where there are enough of them to fill the compute units
  int q_tokens = 1;
  while (q_tokens < kMostQueryTokens && (long long)p.total >= 2048LL * q_tokens) q_tokens *= 2;
  const long long q_blocks = p.q ? (p.total + q_tokens - 1) / q_tokens : 0;
  // a wave a head where the pages alone would not fill the compute units
  const int most = (2 * p.c.H + kWaves - 1) / kWaves;
  const int split = (int)std::max(1LL, std::min((long long)most, 2048 / std::max(pages, 1LL)));
  const size_t lds = (size_t)std::max(p.cu ? p.c.page_tokens : 1, q_tokens) * (p.rot / 2) * sizeof(float2);
  if (lds > 65000) {  // more than the default has to be asked for
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&kda_kv_append_kernel<IO, E4, NB>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((kda_kv_append_kernel<IO, E4, NB>), dim3((unsigned)(pages + (q_blocks + split - 1) / split), split),
                     dim3(kThreads), lds, s, p, (int)pages, q_tokens);
  return hipGetLastError();
}

template <typename IO, bool E4>
hipError_t append_one(const AppendParams& p, hipStream_t s) {
  return p.cu ? append_nb<IO, E4, sizeof(IO) == 2 ? 4 : 2>(p, s) : append_nb<IO, E4, 1>(p, s);
}

// ---- back ---------------------------------------------------------------------------------

constexpr int kReadTokens = 8;
constexpr size_t kLastCache = (size_t)256 << 20;  // bytes of the cache that the dies share

// Stores 16 bytes, past the caches or not.
template <bool PAST>
__device__ __forceinline__ void store16(char* p, const u32x4& x) {
  if constexpr (PAST) __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(p));
  else *reinterpret_cast<u32x4*>(p) = x;
}

// Each lane's 32 bytes a, b of 128 neighbours that four lanes hold, to p: exchanged, so that a store of the four is 64 neighbours.
template <bool PAST>
__device__ __forceinline__ void store32(char* p, const u32x4& a, const u32x4& b, int lane) {
  u32x4 x, y;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t ae = a[e], be = b[e];
    // (quad_perm: lanes 0, 0, 1, 1 and 2, 2, 3, 3 of the four)
    const uint32_t a0 = __builtin_amdgcn_mov_dpp(ae, 0x50, 0xf, 0xf, false), b0 = __builtin_amdgcn_mov_dpp(be, 0x50, 0xf, 0xf, false);
    const uint32_t a1 = __builtin_amdgcn_mov_dpp(ae, 0xfa, 0xf, 0xf, false), b1 = __builtin_amdgcn_mov_dpp(be, 0xfa, 0xf, 0xf, false);
    x[e] = lane & 1 ? b0 : a0;
    y[e] = lane & 1 ? b1 : a1;
  }
  p -= 16 * (lane % 4);
  store16<PAST>(p, x);
  store16<PAST>(p + 64, y);
}

// A lane moves V values (16 bytes of the page) of a token's head: always the same ones, of one token after another.
// Four neighbouring lanes always move neighbours of one row.  Bound by memory: 70,001 tokens of 8 heads of 128, e4m3 to bf16, 91 us
// (4.8 TB/s, two thirds of it stores; 16, 32 and 64 tokens a workgroup 6 to 17% slower); 517 tokens of 4 heads 4.9 us, latency.
template <typename OUT, bool E4, bool PAST>
__global__ __launch_bounds__(kThreads) void kda_kv_read_kernel(ReadParams p) {
  __shared__ int page[kReadTokens], slot[kReadTokens];
  constexpr int V = E4 ? 16 : 8, NB = 4;
  const KvCache& c = p.c;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, t0 = blockIdx.x * kReadTokens, nt = min(kReadTokens, p.total - t0);
  if (wave == 0) {
    const int b0 = last_at_most_wave(p.N, t0, [&](int i) { return (long long)p.cu[i]; });
    if (lane < nt) {
      const int t = t0 + lane;
      int b = b0;
      while (b + 1 < p.N && p.cu[b + 1] <= t) ++b;
      const int begin = clamp_to(p.cu[b], p.total), end = clamp_to(p.cu[b + 1], p.total);
      const long long pos = (p.starts ? max(p.starts[b], 0) : 0) + (long long)(t - begin);
      page[lane] = t >= begin && t < end ? kv_page(c, b, pos / c.page_tokens) : -1;
      slot[lane] = (int)(pos % c.page_tokens);
    }
  }
  __syncthreads();
  const int nk = c.H * c.dk / V, n = nk + c.H * c.dv / V;  // pieces of a token: of its keys, then of its values
  int lanes = 64;                                          // of a wave for one token
  while (lanes / 2 >= n) lanes /= 2;
  const int step = kWaves * (64 / lanes);
  for (int r = lane % lanes; r < n; r += lanes) {
    const bool is_v = r >= nk;
    const int d = is_v ? c.dv : c.dk, j = (is_v ? r - nk : r) * V, h = j / d;
    const size_t at = (is_v ? kv_values(c, h) : kv_keys(c, h)) + (size_t)(j % d) * (E4 ? 1 : 2);
    const size_t sat = kv_scales(c) + 4 * (size_t)((is_v ? c.H : 0) + h);
    OUT* to = static_cast<OUT*>(is_v ? p.v_out : p.k_out) + (size_t)t0 * c.H * d + j;
    for (int t1 = wave * (64 / lanes) + lane / lanes; t1 < nt; t1 += NB * step) {
      u32x4 w[NB];
      float s[NB];
      bool there[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int t = t1 + i * step;
        there[i] = t < nt && page[min(t, nt - 1)] >= 0;
        if (there[i]) {
          const char* base = c.pool + (size_t)page[t] * c.page_bytes;
          w[i] = *reinterpret_cast<const u32x4*>(base + at + (size_t)slot[t] * d * (E4 ? 1 : 2));
          if constexpr (E4) s[i] = *reinterpret_cast<const float*>(base + sat);
        }
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if (!there[i]) continue;
        OUT* y = to + (size_t)(t1 + i * step) * c.H * d;
        if constexpr (E4) {
          f32x4 x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = from_e4m3x4(w[i][e]) * s[i];
          if constexpr (sizeof(OUT) == 2) {
            store32<PAST>(reinterpret_cast<char*>(y), bits_of(x[0], x[1]), bits_of(x[2], x[3]), lane);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) store16<PAST>(reinterpret_cast<char*>(y + 4 * e), __builtin_bit_cast(u32x4, x[e]));
          }
        } else if constexpr (sizeof(OUT) == 2) {
          store16<PAST>(reinterpret_cast<char*>(y), w[i]);
        } else {
          Raw<__bf16> x;
          x.w[0] = w[i];
          const f32x8 z = x.values();
          store32<PAST>(reinterpret_cast<char*>(y), __builtin_bit_cast(u32x4, __builtin_shufflevector(z, z, 0, 1, 2, 3)),
                  __builtin_bit_cast(u32x4, __builtin_shufflevector(z, z, 4, 5, 6, 7)), lane);
        }
      }
    }
  }
}

template <typename OUT, bool E4>
hipError_t read_one(const ReadParams& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.total + kReadTokens - 1) / kReadTokens)), threads(kThreads);
  // Rows that the shared cache could not hold until they are read are stored past it.  Measured on e4m3 pages, us alone and
  // with a pass over the rows behind it: 287 MB 91 (96 through the caches) and 179.5 (181); 66 MB 23 (26), but 65 (58).
  const bool past = (size_t)p.total * p.c.H * (p.c.dk + p.c.dv) * sizeof(OUT) > kLastCache;
  if (past) hipLaunchKernelGGL((kda_kv_read_kernel<OUT, E4, true>), grid, threads, 0, s, p);
  else hipLaunchKernelGGL((kda_kv_read_kernel<OUT, E4, false>), grid, threads, 0, s, p);
  return hipGetLastError();
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
  return out_dtype == 1 ? p.c.e4m3 ? read_one<__bf16, true>(p, s) : read_one<__bf16, false>(p, s)
                        : p.c.e4m3 ? read_one<float, true>(p, s) : read_one<float, false>(p, s);
}

}  // namespace kda
