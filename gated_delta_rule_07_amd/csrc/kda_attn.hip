// Attention over whole prompts, causal, with grouped heads and packed sequences, for gfx950.
//
//   o_i = sum_j p_ij v_j,  p_i = softmax over the keys j <= i + n_k - n_q of scale q_i . k_j
//
// One pass over the keys with a running maximum m and sum l of each query:
//   m' = max(m, max_j s_j),  o <- o 2^(m - m') + sum_j 2^(s_j - m') v_j,  l likewise.
// Scores are formed transposed, S^T = K Q^T, so that a lane holds one query's scores: the maximum
// and the sum are then mostly a lane's own, and P^T as the product leaves it is the operand of O^T = V^T P^T.
#include <algorithm>

#include "kda_kv_device.h"

namespace kda {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// One workgroup's part: tokens [q0, q0 + nq) of the call's queries are the rows from r0 on of sequence b.
struct Part {
  int q0, nq;   // the sequence's queries
  int k0, nk;   // its keys
  int r0;       // the first row of this tile within the sequence
};

// Tile `tile` of tiles of BM rows: sequence b has cu[b + 1] / BM - cu[b] / BM + 1 of them.
template <int BM>
__device__ __forceinline__ bool part_of(const AttnParams& p, int tile, Part& s) {
  int b, j;
  if (p.cu_q) {
    auto first = [&](int i) { return (long long)(clamp_to(p.cu_q[i], p.total_q) / BM) + i; };
    b = last_at_most(p.N, tile, first);
    j = tile - (int)first(b);
    s.q0 = clamp_to(p.cu_q[b], p.total_q);
    s.nq = clamp_to(p.cu_q[b + 1], p.total_q) - s.q0;
    const int* ck = p.cu_k ? p.cu_k : p.cu_q;
    s.k0 = clamp_to(ck[b], p.total_k);
    s.nk = clamp_to(ck[b + 1], p.total_k) - s.k0;
  } else {
    s.nq = p.total_q / p.N;
    s.nk = p.total_k / p.N;
    const int per = (s.nq + BM - 1) / BM;
    b = tile / per;
    j = tile % per;
    s.q0 = b * s.nq;
    s.k0 = b * s.nk;
  }
  // (long sequences' last tiles have the most keys: they go first)
  const int tiles = (s.nq + BM - 1) / BM;
  s.r0 = (tiles - 1 - j) * BM;
  s.nk = max(s.nk, 0);
  return j >= 0 && s.nq > 0 && j < tiles;
}

// ---- every type and head size: fp32 matrix cores -------------------------------------------

constexpr int kRows = 64, kKeys = 32, kPad = 4;

template <typename IO, int DK, int DV>
__global__ __launch_bounds__(256) void kda_attn_plain_kernel(AttnParams p) {
  __shared__ __attribute__((aligned(16))) float sk[kKeys][DK + kPad];
  __shared__ __attribute__((aligned(16))) float sv[DV][kKeys + kPad];  // transposed
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, c = lane % 16, g = lane / 16;
  const int h = blockIdx.y, hk = h / (p.Hq / p.Hk);
  Part s;
  if (!part_of<kRows>(p, blockIdx.x, s)) return;
  const int row = s.r0 + 16 * wave + c;  // this lane's query
  // queries as B operands: values 32 step + 8 g + e
  constexpr int NS = (DK + 31) / 32;
  Frag<float> q[NS];
#pragma unroll
  for (int st = 0; st < NS; ++st) {
    q[st].zero();
    const int i0 = 32 * st + 8 * g;
    if (row < s.nq && i0 < DK) {
      const IO* x = static_cast<const IO*>(p.q) + (size_t)(s.q0 + row) * p.q_stride + (size_t)h * DK + i0;
#pragma unroll
      for (int e = 0; e < 8; ++e) q[st].v[e] = to_f32(x[e]);
    }
  }
  const int shift = s.nk - s.nq;
  const int limit = row < s.nq ? row + shift + 1 : 0;              // this query's keys
  const int last = min(s.r0 + kRows, s.nq) + shift;                // the workgroup's
  const int wfirst = s.r0 + 16 * wave + shift + 1;                 // the least of the wave's rows
  const float scale = p.scale * kLog2e;
  constexpr int NT = DV / 16;
  f32x4 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = (f32x4)0.0f;
  float m = -__builtin_inff(), l = 0.0f;
  for (int k0 = 0; k0 < last; k0 += kKeys) {
    __syncthreads();
    for (int i = tid; i < kKeys * DK; i += 256) {
      const int r = i / DK, e = i % DK;
      sk[r][e] = k0 + r < s.nk ? to_f32(static_cast<const IO*>(p.k)[(size_t)(s.k0 + k0 + r) * p.k_stride + (size_t)hk * DK + e]) : 0.0f;
    }
    for (int i = tid; i < kKeys * DV; i += 256) {
      const int r = i / DV, e = i % DV;
      sv[e][r] = k0 + r < s.nk ? to_f32(static_cast<const IO*>(p.v)[(size_t)(s.k0 + k0 + r) * p.v_stride + (size_t)hk * DV + e]) : 0.0f;
    }
    __syncthreads();
    f32x4 x[2] = {(f32x4)0.0f, (f32x4)0.0f};  // S^T of keys 0..15 and 16..31
#pragma unroll
    for (int st = 0; st < NS; ++st) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        x[u] = mma(lds_frag<float>(&sk[0][0], DK + kPad, 16 * u + c, 32 * st + 8 * g, DK), q[st], x[u]);
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[u][r] = k0 + 16 * u + 4 * g + r < limit ? x[u][r] * scale : -__builtin_inff();
        top = fmaxf(top, x[u][r]);
      }
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float now = fmaxf(m, top), base = now == -__builtin_inff() ? 0.0f : now;
    const float keep = exp2f(m - base);
    m = now;
    l *= keep;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[u][r] = exp2f(x[u][r] - base);
        l += x[u][r];
      }
    }
    const Frag<float> pt = frag_from_tiles<float>(x[0], x[1], 1.0f);
    // Where some of the wave's queries do not see all of the tile, values that are not finite must not reach
    // them as 0 v: each query's keys are then taken by themselves.
    bool odd = false;
    if (wfirst < k0 + kKeys) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Frag<float> a = lds_frag_stacked<float>(&sv[0][0], kKeys + kPad, 16 * t + c, 0, g, kKeys);
#pragma unroll
        for (int e = 0; e < 8; ++e) odd = odd || !(__builtin_fabsf(a.v[e]) < __builtin_inff());
      }
    }
    const bool slow = __any(odd);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      o[t] *= keep;
      Frag<float> a = lds_frag_stacked<float>(&sv[0][0], kKeys + kPad, 16 * t + c, 0, g, kKeys);
      if (!slow) {
        o[t] = mma(a, pt, o[t]);
      } else {
        for (int r = 0; r < 16; ++r) {
          const int lim = __shfl(limit, r);
          Frag<float> b = a;
#pragma unroll
          for (int e = 0; e < 8; ++e) b.v[e] = k0 + (e / 4) * 16 + 4 * g + e % 4 < lim ? a.v[e] : 0.0f;
          const f32x4 y = mma(b, pt, (f32x4)0.0f);
          if (c == r) o[t] += y;
        }
      }
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (row >= s.nq) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t at = (size_t)(s.q0 + row) * p.o_stride + (size_t)h * DV + 4 * g;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const f32x4 y = o[t] * inv;
    if (p.o_f32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(p.o) + at + 16 * t) = y;
    } else {
      bf16x4 z;
#pragma unroll
      for (int r = 0; r < 4; ++r) z[r] = (__bf16)y[r];
      *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(p.o) + at + 16 * t) = z;
    }
  }
}

template <int BM>
unsigned tiles_of(const AttnParams& p) {
  return p.cu_q ? (unsigned)(p.total_q / BM + p.N) : (unsigned)((p.total_q / p.N + BM - 1) / BM * p.N);
}

template <typename IO, int DK, int DV>
hipError_t launch_plain(const AttnParams& p, hipStream_t s) {
  hipLaunchKernelGGL((kda_attn_plain_kernel<IO, DK, DV>), dim3(tiles_of<kRows>(p), p.Hq), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename IO, int DK>
hipError_t pick_dv(const AttnParams& p, hipStream_t s) {
  switch (p.dv) {
    case 16: return launch_plain<IO, DK, 16>(p, s);
    case 32: return launch_plain<IO, DK, 32>(p, s);
    case 64: return launch_plain<IO, DK, 64>(p, s);
    case 128: return launch_plain<IO, DK, 128>(p, s);
  }
  return hipErrorInvalidValue;
}

template <typename IO>
hipError_t pick_dk(const AttnParams& p, hipStream_t s) {
  switch (p.dk) {
    case 16: return pick_dv<IO, 16>(p, s);
    case 32: return pick_dv<IO, 32>(p, s);
    case 64: return pick_dv<IO, 64>(p, s);
    case 128: return pick_dv<IO, 128>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_attn_fwd(const AttnParams& p, int io_dtype, hipStream_t s) {
  if (p.total_q < 1 || p.N < 1) return hipErrorInvalidValue;
  return io_dtype == 1 ? pick_dk<__bf16>(p, s) : pick_dk<float>(p, s);
}

}  // namespace kda
