// Attention over whole prompts, causal, with grouped heads and packed sequences, for gfx950.
//
//   o_i = sum_j p_ij v_j,  p_i = softmax over the keys j <= i + n_k - n_q of scale q_i . k_j
//
// One pass over the keys with a running maximum m and sum l of each query:
//   m' = max(m, max_j s_j),  o <- o 2^(m - m') + sum_j 2^(s_j - m') v_j,  l likewise.
// Scores are formed transposed, S^T = K Q^T, so that a lane holds one query's scores: the maximum
// and the sum are then mostly a lane's own, and P^T as the product leaves it is the operand of O^T = V^T P^T.
#include <algorithm>
#include <type_traits>

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
    b = last_at_most_wave(p.N, tile, first);
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

// Workgroups go to the 8 dies in turn, and what a die's workgroups read is shared in its L2: each die takes whole key heads
// or, where there are fewer than dies (or an odd number of them), every R-th tile of its heads, so that tiles with many keys
// are spread.  Measured on 8,000 tokens, us, against runs of neighbouring tiles a die: 8 heads of queries on 1 of keys
// 175 / 203, 16 on 4 264 / 317, 12 on 3 233 / 293; fp32, 3,000 tokens, 8 on 2 261 against 326 in the order of the heads.
// pair_of returns whether this workgroup has a tile; its heads and tile.
__host__ __device__ inline unsigned dies_of_head(const AttnParams& p) { return 8 / std::min(p.Hk & -p.Hk, 8); }
__host__ __device__ inline unsigned tiles_of_die(const AttnParams& p, unsigned tiles) { return (tiles + dies_of_head(p) - 1) / dies_of_head(p); }
inline dim3 grid_of(const AttnParams& p, unsigned tiles) { return dim3(dies_of_head(p) * p.Hq * tiles_of_die(p, tiles)); }
__device__ __forceinline__ bool pair_of(const AttnParams& p, unsigned tiles, int& h, int& hk, int& tile) {
  const unsigned G = p.Hq / p.Hk, R = dies_of_head(p), per = tiles_of_die(p, tiles), die = blockIdx.x % 8, i = blockIdx.x / 8;
  hk = die / R + 8 / R * (i / (per * G));
  h = hk * G + i % G;
  tile = i % (per * G) / G * R + die % R;
  return (unsigned)tile < tiles;
}

// Four outputs from element `at` of o on.
__device__ __forceinline__ void store4(const AttnParams& p, size_t at, const f32x4& y) {
  if (p.o_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(p.o) + at) = y;
  else *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(p.o) + at) = bf16x4{(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
}

// ---- every type and head size: fp32 matrix cores -------------------------------------------
// The fp32 matrix cores are slow enough for the operands to come straight from the caches into registers: a
// workgroup takes 16 or 32 queries, each of its waves every fourth tile of 32 keys, and they are joined at the end.  So a
// few queries behind a long prefix already fill many waves.  Measured: 391 queries of 8 heads of 64 / 128 behind 3 cached
// prefixes 26 us (eight waves: 29.6), 3,000 tokens of 8 heads of 128 196 us (94 TFLOP/s of 154); bf16, 4,000 tokens of 8 heads of 32 106 us
// (77 TFLOP/s), of 16 86 us (48).  Bound by the matrix
// cores, of which a wave with a SIMD to itself fills three quarters, and by what a compute unit takes from the L2, 32 KB a tile.
//   S^T = K Q^T: a lane holds 8 of every 32 values of a key's row;
//   O^T = V^T P^T: a lane holds DV / 16 neighbouring channels of 8 keys, and tile t of the output is the t-th of them.

constexpr int kKeys = 32, kPlainWaves = 4;

// n neighbouring values as fp32.
template <int N>
__device__ __forceinline__ void load_values(const float* p, float* r) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) r[i + e] = x[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = p[i];
  }
}
template <int N>
__device__ __forceinline__ void load_values(const __bf16* p, float* r) {
  typedef __bf16 vec __attribute__((ext_vector_type(N > 1 ? N : 2)));
  if constexpr (N > 1) {
    const vec x = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int e = 0; e < N; ++e) r[e] = (float)x[e];
  } else {
    r[0] = (float)p[0];
  }
}

// A workgroup takes RT tiles of 16 queries.
template <typename IO, int DK, int DV, int RT>
__global__ __launch_bounds__(64 * kPlainWaves, RT == 1 ? 2 : 1) void kda_attn_plain_kernel(AttnParams p, unsigned tiles) {
  constexpr int NS = (DK + 31) / 32, NT = DV / 16, kRows = 16 * RT;
  __shared__ __attribute__((aligned(16))) float so[kPlainWaves][kRows][DV + 4];
  __shared__ float sm[kPlainWaves][kRows], sl[kPlainWaves][kRows];
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), c = lane % 16, g = lane / 16;
  int h, hk, at;
  Part s;
  if (!pair_of(p, tiles, h, hk, at) || !part_of<kRows>(p, at, s)) return;
  const int shift = s.nk - s.nq;
  const int last = min(s.r0 + kRows, s.nq) + shift;  // the workgroup's keys
  const int least = s.r0 + shift + 1;                // what all of its queries see
  const float scale = p.scale * kLog2e;
  // of the lane's queries, r0 + 16 j + c
  int limit[RT];  // their keys
  f32x4 o[RT][NT];
  float m[RT], l[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int row = s.r0 + 16 * j + c;
    limit[j] = row < s.nq ? row + shift + 1 : 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) o[j][t] = (f32x4)0.0f;
    m[j] = -__builtin_inff(), l[j] = 0.0f;
  }

  const IO* kg = static_cast<const IO*>(p.k) + (size_t)s.k0 * p.k_stride + (size_t)hk * DK;
  const IO* vg = static_cast<const IO*>(p.v) + (size_t)s.k0 * p.v_stride + (size_t)hk * DV;
  Frag<float> q[RT][NS];  // as B operands: values 32 step + 8 g + e
  Frag<float> k[2][NS];
  float v[8][NT];
  // (rows behind the last key: that one again)
  auto keys = [&](int k0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const IO* x = kg + (size_t)min(k0 + 16 * u + c, s.nk - 1) * p.k_stride;
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        const int i0 = 32 * st + 8 * g;
        if (DK % 32 == 0 || i0 < DK) load_values<8>(x + i0, k[u][st].v);
        else k[u][st].zero();
      }
    }
  };
  auto values = [&](int k0) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      load_values<NT>(vg + (size_t)min(k0 + 16 * (e / 4) + 4 * g + e % 4, s.nk - 1) * p.v_stride + NT * c, v[e]);
  };

  // The order of loads and uses is kept (the scheduler would mix them, and then wait for all): a tile's keys are loaded
  // while the last one's values are used, its values while its keys are.
  auto scores = [&](f32x4 (&x)[RT][2]) {  // S^T of keys 0..15 and 16..31
#pragma unroll
    for (int j = 0; j < RT; ++j) x[j][0] = x[j][1] = (f32x4)0.0f;
#pragma unroll
    for (int st = 0; st < NS; ++st)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < RT; ++j) x[j][u] = mma(k[u][st], q[j][st], x[j][u]);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto powers = [&](f32x4 (&x)[2], int j) {
    float top = -__builtin_inff();
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = fmaxf(top, x[u][r]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float now = fmaxf(m[j], top), base = now == -__builtin_inff() ? 0.0f : now;
    const float keep = __builtin_amdgcn_exp2f(m[j] - base);
    m[j] = now;
    l[j] *= keep;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[u][r] = __builtin_amdgcn_exp2f(x[u][r] - base);
        l[j] += x[u][r];
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) o[j][t] *= keep;
    return frag_from_tiles<float>(x[0], x[1], 1.0f);
  };
  int k0 = wave * kKeys;
  if (k0 < last) {
    keys(k0);
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int row = min(s.r0 + 16 * j + c, s.nq - 1);
      const IO* y = static_cast<const IO*>(p.q) + (size_t)(s.q0 + row) * p.q_stride + (size_t)h * DK + 8 * g;
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        if (DK % 32 == 0 || 32 * st + 8 * g < DK) load_values<8>(y + 32 * st, q[j][st].v);
        else q[j][st].zero();
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    values(k0);
    __builtin_amdgcn_sched_barrier(0);
    // (waited for here: a wait inside the loop would wait for the tiles' loads too)
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int st = 0; st < NS; ++st)
#pragma unroll
        for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(q[j][st].v[e]));
    f32x4 x[RT][2];
    Frag<float> pt[RT];
    for (; k0 + kKeys <= least; k0 += kPlainWaves * kKeys) {  // tiles that every query sees whole
      scores(x);
      keys(k0 + kPlainWaves * kKeys);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        x[j][0] *= scale, x[j][1] *= scale;
        pt[j] = powers(x[j], j);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        Frag<float> a;
#pragma unroll
        for (int e = 0; e < 8; ++e) a.v[e] = v[e][t];
#pragma unroll
        for (int j = 0; j < RT; ++j) o[j][t] = mma(a, pt[j], o[j][t]);
      }
      __builtin_amdgcn_sched_barrier(0);
      values(k0 + kPlainWaves * kKeys);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (k0 < last) {  // one that is cut: the borders of up to 32 queries lie in two tiles at most, of two waves
      scores(x);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) x[j][u][r] = k0 + 16 * u + 4 * g + r >= limit[j] ? -__builtin_inff() : x[j][u][r] * scale;
        pt[j] = powers(x[j], j);
      }
      // What no query sees is left out.  Values that are not finite must not reach, as 0 v, queries that do not see them:
      // they are left out too, and counted for each query that does see them: its outputs become NaN.
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        Frag<float> a, n;
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool there = k0 + 16 * (e / 4) + 4 * g + e % 4 < last, fine = __builtin_fabsf(v[e][t]) < __builtin_inff();
          a.v[e] = there & fine ? v[e][t] : 0.0f;
          n.v[e] = there & !fine ? 1.0f : 0.0f;
          odd |= there & !fine;
        }
#pragma unroll
        for (int j = 0; j < RT; ++j) o[j][t] = mma(a, pt[j], o[j][t]);
        if (__builtin_expect(__any(odd), 0)) {
#pragma unroll
          for (int j = 0; j < RT; ++j) {
            Frag<float> see;
#pragma unroll
            for (int e = 0; e < 8; ++e) see.v[e] = k0 + 16 * (e / 4) + 4 * g + e % 4 < limit[j] ? 1.0f : 0.0f;
            const f32x4 y = mma(n, see, (f32x4)0.0f);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[j][t][r] = y[r] > 0.0f ? __builtin_nanf("") : o[j][t][r];
          }
        }
      }
    }
  }

  // join the waves
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    l[j] += __shfl_xor(l[j], 16);
    l[j] += __shfl_xor(l[j], 32);
    if (g == 0) sm[wave][16 * j + c] = m[j], sl[wave][16 * j + c] = l[j];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) so[wave][16 * j + c][NT * (4 * g + r) + t] = o[j][t][r];
  }
  __syncthreads();
  for (int i = tid; i < kRows * DV / 4; i += 64 * kPlainWaves) {
    const int r = i / (DV / 4), e = 4 * (i % (DV / 4));
    if (s.r0 + r >= s.nq) break;
    float top = sm[0][r];
#pragma unroll
    for (int w = 1; w < kPlainWaves; ++w) top = fmaxf(top, sm[w][r]);
    const float base = top == -__builtin_inff() ? 0.0f : top;
    f32x4 y = (f32x4)0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kPlainWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(sm[w][r] - base);
      sum += f * sl[w][r];
      y += f * *reinterpret_cast<const f32x4*>(&so[w][r][e]);
    }
    store4(p, (size_t)(s.q0 + s.r0 + r) * p.o_stride + (size_t)h * DV + e, y * (sum == 0.0f ? 0.0f : 1.0f / sum));
  }
}

// ---- bf16 with heads of 64 and 128 ---------------------------------------------------------
// A wave holds 32 queries, a workgroup of NW waves 32 NW; 64 keys and values at a time are copied
// straight into LDS, two buffers in turn, one barrier a tile.  32x32x16 matrix cores:
//   S^T (64 keys x 32 queries) = K Q^T, K's rows read 16 bytes a lane;
//   O^T (DV x 32) += V^T P^T, V^T read through the LDS transpose (4 keys of 16 channels a group of
//   16 lanes); the keys of a step are taken in the order in which S^T leaves them in a lane.
// LDS rows are dense; their 16-byte pieces are exchanged (xor with bits of the row) so that the lanes of a
// read fall on different banks (no conflicts in the counters).
// Probabilities are rounded to bf16 for the product with V and summed as rounded, in fp32; scores, maxima, sums and outputs are fp32.
// (bf16 outputs are then 0.18 to 0.21% off the definition, their own rounding alone 0.16%.  Probabilities in two bf16 terms, as decode
// has them, are half as many products again: 16,384 tokens 2.87 ms for 2.07, the packed batch 631 us for 484.)
// Measured, 32 + 8 heads of 128: 16,384 tokens 2.02 ms (1.09 PFLOP/s, where a matrix product of 8192^3 reaches 1.36), 24,961 tokens
// in 16 sequences 471 us (0.86).  Bound by the matrix cores and the exponentials beside them: the cores are busy 56% of the
// cycles at a clock that the load holds at 1.8 GHz, vector instructions 43%, with two waves a SIMD to overlap them (256 registers
// each).  The packed batch loses 6% to cut tiles and the rest to the first loads and last stores of its 6,528 workgroups (of 6,752 launched).
// Slower: eight waves and 256 queries a workgroup (packed 620 us), scores a tile ahead of the probabilities (566).

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

constexpr int kTileKeys = 64;
constexpr float kSlack = 8.0f;

// 16 bytes a lane from `src` to dst + 16 lane (dst the same for the wave).  Written out because the
// compiler, which cannot tell the buffer that is filled from the one that is read, would wait for every copy
// before the next LDS read; it writes no register, and tile_barrier() waits for it.
__device__ __forceinline__ void copy16(const char* src, char* dst) {
  const uint32_t at = (uint32_t)(uintptr_t)(lds_void*)dst;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "memory", "m0");
}
// The same from base + off.
__device__ __forceinline__ void copy16(const char* base, uint32_t off, char* dst) {
  const uint32_t at = (uint32_t)(uintptr_t)(lds_void*)dst;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory", "m0");
}
// Every wave's LDS writes are there.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// Every wave's copies have landed, and its reads of the other buffer are done.
__device__ __forceinline__ void tile_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The larger of the two halves' values.
__device__ __forceinline__ float half_max(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto y = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t lo = y[0], hi = y[1];  // (a bit cast of y[1] itself gives y[0])
  return fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}

// Where the 16-byte piece c of row r lies in its row.
template <int D>
__device__ __forceinline__ int key_piece(int r, int c) { return D == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7); }
template <int D>
__device__ __forceinline__ int value_piece(int r, int c) { return D == 128 ? c ^ (4 * (r & 3)) : c ^ (4 * ((r >> 1) & 1)); }

// V^T as an operand: channels [32 i, 32 i + 32) of keys [16 st, 16 st + 16); slot e of half hf is key 8 (e / 4) + 4 hf + e % 4.
template <int DV>
__device__ __forceinline__ bf16x8 value_operand(char* vl, int i, int st, int lane) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  s16x4 y[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 16 * st + 8 * j + 4 * (lane / 32) + lane % 16 / 4;
    const int cc = 4 * i + 2 * (lane / 16 % 2) + lane % 4 / 2;
    y[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(vl + r * (2 * DV) + 16 * value_piece<DV>(r, cc) + 8 * (lane % 2)));
  }
  return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(y[0], y[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// The operands that count the values noted in `bad` (n) for the queries that see them (see); seen: the lane's query's keys of the
// tile; noted(e): whether the byte of piece e was written.
template <int DV, typename F>
__device__ __forceinline__ void counted(const unsigned char* bad, int i, int st, int lane, int seen, bf16x8& n, bf16x8& see, F noted) {
  const int c = lane % 32;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int r = 16 * st + 8 * (e / 4) + 4 * (lane / 32) + e % 4;
    const int piece = r * (DV / 8) + value_piece<DV>(r, 4 * i + c / 8);
    const unsigned bits = noted(piece) ? bad[piece] : 0u;
    n[e] = (__bf16)(float)(bits >> c % 8 & 1);
    see[e] = (__bf16)(r < seen ? 1.0f : 0.0f);
  }
}

// Takes the values of NC pieces of 16 bytes (the at(i)-th of a tile, i < NC) that are not finite out of the tile at vl, and notes them
// in `bad`, a bit each; returns whether there are any (in any lane: only then `bad` is written).  Times 0, every finite value is 0.
template <int NC, typename F>
__device__ __forceinline__ bool take_out(char* vl, unsigned char* bad, F at) {
  u32x4 y[NC];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    y[i] = *reinterpret_cast<const u32x4*>(vl + 16 * at(i));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = y[i][j];
      sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), bf16x2{(__bf16)0.0f, (__bf16)0.0f}, sum, false);
    }
  }
  if (__builtin_expect(!__any(sum != 0.0f), 1)) return false;  // (NaN is not 0 either)
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool lo = (y[i][j] & 0x7f80u) == 0x7f80u, hi = (y[i][j] & 0x7f800000u) == 0x7f800000u;
      bits |= (uint32_t)lo << 2 * j | (uint32_t)hi << (2 * j + 1);
      y[i][j] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
    }
    bad[at(i)] = (unsigned char)bits;
    *reinterpret_cast<u32x4*>(vl + 16 * at(i)) = y[i];
  }
  return true;
}

template <int NW, int DK, int DV>
struct FastCfg {
  static constexpr int BM = 32 * NW;
  static constexpr int NT = 64 * NW;
  static constexpr int KB = kTileKeys * DK * 2, VB = kTileKeys * DV * 2;  // bytes of a tile
  static constexpr int NK = KB / 1024 / NW, NV = VB / 1024 / NW;          // 1 KB copies of a wave
  static constexpr int LDS = 2 * (KB + VB);
  static_assert(NK * NW * 1024 == KB && NV * NW * 1024 == VB, "whole copies");
};

template <int NW, int DK, int DV>
__global__ __launch_bounds__(64 * NW, 2) void kda_attn_kernel(AttnParams p, unsigned tiles) {
  using C = FastCfg<NW, DK, DV>;
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  __shared__ unsigned char bad[C::VB / 16];  // a bit for each value of a tile that is not finite
  __shared__ int some[NW];
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), c = lane % 32, hf = lane / 32;
  int h, hk, at;
  Part s;
  if (!pair_of(p, tiles, h, hk, at) || !part_of<C::BM>(p, at, s)) return;
  const int row = s.r0 + 32 * wave + c;  // this lane's query
  const int shift = s.nk - s.nq;
  const int limit = row < s.nq ? row + shift + 1 : 0;
  const int last = min(s.r0 + C::BM, s.nq) + shift;                       // keys of the workgroup
  const bool live = s.r0 + 32 * wave < s.nq;                               // whether the wave has queries
  const int wlast = live ? min(s.r0 + 32 * wave + 32, s.nq) + shift : 0;   // its keys
  const int wfirst = s.r0 + 32 * wave + shift + 1;                        // its first query's
  const int ntiles = (last + kTileKeys - 1) / kTileKeys;

  const char* kg = reinterpret_cast<const char*>(static_cast<const __bf16*>(p.k) + (size_t)s.k0 * p.k_stride + (size_t)hk * DK);
  const char* vg = reinterpret_cast<const char*>(static_cast<const __bf16*>(p.v) + (size_t)s.k0 * p.v_stride + (size_t)hk * DV);
  // this lane's pieces of a tile: row and offset within the tile's rows
  const uint32_t krow = (uint32_t)(2 * p.k_stride), vrow = (uint32_t)(2 * p.v_stride);  // (bytes; the launch sees to it that a tile's fit)
  uint32_t koff[C::NK], voff[C::NV];
#pragma unroll
  for (int i = 0; i < C::NK; ++i) {
    const int e = (wave * C::NK + i) * 64 + lane, r = e / (DK / 8);
    koff[i] = r * krow + 16 * key_piece<DK>(r, e % (DK / 8));
  }
#pragma unroll
  for (int i = 0; i < C::NV; ++i) {
    const int e = (wave * C::NV + i) * 64 + lane, r = e / (DV / 8);
    voff[i] = r * vrow + 16 * value_piece<DV>(r, e % (DV / 8));
  }
  auto copy = [&](int t, auto buf) {
    char* kl = lds + buf * (C::KB + C::VB);
    char* vl = kl + C::KB;
    const char* kt = kg + (size_t)t * kTileKeys * krow;
    const char* vt = vg + (size_t)t * kTileKeys * vrow;
    if ((t + 1) * kTileKeys <= s.nk) {
#pragma unroll
      for (int i = 0; i < C::NK; ++i) copy16(kt, koff[i], kl + (wave * C::NK + i) * 1024);
#pragma unroll
      for (int i = 0; i < C::NV; ++i) copy16(vt, voff[i], vl + (wave * C::NV + i) * 1024);
    } else {  // rows behind the last key: that one again (nobody sees them)
      const int most = s.nk - 1 - t * kTileKeys;
#pragma unroll
      for (int i = 0; i < C::NK; ++i) {
        const int r = ((wave * C::NK + i) * 64 + lane) / (DK / 8);
        copy16(kt, koff[i] - max(r - most, 0) * krow, kl + (wave * C::NK + i) * 1024);
      }
#pragma unroll
      for (int i = 0; i < C::NV; ++i) {
        const int r = ((wave * C::NV + i) * 64 + lane) / (DV / 8);
        copy16(vt, voff[i] - max(r - most, 0) * vrow, vl + (wave * C::NV + i) * 1024);
      }
    }
  };

  using B0 = std::integral_constant<int, 0>;
  using B1 = std::integral_constant<int, 1>;
  if (ntiles > 0) copy(0, B0{});
  bf16x8 q[DK / 16];
  {
    const __bf16* x = static_cast<const __bf16*>(p.q) + (size_t)(s.q0 + min(row, s.nq - 1)) * p.q_stride + (size_t)h * DK + 8 * hf;
#pragma unroll
    for (int st = 0; st < DK / 16; ++st) q[st] = *reinterpret_cast<const bf16x8*>(x + 16 * st);
    if (p.scale < 0.0f) {  // (so that the largest score has the largest product)
#pragma unroll
      for (int st = 0; st < DK / 16; ++st) q[st] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, q[st]) ^ 0x80008000u);
    }
    // (waited for here: a wait at their use, inside the loop, would wait for the tiles' copies too)
#pragma unroll
    for (int st = 0; st < DK / 16; ++st) asm volatile("" : "+v"(q[st]));
  }
  // (not 0, which would make NaN of masked scores: 1e-30 of any product is as little)
  const float scale = fmaxf(__builtin_fabsf(p.scale) * kLog2e, 1e-30f);
  f32x16 o[DV / 32];
#pragma unroll
  for (int t = 0; t < DV / 32; ++t) o[t] = (f32x16)0.0f;
  float m = -__builtin_inff(), l = 0.0f;
  const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
  const int nfull = max(min((s.r0 + shift + 1) / kTileKeys, ntiles), 0);  // tiles that every query of the workgroup sees whole
  auto tile = [&](int t, auto buf) {
    tile_barrier();
    if (t + 1 < ntiles) copy(t + 1, std::integral_constant<int, 1 - decltype(buf)::value>{});
    const int k0 = t * kTileKeys;
    const char* kl = lds + buf * (C::KB + C::VB);
    char* vl = lds + buf * (C::KB + C::VB) + C::KB;
    bool odd = false;
    if (t >= nfull) {
      // Some queries do not see all of the tile: values that are not finite must not reach them as 0 v.  They are taken
      // out, and noted, a bit each.
      const bool any = take_out<C::NV>(vl, bad, [&](int i) { return (wave * C::NV + i) * 64 + lane; });
      if (lane == 0) some[wave] = any;
      lds_barrier();
#pragma unroll
      for (int w = 0; w < NW; ++w) odd |= some[w] != 0;
    }
    if (k0 >= wlast) return;  // (a wave that is done still copies and waits)
    f32x16 x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      x[u] = (f32x16)0.0f;
      const int r = 32 * u + c;
#pragma unroll
      for (int st = 0; st < DK / 16; ++st) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(kl + r * (2 * DK) + 16 * key_piece<DK>(r, 2 * st + hf));
        x[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[st], x[u], 0, 0, 0);
      }
    }
    const int rel = limit - k0 - 4 * hf;  // the query's keys in the tile, from this half's first on
    if (wfirst < k0 + kTileKeys) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) x[u][r] = 32 * u + 8 * (r / 4) + r % 4 >= rel ? -__builtin_inff() : x[u][r];
    }
    // the maximum of the raw products; it is taken over only when it has grown by 8 in log2, so that outputs
    // are rarely rescaled: powers stay below 2^8, and with them what fp32 sums and bf16 can tell apart
    float top = -__builtin_inff();
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, x[u][r]);
    top = half_max(top) * scale;
    if (__any(top > m + kSlack)) {
      const float now = fmaxf(m, top);
      const float keep = now == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= keep;
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) o[i] *= keep;
    }
    const float base = m == -__builtin_inff() ? 0.0f : -m;
    bf16x8 pt[4];
#pragma unroll
    for (int st = 0; st < 4; ++st) {
#pragma unroll
      for (int e = 0; e < 8; ++e) pt[st][e] = (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(x[st / 2][8 * (st % 2) + e], scale, base));
      // the sum of what the product with V takes: the rounded probabilities, two at a time
#pragma unroll
      for (int e = 0; e < 8; e += 2) l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{pt[st][e], pt[st][e + 1]}, ones, l, false);
    }
#pragma unroll
    for (int st = 0; st < 4; ++st)
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value_operand<DV>(vl, i, st, lane), pt[st], o[i], 0, 0, 0);
    if (__builtin_expect(odd, 0)) {  // outputs of queries that see a value that is not finite: NaN.  The values are counted by a product.
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) {
        f32x16 y = (f32x16)0.0f;
#pragma unroll 1
        for (int st = 0; st < 4; ++st) {
          bf16x8 n, see;
          counted<DV>(bad, i, st, lane, limit - k0, n, see, [&](int e) { return some[e / (64 * C::NV)]; });
          y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(n, see, y, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = y[r] > 0.0f ? __builtin_nanf("") : o[i][r];
      }
    }
  };
  for (int t = 0; t < ntiles; t += 2) {  // (two at a time: the buffers' addresses are constants)
    tile(t, B0{});
    if (t + 1 < ntiles) tile(t + 1, B1{});
  }
  l += __shfl_xor(l, 32);
  if (row >= s.nq) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  char* out = static_cast<char*>(p.o) + ((size_t)(s.q0 + row) * p.o_stride + (size_t)h * DV) * (p.o_f32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < DV / 32; ++i) {
    o[i] *= inv;
    if (p.o_f32) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<f32x4*>(out + 4 * (32 * i + 8 * r + 4 * hf)) = f32x4{o[i][4 * r], o[i][4 * r + 1], o[i][4 * r + 2], o[i][4 * r + 3]};
    } else {
      // halves exchange fours, so that each writes 8 neighbours: 16 bytes
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          a[e] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)o[i][8 * j + 2 * e], (__bf16)o[i][8 * j + 2 * e + 1]});
        const auto x = __builtin_amdgcn_permlane32_swap(a[0], a[2], false, false), y = __builtin_amdgcn_permlane32_swap(a[1], a[3], false, false);
        *reinterpret_cast<u32x4*>(out + 2 * (32 * i + 16 * j + 8 * hf)) = u32x4{x[0], y[0], x[1], y[1]};
      }
    }
  }
}

// ---- the same for few queries ---------------------------------------------------------------
// Where the workgroups above would not fill the compute units -- a short prompt, one prompt of few heads, or a few
// new tokens behind a long prefix -- a workgroup takes 32 queries, and each of its four waves every fourth tile of 32 keys,
// through two buffers of its own in LDS: no barrier until the waves are joined.  Bound by latency: 77 tokens of 8 heads of 64 5.1 us.
// 128 tokens of 32 heads of 128 behind 8,000 cached ones 64 us (0.26 PFLOP/s): 128 workgroups on 256 compute units, and with 131 KB of LDS
// a workgroup one wave a SIMD, whose exponentials and products nothing overlaps.

constexpr int kSplitWaves = 4, kSplitKeys = 32;
constexpr unsigned kFewTiles = 256;  // workgroups of it that fill the compute units

template <int DK, int DV>
__global__ __launch_bounds__(64 * kSplitWaves, 1) void kda_attn_split_kernel(AttnParams p, unsigned tiles) {
  constexpr int KB = kSplitKeys * DK * 2, VB = kSplitKeys * DV * 2, NK = KB / 1024, NV = VB / 1024;
  constexpr int RING = 2 * (KB + VB), JOIN = 32 * (DV + 4) * 4;  // bytes of a wave
  __shared__ __attribute__((aligned(1024))) char lds[kSplitWaves * (RING > JOIN ? RING : JOIN)];
  __shared__ unsigned char bads[kSplitWaves][VB / 16];
  __shared__ float sm[kSplitWaves][32], sl[kSplitWaves][32];
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), c = lane % 32, hf = lane / 32;
  int h, hk, at;
  Part s;
  if (!pair_of(p, tiles, h, hk, at) || !part_of<32>(p, at, s)) return;
  const int row = s.r0 + c, shift = s.nk - s.nq;
  const int limit = row < s.nq ? row + shift + 1 : 0;  // this lane's query's keys
  const int last = min(s.r0 + 32, s.nq) + shift;       // the workgroup's
  const int least = s.r0 + shift + 1;                  // what all of its queries see
  const int ntiles = (last + kSplitKeys - 1) / kSplitKeys;
  char* ring = lds + wave * RING;
  unsigned char* bad = bads[wave];

  const char* kg = reinterpret_cast<const char*>(static_cast<const __bf16*>(p.k) + (size_t)s.k0 * p.k_stride + (size_t)hk * DK);
  const char* vg = reinterpret_cast<const char*>(static_cast<const __bf16*>(p.v) + (size_t)s.k0 * p.v_stride + (size_t)hk * DV);
  const uint32_t krow = (uint32_t)(2 * p.k_stride), vrow = (uint32_t)(2 * p.v_stride);
  auto copy = [&](int t, int buf) {
    const char* kt = kg + (size_t)t * kSplitKeys * krow;
    const char* vt = vg + (size_t)t * kSplitKeys * vrow;
    const int most = s.nk - 1 - t * kSplitKeys;  // (rows behind the last key: that one again)
    char* to = ring + buf * (KB + VB);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int e = i * 64 + lane, r = e / (DK / 8);
      copy16(kt, (uint32_t)min(r, most) * krow + 16 * key_piece<DK>(r, e % (DK / 8)), to + i * 1024);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * 64 + lane, r = e / (DV / 8);
      copy16(vt, (uint32_t)min(r, most) * vrow + 16 * value_piece<DV>(r, e % (DV / 8)), to + KB + i * 1024);
    }
  };
  if (wave < ntiles) copy(wave, 0);
  bf16x8 q[DK / 16];
  const __bf16* qx = static_cast<const __bf16*>(p.q) + (size_t)(s.q0 + min(row, s.nq - 1)) * p.q_stride + (size_t)h * DK + 8 * hf;
#pragma unroll
  for (int st = 0; st < DK / 16; ++st) q[st] = *reinterpret_cast<const bf16x8*>(qx + 16 * st);
  if (p.scale < 0.0f) {  // (so that the largest score has the largest product)
#pragma unroll
    for (int st = 0; st < DK / 16; ++st) q[st] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, q[st]) ^ 0x80008000u);
  }
#pragma unroll
  for (int st = 0; st < DK / 16; ++st) asm volatile("" : "+v"(q[st]));  // (waited for here, not inside the loop)
  const float scale = fmaxf(__builtin_fabsf(p.scale) * kLog2e, 1e-30f);
  const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
  f32x16 o[DV / 32];
#pragma unroll
  for (int t = 0; t < DV / 32; ++t) o[t] = (f32x16)0.0f;
  float m = -__builtin_inff(), l = 0.0f;
  int buf = 0;
  for (int t = wave; t < ntiles; t += kSplitWaves, buf ^= 1) {
    // the reads of the buffer that is filled next are done; then this tile's copies have landed
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (t + kSplitWaves < ntiles) {
      copy(t + kSplitWaves, buf ^ 1);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NK + NV) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    const int k0 = t * kSplitKeys;
    const char* kl = ring + buf * (KB + VB);
    char* vl = ring + buf * (KB + VB) + KB;
    const int rel = limit - k0 - 4 * hf;
    const bool cut = k0 + kSplitKeys > least;
    bool odd = false;
    if (cut) {  // as above: values that are not finite are taken out and noted
      odd = take_out<NV>(vl, bad, [&](int i) { return i * 64 + lane; });
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    f32x16 x = (f32x16)0.0f;
#pragma unroll
    for (int st = 0; st < DK / 16; ++st) {
      const bf16x8 a = *reinterpret_cast<const bf16x8*>(kl + c * (2 * DK) + 16 * key_piece<DK>(c, 2 * st + hf));
      x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[st], x, 0, 0, 0);
    }
    if (cut) {
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = 8 * (r / 4) + r % 4 >= rel ? -__builtin_inff() : x[r];
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, x[r]);
    top = half_max(top) * scale;
    if (__any(top > m + kSlack)) {
      const float now = fmaxf(m, top);
      const float keep = now == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= keep;
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) o[i] *= keep;
    }
    const float base = m == -__builtin_inff() ? 0.0f : -m;
    bf16x8 pt[2];
#pragma unroll
    for (int st = 0; st < 2; ++st) {
#pragma unroll
      for (int e = 0; e < 8; ++e) pt[st][e] = (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(x[8 * st + e], scale, base));
#pragma unroll
      for (int e = 0; e < 8; e += 2) l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{pt[st][e], pt[st][e + 1]}, ones, l, false);
    }
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value_operand<DV>(vl, i, st, lane), pt[st], o[i], 0, 0, 0);
    if (__builtin_expect(odd, 0)) {
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) {
        f32x16 y = (f32x16)0.0f;
#pragma unroll 1
        for (int st = 0; st < 2; ++st) {
          bf16x8 n, see;
          counted<DV>(bad, i, st, lane, limit - k0, n, see, [](int) { return 1; });
          y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(n, see, y, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = y[r] > 0.0f ? __builtin_nanf("") : o[i][r];
      }
    }
  }

  // join the waves, in the memory of the tiles
  l += __shfl_xor(l, 32);
  __syncthreads();
  float* so = reinterpret_cast<float*>(lds);
  if (hf == 0) sm[wave][c] = m, sl[wave][c] = l;
#pragma unroll
  for (int i = 0; i < DV / 32; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<f32x4*>(so + (wave * 32 + c) * (DV + 4) + 32 * i + 8 * r + 4 * hf) =
          f32x4{o[i][4 * r], o[i][4 * r + 1], o[i][4 * r + 2], o[i][4 * r + 3]};
  __syncthreads();
  for (int i = tid; i < 32 * DV / 4; i += 64 * kSplitWaves) {
    const int r = i / (DV / 4), e = 4 * (i % (DV / 4));
    if (s.r0 + r >= s.nq) break;
    float top = sm[0][r];
#pragma unroll
    for (int w = 1; w < kSplitWaves; ++w) top = fmaxf(top, sm[w][r]);
    const float base = top == -__builtin_inff() ? 0.0f : top;
    f32x4 y = (f32x4)0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kSplitWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(sm[w][r] - base);
      sum += f * sl[w][r];
      y += f * *reinterpret_cast<const f32x4*>(so + (w * 32 + r) * (DV + 4) + e);
    }
    store4(p, (size_t)(s.q0 + s.r0 + r) * p.o_stride + (size_t)h * DV + e, y * (sum == 0.0f ? 0.0f : 1.0f / sum));
  }
}

template <int BM>
unsigned tiles_of(const AttnParams& p) {
  return p.cu_q ? (unsigned)(p.total_q / BM + p.N) : (unsigned)((p.total_q / p.N + BM - 1) / BM * p.N);
}

template <int DK, int DV>
hipError_t launch_fast(const AttnParams& p, hipStream_t s) {
  constexpr int NW = 4;
  // Workgroups of 32 queries, whose waves divide the keys, against those of 128, whose waves divide the queries.  By what is
  // measured the first take 4.9 us + 7.1e-3 (600 + keys of a query) for each time that they fill the compute units, the second,
  // while they do not fill them, 5 us + 18.5e-3 for each key of a sequence; with heads of 64 it is 3.5e-3 (400 + keys) and 12.5e-3.
  // us, heads of 128: 77 tokens of 8 heads 6.4 / 7.3; 1,000 tokens of 16 heads 19 / 24, of 32 37 / 26; 3,000 of 8 49 / 59; 8
  // sequences of 300 of 8 heads 21 / 12; behind 8,000 cached tokens 128 of 32 heads 64 / 148.  Heads of 64: 2,000 tokens of
  // 16 heads 24 / 30, 8 sequences of 300 of 8 heads 10.9 / 8.3.
  const unsigned few = tiles_of<32>(p);
  const long long groups = (long long)few * p.Hq, nq = p.total_q / p.N, nk = p.total_k / p.N, seen = nk - std::min(nq, nk) / 2;
  constexpr int FIXED = 200 + (DK + DV) * 25 / 16, TIMES = 1178 - 2 * (DK + DV);  // 600 and 666 = 2.6 kFewTiles; 400 and 922
  if (groups <= kFewTiles || groups * (FIXED + seen) <= TIMES * nk) {
    hipLaunchKernelGGL((kda_attn_split_kernel<DK, DV>), grid_of(p, few), dim3(64 * kSplitWaves), 0, s, p, few);
    return hipGetLastError();
  }
  const unsigned tiles = tiles_of<32 * NW>(p);
  hipLaunchKernelGGL((kda_attn_kernel<NW, DK, DV>), grid_of(p, tiles), dim3(64 * NW), 0, s, p, tiles);
  return hipGetLastError();
}

template <typename IO, int DK, int DV>
hipError_t launch_plain(const AttnParams& p, hipStream_t s) {
  // 32 queries a workgroup take half as much from the L2, but want long sequences, and enough workgroups.  Against 16, us,
  // fp32: 3,000 tokens of 8 + 2 heads of 128 196 / 242, 1,000 (256 workgroups) 44 / 51, 512 behind 1,488 of 16 heads 78 / 106;
  // 20 sequences of 500 196 / 201; 10 of 300 62 / 56, 300 (80 workgroups) 23 / 16; of 8 + 8 heads of 64, 8 of 600 55 / 57.
  const unsigned half = tiles_of<32>(p);
  if (p.total_k / p.N >= 512 && (unsigned long long)half * p.Hq >= 256) {
    hipLaunchKernelGGL((kda_attn_plain_kernel<IO, DK, DV, 2>), grid_of(p, half), dim3(64 * kPlainWaves), 0, s, p, half);
    return hipGetLastError();
  }
  const unsigned tiles = tiles_of<16>(p);
  hipLaunchKernelGGL((kda_attn_plain_kernel<IO, DK, DV, 1>), grid_of(p, tiles), dim3(64 * kPlainWaves), 0, s, p, tiles);
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
  // (64 rows of keys or values have to lie within 2^31 bytes)
  if (io_dtype == 1 && p.dk % 64 == 0 && p.dv % 64 == 0 && std::max(p.k_stride, p.v_stride) < (1LL << 24)) {
    if (p.dk == 128) return p.dv == 128 ? launch_fast<128, 128>(p, s) : launch_fast<128, 64>(p, s);
    return p.dv == 128 ? launch_fast<64, 128>(p, s) : launch_fast<64, 64>(p, s);
  }
  return io_dtype == 1 ? pick_dk<__bf16>(p, s) : pick_dk<float>(p, s);
}

}  // namespace kda
