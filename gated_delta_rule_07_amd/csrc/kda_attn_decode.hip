// Attention of one or a few tokens of each sequence over its cached keys and values, for gfx950.
//
//   o = sum_j p_j v_j,  p = softmax_j(scale q . k_j),  k_j, v_j = scale of their page x code
//
// Every cached byte is read once and multiplied with the K G queries (K tokens, G heads of a group)
// that share it, 16 of them at a time, so the call is bound by those bytes.  A unit is one sequence's head and 16 query rows.
// Short ones are taken whole, a workgroup each.  Else the work is cut into granules of 128 keys, and every workgroup takes an
// equal run of them, whatever the sequences' lengths: a run that holds a unit whole writes its output, others leave (o, m, l) in
// the workspace for a second kernel.  Within a workgroup each wave streams its own 32-key tiles from
// memory into registers -- no LDS and no barrier until a unit ends:
//   S^T = K Q^T with a lane holding 16 bytes of a key's row; P^T as it comes out is the operand of
//   O^T = V^T P^T, whose other operand wants 8 keys' values of one channel in a lane: a lane loads
//   8 channels of 8 keys and transposes them in registers (byte permutes, then the conversion to bf16).
// Codes convert to bf16 exactly; the page's scales multiply scores and probabilities instead.
// fp32 queries are split into three bf16 terms, and so are their probabilities: 24 bits on bf16 matrix cores.
// With bf16 queries the probabilities are two bf16 terms, 16 bits: one took bf16 outputs from 0.17% of the definition, their own
// rounding, to 0.23%.  Against one term long sequences take the same time, short ones up to 0.7 us more (4 of 1,000 tokens 12.0
// us for 11.4, 8 of 2,000 19.1 for 18.1).  Maxima, sums and outputs are fp32 always.
// Measured, 32 + 8 heads of 128 in e4m3: 256 sequences of up to 9,000 tokens 465 us (5.6 TB/s, where reads alone reach 5.2 to 6.3
// and copies 5.4), 4 drafts behind 1,000,003 tokens 362 us (5.6), of which the second kernel takes 7 and 8; one sequence of 903
// tokens of 8 + 2 heads of 64 9.0 us (fp32 queries: the 256 sequences 510 us, the one 10.0), bound by the latency of a chain of loads: lengths, page numbers, keys.  Vector
// instructions (conversions, byte permutes) take 32% of the cycles, the matrix cores 11%.  Slower: four waves a SIMD (they
// spill), 768 workgroups that share the granules (484 and 374 us).
#include <algorithm>

#include "kda_kv_device.h"

namespace kda {
namespace {

constexpr int kTile = 32;         // keys of a wave's turn
constexpr int kWaves = 4;         // waves of a workgroup that shares the granules (and of a join)
constexpr int kMoreWaves = 8;     // of one that takes a unit whole where there are few units
constexpr int kWorkers = 512;     // workgroups that share the granules
constexpr int kLeastRun = 2;      // granules a workgroup takes at least
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;


__host__ __device__ inline int columns(int K, int G) { return (K * G + kAttnColumns - 1) / kAttnColumns; }

// The workspace: for each worker two partial results, then the units that have to be joined.
struct Join {
  int unit, last, slot, unused;  // unit = (b H + head) column tiles + column tile, or -1; the worker that ends it; which part it is here
};
__host__ __device__ inline size_t part_floats(int dv) { return (size_t)kAttnColumns * (dv + 2); }

struct DecodePlan {
  AttnDecodeParams p;
  int G, CT, workers;
  float* parts;  // [workers][2][16 dv + 16 m + 16 l]
  Join* joins;   // [workers]
};

__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); }
__device__ __forceinline__ uint32_t bf16_of_e4m3(uint32_t w, bool hi) {
  return __builtin_bit_cast(uint32_t, hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                         : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}

// Four outputs from element `at` of o on.
__device__ __forceinline__ void store4(const AttnDecodeParams& p, size_t at, const f32x4& y) {
  if (p.o_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(p.o) + at) = y;
  else *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(p.o) + at) = bf16x4{(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
}

// All ones in the bytes (e4m3) or halves (bf16) of w that are not finite.
template <bool E4>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  uint32_t r = 0;
  if constexpr (E4) {
#pragma unroll
    for (int b = 0; b < 4; ++b) r |= (w >> 8 * b & 0x7fu) == 0x7fu ? 0xffu << 8 * b : 0u;
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) r |= (w >> 16 * b & 0x7f80u) == 0x7f80u ? 0xffffu << 16 * b : 0u;
  }
  return r;
}

// Tokens that rows of sequence b attend to, and its granules (0: no row of the table, nothing is written).
__device__ __forceinline__ int tokens_of(const AttnDecodeParams& p, int b) {
  return min(max(p.lens[b], 0), p.c.width * p.c.page_tokens);
}
template <int NW>
__device__ __forceinline__ int granules_of(const AttnDecodeParams& p, int b) {
  const int row = p.c.rows ? p.c.rows[b] : b, n = tokens_of(p, b);
  return row < 0 || row >= p.c.n_rows ? 0 : max(1, (n + NW * kTile - 1) / (NW * kTile));
}

template <bool E4, int DK, int DV>
struct Tile {
  static constexpr int NK = DK * (E4 ? 1 : 2) / 64;  // 16-byte loads of a lane for 16 keys
  static constexpr int NV = DV / 16;                 // channels of a lane
  static constexpr int VW = NV * (E4 ? 1 : 2) / 4;   // dwords of a lane and key
  u32x4 k[2][NK];
  uint32_t v[8][VW];
  float ks[2], vs[2];
  bool there[2];  // whether its halves have pages
};

// The largest of a column's values (in lanes 16 apart).
__device__ __forceinline__ float column_max(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto y = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a = y[0], b = y[1];  // (a bit cast of y[1] itself gives y[0])
  const float z = fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
  const uint32_t w = __builtin_bit_cast(uint32_t, z);
  const auto t = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  const uint32_t c = t[0], d = t[1];
  return fmaxf(__builtin_bit_cast(float, c), __builtin_bit_cast(float, d));
}

// (at least three waves a SIMD are asked for where the registers do without spilling: 110 to 152 of them here; the instances that
// are asked for two have up to 168 with bf16 queries, so three too, and up to 203 with fp32 ones)
template <int NW, int NT, bool E4, int DK, int DV>
__global__ __launch_bounds__(64 * NW, NW == kWaves && NT == 1 && E4 ? 3 : 2) void kda_attn_decode_kernel(DecodePlan a) {
  constexpr int kThreads = 64 * NW, kGranule = NW * kTile;
  using T = Tile<E4, DK, DV>;
  constexpr int NM = DV / 16, NS = DK / 32;
  constexpr int NP = NT == 1 ? 2 : NT;         // bf16 terms of a probability
  constexpr int ES = E4 ? 1 : 2, CW = 4 / ES;  // bytes of an element, elements of a dword
  __shared__ __attribute__((aligned(16))) float so[NW][kAttnColumns][DV + 4];
  __shared__ float sm[NW][kAttnColumns], sl[NW][kAttnColumns];
  __shared__ int swave[NW];
  extern __shared__ int prefix[];  // [B + 1]: granules of the sequences before
  const AttnDecodeParams& p = a.p;
  const KvCache& cache = p.c;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), col = lane % 16, g = lane / 16;
  const int H = cache.H, units = a.CT * H, pt = cache.page_tokens, lg = 31 - __builtin_clz(pt);
  const float scale = p.scale * kLog2e;

  long long at, end, mine;  // this workgroup's granules; where its run begins
  const bool whole = a.workers == 0;
  int b = 0;
  if (whole) {
    b = blockIdx.x / units;
    at = mine = 0;
    end = granules_of<NW>(p, b);
  } else {
    const int each = (p.B + kThreads - 1) / kThreads, i0 = min(tid * each, p.B), i1 = min(i0 + each, p.B);
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += granules_of<NW>(p, i);
    int run = sum;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const int up = __shfl_up(run, m);
      if (lane >= m) run += up;
    }
    if (lane == 63) swave[wave] = run;
    __syncthreads();
    int before = run - sum;
    for (int w = 0; w < wave; ++w) before += swave[w];
    for (int i = i0; i < i1; ++i) {
      prefix[i] = before;
      before += granules_of<NW>(p, i);
    }
    if (tid == kThreads - 1) prefix[p.B] = before;
    __syncthreads();
    const long long total = (long long)prefix[p.B] * units;
    const long long per = max((total + a.workers - 1) / a.workers, (long long)kLeastRun);
    at = mine = min(per * blockIdx.x, total);
    end = min(at + per, total);
    if (tid == 0) a.joins[blockIdx.x] = Join{-1, 0, 0, 0};
    if (at < end) b = last_at_most(p.B, at, [&](int i) { return (long long)prefix[i] * units; });
  }

  while (at < end) {
    // the unit that granule `at` belongs to, and this workgroup's granules [g0, g1) of its n
    int unit, n, g0, g1;
    if (whole) {
      unit = blockIdx.x % units;
      g0 = 0;
      g1 = n = (int)end;
    } else {
      while ((long long)prefix[b + 1] * units <= at) ++b;  // (sequences without a granule)
      n = prefix[b + 1] - prefix[b];
      const long long off = at - (long long)prefix[b] * units;
      unit = (int)(off / n);
      g0 = (int)(off % n);
      g1 = (int)min((long long)n, g0 + (end - at));
    }
    const int h = unit / a.CT, ct = unit % a.CT;
    const int row = __builtin_amdgcn_readfirstlane(cache.rows ? cache.rows[b] : b);
    const int* pages = cache.table + (size_t)row * cache.width;
    const int len = __builtin_amdgcn_readfirstlane(tokens_of(p, b));
    const int cc = kAttnColumns * ct + col, tok = cc / a.G, head = h * a.G + cc % a.G;
    const bool live = tok < p.K;
    const int limit = live ? len - p.K + 1 + tok : len;
    const int least = len - p.K + 1;  // what every row attends to

    // queries as B operands (NT terms): with 16-byte key loads a lane's values are 16 of every 64 in e4m3, 8 of every 32 in bf16
    bf16x8 q[NT][NS];
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      const int i0 = E4 ? 64 * (st / 2) + 16 * g + 8 * (st % 2) : 32 * st + 8 * g;
      const size_t x = (((size_t)b * p.K + (live ? tok : 0)) * p.Hq + (live ? head : 0)) * DK + i0;
      if constexpr (NT == 1) {
        q[0][st] = *reinterpret_cast<const bf16x8*>(static_cast<const __bf16*>(p.q) + x);
      } else {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = static_cast<const float*>(p.q)[x + e];
#pragma unroll
        for (int n3 = 0; n3 < NT; ++n3)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __bf16 t = (__bf16)f[e];
            q[n3][st][e] = t;
            f[e] -= (float)t;
          }
      }
    }
    f32x4 o[NM];
#pragma unroll
    for (int t = 0; t < NM; ++t) o[t] = (f32x4)0.0f;
    float m = -__builtin_inff(), l = 0.0f;

    // Offsets of a lane within a half tile's keys and values; the rest of an address is the wave's.
    const uint32_t koff = (uint32_t)(col * DK * ES + 16 * g), voff = (uint32_t)(4 * g * DV * ES + col * T::VW * 4);
    const size_t kat = kv_keys(cache, h), vat = kv_values(cache, h), sat = kv_scales(cache);
    const int kend = min(g1 * kGranule, len);
    // The pages of a tile's halves, -1 where there is none (behind the sequence a row may name any page).  64 entries of the
    // row at a time lie in the wave's lanes: a load for each tile would be waited for, and with it all tiles in flight.
    struct Pages {
      int p[2];
    };
    int first = -64, entries = 0;
    auto pages_of = [&](int k0) {
      Pages r;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        r.p[u] = -1;
        if (k0 + 16 * u < kend) {
          const int i = (k0 + 16 * u) >> lg;
          if (i >= first + 64) {
            first = i;
            entries = i + lane < cache.width ? pages[i + lane] : -1;
          }
          const int page = __builtin_amdgcn_readlane(entries, i - first);
          r.p[u] = page < cache.n_pages ? page : -1;
        }
      }
      return r;
    };
    auto load = [&](int k0, const Pages& pg) {
      T t;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int slot = (k0 + 16 * u) & (pt - 1);
        t.there[u] = pg.p[u] >= 0;
        const char* base = cache.pool + (size_t)max(pg.p[u], 0) * cache.page_bytes;
        const char* kp = base + kat + (uint32_t)(slot * DK * ES);
        const char* vp = base + vat + (uint32_t)(slot * DV * ES);
#pragma unroll
        for (int i = 0; i < T::NK; ++i) t.k[u][i] = *reinterpret_cast<const u32x4*>(kp + (koff + 64 * i));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const char* x = vp + (voff + r * DV * ES);
          if constexpr (T::VW == 1) {
            t.v[4 * u + r][0] = *reinterpret_cast<const uint32_t*>(x);
          } else if constexpr (T::VW == 2) {
            const u32x2 y = *reinterpret_cast<const u32x2*>(x);
            t.v[4 * u + r][0] = y[0], t.v[4 * u + r][1] = y[1];
          } else {
            const u32x4 y = *reinterpret_cast<const u32x4*>(x);
#pragma unroll
            for (int i = 0; i < 4; ++i) t.v[4 * u + r][i] = y[i];
          }
        }
        t.ks[u] = t.vs[u] = 1.0f;
        if constexpr (E4) {
          const float* sc = reinterpret_cast<const float*>(base + sat);
          t.ks[u] = sc[h];
          t.vs[u] = sc[H + h];
        }
      }
      return t;
    };

    auto compute = [&](int k0, T& cur) {
      // scores of 32 keys
      f32x4 x[2] = {(f32x4)0.0f, (f32x4)0.0f};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int st = 0; st < NS; ++st) {
          u32x4 w;
          if constexpr (E4) {
            const uint32_t lo = cur.k[u][st / 2][2 * (st % 2)], hi = cur.k[u][st / 2][2 * (st % 2) + 1];
            w = u32x4{bf16_of_e4m3(lo, false), bf16_of_e4m3(lo, true), bf16_of_e4m3(hi, false), bf16_of_e4m3(hi, true)};
          } else {
            w = cur.k[u][st];
          }
#pragma unroll
          for (int n3 = NT - 1; n3 >= 0; --n3)
            x[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), q[n3][st], x[u], 0, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) x[u] *= cur.ks[u] * scale;
      const bool partial = k0 + kTile > least || !cur.there[0] || !cur.there[1];  // (the same for the wave)
      if (partial) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          cur.vs[u] = cur.there[u] ? cur.vs[u] : 1.0f;  // (0 times another page's scale could be NaN)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (!cur.there[u] || k0 + 16 * u + 4 * g + r >= limit) x[u][r] = -__builtin_inff();
            if (!cur.there[u] || k0 + 16 * u + 4 * g + r >= len) {  // what nobody sees may hold anything
#pragma unroll
              for (int i = 0; i < T::VW; ++i) cur.v[4 * u + r][i] = 0;
            }
          }
        }
      }
      float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])), fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
      top = column_max(top);
      // (taken over only when it has grown by 8 in log2: powers stay below 2^8, and outputs are rarely rescaled)
      if (__any(top > m + kSlack)) {
        const float now = fmaxf(m, top);
        const float keep = now == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - now);
        m = now;
        l *= keep;
#pragma unroll
        for (int t = 0; t < NM; ++t) o[t] *= keep;
      }
      const float base = m == -__builtin_inff() ? 0.0f : m;
      bf16x8 pt8[NP];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float y = __builtin_amdgcn_exp2f(x[u][r] - base);
          l += y;
          float z = y * cur.vs[u];
#pragma unroll
          for (int n3 = 0; n3 < NP; ++n3) {
            const __bf16 t = (__bf16)z;
            pt8[n3][4 * u + r] = t;
            if (n3 + 1 < NP) z -= (float)t;
          }
        }
      // V^T: 8 keys of channel NV col + t in a lane, a dword of each key's channels at a time
      auto values = [&](int i, bf16x8* vt) {
        u32x4 w[CW];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t x0 = cur.v[2 * r][i], x1 = cur.v[2 * r + 1][i];
          if constexpr (E4) {
            const uint32_t lo = perm(x1, x0, 0x05010400u), hi = perm(x1, x0, 0x07030602u);
            w[0][r] = bf16_of_e4m3(lo, false);
            w[1][r] = bf16_of_e4m3(lo, true);
            w[2][r] = bf16_of_e4m3(hi, false);
            w[3][r] = bf16_of_e4m3(hi, true);
          } else {
            w[0][r] = perm(x1, x0, 0x05040100u);
            w[1][r] = perm(x1, x0, 0x07060302u);
          }
        }
#pragma unroll
        for (int e = 0; e < CW; ++e) vt[e] = __builtin_bit_cast(bf16x8, w[e]);
      };
      if (partial && p.K > 1) {
        // Values that are not finite must not reach, as 0 v, drafted tokens that do not see them: they are taken
        // out, and counted for each token that does see them: its outputs become NaN.
        bool odd = false;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < T::VW; ++i) odd |= not_finite<E4>(cur.v[j][i]) != 0;
        if (__builtin_expect(__any(odd), 0)) {
          bf16x8 see;
#pragma unroll
          for (int e = 0; e < 8; ++e) see[e] = (__bf16)(k0 + 16 * (e / 4) + 4 * g + e % 4 < limit ? 1.0f : 0.0f);
#pragma unroll
          for (int i = 0; i < T::VW; ++i) {
            uint32_t keep[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // their bits in place of the values
              const uint32_t bad = not_finite<E4>(cur.v[j][i]);
              keep[j] = cur.v[j][i] & ~bad;
              cur.v[j][i] = bad & (E4 ? 0x38383838u : 0x3f803f80u);  // 1.0 where it is not finite
            }
            bf16x8 n[CW];
            values(i, n);
#pragma unroll
            for (int e = 0; e < CW; ++e) {
              const f32x4 y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n[e], see, (f32x4)0.0f, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < 4; ++r) o[CW * i + e][r] = y[r] > 0.0f ? __builtin_nanf("") : o[CW * i + e][r];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) cur.v[j][i] = keep[j];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < T::VW; ++i) {
        bf16x8 vt[CW];
        values(i, vt);
#pragma unroll
        for (int e = 0; e < CW; ++e)
#pragma unroll
          for (int n3 = NP - 1; n3 >= 0; --n3)
            o[CW * i + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt[e], pt8[n3], o[CW * i + e], 0, 0, 0);
      }
    };
    int k0 = g0 * kGranule + kTile * wave;
    // (the waves of a SIMD overlap one's loads with another's work: tiles loaded ahead take registers and make the code longer,
    // and were slower: 447 against 431 us on 128 sequences of up to 6,000 tokens in bf16, 10.0 against 9.3 on one of 903)
    Pages pg = pages_of(k0);
    for (; k0 < kend; k0 += kGranule) {
      T cur = load(k0, pg);
      pg = pages_of(k0 + kGranule);  // (a turn before their tile's loads need them)
      compute(k0, cur);
    }

    // join the waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) sm[wave][col] = m, sl[wave][col] = l;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int t = 0; t < NM; t += 4)
        *reinterpret_cast<f32x4*>(&so[wave][col][NM * (4 * g + r) + t]) = f32x4{o[t][r], o[t + 1][r], o[t + 2][r], o[t + 3][r]};
    __syncthreads();
    const bool complete = g0 == 0 && g1 == n;
    float* part = nullptr;
    if (!complete) {
      part = a.parts + (2 * (size_t)blockIdx.x + (at == mine ? 0 : 1)) * part_floats(DV);
      if (tid == 0 && g0 == 0) {  // the unit begins here and ends with another worker
        const long long per = max(((long long)prefix[p.B] * units + a.workers - 1) / a.workers, (long long)kLeastRun);
        a.joins[blockIdx.x] = Join{b * units + unit, (int)((at + n - 1) / per), at == mine ? 0 : 1, 0};
      }
    }
    for (int i = tid; i < kAttnColumns * DV / 4; i += kThreads) {
      const int c = i / (DV / 4), d = 4 * (i % (DV / 4));
      float top = sm[0][c];
#pragma unroll
      for (int w = 1; w < NW; ++w) top = fmaxf(top, sm[w][c]);
      const float base = top == -__builtin_inff() ? 0.0f : top;
      f32x4 y = (f32x4)0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = __builtin_amdgcn_exp2f(sm[w][c] - base);
        sum += f * sl[w][c];
        y += f * *reinterpret_cast<const f32x4*>(&so[w][c][d]);
      }
      if (!complete) {
        *reinterpret_cast<f32x4*>(part + c * DV + d) = y;
        if (d == 0) part[kAttnColumns * DV + c] = top, part[kAttnColumns * (DV + 1) + c] = sum;
        continue;
      }
      const int c2 = kAttnColumns * ct + c, tk = c2 / a.G;
      if (tk >= p.K) continue;
      y *= sum == 0.0f ? 0.0f : 1.0f / sum;
      store4(p, (((size_t)b * p.K + tk) * p.Hq + h * a.G + c2 % a.G) * DV + d, y);
    }
    __syncthreads();
    at += g1 - g0;
  }
}

// Joins the parts of a unit that several workers share: a workgroup a row of queries.  DV / 4 lanes hold a row, the
// groups of lanes take the parts in turn, so that the parts of even a long unit are in flight together.
template <int DV>
__global__ __launch_bounds__(256) void kda_attn_join_kernel(DecodePlan a) {
  constexpr int NL = DV / 4, NG = 256 / NL, AHEAD = 8;
  constexpr int NP = (kWorkers + 255) / 256;  // parts of a thread
  __shared__ float sf[256 * NP], st[4], sl[4];
  __shared__ __attribute__((aligned(16))) float sy[NG][DV];
  const int w0 = blockIdx.x, tid = threadIdx.x, lane = tid % 64, c = blockIdx.y, e = 4 * (tid % NL), gr = tid / NL;
  const Join j = a.joins[w0];
  if (j.unit < 0) return;
  const AttnDecodeParams& p = a.p;
  const int units = a.CT * p.c.H, b = j.unit / units, h = j.unit % units / a.CT, ct = j.unit % a.CT;
  const int c2 = kAttnColumns * ct + c, tk = c2 / a.G, n = j.last - w0 + 1;
  if (tk >= p.K) return;
  // worker w0's part is its first or its second, the others' their first
  auto part = [&](int i) { return a.parts + (2 * (size_t)(w0 + i) + (i == 0 ? j.slot : 0)) * part_floats(DV); };
  // thread i has the maxima and sums of the parts i, i + 256, ..; the first outputs are on their way meanwhile
  float most[NP], sums[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = tid + 256 * k;
    const float* x = part(min(i, n - 1)) + kAttnColumns * DV + c;
    most[k] = i < n ? x[0] : -__builtin_inff();
    sums[k] = i < n ? x[kAttnColumns] : 0.0f;
  }
  auto output = [&](int i) { return *reinterpret_cast<const f32x4*>(part(i) + c * DV + e); };
  f32x4 first[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) first[k] = output(min(gr + k * NG, n - 1));
  float top = most[0];
#pragma unroll
  for (int k = 1; k < NP; ++k) top = fmaxf(top, most[k]);
#pragma unroll
  for (int m = 1; m < 64; m *= 2) top = fmaxf(top, __shfl_xor(top, m));
  if (lane == 0) st[tid / 64] = top;
  __syncthreads();
  top = fmaxf(fmaxf(st[0], st[1]), fmaxf(st[2], st[3]));
  const float base = top == -__builtin_inff() ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const float f = __builtin_amdgcn_exp2f(most[k] - base);
    sf[tid + 256 * k] = f;
    sum += f * sums[k];
  }
  __syncthreads();
  f32x4 y = (f32x4)0.0f;
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (gr + k * NG < n) y += sf[gr + k * NG] * first[k];
#pragma unroll 8
  for (int i = gr + AHEAD * NG; i < n; i += NG) y += sf[i] * output(i);
#pragma unroll
  for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
  if (lane == 0) sl[tid / 64] = sum;
  *reinterpret_cast<f32x4*>(&sy[gr][e]) = y;
  __syncthreads();
  if (tid >= NL) return;
  sum = sl[0] + sl[1] + sl[2] + sl[3];
#pragma unroll
  for (int i = 1; i < NG; ++i) y += *reinterpret_cast<const f32x4*>(&sy[i][e]);
  store4(p, (((size_t)b * p.K + tk) * p.Hq + h * a.G + c2 % a.G) * DV + e, y * (sum == 0.0f ? 0.0f : 1.0f / sum));
}

// Whether a call takes its units whole, a workgroup each: no workspace and no second launch.  It knows what rows of the table
// hold, not how long the sequences are: longer rows are shared, lest one long sequence among short ones be one workgroup's.
// With 32 + 8 heads of 128 in e4m3, whole against shared, us: 1 sequence (8 units) of 1,000 tokens 11.7 / 12.3, of 1,500 15.1 /
// 12.3; 4 of 1,000 12.0 / 12.9, of 1,500 15.6 / 14.1; 8 of 1,500 16.0 / 16.0, of 2,000 19.2 / 18.2; 16 of 2,000 19.4 / 22.9, of
// 4,000 36.7 / 36.0; 20 of 4,000 38 / 45; 64 of 4,000 92 / 96; 256 of 300 to 9,000 512 / 471.
bool takes_whole(long long tokens, long long units) {
  return tokens <= 1280 || (tokens <= 2048 && units >= 64) || (tokens <= 4096 && units >= 128);
}
bool takes_whole(int B, int K, int Hq, int H, int page_tokens, int width) {
  return takes_whole((long long)page_tokens * width, (long long)B * columns(K, Hq / H) * H);
}

template <int NT, bool E4, int DK, int DV>
hipError_t launch_one(const AttnDecodeParams& p, hipStream_t s) {
  DecodePlan a;
  a.p = p;
  a.G = p.Hq / p.c.H;
  a.CT = columns(p.K, a.G);
  const bool whole = takes_whole(p.B, p.K, p.Hq, p.c.H, p.c.page_tokens, p.c.width);
  a.workers = whole ? 0 : kWorkers;
  a.parts = static_cast<float*>(p.ws);
  a.joins = whole ? nullptr : reinterpret_cast<Join*>(a.parts + 2 * (size_t)kWorkers * part_floats(DV));
  if (whole) {
    const unsigned grid = (unsigned)p.B * a.CT * p.c.H;
    // no more workgroups than compute units: more waves each
    if (grid <= 256) hipLaunchKernelGGL((kda_attn_decode_kernel<kMoreWaves, NT, E4, DK, DV>), dim3(grid), dim3(64 * kMoreWaves), 0, s, a);
    else hipLaunchKernelGGL((kda_attn_decode_kernel<kWaves, NT, E4, DK, DV>), dim3(grid), dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((kda_attn_decode_kernel<kWaves, NT, E4, DK, DV>), dim3(kWorkers), dim3(64 * kWaves),
                     sizeof(int) * ((size_t)p.B + 1), s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int rows = std::min(kAttnColumns, p.K * a.G);
  hipLaunchKernelGGL((kda_attn_join_kernel<DV>), dim3(kWorkers, rows), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int NT, bool E4>
hipError_t pick_dims(const AttnDecodeParams& p, hipStream_t s) {
  if (p.c.dk == 128) return p.c.dv == 128 ? launch_one<NT, E4, 128, 128>(p, s) : launch_one<NT, E4, 128, 64>(p, s);
  return p.c.dv == 128 ? launch_one<NT, E4, 64, 128>(p, s) : launch_one<NT, E4, 64, 64>(p, s);
}

}  // namespace

size_t attn_decode_workspace(int B, int K, int Hq, int H, int dv, int page_tokens, int width) {
  if (takes_whole(B, K, Hq, H, page_tokens, width)) return 0;
  return (size_t)kWorkers * (2 * part_floats(dv) * sizeof(float) + sizeof(Join));
}

hipError_t launch_attn_decode(const AttnDecodeParams& p, int q_dtype, hipStream_t s) {
  const KvCache& c = p.c;
  if (p.B < 1 || p.K < 1 || c.H < 1 || p.Hq % c.H || (c.dk != 64 && c.dk != 128) || (c.dv != 64 && c.dv != 128) ||
      c.page_tokens % 16)
    return hipErrorInvalidValue;
  if (q_dtype == 1) return c.e4m3 ? pick_dims<1, true>(p, s) : pick_dims<1, false>(p, s);
  return c.e4m3 ? pick_dims<3, true>(p, s) : pick_dims<3, false>(p, s);
}

}  // namespace kda
