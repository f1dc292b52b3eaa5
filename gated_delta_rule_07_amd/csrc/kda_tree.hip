// Trees of drafted tokens for KDA on gfx950: verify a whole tree against each
// cached state, then commit its accepted path.
//
// Node t of a tree follows its parent's state (the cached state S at the root):
//   S_t = Diag(alpha_t) S_parent + k_t u_t^T,   o_t = S_t^T q_t,
//   u_t = beta_t (v_t - (Diag(alpha_t) S_parent)^T k_t).
// With P_t the product of the alphas on the path from the root to t, and G_ts
// that of the alphas after the ancestor s up to t (per key channel), unrolling
// the path gives
//   x_t = S^T (P_t k_t) + sum_{s above t} c_ts u_s,   c_ts = sum_i k_s G_ts k_t,
//   u_t = beta_t (v_t - x_t),
//   o_t = S^T (P_t q_t) + sum_{s above t} d_ts u_s + (k_t . q_t) u_t,
//                                                     d_ts = sum_i k_s G_ts q_t,
// so S is read once and meets 2K vectors, and what the nodes do to one another
// is scalars.  G_ts is a running product along the path: no division, so a
// channel that has decayed to nothing (or alpha = 0) needs no care.
//
// kda_tree_verify_kernel, one workgroup of four waves per (sequence, head):
//   1. the keys, queries and decays of the tree's nodes, the state and the values
//      are loaded, all in flight at once; the first three go to LDS;
//   2. one group of d_k / 8 lanes per node walks up its path: c, d and P_t;
//   3. the 2K x d_k by d_k x d_v product runs on the fp32 matrix cores.  Each wave
//      owns d_v / 4 columns and holds the state as the B operand straight from
//      its loads; the A operands P_t k_t and P_t q_t are formed as they are read;
//   4. each wave substitutes through its columns, level after level of the tree,
//      on the values as the matrix cores left them: a lane holds every fourth
//      run of four nodes.  The nodes of a level write their u to LDS, and every
//      node below takes the term of its ancestor there, so a level costs one
//      exchange however long the paths are.
#include "kda_device.h"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kTreeThreads = 256;

template <typename IO, int DK, int DV>
struct TCfg {
  static constexpr int NTL = DV >= 128 ? 2 : 1;        // 16-column tiles of a state wave
  static constexpr int CW = 16 * NTL;                  // its columns
  static constexpr int NW = DV / CW;                   // state waves (of 4)
  // a node's row in LDS: key, query, decays, and 16 bytes by which 16 rows cover all banks
  static constexpr int QAT = DK * (int)sizeof(IO), AAT = 2 * QAT, ROW = AAT + DK * 4 + 16;
  static constexpr int GL = DK / 8;                    // lanes of a node's group
  static constexpr int GROUPS = kTreeThreads / GL;
  static_assert(NW <= 4 && NW * CW == DV, "state waves");
};

// The verify kernel's LDS, in bytes, for K nodes.  Row K stands for the state the tree
// starts from: no key, and no decay.  u takes the place of the rows.
struct TLay {
  int rows, u, cd, anc, self, beta, par, depth, total;
  __host__ __device__ static int r16(int n) { return (n + 15) & ~15; }
  __host__ __device__ TLay(int K, int row, int dv) {
    const int pairs = K * (K - 1) / 2;
    rows = u = 0;
    cd = r16((K + 1) * (row > dv * 4 ? row : dv * 4));
    anc = cd + r16(8 * pairs);
    self = anc + r16(pairs);
    beta = self + r16(4 * K);
    par = beta + r16(4 * K);
    depth = par + r16(4 * K + 4);
    total = depth + r16(4 * K);
  }
};

// beta_t c, d and the ancestor of node t's hop j upwards (0: its parent; j < t) stand at
// first_pair(t) + j.
__device__ __forceinline__ int first_pair(int t) { return t * (t - 1) / 2; }

// The sum of x over each aligned group of G lanes, in every one of them.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  const int y = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true);
  return x + __builtin_bit_cast(float, y);
}
template <int G>
__device__ __forceinline__ float group_sum(float x) {
  static_assert(G == 2 || G == 4 || G == 8 || G == 16, "lanes of a group");
  x = add_dpp<0xB1>(x);                          // lane ^ 1
  if constexpr (G >= 4) x = add_dpp<0x4E>(x);    // lane ^ 2
  if constexpr (G >= 8) x = add_dpp<0x141>(x);   // the other four of eight
  if constexpr (G >= 16) x = add_dpp<0x140>(x);  // the other eight of sixteen
  return x;
}

__device__ __forceinline__ f32x4 lds4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 lds4(const __bf16* p) {
  const u32x2 w = *reinterpret_cast<const u32x2*>(p);
  return f32x4{__builtin_bit_cast(float, w.x << 16), __builtin_bit_cast(float, w.x & 0xffff0000u),
               __builtin_bit_cast(float, w.y << 16), __builtin_bit_cast(float, w.y & 0xffff0000u)};
}

// A barrier that waits for LDS only: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// What this wave wrote to LDS is seen by its own later reads.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <typename IO, int DK, int DV, int MAXK>
__global__ __launch_bounds__(kTreeThreads, MAXK <= 32 ? 3 : 1) void kda_tree_verify_kernel(TreeParams p) {
  using C = TCfg<IO, DK, DV>;
  extern __shared__ u32x4 tree_lds[];
  char* sm = reinterpret_cast<char*>(tree_lds);
  const int K = p.K, tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const TLay L(K, C::ROW, DV);
  const int b = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int n = p.n_nodes ? min(max(p.n_nodes[b], 0), K) : K;
  const int page = p.pages ? p.pages[b] : b;
  if (n == 0 || !page_ok(page, p.n_pages)) return;
  const size_t row0 = (size_t)b * K * p.H + h;  // node t: row row0 + t H of the [B][K][H][d] arrays

  // keys, queries and decays, 16 bytes a load (indices clamped into the tree's rows, and
  // no branch: one around a load makes the compiler wait for it)
  constexpr int CK = DK * (int)sizeof(IO) / 16, CA = DK * 4 / 16;  // loads of a row
  constexpr int EK = (MAXK * CK + kTreeThreads - 1) / kTreeThreads, EA = (MAXK * CA + kTreeThreads - 1) / kTreeThreads;
  u32x4 rk[EK], rq[EK];
  f32x4 ra[EA];
  const int tn = min(tid, n - 1);
  const int up = p.parents[(size_t)b * K + tn];
  const float bt = p.beta[row0 + (size_t)tn * p.H];
#pragma unroll
  for (int j = 0; j < EK; ++j) {
    const unsigned e = min(tid + j * kTreeThreads, n * CK - 1);
    const size_t at = (row0 + (size_t)(e / CK) * p.H) * (DK * sizeof(IO)) + 16 * (e % CK);
    rk[j] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p.k) + at);
    rq[j] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p.q) + at);
  }
#pragma unroll
  for (int j = 0; j < EA; ++j) {
    const unsigned e = min(tid + j * kTreeThreads, n * CA - 1);
    ra[j] = *reinterpret_cast<const f32x4*>(p.alpha + (row0 + (size_t)(e / CA) * p.H) * DK + 4 * (e % CA));
  }
  __builtin_amdgcn_sched_barrier(0);  // (loads are counted in order: the small ones come first)

  // the state, as the matrix cores' B operand: slot (lg, e) of step kk is row 16 kk + 4 lg + e
  typedef float colf __attribute__((ext_vector_type(C::NTL)));
  typedef IO colio __attribute__((ext_vector_type(C::NTL)));
  const int ln = lane % 16, lg = lane / 16;
  const bool stw = C::NW == 4 || wave < C::NW;  // a state wave (the others load what the last one does)
  const int col = C::CW * min(wave, C::NW - 1) + C::NTL * ln;  // its lane's first column
  constexpr int NT = (MAXK + 15) / 16;
  colf s[DK / 16][4];
  colio rv[NT][4];
  const float* S = p.pool + ((size_t)page * p.H + h) * DK * DV + col;
#pragma unroll
  for (int kk = 0; kk < DK / 16; ++kk)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[kk][e] = *reinterpret_cast<const colf*>(S + (size_t)(16 * kk + 4 * lg + e) * DV);
#pragma unroll
  for (int m = 0; m < NT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      rv[m][r] = *reinterpret_cast<const colio*>(
          static_cast<const IO*>(p.v) + (row0 + (size_t)min(16 * m + 4 * lg + r, n - 1) * p.H) * DV + col);
  }
  __builtin_amdgcn_sched_barrier(0);

  int* par = reinterpret_cast<int*>(sm + L.par);
  float* beta = reinterpret_cast<float*>(sm + L.beta);
  if (tid < n) {
    par[tid] = up >= 0 && up < tid ? up : K;
    beta[tid] = bt;
  }
  if (tid == 0) par[K] = K;
  // (24-bit products: a 32-bit one becomes a 64-bit multiply-add whose unused half may
  // wait for a load)
  auto row = [&](int t) { return sm + L.rows + __umul24(t, C::ROW); };
  auto krow = [&](int t) { return reinterpret_cast<const IO*>(row(t)); };
  auto qrow = [&](int t) { return reinterpret_cast<const IO*>(row(t) + C::QAT); };
  auto arow = [&](int t) { return reinterpret_cast<float*>(row(t) + C::AAT); };
  for (int i = tid; i < DK; i += kTreeThreads) {
    const_cast<IO*>(krow(K))[i] = (IO)0.0f;
    arow(K)[i] = 1.0f;
  }
#pragma unroll
  for (int j = 0; j < EK; ++j) {
    const unsigned e = min(tid + j * kTreeThreads, n * CK - 1);  // (a clamped index stores what is there)
    *reinterpret_cast<u32x4*>(row(e / CK) + 16 * (e % CK)) = rk[j];
    *reinterpret_cast<u32x4*>(row(e / CK) + C::QAT + 16 * (e % CK)) = rq[j];
  }
#pragma unroll
  for (int j = 0; j < EA; ++j) {
    const unsigned e = min(tid + j * kTreeThreads, n * CA - 1);
    *reinterpret_cast<f32x4*>(row(e / CA) + C::AAT + 16 * (e % CA)) = ra[j];
  }
  lds_barrier();

  // up each node's path; a lane holds channels 4 gl + {0..3} and DK/2 + 4 gl + {0..3}, and
  // reads the next ancestor's row while it works on one
  constexpr int NPG = (MAXK + C::GROUPS - 1) / C::GROUPS;
  const int gl = tid % C::GL, grp = tid / C::GL;
  const int i0 = 4 * gl, i1 = DK / 2 + 4 * gl;
  f32x4 P[NPG][2];
  float2* cd = reinterpret_cast<float2*>(sm + L.cd);
  unsigned char* anc = reinterpret_cast<unsigned char*>(sm + L.anc);
  float* self = reinterpret_cast<float*>(sm + L.self);
  int* depth = reinterpret_cast<int*>(sm + L.depth);
#pragma unroll
  for (int it = 0; it < NPG; ++it) {
    const int t = it * C::GROUPS + grp;
    if (t >= n) continue;
    int r = par[t];
    const f32x4 k0 = lds4(krow(t) + i0), k1 = lds4(krow(t) + i1);
    const f32x4 q0 = lds4(qrow(t) + i0), q1 = lds4(qrow(t) + i1);
    f32x4 g0 = lds4(arow(t) + i0), g1 = lds4(arow(t) + i1);
    f32x4 kr0 = lds4(krow(r) + i0), kr1 = lds4(krow(r) + i1), ar0 = lds4(arow(r) + i0), ar1 = lds4(arow(r) + i1);
    int rn = par[r];
    const float be = beta[t];
    float dt = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) dt += k0[e] * q0[e] + k1[e] * q1[e];
    dt = group_sum<C::GL>(dt);
    int at = first_pair(t);
    while (r < K) {
      const f32x4 w0 = g0 * kr0, w1 = g1 * kr1;
      g0 *= ar0;
      g1 *= ar1;
      const unsigned char who = (unsigned char)r;
      r = rn;
      kr0 = lds4(krow(r) + i0);
      kr1 = lds4(krow(r) + i1);
      ar0 = lds4(arow(r) + i0);
      ar1 = lds4(arow(r) + i1);
      rn = par[r];
      float cs = 0.0f, ds = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs += w0[e] * k0[e];
        ds += w0[e] * q0[e];
        cs += w1[e] * k1[e];
        ds += w1[e] * q1[e];
      }
      cs = group_sum<C::GL>(cs);
      ds = group_sum<C::GL>(ds);
      if (gl == 0) {
        cd[at] = float2{be * cs, ds};
        anc[at] = who;
      }
      ++at;
    }
    if (gl == 0) {
      self[t] = dt;
      depth[t] = at - first_pair(t);
    }
    P[it][0] = g0;
    P[it][1] = g1;
  }
  lds_barrier();
  // P takes the decays' place
#pragma unroll
  for (int it = 0; it < NPG; ++it) {
    const int t = it * C::GROUPS + grp;
    if (t >= n) continue;
    *reinterpret_cast<f32x4*>(arow(t) + i0) = P[it][0];
    *reinterpret_cast<f32x4*>(arow(t) + i1) = P[it][1];
  }
  lds_barrier();

  // products with the state: x (of the keys) and y (of the queries), of node 16 m + 4 lg + r
  f32x4 xa[NT][C::NTL], ya[NT][C::NTL];
#pragma unroll
  for (int m = 0; m < NT; ++m)
#pragma unroll
    for (int j = 0; j < C::NTL; ++j) xa[m][j] = ya[m][j] = (f32x4)0.0f;
  if (stw) {
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      if (16 * m >= n) continue;
      const int t = min(16 * m + ln, n - 1);  // (a row past the last node only feeds its own row of the result)
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        const int i = 16 * kk + 4 * lg;
        const f32x4 pt = lds4(arow(t) + i);
        const f32x4 pk = pt * lds4(krow(t) + i), pq = pt * lds4(qrow(t) + i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < C::NTL; ++j) {
            xa[m][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(pk[e], s[kk][e][j], xa[m][j], 0, 0, 0);
            ya[m][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(pq[e], s[kk][e][j], ya[m][j], 0, 0, 0);
          }
      }
    }
  }
  lds_barrier();  // keys, queries and decays are done with: u takes their place
  if (!stw) return;

  // substitution, a level of the tree at a time: x, from beta (v - x) on, is a node's u
  // as soon as the levels above it are done
  float* us = reinterpret_cast<float*>(sm + L.u) + (size_t)(K + 1) * C::CW * wave + C::NTL * ln;  // [K + 1][CW] of this wave
  float x[NT][4][C::NTL], y[NT][4][C::NTL];
  int dep[NT][4], top[NT][4];  // a node's depth, and where its hop to the root stands in cd and anc
  int deepest = 0;
#pragma unroll
  for (int m = 0; m < NT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * m + 4 * lg + r, tc = min(t, n - 1);
      dep[m][r] = t < n ? depth[tc] : -1;
      deepest = max(deepest, dep[m][r]);
      top[m][r] = first_pair(tc) + max(dep[m][r], 0) - 1;
      const float be = beta[tc];
#pragma unroll
      for (int j = 0; j < C::NTL; ++j) {
        x[m][r][j] = be * (to_f32(rv[m][r][j]) - xa[m][j][r]);
        y[m][r][j] = ya[m][j][r];
      }
    }
  }
  deepest = max(deepest, __shfl_xor(deepest, 16));
  deepest = max(deepest, __shfl_xor(deepest, 32));
  // (no branches on single nodes: every load of a level is in flight at once.  What a node
  // writes before its level is written again there, row K is a spare, and a node at or above
  // the level reads some pair and row and drops them)
  for (int lev = 0; lev < deepest; ++lev) {
#pragma unroll
    for (int m = 0; m < NT; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        colf w;
#pragma unroll
        for (int j = 0; j < C::NTL; ++j) w[j] = x[m][r][j];
        *reinterpret_cast<colf*>(us + min(16 * m + 4 * lg + r, K) * C::CW) = w;
      }
    }
    wave_lds_order();
    float2 w[NT][4];
    int row[NT][4];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = max(top[m][r] - lev, 0);
        w[m][r] = cd[at];
        row[m][r] = anc[at];
      }
    }
#pragma unroll
    for (int m = 0; m < NT; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool below = dep[m][r] > lev;
        const colf ua = *reinterpret_cast<const colf*>(us + (below ? row[m][r] : 0) * C::CW);
#pragma unroll
        for (int j = 0; j < C::NTL; ++j) {
          x[m][r][j] = below ? x[m][r][j] - w[m][r].x * ua[j] : x[m][r][j];
          y[m][r][j] = below ? y[m][r][j] + w[m][r].y * ua[j] : y[m][r][j];
        }
      }
    }
    wave_lds_order();
  }
#pragma unroll
  for (int m = 0; m < NT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * m + 4 * lg + r;
      if (t >= n) continue;
      const float se = self[t];
      colf ut, ot;
#pragma unroll
      for (int j = 0; j < C::NTL; ++j) {
        ut[j] = x[m][r][j];
        ot[j] = y[m][r][j] + se * x[m][r][j];
      }
      const size_t at = (row0 + (size_t)t * p.H) * DV + col;
      *reinterpret_cast<colf*>(p.u + (((size_t)b * p.H + h) * K + t) * DV + col) = ut;
      if (p.o_f32) {
        *reinterpret_cast<colf*>(static_cast<float*>(p.o) + at) = ot;
      } else {
        typedef __bf16 colb __attribute__((ext_vector_type(C::NTL)));
        colb ob;
#pragma unroll
        for (int j = 0; j < C::NTL; ++j) ob[j] = (__bf16)ot[j];
        *reinterpret_cast<colb*>(static_cast<__bf16*>(p.o) + at) = ob;
      }
    }
  }
}

// Commit: each thread owns a float4 column group and DK/RG rows, as the decode
// step; with the accepted path t_1 .. t_j from the root,
//   S' = Diag(P_j) S + sum_m Diag(prod_{l>m} alpha_{t_l}) k_{t_m} u_{t_m}^T.
template <int DK, int DV>
struct MCfg {
  static constexpr int NCG = DV / 4;
  static constexpr int RG = (256 / NCG < DK) ? 256 / NCG : DK;
  static constexpr int NT = NCG * RG;
  static constexpr int RPT = DK / RG;
  static_assert(NT % 64 == 0 && NT <= 256, "block shape");
};

template <typename IO, int DK, int DV>
__global__ __launch_bounds__(256) void kda_tree_commit_kernel(TreeCommitParams p) {
  using C = MCfg<DK, DV>;
  extern __shared__ float coef[];  // [K][DK]: k_t times the decays after t, for the path's tokens, last first
  __shared__ float pj[DK];
  __shared__ int par[kMaxTree], path[kMaxTree + 1], srace[C::NT / 64];
  const int tid = threadIdx.x, K = p.K;
  const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H;
  const int in = p.pages_in ? p.pages_in[b] : b;
  const int out = p.pages_out ? p.pages_out[b] : in;
  if (!page_ok(in, p.n_pages) || !page_ok(out, p.n_pages)) return;
  const int n = p.n_nodes ? min(max(p.n_nodes[b], 0), K) : K;
  int last = p.last[b];
  if (last < 0 || last >= n) last = -1;
  if (last < 0 && in == out) return;

  const int cg = tid % C::NCG, rg = tid / C::NCG;
  const float* S = p.pool + ((size_t)in * p.H + h) * DK * DV;
  float* So = p.pool + ((size_t)out * p.H + h) * DK * DV;
  f32x4 s[C::RPT];
#pragma unroll
  for (int r = 0; r < C::RPT; ++r) s[r] = *reinterpret_cast<const f32x4*>(S + (size_t)(rg + C::RG * r) * DV + 4 * cg);
  const bool races = __any(page_races(p.pages_in, p.pages_out, p.n_pages, p.B, b, in, out, tid, C::NT));
  if (tid % 64 == 0) srace[tid / 64] = races;
  if (tid < K) {
    const int up = p.parents[(size_t)b * K + tid];
    par[tid] = up >= -1 && up < tid ? up : -1;
  }
  __syncthreads();
  int skip = 0;
#pragma unroll
  for (int w = 0; w < C::NT / 64; ++w) skip |= srace[w];
  if (skip) return;  // (the same for the whole workgroup)
  if (tid == 0) {
    int j = 0;
    for (int t = last; t >= 0; t = par[t]) path[j++] = t;
    path[kMaxTree] = j;
  }
  __syncthreads();
  const int j = path[kMaxTree];
  for (int i = tid; i < DK; i += C::NT) {
    float run = 1.0f;
    for (int m = 0; m < j; ++m) {
      const size_t row = ((size_t)b * K + path[m]) * p.H + h;
      coef[m * DK + i] = to_f32(static_cast<const IO*>(p.k)[row * DK + i]) * run;
      run *= p.alpha[row * DK + i];
    }
    pj[i] = run;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < C::RPT; ++r) s[r] *= pj[rg + C::RG * r];
  for (int m = 0; m < j; ++m) {
    const f32x4 ut = *reinterpret_cast<const f32x4*>(p.u + ((size_t)bh * K + path[m]) * DV + 4 * cg);
#pragma unroll
    for (int r = 0; r < C::RPT; ++r) s[r] += coef[m * DK + rg + C::RG * r] * ut;
  }
#pragma unroll
  for (int r = 0; r < C::RPT; ++r)
    __builtin_nontemporal_store(s[r], reinterpret_cast<f32x4*>(So + (size_t)(rg + C::RG * r) * DV + 4 * cg));
}

template <typename IO, int DK, int DV, int MAXK>
hipError_t verify_k(const TreeParams& p, hipStream_t s) {
  using C = TCfg<IO, DK, DV>;
  const int lds = TLay(p.K, C::ROW, DV).total;
  if (lds > 65536) {  // more than the default has to be asked for
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&kda_tree_verify_kernel<IO, DK, DV, MAXK>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((kda_tree_verify_kernel<IO, DK, DV, MAXK>), dim3((unsigned)(p.B * p.H)), dim3(kTreeThreads), lds, s, p);
  return hipGetLastError();
}

template <typename IO, int DK, int DV>
hipError_t verify_one(const TreeParams& p, hipStream_t s) {
  if (p.K <= 16) return verify_k<IO, DK, DV, 16>(p, s);
  if (p.K <= 32) return verify_k<IO, DK, DV, 32>(p, s);
  return verify_k<IO, DK, DV, kMaxTree>(p, s);
}
template <typename IO, int DK, int DV>
hipError_t commit_one(const TreeCommitParams& p, hipStream_t s) {
  hipLaunchKernelGGL((kda_tree_commit_kernel<IO, DK, DV>), dim3((unsigned)(p.B * p.H)), dim3(MCfg<DK, DV>::NT),
                     (size_t)p.K * DK * sizeof(float), s, p);
  return hipGetLastError();
}

template <class P>
using tree_fn = hipError_t (*)(const P&, hipStream_t);

template <typename IO, int DK, int DV>
struct VerifyF {
  static constexpr tree_fn<TreeParams> fn = &verify_one<IO, DK, DV>;
};
template <typename IO, int DK, int DV>
struct CommitF {
  static constexpr tree_fn<TreeCommitParams> fn = &commit_one<IO, DK, DV>;
};

template <class P, template <typename, int, int> class F, typename IO, int DK>
tree_fn<P> pick_dv(int dv) {
  switch (dv) {
    case 16: return F<IO, DK, 16>::fn;
    case 32: return F<IO, DK, 32>::fn;
    case 64: return F<IO, DK, 64>::fn;
    case 128: return F<IO, DK, 128>::fn;
    default: return nullptr;
  }
}

template <class P, template <typename, int, int> class F, typename IO>
tree_fn<P> pick_dk(int dk, int dv) {
  switch (dk) {
    case 16: return pick_dv<P, F, IO, 16>(dv);
    case 32: return pick_dv<P, F, IO, 32>(dv);
    case 64: return pick_dv<P, F, IO, 64>(dv);
    case 128: return pick_dv<P, F, IO, 128>(dv);
    default: return nullptr;
  }
}

template <class P, template <typename, int, int> class F>
tree_fn<P> pick(int io_dtype, int dk, int dv) {
  if (io_dtype == 1) return pick_dk<P, F, __bf16>(dk, dv);
  if (io_dtype == 0) return pick_dk<P, F, float>(dk, dv);
  return nullptr;
}

}  // namespace

bool tree_supported(int io_dtype, int dk, int dv) { return pick<TreeParams, VerifyF>(io_dtype, dk, dv) != nullptr; }

hipError_t launch_tree_verify(const TreeParams& p, int io_dtype, hipStream_t s) {
  const tree_fn<TreeParams> f = pick<TreeParams, VerifyF>(io_dtype, p.dk, p.dv);
  if (!f || p.K < 1 || p.K > kMaxTree) return hipErrorInvalidValue;
  return f(p, s);
}

hipError_t launch_tree_commit(const TreeCommitParams& p, int io_dtype, hipStream_t s) {
  const tree_fn<TreeCommitParams> f = pick<TreeCommitParams, CommitF>(io_dtype, p.dk, p.dv);
  if (!f || p.K < 1 || p.K > kMaxTree) return hipErrorInvalidValue;
  return f(p, s);
}

}  // namespace kda
