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
// kda_tree_verify_kernel, one workgroup of eight waves per (sequence, head):
//   1. the keys, queries and decays of the tree's nodes, the state and the values
//      are loaded, all in flight at once; the first three go to LDS;
//   2. one group of d_k / 8 lanes per node walks up its path with the node's key
//      and query, decayed on the way: c, d, and at the root P_t k_t and P_t q_t, which
//      take the place of the rows in LDS.  c and d fill two K x K matrices, C (beta_t c, strictly below the diagonal because a
//      node follows its parent) and D (d, with k_t . q_t on it), zero elsewhere;
//   3. the 2K x d_k by d_k x d_v product runs on the fp32 matrix cores.  Each wave
//      owns 16 columns and holds the state as the B operand straight from
//      its loads;
//   4. U = (I + C)^-1 beta (V - X) and O = Y + D U, in blocks of 16 nodes, on the
//      matrix cores too: the 16 x 16 inverses on the diagonal are one lane per
//      column, and a block's result, as the matrix cores leave it, is the next
//      product's B operand.  (Substituting level after level of the tree through
//      LDS instead took 8 of 20 us on deep trees of 63 nodes.)
//      Zero times a value that is not finite would spread one node's NaN to nodes
//      that do not follow it, so from a block on whose right-hand sides or u pass 1e18 (as any
//      do where C, D, an inverse or an input has left fp32) a wave takes the sums along the paths.
//
// Measured, 64 sequences of 32 heads of 128, trees of 24 to 32 nodes 6 deep, bf16: 84 us (78 at best),
// for 252 MB (47 us at a copy's rate) and 256 + 48 fp32 matrix instructions a wave pair, 35 us
// of the matrix cores at the 2.2 GHz that the launch runs at.  The loads alone take 40 us,
// and the kernel without the first product 58 us: what is lost is overlap, two workgroups
// of 47 KB of LDS and 64 KB of state in registers a compute unit.  Trees of 63 nodes, 12 deep, on
// 120 fp32 states of 64 x 64: 13.7 us (33.7 us substituting node after node).  One tree of 8
// nodes on 8 states: 7.4 us.  Tried and no faster on the first, where this form took
// 80 us then: four waves with two column tiles each and three workgroups a compute unit (81 us, and 15.0 and 8.0 us on the others), a
// persistent grid that loads the next state during the substitution (96 us), registers
// cut to 80 for three workgroups of eight waves (105 us, spills).
//
// kda_tree_commit_kernel reads and writes a state as the decode step does: 45 us for the 2,048
// states above (275 MB, 6.1 TB/s with what the verify left in the caches).  It looks over the other
// sequences' pages as that step does: 4,096 x 8 states of 16 x 16 take 109 us.
#include "kda_device.h"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kTreeThreads = 512;
constexpr int kInvRow = 20, kInvBytes = 16 * kInvRow * 4;  // a 16 x 16 inverse, rows 4 banks apart

template <typename IO, int DK, int DV>
struct TCfg {
  static constexpr int CW = 16;                        // columns of a state wave
  static constexpr int NW = DV / CW;                   // state waves (of 8)
  // a node's row in LDS: key, query, decays, and 16 bytes by which 16 rows cover all banks
  static constexpr int QAT = DK * (int)sizeof(IO), AAT = 2 * QAT, ROW = AAT + DK * 4 + 16;
  static constexpr int PROW = 8 * DK + 16;             // the same of a row of P_t k_t and P_t q_t
  static constexpr int GL = DK / 8;                    // lanes of a node's group
  static constexpr int GROUPS = kTreeThreads / GL;
  static_assert(NW <= kTreeThreads / 64 && NW * CW == DV, "state waves");
};

// The verify kernel's LDS, in bytes, for K nodes.  Row K stands for the state the tree
// starts from: no key, and no decay.  u takes the place of the rows.
struct TLay {
  int rows, u, c, d, inv, beta, par, flag, total;
  __host__ __device__ static int r16(int n) { return (n + 15) & ~15; }
  // mrow: the bytes of a row of C and D; nblk: 16-node blocks
  __host__ __device__ TLay(int K, int row, int dv, int mrow, int nblk) {
    rows = u = 0;
    c = r16((K + 1) * row > K * dv * 4 ? (K + 1) * row : K * dv * 4);
    d = c + 16 * nblk * mrow;
    inv = d + 16 * nblk * mrow;
    beta = inv + nblk * kInvBytes;
    par = beta + r16(4 * K);
    flag = par + r16(4 * K + 4);
    total = flag + 16;
  }
};

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

// Entries of C and D, right-hand sides and write vectors up to here take the products with C, D and the
// inverses: sums of 64 products of two of them stay inside fp32.
constexpr float kPlain = 1e18f;

template <typename IO, int DK, int DV, int MAXK>
__global__ __launch_bounds__(kTreeThreads, MAXK <= 32 ? 4 : 2) void kda_tree_verify_kernel(TreeParams p) {
  using C = TCfg<IO, DK, DV>;
  extern __shared__ u32x4 tree_lds[];
  char* sm = reinterpret_cast<char*>(tree_lds);
  const int K = p.K, tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  constexpr int NT = (MAXK + 15) / 16, MROW = 16 * NT + 4;  // blocks of 16 nodes; floats between rows of C and D
  const TLay L(K, C::ROW, DV, 4 * MROW, NT);
  const int b = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int n = p.n_nodes ? min(max(p.n_nodes[b], 0), K) : K;
  const int page = p.pages ? p.pages[b] : b;
  if (n == 0 || !page_ok(page, p.n_pages)) return;
  // node t: row row0 + t H of the [B][K][H][d] arrays; within a sequence 32 bits of bytes
  const size_t row0 = (size_t)b * K * p.H + h;
  const char* qb = static_cast<const char*>(p.q) + row0 * (DK * sizeof(IO));
  const char* kb = static_cast<const char*>(p.k) + row0 * (DK * sizeof(IO));
  const char* ab = reinterpret_cast<const char*>(p.alpha + row0 * DK);
  const char* vb = static_cast<const char*>(p.v) + row0 * (DV * sizeof(IO));
  const unsigned H = p.H;

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
    const unsigned at = e / CK * H * (unsigned)(DK * sizeof(IO)) + 16 * (e % CK);
    rk[j] = *reinterpret_cast<const u32x4*>(kb + at);
    rq[j] = *reinterpret_cast<const u32x4*>(qb + at);
  }
#pragma unroll
  for (int j = 0; j < EA; ++j) {
    const unsigned e = min(tid + j * kTreeThreads, n * CA - 1);
    ra[j] = *reinterpret_cast<const f32x4*>(ab + (e / CA * H * (unsigned)(DK * 4) + 16 * (e % CA)));
  }
  __builtin_amdgcn_sched_barrier(0);  // (loads are counted in order: the small ones come first)

  // the state, as the matrix cores' B operand: slot (lg, e) of step kk is row 16 kk + 4 lg + e
  const int ln = lane % 16, lg = lane / 16;
  const bool stw = C::NW == kTreeThreads / 64 || wave < C::NW;  // a state wave (the others load what the last one does)
  const int col = C::CW * min(wave, C::NW - 1) + ln;  // its lane's column
  float s[DK / 16][4];
  IO rv[NT][4];
  const float* S = p.pool + ((size_t)page * p.H + h) * DK * DV + col;
#pragma unroll
  for (int kk = 0; kk < DK / 16; ++kk)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[kk][e] = S[(size_t)(16 * kk + 4 * lg + e) * DV];
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
  float* cm = reinterpret_cast<float*>(sm + L.c);
  float* dm = reinterpret_cast<float*>(sm + L.d);
  int* flag = reinterpret_cast<int*>(sm + L.flag);
  if (tid == 0) *flag = 0;
#pragma unroll
  for (int i = 0; i < (2 * 16 * NT * MROW / 4 + kTreeThreads - 1) / kTreeThreads; ++i)
    if (tid + i * kTreeThreads < 2 * 16 * NT * MROW / 4) reinterpret_cast<f32x4*>(cm)[tid + i * kTreeThreads] = (f32x4)0.0f;
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

  // up each node's path; a lane holds channels 4 gl + {0..3} and DK/2 + 4 gl + {0..3} of
  // the node's key and query, decayed so far
  constexpr int NPG = (MAXK + C::GROUPS - 1) / C::GROUPS;
  const int gl = tid % C::GL, grp = tid / C::GL;
  const int i0 = 4 * gl, i1 = DK / 2 + 4 * gl;
  f32x4 pk[NPG][2], pq[NPG][2];
#pragma unroll
  for (int it = 0; it < NPG; ++it) {
    const int t = it * C::GROUPS + grp;
    if (t >= n) continue;
    int r = par[t];
    f32x4 k0 = lds4(krow(t) + i0), k1 = lds4(krow(t) + i1), q0 = lds4(qrow(t) + i0), q1 = lds4(qrow(t) + i1);
    const f32x4 a0 = lds4(arow(t) + i0), a1 = lds4(arow(t) + i1);
    const float be = beta[t];
    float dt = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dt += k0[e] * q0[e];
      dt += k1[e] * q1[e];
    }
    dt = group_sum<C::GL>(dt);
    k0 *= a0, k1 *= a1, q0 *= a0, q1 *= a1;
    bool fine = true;
    while (r < K) {
      const f32x4 kr0 = lds4(krow(r) + i0), kr1 = lds4(krow(r) + i1);
      const f32x4 ar0 = lds4(arow(r) + i0), ar1 = lds4(arow(r) + i1);
      const int at = t * MROW + r;
      r = par[r];
      float cs = 0.0f, ds = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs += k0[e] * kr0[e];
        ds += q0[e] * kr0[e];
        cs += k1[e] * kr1[e];
        ds += q1[e] * kr1[e];
      }
      k0 *= ar0, k1 *= ar1, q0 *= ar0, q1 *= ar1;
      cs = be * group_sum<C::GL>(cs);
      ds = group_sum<C::GL>(ds);
      if (gl == 0) {
        cm[at] = cs;
        dm[at] = ds;
      }
      fine &= fabsf(cs) <= kPlain && fabsf(ds) <= kPlain;
    }
    if (gl == 0) {
      dm[t * MROW + t] = dt;
      if (!(fine && fabsf(dt) <= kPlain)) *flag = 1;
    }
    pk[it][0] = k0, pk[it][1] = k1, pq[it][0] = q0, pq[it][1] = q1;
  }
  lds_barrier();
  // P_t k_t and P_t q_t take the rows' place
  auto prow = [&](int t) { return reinterpret_cast<float*>(sm + L.rows + __umul24(t, C::PROW)); };
#pragma unroll
  for (int it = 0; it < NPG; ++it) {
    const int t = it * C::GROUPS + grp;
    if (t >= n) continue;
    *reinterpret_cast<f32x4*>(prow(t) + i0) = pk[it][0];
    *reinterpret_cast<f32x4*>(prow(t) + i1) = pk[it][1];
    *reinterpret_cast<f32x4*>(prow(t) + DK + i0) = pq[it][0];
    *reinterpret_cast<f32x4*>(prow(t) + DK + i1) = pq[it][1];
  }
  lds_barrier();

  // the values, on their way while the products run
#pragma unroll
  for (int m = 0; m < NT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      rv[m][r] = *reinterpret_cast<const IO*>(
          vb + ((unsigned)min(16 * m + 4 * lg + r, n - 1) * H * (unsigned)(DV * sizeof(IO)) + (unsigned)(col * sizeof(IO))));
  }
  // wave m inverts I + C of block m: column ln of the inverse, row after row
  if (wave < NT && 16 * wave < n) {
    const float* cb = cm + 16 * wave * MROW + 16 * wave;
    float inv[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      float a = t == ln ? 1.0f : 0.0f;
#pragma unroll
      for (int e = 0; e < t; e += 4) {
        const f32x4 c4 = *reinterpret_cast<const f32x4*>(cb + t * MROW + e);
#pragma unroll
        for (int f = 0; f < 4; ++f)
          if (e + f < t) a -= c4[f] * inv[e + f];
      }
      inv[t] = a;
    }
    float* to = reinterpret_cast<float*>(sm + L.inv + wave * kInvBytes) + ln;
    if (lg == 0) {
#pragma unroll
      for (int t = 0; t < 16; ++t) to[t * kInvRow] = inv[t];
    }
  }

  // products with the state: x (of the keys) and y (of the queries), of node 16 m + 4 lg + r
  f32x4 xa[NT], ya[NT];
#pragma unroll
  for (int m = 0; m < NT; ++m) xa[m] = ya[m] = (f32x4)0.0f;
  if (stw) {
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      if (16 * m >= n) continue;
      const int t = min(16 * m + ln, n - 1);  // (a row past the last node only feeds its own row of the result)
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        const int i = 16 * kk + 4 * lg;
        const f32x4 ak = lds4(prow(t) + i), aq = lds4(prow(t) + DK + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xa[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(ak[e], s[kk][e], xa[m], 0, 0, 0);
          ya[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(aq[e], s[kk][e], ya[m], 0, 0, 0);
        }
      }
    }
  }
  lds_barrier();  // keys, queries and decays are done with: u takes their place
  if (!stw) return;

  bool fine = *flag == 0;
#pragma unroll
  for (int m = 0; m < NT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * m + 4 * lg + r;
      const float be = beta[min(t, n - 1)];
      const float x = be * (to_f32(rv[m][r]) - xa[m][r]);
      xa[m][r] = t < n ? x : 0.0f;
      fine &= fabsf(xa[m][r]) <= kPlain;
    }
  }
  // block after block of nodes: xa turns into u, ya into o, as long as u stays below kPlain too (it grows by up to
  // |c| a level, and the inverses with it: an entry that has left fp32 makes its row of um infinite or NaN)
  bool plain = __all(fine);
  int done = 0;  // blocks whose u and o stand
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    if (16 * m >= n || !plain) continue;
    const float* crow = cm + (16 * m + ln) * MROW + 4 * lg;
    const float* drow = dm + (16 * m + ln) * MROW + 4 * lg;
#pragma unroll
    for (int mm = 0; mm < m; ++mm) {
      const f32x4 c4 = *reinterpret_cast<const f32x4*>(crow + 16 * mm), d4 = *reinterpret_cast<const f32x4*>(drow + 16 * mm);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        xa[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(-c4[r], xa[mm][r], xa[m], 0, 0, 0);
        ya[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(d4[r], xa[mm][r], ya[m], 0, 0, 0);
      }
    }
    const f32x4 i4 = *reinterpret_cast<const f32x4*>(sm + L.inv + m * kInvBytes + 4 * (ln * kInvRow + 4 * lg));
    const f32x4 d4 = *reinterpret_cast<const f32x4*>(drow + 16 * m);
    f32x4 um = (f32x4)0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) um = __builtin_amdgcn_mfma_f32_16x16x4f32(i4[r], xa[m][r], um, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) fine &= fabsf(um[r]) <= kPlain;
    plain = __all(fine);
    if (!plain) continue;
    done = m + 1;
    xa[m] = um;
#pragma unroll
    for (int r = 0; r < 4; ++r) ya[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(d4[r], um[r], ya[m], 0, 0, 0);
  }
  if (!plain) {
    // from the block that was not plain on node after node, along its path: [K][CW] of this wave in LDS.  That block's xa
    // and ya hold the products with the blocks before it already, the later blocks' none.
    const int t0 = 16 * done;
    float* us = reinterpret_cast<float*>(sm + L.u) + (size_t)K * C::CW * wave;
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (16 * m + 4 * lg + r < n) us[(16 * m + 4 * lg + r) * C::CW + ln] = xa[m][r];
    wave_lds_order();
    for (int t = t0; t < n; ++t) {
      const int from = t < t0 + 16 ? t0 : 0;
      if (lane < C::CW) {
        float x = us[t * C::CW + lane];
        for (int a = par[t]; a < K && a >= from; a = par[a]) x -= cm[t * MROW + a] * us[a * C::CW + lane];
        us[t * C::CW + lane] = x;
      }
      wave_lds_order();
    }
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const int from = m == done ? t0 : 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * m + 4 * lg + r;
        if (m < done || t >= n) continue;
        for (int a = t; a < K && a >= from; a = par[a]) ya[m][r] += dm[t * MROW + a] * us[a * C::CW + ln];
        xa[m][r] = us[t * C::CW + ln];
      }
    }
  }
  float* ub = p.u + ((size_t)b * p.H + h) * K * DV;
#pragma unroll
  for (int m = 0; m < NT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * m + 4 * lg + r;
      if (t >= n) continue;
      const unsigned at = (unsigned)t * H * DV + col;
      ub[t * DV + col] = xa[m][r];
      if (p.o_f32) (static_cast<float*>(p.o) + row0 * DV)[at] = ya[m][r];
      else (static_cast<__bf16*>(p.o) + row0 * DV)[at] = (__bf16)ya[m][r];
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
  constexpr int NT = (MAXK + 15) / 16;
  const int lds = TLay(p.K, C::ROW, DV, 4 * (16 * NT + 4), NT).total;
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
