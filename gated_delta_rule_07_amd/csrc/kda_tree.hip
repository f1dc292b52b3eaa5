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
//   1. keys, queries and decays of the tree's nodes go to LDS, the state to
//      registers, all loads in flight at once;
//   2. one group of d_k / 8 lanes per node walks up its path: c, d and P_t;
//   3. the 2K x d_k by d_k x d_v product runs on the fp32 matrix cores.  Each wave
//      owns d_v / 4 columns and holds the state as the B operand straight from
//      its loads; the A operands P_t k_t and P_t q_t are formed as they are read;
//   4. each wave substitutes through its columns level by level.  Nodes of one
//      level do not depend on each other and are spread over the wave's lanes.
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
  static constexpr int SUB = 64 / CW;                  // nodes one wave substitutes at once
  static constexpr int PAD = 16;                       // bytes between LDS rows: 16 rows cover all banks
  static constexpr int KROW = DK * (int)sizeof(IO) + PAD;
  static constexpr int AROW = DK * 4 + PAD;
  static constexpr int GL = DK / 8;                    // lanes of a node's group
  static constexpr int GROUPS = kTreeThreads / GL;
  static_assert(NW <= 4 && NW * CW == DV, "state waves");
};

// The verify kernel's LDS, in bytes, for K nodes.  x (the 2K products with the
// state) takes the place of the keys, queries and decays.
struct TLay {
  int k, q, a, x, cd, anc, self, beta, par, depth, slot, total;
  __host__ __device__ static int r16(int n) { return (n + 15) & ~15; }
  __host__ __device__ TLay(int K, int krow, int arow, int dv) {
    const int pairs = K * (K - 1) / 2;
    k = 0;
    q = k + K * krow;
    a = q + K * krow;
    x = 0;
    int o = a + K * arow;
    if (o < 2 * K * dv * 4) o = 2 * K * dv * 4;
    cd = r16(o);
    anc = cd + r16(8 * pairs);
    self = anc + r16(pairs);
    beta = self + r16(4 * K);
    par = beta + r16(4 * K);
    depth = par + r16(4 * K);
    slot = depth + r16(4 * K);
    total = slot + 4 * kMaxTree + 16;  // at most 4 K slots (levels padded to whole turns), and their number
  }
};

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int m = 1; m < G; m *= 2) x += __shfl_xor(x, m);
  return x;
}

__device__ __forceinline__ f32x4 lds4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 lds4(const __bf16* p) {
  const u32x2 w = *reinterpret_cast<const u32x2*>(p);
  return f32x4{__builtin_bit_cast(float, w.x << 16), __builtin_bit_cast(float, w.x & 0xffff0000u),
               __builtin_bit_cast(float, w.y << 16), __builtin_bit_cast(float, w.y & 0xffff0000u)};
}

template <typename IO, int DK, int DV, int MAXK>
__global__ __launch_bounds__(kTreeThreads) void kda_tree_verify_kernel(TreeParams p) {
  using C = TCfg<IO, DK, DV>;
  extern __shared__ u32x4 tree_lds[];
  char* sm = reinterpret_cast<char*>(tree_lds);
  const int K = p.K, tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const TLay L(K, C::KROW, C::AROW, DV);
  const int b = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int n = p.n_nodes ? min(max(p.n_nodes[b], 0), K) : K;
  const int page = p.pages ? p.pages[b] : b;
  if (n == 0 || !page_ok(page, p.n_pages)) return;
  const size_t row0 = (size_t)b * K * p.H + h;  // node t: row row0 + t H of the [B][K][H][d] arrays

  int* par = reinterpret_cast<int*>(sm + L.par);
  float* beta = reinterpret_cast<float*>(sm + L.beta);
  if (tid < n) {
    const int up = p.parents[(size_t)b * K + tid];
    par[tid] = up >= -1 && up < tid ? up : -1;
    beta[tid] = p.beta[row0 + (size_t)tid * p.H];
  }
  // keys, queries and decays, 16 bytes a load, then the state
  constexpr int CK = DK * (int)sizeof(IO) / 16, CA = DK * 4 / 16;  // loads of a row
  for (int e = tid; e < n * CK; e += kTreeThreads) {
    const int t = e / CK, c = 16 * (e % CK);
    const size_t at = (row0 + (size_t)t * p.H) * DK * sizeof(IO) + c;
    *reinterpret_cast<u32x4*>(sm + L.k + t * C::KROW + c) = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p.k) + at);
    *reinterpret_cast<u32x4*>(sm + L.q + t * C::KROW + c) = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p.q) + at);
  }
  for (int e = tid; e < n * CA; e += kTreeThreads) {
    const int t = e / CA, c = e % CA;
    *reinterpret_cast<f32x4*>(sm + L.a + t * C::AROW + 16 * c) =
        *reinterpret_cast<const f32x4*>(p.alpha + (row0 + (size_t)t * p.H) * DK + 4 * c);
  }
  const int ln = lane % 16, lg = lane / 16;
  const bool stw = wave < C::NW;  // a state wave
  const int col = C::CW * wave + C::NTL * ln;  // its lane's first column
  float s[DK / 16][4][C::NTL];  // rows 16 kk + 4 lg + e
  if (stw) {
    const float* S = p.pool + ((size_t)page * p.H + h) * DK * DV + col;
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        typedef float row __attribute__((ext_vector_type(C::NTL)));
        const row w = *reinterpret_cast<const row*>(S + (size_t)(16 * kk + 4 * lg + e) * DV);
#pragma unroll
        for (int j = 0; j < C::NTL; ++j) s[kk][e][j] = w[j];
      }
  }
  __syncthreads();

  auto krow = [&](int t) { return reinterpret_cast<const IO*>(sm + L.k + t * C::KROW); };
  auto qrow = [&](int t) { return reinterpret_cast<const IO*>(sm + L.q + t * C::KROW); };
  auto arow = [&](int t) { return reinterpret_cast<float*>(sm + L.a + t * C::AROW); };

  // up each node's path; a lane holds channels 4 gl + {0..3} and DK/2 + 4 gl + {0..3}
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
    const f32x4 k0 = lds4(krow(t) + i0), k1 = lds4(krow(t) + i1);
    const f32x4 q0 = lds4(qrow(t) + i0), q1 = lds4(qrow(t) + i1);
    f32x4 g0 = lds4(arow(t) + i0), g1 = lds4(arow(t) + i1);
    float dt = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) dt += k0[e] * q0[e] + k1[e] * q1[e];
    dt = group_sum<C::GL>(dt);
    const int off = t * (t - 1) / 2;
    int hops = 0;
    for (int r = par[t]; r >= 0; r = par[r], ++hops) {
      const f32x4 w0 = g0 * lds4(krow(r) + i0), w1 = g1 * lds4(krow(r) + i1);
      float cs = 0.0f, ds = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs += w0[e] * k0[e] + w1[e] * k1[e];
        ds += w0[e] * q0[e] + w1[e] * q1[e];
      }
      cs = group_sum<C::GL>(cs);
      ds = group_sum<C::GL>(ds);
      if (gl == 0) {
        cd[off + hops] = float2{cs, ds};
        anc[off + hops] = (unsigned char)r;
      }
      g0 *= lds4(arow(r) + i0);
      g1 *= lds4(arow(r) + i1);
    }
    if (gl == 0) {
      self[t] = dt;
      depth[t] = hops;
    }
    P[it][0] = g0;
    P[it][1] = g1;
  }
  __syncthreads();
  // P takes the decays' place
#pragma unroll
  for (int it = 0; it < NPG; ++it) {
    const int t = it * C::GROUPS + grp;
    if (t >= n) continue;
    *reinterpret_cast<f32x4*>(arow(t) + i0) = P[it][0];
    *reinterpret_cast<f32x4*>(arow(t) + i1) = P[it][1];
  }
  // the order of substitution: level after level, each padded to whole turns of SUB nodes
  signed char* slot = reinterpret_cast<signed char*>(sm + L.slot);
  int* nslots = reinterpret_cast<int*>(sm + L.slot + 4 * kMaxTree);
  if (wave == 3) {
    const int dpt = lane < n ? depth[lane] : -1;
    for (int e = lane; e < 4 * kMaxTree; e += 64) slot[e] = -1;
    int base = 0, left = n;
    for (int lev = 0; left > 0; ++lev) {
      const unsigned long long m = __ballot(dpt == lev);
      if (dpt == lev) slot[base + __popcll(m & ((1ull << lane) - 1))] = (signed char)lane;
      const int cnt = __popcll(m);
      left -= cnt;
      base += (cnt + C::SUB - 1) / C::SUB * C::SUB;
    }
    if (lane == 0) *nslots = base;
  }
  __syncthreads();

  // products with the state
  constexpr int NT = (MAXK + 15) / 16;
  f32x4 xk[NT][C::NTL], xq[NT][C::NTL];
#pragma unroll
  for (int m = 0; m < NT; ++m)
#pragma unroll
    for (int j = 0; j < C::NTL; ++j) xk[m][j] = xq[m][j] = (f32x4)0.0f;
  if (stw) {
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) {
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        if (16 * m >= n) continue;
        const int t = min(16 * m + ln, n - 1);  // (a row past the last node only feeds its own row of the result)
        const int i = 16 * kk + 4 * lg;
        const f32x4 pt = lds4(arow(t) + i);
        const f32x4 pk = pt * lds4(krow(t) + i), pq = pt * lds4(qrow(t) + i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < C::NTL; ++j) {
            xk[m][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(pk[e], s[kk][e][j], xk[m][j], 0, 0, 0);
            xq[m][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(pq[e], s[kk][e][j], xq[m][j], 0, 0, 0);
          }
      }
    }
  }
  __syncthreads();  // keys, queries and decays are done with: x takes their place
  if (!stw) return;
  float* x = reinterpret_cast<float*>(sm + L.x);
#pragma unroll
  for (int m = 0; m < NT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * m + 4 * lg + r;
      if (t >= n) continue;
      const IO* v = static_cast<const IO*>(p.v) + (row0 + (size_t)t * p.H) * DV + col;
#pragma unroll
      for (int j = 0; j < C::NTL; ++j) {
        x[t * DV + col + j] = to_f32(v[j]) - xk[m][j][r];
        x[(K + t) * DV + col + j] = xq[m][j][r];
      }
    }
  }
  // (from here on a wave only reads what it wrote itself)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();

  const int c = C::CW * wave + lane % C::CW, sub = lane / C::CW;
  const int turns = *nslots / C::SUB;
  for (int i = 0; i < turns; ++i) {
    const int t = slot[i * C::SUB + sub];
    if (t >= 0) {
      float xt = x[t * DV + c], yt = x[(K + t) * DV + c];
      const int off = t * (t - 1) / 2, hops = depth[t];
#pragma unroll 4
      for (int j = 0; j < hops; ++j) {
        const float2 w = cd[off + j];
        const float us = x[(int)anc[off + j] * DV + c];
        xt -= w.x * us;
        yt += w.y * us;
      }
      const float ut = beta[t] * xt;
      yt += self[t] * ut;
      x[t * DV + c] = ut;
      const size_t orow = row0 + (size_t)t * p.H;
      if (p.o_f32) static_cast<float*>(p.o)[orow * DV + c] = yt;
      else static_cast<__bf16*>(p.o)[orow * DV + c] = (__bf16)yt;
      p.u[(((size_t)b * p.H + h) * K + t) * DV + c] = ut;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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
  const int lds = TLay(p.K, C::KROW, C::AROW, DV).total;
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
