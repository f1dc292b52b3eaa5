// libkda C ABI: the calls around the recurrence -- norms of queries and keys, the
// cache of state pages, decode on pages and trees of drafted tokens.
//
// Every check runs before any HIP call, so invalid arguments return a status
// without touching the device.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kda_check.h"
#include "kda_launch.h"

namespace {

using namespace kda::check;

static_assert(kda::kMaxTree == KDA_MAX_TREE && kda::kMaxPages == KDA_MAX_PAGES && kda::kMaxForks == KDA_MAX_FORKS &&
                  kda::kMaxPagedSeqs == KDA_MAX_PAGED_SEQS,
              "limits of the header");

// One workgroup of up to 512 threads for each of B H states, fewer than 2^32 threads in all.
bool states_ok(int B, int H) { return (long long)B * H <= (1LL << 22); }

bool table_ok(int n_rows, int width, int n_pages) {
  return n_rows >= 1 && width >= 1 && (long long)n_rows * width <= (1LL << 26) && n_pages >= 1 && n_pages <= KDA_MAX_PAGES;
}

}  // namespace

extern "C" {

kda_status kda_qk_norm(const void* q, long long q_stride, const void* k, long long k_stride, kda_dtype dtype,
                       kda_norm norm, const float* q_weight, const float* k_weight, float eps, float q_scale,
                       const int* positions, const float* inv_freq, int rot, kda_pairing pairing,
                       void* q_out, long long q_out_stride, void* k_out, long long k_out_stride,
                       kda_dtype out_dtype, int n, int H_q, int H_k, int d, hipStream_t stream) {
  if (!dtype_ok(raw_enum(dtype)) || !dtype_ok(raw_enum(out_dtype))) return KDA_ERR_DTYPE;
  const int nm = raw_enum(norm), pr = raw_enum(pairing);
  if ((nm != KDA_NORM_L2 && nm != KDA_NORM_RMS) || (pr != KDA_PAIR_HALVES && pr != KDA_PAIR_ADJACENT)) return KDA_ERR_DTYPE;
  if (n < 0 || H_q < 1 || H_k < 0) return KDA_ERR_SHAPE;
  if (d < 8 || d > 256 || d % 8 || rot < 0 || rot > d || rot % 16) return KDA_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f && eps <= 3.4028235e38f)) return KDA_ERR_SHAPE;
  const long long heads = (long long)H_q + H_k;
  if (heads > (1 << 20) || (long long)n * heads > (1LL << 40) / 256) return KDA_ERR_SHAPE;
  if (n == 0) return KDA_OK;
  if (n > 1) {
    const long long lim = 1LL << 40;  // (n rows of it stay far below 2^63 elements' bytes)
    if (q_stride < (long long)H_q * d || q_out_stride < (long long)H_q * d || q_stride > lim / n || q_out_stride > lim / n)
      return KDA_ERR_SHAPE;
    if (H_k && (k_stride < (long long)H_k * d || k_out_stride < (long long)H_k * d || k_stride > lim / n || k_out_stride > lim / n))
      return KDA_ERR_SHAPE;
  } else {
    q_stride = q_out_stride = (long long)H_q * d;  // (one row: its stride is not used)
    k_stride = k_out_stride = (long long)H_k * d;
  }
  if (!q || !q_out || (H_k && (!k || !k_out)) || (rot && (!positions || !inv_freq))) return KDA_ERR_NULL;
  if (!H_k) k = k_out = nullptr, k_weight = nullptr, k_stride = k_out_stride = 0;
  if (!rot) positions = nullptr, inv_freq = nullptr;
  const int io = io_of(raw_enum(dtype)), oo = io_of(raw_enum(out_dtype));
  const unsigned long long es = io ? 2 : 4, eo = oo ? 2 : 4;
  const void* ptrs[] = {q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out};
  for (const void* ptr : ptrs)
    if (ptr && !aligned16(ptr)) return KDA_ERR_MISALIGNED;
  if ((q_stride * es) % 16 || (k_stride * es) % 16 || (q_out_stride * eo) % 16 || (k_out_stride * eo) % 16)
    return KDA_ERR_MISALIGNED;

  const unsigned long long un = (unsigned long long)n;
  auto rows = [&](const void* ptr, int H, unsigned long long e, long long st) {
    return Rows{reinterpret_cast<uintptr_t>(ptr), ptr ? un : 0, (unsigned long long)H * d * e, (unsigned long long)st * e};
  };
  const Rows rq = rows(q, H_q, es, q_stride), rk = rows(k, H_k, es, k_stride);
  const Rows oq = rows(q_out, H_q, eo, q_out_stride), ok = rows(k_out, H_k, eo, k_out_stride);
  const bool q_same = q_out == q && io == oo && q_out_stride == q_stride;
  const bool k_same = k_out && k_out == k && io == oo && k_out_stride == k_stride;
  if ((!q_same && rows_overlap(oq, rq)) || (!k_same && rows_overlap(ok, rk)) || rows_overlap(oq, rk) ||
      rows_overlap(ok, rq) || rows_overlap(oq, ok))
    return KDA_ERR_ALIAS;
  const Span small[] = {opt_span(q_weight, 4 * (size_t)d), opt_span(k_weight, 4 * (size_t)d),
                        opt_span(positions, 4 * (size_t)n), opt_span(inv_freq, 2 * (size_t)rot)};
  for (const Span& s : small) {
    const Rows r{s.lo, s.hi > s.lo ? 1ull : 0ull, s.hi - s.lo, s.hi - s.lo};
    if (rows_overlap(oq, r) || rows_overlap(ok, r)) return KDA_ERR_ALIAS;
  }
  const kda::HeadsParams p{q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, q_weight, k_weight,
                           positions, inv_freq, eps, q_scale, nm == KDA_NORM_RMS, pr == KDA_PAIR_ADJACENT, rot,
                           n, H_q, H_k, d};
  return launched(kda::launch_heads(p, io, oo, stream));
}

kda_status kda_cache_fork(int* table, int* ref, const int* parents, const int* children, int* moves, int* n_moves,
                          int n, int n_private, int n_rows, int width, int n_pages, hipStream_t stream) {
  if (!table_ok(n_rows, width, n_pages) || n < 0 || n > KDA_MAX_FORKS || n_private < 0 || n_private > width)
    return KDA_ERR_SHAPE;
  // one workgroup looks through n rows, and one thread through a row's private entries
  if ((long long)n * width > (1LL << 26) || n_private > KDA_MAX_PAGES) return KDA_ERR_SHAPE;
  if (!table || !ref || !n_moves || (n > 0 && (!parents || !children || (n_private > 0 && !moves)))) return KDA_ERR_NULL;
  const void* ptrs[] = {table, ref, parents, children, moves, n_moves};
  for (const void* ptr : ptrs)
    if (ptr && !aligned16(ptr)) return KDA_ERR_MISALIGNED;
  const Span st = span(table, (size_t)n_rows * width * 4), sr = span(ref, (size_t)n_pages * 4),
             sm = opt_span(moves, (size_t)n * n_private * 8), sn = span(n_moves, 4);
  const Span ins[] = {opt_span(parents, (size_t)n * 4), opt_span(children, (size_t)n * 4)};
  const Span outs[] = {st, sr, sm, sn};
  for (int i = 0; i < 4; ++i) {
    if (any_overlap(outs[i], ins)) return KDA_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return KDA_ERR_ALIAS;
  }
  const kda::ForkParams p{table, ref, parents, children, moves, n_moves, n, n_private, n_rows, width, n_pages};
  return launched(kda::launch_cache_fork(p, stream));
}

kda_status kda_cache_free(int* table, int* ref, const int* rows, int n, int n_rows, int width, int n_pages,
                          hipStream_t stream) {
  if (!table_ok(n_rows, width, n_pages) || n < 0 || (long long)n * width > (1LL << 31)) return KDA_ERR_SHAPE;
  if (!table || !ref || (n > 0 && !rows)) return KDA_ERR_NULL;
  if (!aligned16(table) || !aligned16(ref) || !aligned16(rows)) return KDA_ERR_MISALIGNED;
  const Span st = span(table, (size_t)n_rows * width * 4), sr = span(ref, (size_t)n_pages * 4),
             sl = opt_span(rows, (size_t)n * 4);
  if (overlap(st, sr) || overlap(st, sl) || overlap(sr, sl)) return KDA_ERR_ALIAS;
  if (n == 0) return KDA_OK;
  return launched(kda::launch_cache_free(table, ref, rows, n, n_rows, width, n_pages, stream));
}

kda_status kda_cache_compact(const int* table, const int* ref, int* table_out, int* ref_out, int* moves, int* n_moves,
                             int* n_live, int n_rows, int width, int n_pages, hipStream_t stream) {
  if (!table_ok(n_rows, width, n_pages)) return KDA_ERR_SHAPE;
  if (!table || !ref || !table_out || !ref_out || !moves || !n_moves || !n_live) return KDA_ERR_NULL;
  const void* ptrs[] = {table, ref, table_out, ref_out, moves, n_moves, n_live};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return KDA_ERR_MISALIGNED;
  const size_t tb = (size_t)n_rows * width * 4, rb = (size_t)n_pages * 4;
  const Span ti = span(table, tb), ri = span(ref, rb);
  const Span outs[] = {span(table_out, tb), span(ref_out, rb), span(moves, (size_t)std::max(n_pages / 2, 1) * 8),
                       span(n_moves, 4), span(n_live, 4)};
  for (int i = 0; i < 5; ++i) {
    if (!(i == 0 && table_out == table) && overlap(outs[i], ti)) return KDA_ERR_ALIAS;
    if (!(i == 1 && ref_out == ref) && overlap(outs[i], ri)) return KDA_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return KDA_ERR_ALIAS;
  }
  const kda::CompactParams p{table, ref, table_out, ref_out, moves, n_moves, n_live, n_rows, width, n_pages};
  return launched(kda::launch_cache_compact(p, stream));
}

kda_status kda_cache_copy(const void* src, void* dst, size_t page_bytes, int n_layers, int n_src_pages, int n_dst_pages,
                          const int* moves, const int* n_moves, int max_moves, hipStream_t stream) {
  if (page_bytes < 1 || page_bytes > ((size_t)1 << 36) || n_layers < 1 || n_layers > 65536 || n_src_pages < 1 ||
      n_src_pages > KDA_MAX_PAGES || n_dst_pages < 1 || n_dst_pages > KDA_MAX_PAGES || max_moves < 0 ||
      max_moves > KDA_MAX_PAGES)
    return KDA_ERR_SHAPE;
  if (page_bytes % 16) return KDA_ERR_MISALIGNED;
  const size_t most = (size_t)std::max(n_src_pages, n_dst_pages) * n_layers;  // <= 2^32
  if (page_bytes > ((size_t)1 << 46) / most) return KDA_ERR_SHAPE;
  if (!src || !dst || (max_moves > 0 && !moves)) return KDA_ERR_NULL;
  const void* ptrs[] = {src, dst, moves, n_moves};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return KDA_ERR_MISALIGNED;
  const Span ss = span(src, page_bytes * n_layers * n_src_pages), sd = span(dst, page_bytes * n_layers * n_dst_pages);
  const bool same = src == dst && n_src_pages == n_dst_pages;
  const Span lists[] = {opt_span(moves, (size_t)max_moves * 8), opt_span(n_moves, 4)};
  if ((!same && overlap(ss, sd)) || any_overlap(sd, lists)) return KDA_ERR_ALIAS;
  if (max_moves == 0) return KDA_OK;
  const kda::CopyParams p{static_cast<const char*>(src), static_cast<char*>(dst), page_bytes, n_layers, n_src_pages,
                          n_dst_pages, moves, n_moves, max_moves, same};
  return launched(kda::launch_cache_copy(p, stream));
}

kda_status kda_decode_step_paged(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const float* alpha,
                                 const void* z, const float* A, const float* beta, float* pool, int n_pages,
                                 const int* pages_in, const int* pages_out, void* o, kda_dtype o_dtype, int B, int H,
                                 int d_k, int d_v, hipStream_t stream) {
  if (!dtype_ok(raw_enum(qkv_dtype)) || !dtype_ok(raw_enum(o_dtype))) return KDA_ERR_DTYPE;
  if (B < 1 || B > KDA_MAX_PAGED_SEQS || H < 1 || n_pages < 1 || n_pages > KDA_MAX_PAGES) return KDA_ERR_SHAPE;
  if (!dim_ok(d_k) || !dim_ok(d_v)) return KDA_ERR_UNSUPPORTED;
  if (!states_ok(B, H) || !sizes_ok(n_pages, 1, H, d_k, d_v)) return KDA_ERR_SHAPE;
  if (alpha) z = nullptr, A = nullptr;
  if (!q || !k || !v || (!alpha && (!z || !A)) || !beta || !pool || !pages_in || !o) return KDA_ERR_NULL;
  const void* ptrs[] = {q, k, v, alpha, z, A, beta, pool, pages_in, pages_out, o};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return KDA_ERR_MISALIGNED;
  const int io = io_of(raw_enum(qkv_dtype));
  if (!kda::decode_supported(io, d_k, d_v)) return KDA_ERR_UNSUPPORTED;
  const size_t esz = io ? 2 : 4, osz = io_of(raw_enum(o_dtype)) ? 2 : 4, nbh = (size_t)B * H;
  const Span so = span(o, nbh * d_v * osz), sp = span(pool, (size_t)n_pages * H * d_k * d_v * 4);
  const Span ins[] = {span(q, nbh * d_k * esz), span(k, nbh * d_k * esz), span(v, nbh * d_v * esz),
                      opt_span(alpha, nbh * d_k * 4), opt_span(z, nbh * d_k * esz), opt_span(A, (size_t)H * 4),
                      span(beta, nbh * 4), span(pages_in, (size_t)B * 4), opt_span(pages_out, (size_t)B * 4)};
  if (overlap(so, sp) || any_overlap(so, ins) || any_overlap(sp, ins)) return KDA_ERR_ALIAS;
  const kda::DecodeParams p{q, k, v, alpha, beta, pool, o, B, H, d_k, d_v, io_of(raw_enum(o_dtype)) ? 0 : 1, z, A,
                            pages_in, pages_out, n_pages};
  return launched(kda::launch_decode(p, io, stream));
}

kda_status kda_tree_verify(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const float* alpha,
                           const float* beta, const float* pool, int n_pages, const int* pages, const int* parents,
                           const int* n_nodes, void* o, kda_dtype o_dtype, float* u, int B, int K, int H, int d_k,
                           int d_v, hipStream_t stream) {
  if (!dtype_ok(raw_enum(qkv_dtype)) || !dtype_ok(raw_enum(o_dtype))) return KDA_ERR_DTYPE;
  if (B < 1 || H < 1 || K < 1 || K > KDA_MAX_TREE || n_pages < 1 || n_pages > KDA_MAX_PAGES) return KDA_ERR_SHAPE;
  if (!dim_ok(d_k) || !dim_ok(d_v)) return KDA_ERR_UNSUPPORTED;
  if (!states_ok(B, H) || !sizes_ok(n_pages, 1, H, d_k, d_v) || (!pages && n_pages < B)) return KDA_ERR_SHAPE;
  if ((long long)K * H * std::max(d_k, d_v) >= (1LL << 30)) return KDA_ERR_SHAPE;  // (offsets within a sequence)
  if (!q || !k || !v || !alpha || !beta || !pool || !parents || !o || !u) return KDA_ERR_NULL;
  const void* ptrs[] = {q, k, v, alpha, beta, pool, pages, parents, n_nodes, o, u};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return KDA_ERR_MISALIGNED;
  const int io = io_of(raw_enum(qkv_dtype));
  if (!kda::tree_supported(io, d_k, d_v)) return KDA_ERR_UNSUPPORTED;
  const size_t esz = io ? 2 : 4, osz = io_of(raw_enum(o_dtype)) ? 2 : 4, ntok = (size_t)B * K * H;
  const Span so = span(o, ntok * d_v * osz), su = span(u, ntok * d_v * 4);
  const Span ins[] = {span(q, ntok * d_k * esz), span(k, ntok * d_k * esz), span(v, ntok * d_v * esz),
                      span(alpha, ntok * d_k * 4), span(beta, ntok * 4),
                      span(pool, (size_t)n_pages * H * d_k * d_v * 4), opt_span(pages, (size_t)B * 4),
                      span(parents, (size_t)B * K * 4), opt_span(n_nodes, (size_t)B * 4)};
  if (overlap(so, su) || any_overlap(so, ins) || any_overlap(su, ins)) return KDA_ERR_ALIAS;
  const kda::TreeParams p{q, k, v, alpha, beta, pool, pages, parents, n_nodes, o, u, n_pages, B, K, H, d_k, d_v,
                          io_of(raw_enum(o_dtype)) ? 0 : 1};
  return launched(kda::launch_tree_verify(p, io, stream));
}

kda_status kda_tree_commit(const void* k, kda_dtype qkv_dtype, const float* alpha, const float* u, const int* parents,
                           const int* n_nodes, const int* last, float* pool, int n_pages, const int* pages_in,
                           const int* pages_out, int B, int K, int H, int d_k, int d_v, hipStream_t stream) {
  if (!dtype_ok(raw_enum(qkv_dtype))) return KDA_ERR_DTYPE;
  if (B < 1 || B > KDA_MAX_PAGED_SEQS || H < 1 || K < 1 || K > KDA_MAX_TREE || n_pages < 1 || n_pages > KDA_MAX_PAGES)
    return KDA_ERR_SHAPE;
  if (!dim_ok(d_k) || !dim_ok(d_v)) return KDA_ERR_UNSUPPORTED;
  if (!states_ok(B, H) || !sizes_ok(n_pages, 1, H, d_k, d_v) || (!pages_in && n_pages < B)) return KDA_ERR_SHAPE;
  if (!k || !alpha || !u || !parents || !last || !pool) return KDA_ERR_NULL;
  const void* ptrs[] = {k, alpha, u, parents, n_nodes, last, pool, pages_in, pages_out};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return KDA_ERR_MISALIGNED;
  const int io = io_of(raw_enum(qkv_dtype));
  if (!kda::tree_supported(io, d_k, d_v)) return KDA_ERR_UNSUPPORTED;
  const size_t esz = io ? 2 : 4, ntok = (size_t)B * K * H;
  const Span sp = span(pool, (size_t)n_pages * H * d_k * d_v * 4);
  const Span ins[] = {span(k, ntok * d_k * esz), span(alpha, ntok * d_k * 4), span(u, ntok * d_v * 4),
                      span(parents, (size_t)B * K * 4), opt_span(n_nodes, (size_t)B * 4), span(last, (size_t)B * 4),
                      opt_span(pages_in, (size_t)B * 4), opt_span(pages_out, (size_t)B * 4)};
  if (any_overlap(sp, ins)) return KDA_ERR_ALIAS;
  const kda::TreeCommitParams p{k, alpha, u, parents, n_nodes, last, pool, pages_in, pages_out, n_pages, B, K, H, d_k, d_v};
  return launched(kda::launch_tree_commit(p, io, stream));
}

}  // extern "C"
