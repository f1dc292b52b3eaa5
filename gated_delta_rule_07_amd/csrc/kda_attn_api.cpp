// libkda C ABI: the attention layers beside the recurrent ones -- attention over prompts,
// keys and values on pages, and attention over those.
//
// Every check runs before any HIP call, so invalid arguments return a status
// without touching the device.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kda_check.h"
#include "kda_launch.h"

namespace {

using namespace kda::check;

typedef unsigned long long u64;

bool head_dim_ok(int d) { return d == 64 || d == 128; }
bool kv_dtype_ok(int t) { return t == KDA_BF16 || t == KDA_E4M3; }
bool heads_ok(int Hq, int Hk) {
  return Hq >= 1 && Hk >= 1 && Hq <= KDA_MAX_HEADS && Hk <= KDA_MAX_HEADS && Hq % Hk == 0;
}
bool page_tokens_ok(int t) { return t == 16 || t == 32 || t == 64 || t == 128; }
size_t page_bytes(int kv, int pt, int H, int dk, int dv) {
  const size_t values = (size_t)H * pt * (dk + dv);
  return kv == KDA_E4M3 ? values + ((size_t)H * 8 + 15) / 16 * 16 : values * 2;
}

// Status of what the calls on pages share, and the cache as the kernels take it.
kda_status cache_of(const void* pool, int kv, int n_pages, int pt, const int* table, int n_rows, int width, const int* rows,
                    int N, int H, int dk, int dv, kda::KvCache* c) {
  if (!kv_dtype_ok(kv)) return KDA_ERR_DTYPE;
  if (N < 1 || N > KDA_MAX_PAGED_SEQS || H < 1 || H > KDA_MAX_HEADS || n_pages < 1 || n_pages > KDA_MAX_PAGES || n_rows < 1 ||
      width < 1 || (long long)n_rows * width > (1LL << 26))
    return KDA_ERR_SHAPE;
  if (!page_tokens_ok(pt) || !head_dim_ok(dk) || !head_dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
  if ((long long)width * pt >= (1LL << 31) || (!rows && N > n_rows)) return KDA_ERR_SHAPE;
  if (!pool || !table) return KDA_ERR_NULL;
  if (!aligned16(pool) || !aligned16(table) || !aligned16(rows)) return KDA_ERR_MISALIGNED;
  *c = kda::KvCache{static_cast<char*>(const_cast<void*>(pool)), page_bytes(kv, pt, H, dk, dv), table, rows, n_pages, pt,
                    n_rows, width, H, dk, dv, kv == KDA_E4M3};
  return KDA_OK;
}

Span pool_span(const kda::KvCache& c) { return span(c.pool, c.page_bytes * c.n_pages); }
Rows flat(const Span& s) { return Rows{s.lo, s.hi > s.lo ? 1ull : 0ull, s.hi - s.lo, s.hi - s.lo}; }
Rows rows_of(const void* p, int n, int H, int d, u64 e, long long stride) {
  return Rows{reinterpret_cast<uintptr_t>(p), p ? (u64)n : 0, (u64)H * d * e, (u64)stride * e};
}
// Row strides of n rows of H d elements: KDA_OK, or what is wrong.  One row's stride is not used.
kda_status stride_ok(long long* stride, int n, int H, int d, int e) {
  if (n <= 1) *stride = (long long)H * d;
  if (*stride < (long long)H * d || *stride > (1LL << 40) / std::max(n, 1)) return KDA_ERR_SHAPE;
  return *stride * e % 16 ? KDA_ERR_MISALIGNED : KDA_OK;
}
bool finite(float x) { return x - x == 0.0f; }
// Decode counts a row's tokens in 32 bits, rounded up to runs of up to 256 and with a run ahead.
bool decode_row_ok(int width, int pt) { return (long long)width * pt <= (1LL << 31) - 512; }

}  // namespace

extern "C" {

kda_status kda_attn_fwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                        long long v_stride, kda_dtype dtype, float scale, const int* cu_seqlens,
                        const int* cu_seqlens_k, int N, int total_q, int total_k, void* o, long long o_stride,
                        kda_dtype o_dtype, int H_q, int H_kv, int d_k, int d_v, hipStream_t stream) {
  if (!dtype_ok(raw_enum(dtype)) || !dtype_ok(raw_enum(o_dtype))) return KDA_ERR_DTYPE;
  if (N < 1 || N > KDA_MAX_CALL_TOKENS || total_q < 0 || total_k < 0 || total_q > KDA_MAX_CALL_TOKENS ||
      total_k > KDA_MAX_CALL_TOKENS || !heads_ok(H_q, H_kv) || !finite(scale))
    return KDA_ERR_SHAPE;
  if (!dim_ok(d_k) || !dim_ok(d_v)) return KDA_ERR_UNSUPPORTED;
  if (!cu_seqlens && cu_seqlens_k) return KDA_ERR_NULL;
  if (!cu_seqlens && (total_q % N || total_k % N)) return KDA_ERR_SHAPE;
  if (cu_seqlens && !cu_seqlens_k && total_q != total_k) return KDA_ERR_SHAPE;
  // fewer than 2^32 threads: 256 for each head and 16 rows, each sequence's rounded up, and all rounded up to 8
  if (((long long)total_q / 64 + N + 2) * H_q > (1LL << 22)) return KDA_ERR_SHAPE;
  if (total_q == 0) return KDA_OK;
  if (!q || !o || (total_k > 0 && (!k || !v))) return KDA_ERR_NULL;
  const int io = io_of(raw_enum(dtype)), oo = io_of(raw_enum(o_dtype));
  const int es = io ? 2 : 4, eo = oo ? 2 : 4;
  if (!total_k) k = v = nullptr;
  const void* ptrs[] = {q, k, v, o, cu_seqlens, cu_seqlens_k};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
  const kda_status st[] = {stride_ok(&q_stride, total_q, H_q, d_k, es), stride_ok(&k_stride, total_k, H_kv, d_k, es),
                           stride_ok(&v_stride, total_k, H_kv, d_v, es), stride_ok(&o_stride, total_q, H_q, d_v, eo)};
  for (kda_status x : st)
    if (x != KDA_OK) return x;
  const Rows ro = rows_of(o, total_q, H_q, d_v, eo, o_stride);
  const Rows ins[] = {rows_of(q, total_q, H_q, d_k, es, q_stride), rows_of(k, total_k, H_kv, d_k, es, k_stride),
                      rows_of(v, total_k, H_kv, d_v, es, v_stride), flat(opt_span(cu_seqlens, ((size_t)N + 1) * 4)),
                      flat(opt_span(cu_seqlens_k, ((size_t)N + 1) * 4))};
  for (const Rows& r : ins)
    if (rows_overlap(ro, r)) return KDA_ERR_ALIAS;
  const kda::AttnParams p{q, k, v, o, q_stride, k_stride, v_stride, o_stride, cu_seqlens, cu_seqlens_k, N, total_q, total_k,
                          H_q, H_kv, d_k, d_v, oo ? 0 : 1, scale};
  return launched(kda::launch_attn_fwd(p, io, stream));
}

kda_status kda_kv_page_bytes(kda_dtype kv_dtype, int page_tokens, int H_kv, int d_k, int d_v, size_t* bytes) {
  if (!kv_dtype_ok(raw_enum(kv_dtype))) return KDA_ERR_DTYPE;
  if (H_kv < 1 || H_kv > KDA_MAX_HEADS) return KDA_ERR_SHAPE;
  if (!page_tokens_ok(page_tokens) || !head_dim_ok(d_k) || !head_dim_ok(d_v)) return KDA_ERR_UNSUPPORTED;
  if (!bytes) return KDA_ERR_NULL;
  *bytes = page_bytes(raw_enum(kv_dtype), page_tokens, H_kv, d_k, d_v);
  return KDA_OK;
}

kda_status kda_kv_append(const void* k, long long k_stride, const void* v, long long v_stride, const void* q,
                         long long q_stride, kda_dtype dtype, const int* positions, const float* inv_freq, int rot,
                         kda_pairing pairing, void* q_out, long long q_out_stride, void* k_out,
                         long long k_out_stride, void* pool, kda_dtype kv_dtype, int n_pages, int page_tokens,
                         const int* table, int n_rows, int width, const int* rows, const int* lens,
                         const int* cu_seqlens, int N, int total, int H_q, int H_kv, int d_k, int d_v,
                         hipStream_t stream) {
  const int pr = raw_enum(pairing);
  if (!dtype_ok(raw_enum(dtype)) || (pr != KDA_PAIR_HALVES && pr != KDA_PAIR_ADJACENT)) return KDA_ERR_DTYPE;
  if (total < 0 || total > KDA_MAX_CALL_TOKENS || (!cu_seqlens && total != N)) return KDA_ERR_SHAPE;
  kda::KvCache c;
  const kda_status bad = cache_of(pool, raw_enum(kv_dtype), n_pages, page_tokens, table, n_rows, width, rows, N, H_kv, d_k, d_v, &c);
  if (bad != KDA_OK) return bad;
  if (!q) H_q = H_kv;
  if (!heads_ok(H_q, H_kv)) return KDA_ERR_SHAPE;
  if (rot < 0 || rot > d_k || rot % 16) return KDA_ERR_UNSUPPORTED;
  if (total == 0) return KDA_OK;
  if (!k || !v || !lens || (q && !q_out) || (!q && q_out) || (rot && !inv_freq)) return KDA_ERR_NULL;
  if (!rot) inv_freq = nullptr, positions = nullptr;
  const int io = io_of(raw_enum(dtype)), es = io ? 2 : 4;
  const void* ptrs[] = {k, v, q, positions, inv_freq, q_out, k_out, lens, cu_seqlens};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
  if (!q) q_stride = q_out_stride = (long long)H_q * d_k;
  if (!k_out) k_out_stride = (long long)H_kv * d_k;
  const kda_status st[] = {stride_ok(&k_stride, total, H_kv, d_k, es), stride_ok(&v_stride, total, H_kv, d_v, es),
                           stride_ok(&q_stride, total, H_q, d_k, es), stride_ok(&q_out_stride, total, H_q, d_k, es),
                           stride_ok(&k_out_stride, total, H_kv, d_k, es)};
  for (kda_status x : st)
    if (x != KDA_OK) return x;
  const Rows rq = rows_of(q, total, H_q, d_k, es, q_stride), rk = rows_of(k, total, H_kv, d_k, es, k_stride),
             rv = rows_of(v, total, H_kv, d_v, es, v_stride), oq = rows_of(q_out, total, H_q, d_k, es, q_out_stride),
             ok = rows_of(k_out, total, H_kv, d_k, es, k_out_stride), op = flat(pool_span(c));
  const bool q_same = q_out && q_out == q && q_out_stride == q_stride, k_same = k_out && k_out == k && k_out_stride == k_stride;
  if ((!q_same && rows_overlap(oq, rq)) || rows_overlap(oq, rk) || rows_overlap(oq, rv) || (!k_same && rows_overlap(ok, rk)) ||
      rows_overlap(ok, rq) || rows_overlap(ok, rv) || rows_overlap(oq, ok) || rows_overlap(op, rq) || rows_overlap(op, rk) ||
      rows_overlap(op, rv) || rows_overlap(op, oq) || rows_overlap(op, ok))
    return KDA_ERR_ALIAS;
  const Span small[] = {opt_span(positions, 4 * (size_t)total), opt_span(inv_freq, 2 * (size_t)rot), span(lens, 4 * (size_t)N),
                        opt_span(cu_seqlens, 4 * ((size_t)N + 1)), span(table, 4 * (size_t)n_rows * width),
                        opt_span(rows, 4 * (size_t)N)};
  for (const Span& s : small)
    if (rows_overlap(op, flat(s)) || rows_overlap(oq, flat(s)) || rows_overlap(ok, flat(s))) return KDA_ERR_ALIAS;
  const kda::AppendParams p{c, k, v, q, k_out, q_out, k_stride, v_stride, q_stride, k_out_stride, q_out_stride, lens, cu_seqlens,
                            positions, inv_freq, rot, pr == KDA_PAIR_ADJACENT, N, total, H_q};
  return launched(kda::launch_kv_append(p, io, stream));
}

kda_status kda_kv_read(const void* pool, kda_dtype kv_dtype, int n_pages, int page_tokens, const int* table, int n_rows,
                       int width, const int* rows, const int* starts, const int* cu_seqlens, void* k_out, void* v_out,
                       kda_dtype out_dtype, int N, int total, int H_kv, int d_k, int d_v, hipStream_t stream) {
  if (!dtype_ok(raw_enum(out_dtype))) return KDA_ERR_DTYPE;
  if (total < 0 || total > KDA_MAX_CALL_TOKENS) return KDA_ERR_SHAPE;
  kda::KvCache c;
  const kda_status bad = cache_of(pool, raw_enum(kv_dtype), n_pages, page_tokens, table, n_rows, width, rows, N, H_kv, d_k, d_v, &c);
  if (bad != KDA_OK) return bad;
  if (total == 0) return KDA_OK;
  if (!cu_seqlens || !k_out || !v_out) return KDA_ERR_NULL;
  const void* ptrs[] = {starts, cu_seqlens, k_out, v_out};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
  const int oo = io_of(raw_enum(out_dtype));
  const size_t row = (size_t)total * H_kv * (oo ? 2 : 4);
  const Span sk = span(k_out, row * d_k), sv = span(v_out, row * d_v);
  const Span ins[] = {pool_span(c), span(table, 4 * (size_t)n_rows * width), opt_span(rows, 4 * (size_t)N),
                      opt_span(starts, 4 * (size_t)N), span(cu_seqlens, 4 * ((size_t)N + 1))};
  if (overlap(sk, sv) || any_overlap(sk, ins) || any_overlap(sv, ins)) return KDA_ERR_ALIAS;
  const kda::ReadParams p{c, cu_seqlens, starts, k_out, v_out, N, total};
  return launched(kda::launch_kv_read(p, oo, stream));
}

kda_status kda_attn_decode_plan(kda_dtype kv_dtype, int page_tokens, int width, int B, int K, int H_q, int H_kv, int d_k,
                                int d_v, size_t* workspace_bytes) {
  if (!kv_dtype_ok(raw_enum(kv_dtype))) return KDA_ERR_DTYPE;
  if (B < 1 || B > KDA_MAX_PAGED_SEQS || K < 1 || K > KDA_MAX_ATTN_TOKENS || width < 1 || !heads_ok(H_q, H_kv)) return KDA_ERR_SHAPE;
  if (!page_tokens_ok(page_tokens) || !head_dim_ok(d_k) || !head_dim_ok(d_v)) return KDA_ERR_UNSUPPORTED;
  if (!decode_row_ok(width, page_tokens)) return KDA_ERR_SHAPE;
  if (!workspace_bytes) return KDA_ERR_NULL;
  *workspace_bytes = kda::attn_decode_workspace(B, K, H_q, H_kv, d_v, page_tokens, width);
  return KDA_OK;
}

kda_status kda_attn_decode(const void* q, kda_dtype q_dtype, float scale, const void* pool, kda_dtype kv_dtype, int n_pages,
                           int page_tokens, const int* table, int n_rows, int width, const int* rows, const int* lens,
                           void* o, kda_dtype o_dtype, void* workspace, size_t workspace_bytes, int B, int K, int H_q,
                           int H_kv, int d_k, int d_v, hipStream_t stream) {
  if (!dtype_ok(raw_enum(q_dtype)) || !dtype_ok(raw_enum(o_dtype))) return KDA_ERR_DTYPE;
  if (K < 1 || K > KDA_MAX_ATTN_TOKENS || !heads_ok(H_q, H_kv) || !finite(scale)) return KDA_ERR_SHAPE;
  kda::KvCache c;
  const kda_status bad = cache_of(pool, raw_enum(kv_dtype), n_pages, page_tokens, table, n_rows, width, rows, B, H_kv, d_k, d_v, &c);
  if (bad != KDA_OK) return bad;
  // 32-bit counts: granules of 128 tokens over the sequences, and threads (a workgroup of up to 512 for each unit)
  if (!decode_row_ok(width, page_tokens) || (long long)B * (((long long)width * page_tokens + 127) / 128) >= (1LL << 31) ||
      (long long)B * K * H_q > (1LL << 22))
    return KDA_ERR_SHAPE;
  const size_t need = kda::attn_decode_workspace(B, K, H_q, H_kv, d_v, page_tokens, width);
  if (!q || !lens || !o || (need && !workspace)) return KDA_ERR_NULL;
  if (need && workspace_bytes < need) return KDA_ERR_SHAPE;
  if (!need) workspace = nullptr;
  const void* ptrs[] = {q, lens, o, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
  const int io = io_of(raw_enum(q_dtype)), oo = io_of(raw_enum(o_dtype));
  const size_t n = (size_t)B * K * H_q;
  const Span so = span(o, n * d_v * (oo ? 2 : 4)), sw = opt_span(workspace, need);
  const Span ins[] = {span(q, n * d_k * (io ? 2 : 4)), pool_span(c), span(table, 4 * (size_t)n_rows * width),
                      opt_span(rows, 4 * (size_t)B), span(lens, 4 * (size_t)B)};
  if (overlap(so, sw) || any_overlap(so, ins) || any_overlap(sw, ins)) return KDA_ERR_ALIAS;
  const kda::AttnDecodeParams p{c, q, lens, o, workspace, B, K, H_q, oo ? 0 : 1, scale};
  return launched(kda::launch_attn_decode(p, io, stream));
}

}  // extern "C"
