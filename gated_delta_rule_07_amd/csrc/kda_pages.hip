// The cache of state pages for gfx950: rows of a page table forked, freed and
// packed, and pages copied.
//
// Tables, reference counts and move lists are some KB, read and written once by
// one workgroup (free: one thread per entry), so those calls cost a launch and a
// few passes' latency.  Everything that has an order -- which free page a fork
// gets, which hole a page moves to -- comes from prefix sums over the pages and
// forks, never from the order of atomics, so the same inputs give the same pages.
// Copying the pages is bound by HBM: each page is read once and written once.
//
// Measured: 1 and 64 forks over 64 and 160 pages 5.2 and 8 to 9.5 us, packing 97 pages under a
// table of 96 entries 5.2 us, freeing 64 rows 3.4 to 5.2 us.
#include <algorithm>

#include "kda_device.h"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kMetaThreads = 1024;
constexpr int kMetaWaves = kMetaThreads / 64;

// Exclusive prefix sum of x over the workgroup's threads; *total: the sum.
// Every thread calls it; `sums` holds kMetaWaves ints.
__device__ __forceinline__ int block_scan(int x, int* sums, int* total) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int v = x;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const int y = __shfl_up(v, m);
    if (lane >= m) v += y;
  }
  __syncthreads();  // (the last call's sums have been read)
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kMetaWaves; ++w) {
    const int s = sums[w];
    before += w < wave ? s : 0;
    all += s;
  }
  *total = all;
  return before + v - x;
}

__global__ __launch_bounds__(kMetaThreads) void kda_cache_fork_kernel(ForkParams p) {
  __shared__ int sums[kMetaWaves];
  __shared__ __align__(16) int child[kMaxForks];  // the row a fork may start, -1: refused
  __shared__ int taken[kMaxForks];  // that row holds a page
  const int tid = threadIdx.x;
  int par = -2, ch = -1;
  if (tid < p.n) {
    par = p.parents[tid];
    ch = p.children[tid];
    if (ch < 0 || ch >= p.n_rows || par < -1 || par >= p.n_rows) ch = -1;
  }
  child[tid] = ch;
  taken[tid] = 0;
  __syncthreads();
  // children's rows that hold a page
  const long long entries = (long long)p.n * p.width;
  for (long long e = tid; e < entries; e += kMetaThreads) {
    const int i = (int)(e / p.width), c = child[i];
    if (c >= 0 && page_ok(p.table[(size_t)c * p.width + e % p.width], p.n_pages)) taken[i] = 1;
  }
  __syncthreads();
  bool ok = ch >= 0 && !taken[tid];
  __syncthreads();
  if (!ok) child[tid] = -1;
  __syncthreads();
  // the first fork that names a child has it; a parent that is itself started
  // here was an empty row before the call
  bool empty = false;
  if (ok) {
    for (int j = 0; j < p.n; j += 4) {  // (past the last fork: -1)
      const int4 c = *reinterpret_cast<const int4*>(child + j);
      const int cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ok &= !(j + e < tid && cs[e] == ch);
        empty |= cs[e] >= 0 && cs[e] == par;
      }
    }
  }
  int need = 0;
  if (ok && !empty) {
    if (par < 0) need = p.n_private;
    else
      for (int w = 0; w < p.n_private; ++w) need += page_ok(p.table[(size_t)par * p.width + w], p.n_pages);
  }
  int wanted = 0;
  const int at = block_scan(need, sums, &wanted);

  // the lowest free pages, as many as are wanted (moves has room for them all)
  int found = 0;
  for (int base = 0; base < p.n_pages && found < wanted; base += kMetaThreads) {
    const int page = base + tid;
    const int is_free = page < p.n_pages && p.ref[page] <= 0;
    int here = 0;
    const int rank = found + block_scan(is_free, sums, &here);
    if (is_free && rank < wanted) p.moves[2 * rank + 1] = page;
    found += here;
  }
  found = min(found, wanted);
  __syncthreads();  // (the pages listed are seen by all threads from here on)
  const bool served = ok && at + need <= found;
  int used = 0;
  (void)block_scan(served ? need : 0, sums, &used);
  if (tid == 0) *p.n_moves = used;
  for (int r = tid; r < used; r += kMetaThreads) p.ref[p.moves[2 * r + 1]] = 1;
  // children's first entries
  if (served) {
    int r = at;
    for (int w = 0; w < p.n_private; ++w) {
      int page = -1;
      const int from = par < 0 || empty ? -1 : p.table[(size_t)par * p.width + w];
      if (!empty && (par < 0 || page_ok(from, p.n_pages))) {
        page = p.moves[2 * r + 1];
        p.moves[2 * r] = from;
        ++r;
      }
      p.table[(size_t)ch * p.width + w] = page;
    }
  }
  // and the pages they share
  child[tid] = served ? ch : -1;
  taken[tid] = served && !empty ? par : -1;
  __syncthreads();
  const int shared = p.width - p.n_private;
  for (long long e = tid; e < (long long)p.n * shared; e += kMetaThreads) {
    const int i = (int)(e / shared), w = p.n_private + (int)(e % shared);
    if (child[i] < 0) continue;
    int page = taken[i] < 0 ? -1 : p.table[(size_t)taken[i] * p.width + w];
    if (page_ok(page, p.n_pages)) atomicAdd(&p.ref[page], 1);
    else page = -1;
    p.table[(size_t)child[i] * p.width + w] = page;
  }
}

__global__ __launch_bounds__(256) void kda_cache_free_kernel(int* table, int* ref, const int* rows, int n, int n_rows,
                                                             int width, int n_pages) {
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= (long long)n * width) return;
  const int row = rows[e / width];
  if (row < 0 || row >= n_rows) return;
  // an entry is taken out once however often its row is listed
  const int page = atomicExch(&table[(size_t)row * width + e % width], -1);
  if (!page_ok(page, n_pages)) return;
  int old = ref[page];
  while (old > 0) {
    const int seen = atomicCAS(&ref[page], old, old - 1);
    if (seen == old) break;
    old = seen;
  }
}

// The index of x in moves[.][which], ascending, of n entries; -1: not there.
__device__ __forceinline__ int find_move(const int* moves, int n, int which, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (moves[2 * mid + which] < x) lo = mid + 1;
    else hi = mid;
  }
  return lo < n && moves[2 * lo + which] == x ? lo : -1;
}

// The table after the n moves: what a page became follows from the moves alone.
__device__ __forceinline__ void rename_entries(const CompactParams& p, int n, int live, long long first, long long step) {
  const long long entries = (long long)p.n_rows * p.width;
  for (long long e = first; e < entries; e += step) {
    const int page = p.table[e];
    int now = -1;
    if (page_ok(page, p.n_pages)) {
      if (page < live) now = find_move(p.moves, n, 1, page) < 0 ? page : -1;
      else {
        const int m = find_move(p.moves, n, 0, page);
        if (m >= 0) now = p.moves[2 * m + 1];
      }
    }
    p.table_out[e] = now;
  }
}

// Tables of at most two entries a thread are renamed by the one workgroup that packs the pages, larger ones by a launch of
// their own.  Measured in a graph, one launch against two: with 97 pages 5.5 against 6.1 us for 96 entries, 6.9 against 7.4
// for 1,026, 7.3 against 7.3 for 2,048, 18.7 against 7.4 for 8,192; with 1,024 pages 6.4 against 7.3, 8.0 against 8.6, 9.8
// against 8.8 and 26.6 against 9.1.
constexpr long long kSmallTable = 2 * kMetaThreads;

__global__ __launch_bounds__(kMetaThreads) void kda_cache_compact_kernel(CompactParams p) {
  __shared__ int sums[kMetaWaves];
  const int tid = threadIdx.x;
  int mine = 0;
  for (int page = tid; page < p.n_pages; page += kMetaThreads) mine += p.ref[page] > 0;
  int live = 0;
  (void)block_scan(mine, sums, &live);
  // below `live` the holes, above it the pages that move: as many of one as of the other
  int holes = 0, movers = 0;
  for (int base = 0; base < p.n_pages; base += kMetaThreads) {
    const int page = base + tid;
    const bool held = page < p.n_pages && p.ref[page] > 0;
    const int hole = page < live && !held, mover = page >= live && held;
    int h = 0, m = 0;
    const int hr = holes + block_scan(hole, sums, &h);
    const int mr = movers + block_scan(mover, sums, &m);
    if (hole) p.moves[2 * hr + 1] = page;
    if (mover) p.moves[2 * mr] = page;
    holes += h;
    movers += m;
  }
  if (tid == 0) {
    *p.n_moves = movers;
    *p.n_live = live;
  }
  __syncthreads();
  // (in place, the refs read here are those of pages at or above `live`, the ones
  // written are holes)
  for (int r = tid; r < movers; r += kMetaThreads) p.ref_out[p.moves[2 * r + 1]] = p.ref[p.moves[2 * r]];
  __syncthreads();
  for (int page = tid; page < p.n_pages; page += kMetaThreads) {
    if (page >= live) p.ref_out[page] = 0;
    else if (p.ref[page] > 0) p.ref_out[page] = p.ref[page];  // (in place, a filled hole writes itself)
  }
  if ((long long)p.n_rows * p.width <= kSmallTable) rename_entries(p, movers, live, tid, kMetaThreads);
}

__global__ __launch_bounds__(256) void kda_cache_rename_kernel(CompactParams p) {
  rename_entries(p, *p.n_moves, *p.n_live, (long long)blockIdx.x * 256 + threadIdx.x, (long long)gridDim.x * 256);
}

// A unit is one tile of one move on one layer, moves within a layer; a workgroup
// takes every so-manieth, so that workgroups that run together copy tiles that lie
// together (40 pages of 2 MiB on 8 layers: 247 us, 5.4 TB/s, against 267 us with a run
// of tiles for each workgroup).  Which moves race is settled by every workgroup
// for itself, with one pass over the list: a bit for each page that is a
// destination, and one for each that is so more than once.  Long lists of small pages pay
// for that pass: 4,096 moves of 64 KiB between two pools 91 us (5.9 TB/s), 16,384 of 16 KiB 110 us
// (4.9), 65,536 of 4 KiB 201 us (2.7) and of 256 bytes 157 us.  A source that several moves name is
// read for each of them, from the caches where they still hold it: 64 copies of 16 pages of 2 MiB
// on 8 layers fetch 0.86 GB, 3.2 times the pages' 0.27, in 282 to 292 us.
constexpr int kTile = 16384;
constexpr int kCopyThreads = 256;
constexpr int kPageWords = kMaxPages / 32;

__device__ __forceinline__ bool move_valid(const CopyParams& p, int from, int to) {
  return page_ok(to, p.n_dst) && (from == -1 || page_ok(from, p.n_src)) && !(p.same && from == to);
}

__global__ __launch_bounds__(kCopyThreads) void kda_cache_copy_kernel(CopyParams p) {
  __shared__ unsigned once[kPageWords], twice[kPageWords];
  const int tid = threadIdx.x;
  const int n = p.n_moves ? min(max(*p.n_moves, 0), p.max_moves) : p.max_moves;
  const long long tiles = (long long)((p.page_bytes + kTile - 1) / kTile);
  const long long units = (long long)p.n_layers * n * tiles;
  if (blockIdx.x >= units) return;
  for (int w = tid; w < (p.n_dst + 31) / 32; w += kCopyThreads) once[w] = twice[w] = 0;
  __syncthreads();
  for (int j = tid; j < n; j += kCopyThreads) {
    const int from = p.moves[2 * j], to = p.moves[2 * j + 1];
    if (!move_valid(p, from, to)) continue;
    const unsigned bit = 1u << (to % 32);
    if (atomicOr(&once[to / 32], bit) & bit) atomicOr(&twice[to / 32], bit);
  }
  __syncthreads();
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long layer = u / (n * tiles);
    const int j = (int)(u / tiles % n);
    const int from = p.moves[2 * j], to = p.moves[2 * j + 1];
    if (!move_valid(p, from, to) || (twice[to / 32] >> (to % 32) & 1)) continue;
    if (p.same && from >= 0 && (once[from / 32] >> (from % 32) & 1)) continue;
    const size_t off = (size_t)(u % tiles) * kTile;
    const int vecs = (int)(min((size_t)kTile, p.page_bytes - off) / 16);
    u32x4* d = reinterpret_cast<u32x4*>(p.dst + ((size_t)layer * p.n_dst + to) * p.page_bytes + off);
    if (from < 0) {
      for (int v = tid; v < vecs; v += kCopyThreads) __builtin_nontemporal_store((u32x4)0u, d + v);
      continue;
    }
    const u32x4* s = reinterpret_cast<const u32x4*>(p.src + ((size_t)layer * p.n_src + from) * p.page_bytes + off);
    if (vecs == kTile / 16) {
      u32x4 x[kTile / 16 / kCopyThreads];
#pragma unroll
      for (int e = 0; e < kTile / 16 / kCopyThreads; ++e) x[e] = s[tid + e * kCopyThreads];
#pragma unroll
      for (int e = 0; e < kTile / 16 / kCopyThreads; ++e) __builtin_nontemporal_store(x[e], d + tid + e * kCopyThreads);
    } else {
      for (int v = tid; v < vecs; v += kCopyThreads) __builtin_nontemporal_store(s[v], d + v);
    }
  }
}

}  // namespace

hipError_t launch_cache_fork(const ForkParams& p, hipStream_t s) {
  if (p.n > kMaxForks || p.n_pages > kMaxPages) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kda_cache_fork_kernel, dim3(1), dim3(kMetaThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_cache_free(int* table, int* ref, const int* rows, int n, int n_rows, int width, int n_pages,
                             hipStream_t s) {
  const long long entries = (long long)n * width;
  hipLaunchKernelGGL(kda_cache_free_kernel, dim3((unsigned)((entries + 255) / 256)), dim3(256), 0, s, table, ref, rows,
                     n, n_rows, width, n_pages);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const CompactParams& p, hipStream_t s) {
  if (p.n_pages > kMaxPages) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kda_cache_compact_kernel, dim3(1), dim3(kMetaThreads), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const long long entries = (long long)p.n_rows * p.width;
  if (entries <= kSmallTable) return hipSuccess;
  const unsigned grid = (unsigned)std::min((entries + 255) / 256, (long long)2048);
  hipLaunchKernelGGL(kda_cache_rename_kernel, dim3(grid), dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_cache_copy(const CopyParams& p, hipStream_t s) {
  if (p.n_src > kMaxPages || p.n_dst > kMaxPages || p.max_moves < 1) return hipErrorInvalidValue;
  const long long units = (long long)p.n_layers * p.max_moves * (long long)((p.page_bytes + kTile - 1) / kTile);
  const unsigned grid = (unsigned)std::min(units, (long long)2048);
  hipLaunchKernelGGL(kda_cache_copy_kernel, dim3(grid), dim3(kCopyThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace kda
