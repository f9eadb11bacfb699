// Compaction of a page pool and copies of whole pages.
//
// Compaction.  The pages that a table names, L of them, are to have the ids 0
// .. L - 1.  Those that have such an id stay; the i-th lowest of the others
// goes to the i-th lowest id below L that is free.  So pages are read at ids
// from L on and written at ids below L, and the copies need no order.
//
// One cluster of eight CTAs does it in one launch.  A bit a page, in the CTAs'
// shared memory (a range of ids each), is set for every entry of the table; the
// bits' counts, summed over threads and CTAs, give L and every id's rank among
// the live or the free; a second pass over the table renames.  Latency bounds it:
// two passes over the table and six barriers of the cluster.  Measured (GB300): 344
// live pages of 382, 8 x 64 entries, with the copies of 34 pages of 4 heads 11.4 to 12 us
// a call among others.  (A map in memory instead of the bits, one CTA that scans it, four
// launches: 15.1.)
//
// Copies.  A warp takes a (pair, KV head) and ends, so that no load waits for the
// stores before it.  Bound by HBM: 4.4K pages of 8 heads, 1.14 GB read and written,
// 165 us, 6.93 TB/s, a little above the rate of a plain copy.  (Warps that walk over
// the pairs: 180.)
#include <algorithm>

#include <cooperative_groups.h>

#include "kv16.cuh"

namespace oscar {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kEntries = 4;      // of a thread in flight

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
page_compact_kernel(const int32_t* table, int32_t* new_table, long long entries, int n_pages,
                    int words, int2* moves, int32_t* counts, int32_t* map, unsigned* status) {
  extern __shared__ unsigned bits[];        // [words]: ids from rank * 32 * words on
  __shared__ int scan[kThreads / 32], totals[kCluster], s_below;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)cluster.block_rank();
  for (int i = tid; i < words; i += kThreads) bits[i] = 0u;
  cluster.sync();
  const long long first = (long long)rank * kThreads + tid, step = (long long)kCluster * kThreads;
  for (long long e0 = first; e0 < entries; e0 += step * kEntries) {
    int id[kEntries];
#pragma unroll
    for (int u = 0; u < kEntries; ++u) id[u] = e0 + u * step < entries ? table[e0 + u * step] : -1;
#pragma unroll
    for (int u = 0; u < kEntries; ++u) {
      if (id[u] < 0) continue;
      if (id[u] >= n_pages) {
        record_error(status, kDevErrBadPaged);
        continue;
      }
      const int w = id[u] >> 5, owner = w / words;
      atomicOr(cluster.map_shared_rank(bits, owner) + (w - owner * words), 1u << (id[u] & 31));
    }
  }
  cluster.sync();

  // live pages before this thread's words [w0, w1)
  const int each = (words + kThreads - 1) / kThreads;
  const int w0 = min(tid * each, words), w1 = min(w0 + each, words);
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += y;
  }
  if (lane == 31) scan[warp] = sum;
  __syncthreads();
  int before = sum - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  if (tid < kCluster) cluster.map_shared_rank(totals, tid)[rank] = total;
  cluster.sync();
  int live = 0;
  for (int r = 0; r < kCluster; ++r) {
    if (r < rank) before += totals[r];
    live += totals[r];
  }
  // how many of them have ids below `live`: known where that id's bit is
  const int base = rank * words;            // the CTA's first word
  if (live >= kCluster * words * 32) {
    if (tid == 0) s_below = live;
  } else if (live / 32 >= base + w0 && live / 32 < base + w1) {
    int n = before;
    for (int w = base + w0; w < live / 32; ++w) n += __popc(bits[w - base]);
    n += __popc(bits[live / 32 - base] & ((1u << (live % 32)) - 1));
    for (int r = 0; r < kCluster; ++r) *cluster.map_shared_rank(&s_below, r) = n;
  }
  cluster.sync();
  const int n_moves = live - s_below;
  int n = before;                           // live pages before the word
  for (int w = w0; w < w1; ++w) {
    const unsigned x = bits[w];
    const int id0 = (base + w) * 32;
    // free ids below `live`, live ids from it on
    const int split = min(max(live - id0, 0), 32);
    const unsigned below = split == 32 ? ~0u : (1u << split) - 1;
    for (unsigned f = ~x & below; f; f &= f - 1) {
      const int i = __ffs(f) - 1;
      moves[id0 + i - n - __popc(x & ((1u << i) - 1))].y = id0 + i;
    }
    for (unsigned f = x & ~below; f; f &= f - 1) {
      const int i = __ffs(f) - 1;
      moves[n + __popc(x & ((1u << i) - 1)) - s_below].x = id0 + i;
    }
    n += __popc(x);
  }
  __threadfence();
  cluster.sync();
  for (long long i = first; i < n_pages / 2; i += step) {
    if (i < n_moves) {
      const int2 m = __ldcg(moves + i);
      map[m.x] = m.y;
    } else {
      moves[i] = make_int2(-1, -1);
    }
  }
  if (first == 0) counts[0] = n_moves, counts[1] = live;
  __threadfence();
  cluster.sync();
  for (long long e0 = first; e0 < entries; e0 += step * kEntries) {
    int id[kEntries];
#pragma unroll
    for (int u = 0; u < kEntries; ++u) id[u] = e0 + u * step < entries ? table[e0 + u * step] : -1;
#pragma unroll
    for (int u = 0; u < kEntries; ++u)
      if (id[u] >= live && id[u] < n_pages) id[u] = __ldcg(map + id[u]);
#pragma unroll
    for (int u = 0; u < kEntries; ++u)
      if (e0 + u * step < entries) new_table[e0 + u * step] = id[u];
  }
}

constexpr int kCopyThreads = 128;
constexpr int kTokens = 8;    // tokens of a warp in flight

// Lanes 0-15 the keys' 16-byte pieces, lanes 16-31 the values'.
__global__ void __launch_bounds__(kCopyThreads)
kv16_copy_pages_kernel(const Kv16 src, const Kv16 dst, const int2* __restrict__ pairs,
                       const int32_t* __restrict__ n_pairs, int max_pairs) {
  const int n = __ldg(n_pairs), lane = threadIdx.x & 31;
  const long long gid = (long long)blockIdx.x * kCopyThreads + threadIdx.x;
  if (n < 0 || n > max_pairs) {
    if (gid == 0) record_error(src.status, kDevErrBadPaged);
    return;
  }
  const long long u = gid >> 5;
  if (u >= (long long)n * src.Hkv) return;
  const int2 pair = __ldg(pairs + u / src.Hkv);
  const int h = (int)(u % src.Hkv);
  if ((unsigned)pair.x >= (unsigned)src.n_pages || (unsigned)pair.y >= (unsigned)dst.n_pages) {
    if (lane == 0) record_error(src.status, kDevErrBadPaged);
    return;
  }
  const long long s0 = ((long long)pair.x * src.Hkv + h) * kPage;
  const long long d0 = ((long long)pair.y * src.Hkv + h) * kPage;
  const uint4* s = reinterpret_cast<const uint4*>(lane >= 16 ? src.v : src.k) + s0 * 16 + (lane & 15);
  uint4* d = reinterpret_cast<uint4*>(lane >= 16 ? dst.v : dst.k) + d0 * 16 + (lane & 15);
  for (int t0 = 0; t0 < kPage; t0 += kTokens) {
    uint4 x[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) x[i] = __ldcs(s + (t0 + i) * 16);
#pragma unroll
    for (int i = 0; i < kTokens; ++i) d[(t0 + i) * 16] = x[i];
  }
  if (dst.weight) dst.weight[d0 + lane] = src.weight[s0 + lane];
}

// Packed pages, as 16-byte pieces: a warp takes 256 of a pair's.
constexpr int kPieces = 256;
__global__ void __launch_bounds__(kCopyThreads)
paged_copy_pages_kernel(uint4* pages, int n_pages, int pieces, const int2* __restrict__ pairs,
                        const int32_t* __restrict__ n_pairs, int max_pairs, unsigned* status) {
  const int n = __ldg(n_pairs), lane = threadIdx.x & 31;
  const long long gid = (long long)blockIdx.x * kCopyThreads + threadIdx.x;
  if (n < 0 || n > max_pairs) {
    if (gid == 0) record_error(status, kDevErrBadPaged);
    return;
  }
  const int parts = (pieces + kPieces - 1) / kPieces;
  const long long u = gid >> 5;
  if (u >= (long long)n * parts) return;
  const int2 pair = __ldg(pairs + u / parts);
  if ((unsigned)pair.x >= (unsigned)n_pages || (unsigned)pair.y >= (unsigned)n_pages) {
    if (lane == 0) record_error(status, kDevErrBadPaged);
    return;
  }
  const int i0 = (int)(u % parts) * kPieces + lane;
  const uint4* s = pages + (long long)pair.x * pieces;
  uint4* d = pages + (long long)pair.y * pieces;
  uint4 x[kPieces / 32];
#pragma unroll
  for (int i = 0; i < kPieces / 32; ++i)
    if (i0 + 32 * i < pieces) x[i] = __ldcs(s + i0 + 32 * i);
#pragma unroll
  for (int i = 0; i < kPieces / 32; ++i)
    if (i0 + 32 * i < pieces) d[i0 + 32 * i] = x[i];
}

// Words of the bits of one CTA.
int compact_words(int n_pages) { return (n_pages + 32 * kCluster - 1) / (32 * kCluster); }

}  // namespace

static_assert((kMaxPages / 32 + kCluster - 1) / kCluster * 4 <= 224 * 1024, "bits of a CTA");

size_t page_compact_ws_bytes(int n_pages) { return (size_t)n_pages * sizeof(int32_t); }

cudaError_t launch_page_compact(const int32_t* table, int32_t* new_table, long long entries,
                                int n_pages, int32_t* moves, int32_t* counts, void* ws,
                                unsigned* status, cudaStream_t s) {
  const int words = compact_words(n_pages), smem = words * (int)sizeof(unsigned);
  const cudaError_t e =
      allow_shared(page_compact_kernel, compact_words(kMaxPages) * sizeof(unsigned));
  if (e != cudaSuccess) return e;
  page_compact_kernel<<<kCluster, kThreads, smem, s>>>(table, new_table, entries, n_pages, words,
                                                       reinterpret_cast<int2*>(moves), counts,
                                                       static_cast<int32_t*>(ws), status);
  return cudaGetLastError();
}

cudaError_t launch_kv16_copy_pages(const Kv16& src, const Kv16& dst, const int32_t* pairs,
                                   const int32_t* n_pairs, int max_pairs, cudaStream_t s) {
  const long long ctas = ((long long)max_pairs * src.Hkv * 32 + kCopyThreads - 1) / kCopyThreads;
  kv16_copy_pages_kernel<<<(int)ctas, kCopyThreads, 0, s>>>(
      src, dst, reinterpret_cast<const int2*>(pairs), n_pairs, max_pairs);
  return cudaGetLastError();
}

cudaError_t launch_paged_copy_pages(uint8_t* pages, int n_pages, int page_bytes,
                                    const int32_t* pairs, const int32_t* n_pairs, int max_pairs,
                                    unsigned* status, cudaStream_t s) {
  const int pieces = page_bytes / 16, parts = (pieces + kPieces - 1) / kPieces;
  const long long ctas = ((long long)max_pairs * parts * 32 + kCopyThreads - 1) / kCopyThreads;
  paged_copy_pages_kernel<<<(int)ctas, kCopyThreads, 0, s>>>(
      reinterpret_cast<uint4*>(pages), n_pages, pieces, reinterpret_cast<const int2*>(pairs),
      n_pairs, max_pairs, status);
  return cudaGetLastError();
}

}  // namespace oscar
