// Compaction of a page pool and copies of whole pages.
//
// Compaction.  The pages that a table names, L of them, are to have the ids 0
// .. L - 1.  Those that have such an id stay; the i-th lowest of the others
// goes to the i-th lowest id below L that is free.  So pages are read at ids
// from L on and written at ids below L, and the copies need no order.
#include <algorithm>

#include "kv16.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256;
constexpr int kScanThreads = 1024;

__global__ void __launch_bounds__(kThreads)
page_mark_kernel(const int32_t* __restrict__ table, long long entries, int n_pages, int32_t* map,
                 unsigned* status) {
  for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < entries;
       e += (long long)gridDim.x * kThreads) {
    const int id = table[e];
    if (id >= n_pages) record_error(status, kDevErrBadPaged);
    else if (id >= 0) map[id] = 1;
  }
}

// Exclusive sum over the CTA of x; *total gets the whole.
__device__ int cta_scan(int x, int* scan, int* total) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += z;
  }
  if (lane == 31) scan[warp] = y;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kScanThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    all += scan[w];
  }
  __syncthreads();
  *total = all;
  return before + y - x;
}

// map: 1 where a page is live -> its new id.  One CTA.
__global__ void __launch_bounds__(kScanThreads)
page_plan_kernel(int n_pages, int32_t* map, int2* moves, int32_t* counts) {
  __shared__ int scan[kScanThreads / 32];
  const int tid = threadIdx.x;
  int total, live = 0;
  for (int i = tid; i < n_pages; i += kScanThreads) live += map[i];
  cta_scan(live, scan, &live);
  int high = 0, low = 0;      // live pages from L on, free ids below L, so far
  for (int i0 = 0; i0 < n_pages; i0 += kScanThreads) {
    const int i = i0 + tid;
    const bool in = i < n_pages, used = in && map[i] != 0;
    const bool mover = used && i >= live, hole = in && !used && i < live;
    const int before = cta_scan(mover || hole ? 1 : 0, scan, &total);
    // a round of ids may hold both kinds: the holes are those below L
    const int holes = cta_scan(hole ? 1 : 0, scan, &total) , n_holes = total;
    const int movers = before - (mover ? n_holes : holes);
    if (hole) moves[low + holes].y = i;
    if (mover) moves[high + movers].x = i;
    int n_movers;
    cta_scan(mover ? 1 : 0, scan, &n_movers);
    low += n_holes;
    high += n_movers;
  }
  __syncthreads();
  for (int i = tid; i < n_pages; i += kScanThreads) map[i] = i;
  __syncthreads();
  for (int i = tid; i < n_pages / 2; i += kScanThreads) {
    if (i < high) map[moves[i].x] = moves[i].y;
    else moves[i] = make_int2(-1, -1);
  }
  if (tid == 0) counts[0] = high, counts[1] = live;
}

__global__ void __launch_bounds__(kThreads)
page_rename_kernel(const int32_t* table, int32_t* new_table, long long entries, int n_pages,
                   const int32_t* __restrict__ map) {
  for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < entries;
       e += (long long)gridDim.x * kThreads) {
    const int id = table[e];
    new_table[e] = id >= 0 && id < n_pages ? map[id] : id;
  }
}

constexpr int kCopyThreads = 128;
constexpr int kTokens = 8;    // tokens of a warp in flight

// A warp takes a (pair, KV head): lanes 0-15 the keys' 16-byte pieces, lanes
// 16-31 the values'.
__global__ void __launch_bounds__(kCopyThreads)
kv16_copy_pages_kernel(const Kv16 src, const Kv16 dst, const int2* __restrict__ pairs,
                       const int32_t* __restrict__ n_pairs, int max_pairs) {
  const int n = __ldg(n_pairs), lane = threadIdx.x & 31;
  const long long gid = (long long)blockIdx.x * kCopyThreads + threadIdx.x;
  if (n < 0 || n > max_pairs) {
    if (gid == 0) record_error(src.status, kDevErrBadPaged);
    return;
  }
  const long long units = (long long)n * src.Hkv;
  for (long long u = gid >> 5; u < units; u += (long long)gridDim.x * (kCopyThreads / 32)) {
    const int2 pair = __ldg(pairs + u / src.Hkv);
    const int h = (int)(u % src.Hkv);
    if ((unsigned)pair.x >= (unsigned)src.n_pages || (unsigned)pair.y >= (unsigned)dst.n_pages) {
      if (lane == 0) record_error(src.status, kDevErrBadPaged);
      continue;
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
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 152;
  return sms;
}

}  // namespace

size_t page_compact_ws_bytes(int n_pages) { return (size_t)n_pages * sizeof(int32_t); }

cudaError_t launch_page_compact(const int32_t* table, int32_t* new_table, long long entries,
                                int n_pages, int32_t* moves, int32_t* counts, void* ws,
                                unsigned* status, int* launches, cudaStream_t s) {
  int32_t* map = static_cast<int32_t*>(ws);
  *launches = 0;
  cudaError_t e = cudaMemsetAsync(map, 0, page_compact_ws_bytes(n_pages), s);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long long>((entries + kThreads - 1) / kThreads, 8LL * sm_count());
  page_mark_kernel<<<grid, kThreads, 0, s>>>(table, entries, n_pages, map, status);
  page_plan_kernel<<<1, kScanThreads, 0, s>>>(n_pages, map, reinterpret_cast<int2*>(moves), counts);
  page_rename_kernel<<<grid, kThreads, 0, s>>>(table, new_table, entries, n_pages, map);
  *launches = 3;
  return cudaGetLastError();
}

cudaError_t launch_kv16_copy_pages(const Kv16& src, const Kv16& dst, const int32_t* pairs,
                                   const int32_t* n_pairs, int max_pairs, cudaStream_t s) {
  const long long warps = (long long)max_pairs * src.Hkv;
  const int grid = (int)std::min<long long>((warps * 32 + kCopyThreads - 1) / kCopyThreads,
                                            16LL * sm_count());
  kv16_copy_pages_kernel<<<grid, kCopyThreads, 0, s>>>(
      src, dst, reinterpret_cast<const int2*>(pairs), n_pairs, max_pairs);
  return cudaGetLastError();
}

}  // namespace oscar
