// Eviction by accumulated weight: the kept positions of every (sequence, KV
// head), then the copy of the kept tokens into another cache.
//
// Choice.  The keep_top largest weights between the first and the recent
// tokens, lower positions first among equals.  A weight becomes a 32-bit key
// of the same order; three rounds of counting (11, 11 and 10 bits) find the
// key of the last one kept and how many of its equals are kept.  One more pass
// numbers the kept tokens in order of position.
//
// A row is worked by a cluster of 1 to 8 CTAs, each with a run of the row's
// tokens, whose keys it reads once and holds in shared memory (rows too long
// for that are read again in each pass).  The CTAs add up one another's counts
// through distributed shared memory and come to the same key; integer counts,
// so the choice does not depend on any order.
//
// The copy is bound by its bytes, 1 KB per kept token read and written.
//
// Measured (GB300): 64 rows of 10K to 32K tokens cut to 2048: choice 21.6 us,
// copy 23.2 (floor of both 21); 16 rows of 2176: 8.2 + 5.3 us, latency.
#include <algorithm>

#include "kv16.cuh"

namespace oscar {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// Orders as the float does (-0 with +0); a NaN of either sign is the largest.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kKeysMost = 48 * 1024;     // keys that a CTA holds
constexpr int kLoads = 8;                // pages that a warp has in flight

__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// The int at the same place in the shared memory of another CTA of the cluster.
__device__ __forceinline__ int peer_int(const int* p, int rank) {
  unsigned far;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(far) : "memory");
  return v;
}

// *p += v in shared memory.  With v not known to be 1 the compiler leaves the
// adding to the memory; of a constant 1 it makes a loop over the warp's distinct
// addresses, which for keys this spread took most of the kernel's time.
__device__ __forceinline__ void count_up(int* p, int v) {
  asm volatile("red.relaxed.cta.shared::cta.add.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v)
               : "memory");
}

// HELD: a CTA's keys fit in its dynamic shared memory.
template <bool HELD>
__global__ void __launch_bounds__(kSelThreads)
kv16_select_kernel(const Kv16 c, int max_tok, int first, int recent, int top, int cluster,
                   int32_t* counts, int32_t* kept) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kBins];
  __shared__ int s_scan[2][kSelWarps];
  __shared__ int s_total[2];
  __shared__ int s_bin, s_need;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % cluster, row = blockIdx.x / cluster;
  const int b = row / c.Hkv, h = row - b * c.Hkv;
  const int keep = first + recent + top;
  int32_t* out = kept + (long long)row * keep;
  const int n = kv16_length(c, b, max_tok);
  if (n < 0 && tid == 0) record_error(c.status, kDevErrBadPaged);
  if (rank == 0 && tid == 0) counts[row] = min(n, keep);
  if (n <= keep) {     // the whole cluster leaves
    for (int i = rank * kSelThreads + tid; i < keep; i += cluster * kSelThreads)
      out[i] = i < n ? i : -1;
    return;
  }
  for (int i = rank * kSelThreads + tid; i < first; i += cluster * kSelThreads) out[i] = i;
  for (int i = rank * kSelThreads + tid; i < recent; i += cluster * kSelThreads)
    out[first + top + i] = n - recent + i;
  if (top == 0) return;

  // of the tokens to choose from, [first, n - recent), this CTA's are those of
  // the pages [page0, page0 + pages): place i is token 32 page0 + i, and the
  // places [from, from + len) count
  const int end = n - recent, all0 = first / kPage, all = (end + kPage - 1) / kPage - all0;
  const int page0 = all0 + (int)((long long)all * rank / cluster);
  const int pages = all0 + (int)((long long)all * (rank + 1) / cluster) - page0;
  const int from = max(first - page0 * kPage, 0);
  const int len = max(min(end - page0 * kPage, pages * kPage) - from, 0);
  bool bad = false;
  // kLoads pages of a warp at once: a lane each finds its page, then all lanes
  // read every page's 32 weights
  auto read_pages = [&](int q, uint32_t (&k)[kLoads]) {
    int row = 0;
    if (lane < kLoads && q + lane < pages) {
      row = kv16_block_row(c, b, h, page0 + q + lane);
      bad |= row < 0;
    }
    const float* at[kLoads];
    float w[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      // (a contiguous row may end inside its last page)
      const int r = max(__shfl_sync(0xffffffffu, row, u), 0);
      const bool counts = (unsigned)((q + u) * kPage + lane - from) < (unsigned)len;
      at[u] = c.weight + (counts ? (long long)r + lane : 0);
    }
    // in this order: left to itself the compiler waits for each before the next
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(w[u]) : "l"(at[u]));
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      k[u] = __shfl_sync(0xffffffffu, row, u) < 0 ? 0u : order_key(w[u]);
  };
  auto pages_at = [&](int q, uint32_t (&k)[kLoads]) {
    if (HELD) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) k[u] = keys[min(q + u, pages - 1) * kPage + lane];
    } else {
      read_pages(q, k);
    }
  };
  // each warp a run of the pages
  const int per = (pages + kSelWarps - 1) / kSelWarps;
  const int p0 = min(pages, warp * per), p1 = min(pages, p0 + per);
  auto mine = [&](int q) { return q < p1 && (unsigned)(q * kPage + lane - from) < (unsigned)len; };
  if (HELD)
    for (int q = p0; q < p1; q += kLoads) {
      uint32_t k[kLoads];
      read_pages(q, k);
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        if (q + u < p1) keys[(q + u) * kPage + lane] = k[u];
    }

  // the key of the last kept token, found from its top bits down
  uint32_t prefix = 0, mask = 0;
  int need = top, one;
  asm volatile("mov.u32 %0, 1;" : "=r"(one));
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const int bins = round == 2 ? 1024 : 2048;
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int q = p0; q < p1; q += kLoads) {
      uint32_t k[kLoads];
      pages_at(q, k);
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        if (mine(q + u) && (k[u] & mask) == prefix)
          count_up(&hist[(k[u] >> shift) & (bins - 1)], one);
    }
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    // the bin in which the count from above reaches `need`: a thread takes
    // two bins, highest first
    const int b0 = kBins - 1 - 2 * tid;
    int c0 = 0, c1 = 0;
    for (int r = 0; r < cluster; ++r) {
      c0 += cluster > 1 ? peer_int(hist + b0, r) : hist[b0];
      c1 += cluster > 1 ? peer_int(hist + b0 - 1, r) : hist[b0 - 1];
    }
    int x = c0 + c1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) s_scan[0][warp] = x;
    __syncthreads();
    if (warp == 0) {
      int y = s_scan[0][lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) y += z;
      }
      s_scan[0][lane] = y;
    }
    __syncthreads();
    const int above = x - c0 - c1 + (warp ? s_scan[0][warp - 1] : 0);
    if (above < need && above + c0 + c1 >= need) {
      const bool second = above + c0 < need;
      s_bin = second ? b0 - 1 : b0;
      s_need = need - above - (second ? c0 : 0);
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    need = s_need;
    // the others have read this CTA's counts
    if (cluster > 1) cluster_sync();
    else __syncthreads();
  }
  // number the kept tokens
  int gt = 0, eq = 0;
  for (int q = p0; q < p1; q += kLoads) {
    uint32_t k[kLoads];
    pages_at(q, k);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      gt += mine(q + u) && k[u] > prefix;
      eq += mine(q + u) && k[u] == prefix;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_scan[0][warp] = gt;
    s_scan[1][warp] = eq;
  }
  __syncthreads();
  if (tid < 2) {
    int t = 0;
    for (int w = 0; w < kSelWarps; ++w) t += s_scan[tid][w];
    s_total[tid] = t;
  }
  gt = eq = 0;
  for (int w = 0; w < warp; ++w) {
    gt += s_scan[0][w];
    eq += s_scan[1][w];
  }
  if (cluster > 1) {
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      gt += peer_int(&s_total[0], r);
      eq += peer_int(&s_total[1], r);
    }
  }
  const uint32_t below = (1u << lane) - 1;
  for (int q = p0; q < p1; q += kLoads) {
    uint32_t k[kLoads];
    pages_at(q, k);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const uint32_t mg = __ballot_sync(0xffffffffu, mine(q + u) && k[u] > prefix);
      const uint32_t me = __ballot_sync(0xffffffffu, mine(q + u) && k[u] == prefix);
      const int g_here = gt + __popc(mg & below), e_here = eq + __popc(me & below);
      if (((mg >> lane) & 1) || (((me >> lane) & 1) && e_here < need))
        out[first + g_here + min(e_here, need)] = (page0 + q + u) * kPage + lane;
      gt += __popc(mg);
      eq += __popc(me);
    }
  }
  if (bad) record_error(c.status, kDevErrBadPaged);
  if (cluster > 1) cluster_sync();     // the others have read this CTA's totals
}

constexpr int kCopyThreads = 128;
constexpr int kCopyTokens = 8;    // tokens of a warp, all in flight

// A warp copies kCopyTokens kept tokens of one row: lanes 0-15 the key's
// 16-byte pieces, lanes 16-31 the value's.
__global__ void __launch_bounds__(kCopyThreads)
kv16_copy_kernel(const Kv16 c, const Kv16 d, int keep, const int32_t* counts,
                 const int32_t* kept) {
  const int lane = threadIdx.x & 31;
  const int per_row = (keep + kCopyTokens - 1) / kCopyTokens;
  const int w = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
  const int row = w / per_row;
  if (row >= c.B * c.Hkv) return;
  const int b = row / c.Hkv, h = row - b * c.Hkv;
  const int i0 = (w - row * per_row) * kCopyTokens;
  cudaGridDependencySynchronize();  // the choice is complete and its writes visible
  const int n = counts[row];
  if (h == 0 && i0 == 0 && lane == 0 && n >= 0) d.n_tok[b] = n;
  int src = -1, dst = -1;
  if (lane < kCopyTokens && i0 + lane < n) {
    const int j = kept[(long long)row * keep + i0 + lane];
    src = kv16_block_row(c, b, h, j / kPage);
    dst = kv16_block_row(d, b, h, (i0 + lane) / kPage);
    if (src < 0 || dst < 0) {
      record_error(c.status, kDevErrBadPaged);
      src = -1;
    } else {
      src += j % kPage;
      dst += (i0 + lane) % kPage;
      if (d.weight) d.weight[dst] = c.weight[src];
    }
  }
  const uint4* from = reinterpret_cast<const uint4*>(lane < 16 ? c.k : c.v) + (lane & 15);
  uint4* to = reinterpret_cast<uint4*>(lane < 16 ? d.k : d.v) + (lane & 15);
  uint4 x[kCopyTokens];
#pragma unroll
  for (int i = 0; i < kCopyTokens; ++i) {
    const int s = __shfl_sync(0xffffffffu, src, i);
    if (s >= 0) x[i] = __ldg(from + (long long)s * 16);
  }
#pragma unroll
  for (int i = 0; i < kCopyTokens; ++i) {
    const int s = __shfl_sync(0xffffffffu, src, i), t = __shfl_sync(0xffffffffu, dst, i);
    if (s >= 0) to[(long long)t * 16] = x[i];
  }
}

}  // namespace

cudaError_t launch_kv16_evict(const Kv16& src, const Kv16& dst, int max_tok, int keep_first,
                              int keep_recent, int keep_top, int32_t* kept, void* ws,
                              cudaStream_t s) {
  const int rows = src.B * src.Hkv, keep = keep_first + keep_recent + keep_top;
  int32_t* counts = static_cast<int32_t*>(ws);
  if (!kept) kept = counts + (((size_t)rows + 3) / 4) * 4;
  // CTAs per row: as many as it takes to hold the row's keys, and more while
  // that leaves no SM with two and each 8192 tokens (64 rows of 32K tokens: 27.8
  // us with one CTA a row, 21.6 with two).  Smaller shares are slower: a cluster's
  // barriers and remote reads then cost more than the counting that they save
  // (eight CTAs a row, on top of one another: 146 us).
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int most = std::min(max_tok, src.cap);
  int cluster = 1;
  while (cluster < 8 && (most / cluster > kKeysMost - 2 * kPage ||
                         (2LL * rows * cluster <= sms && most / cluster >= 8192)))
    cluster *= 2;
  const int held = (most / kPage / cluster + 2) * kPage;
  const auto select = held <= kKeysMost ? kv16_select_kernel<true> : kv16_select_kernel<false>;
  const size_t smem = held <= kKeysMost ? (size_t)held * sizeof(uint32_t) : 0;
  e = allow_shared(select, kKeysMost * sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  if ((long long)rows * cluster > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * cluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, select, src, max_tok, keep_first, keep_recent, keep_top, cluster,
                         counts, kept);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)rows * ((keep + kCopyTokens - 1) / kCopyTokens);
  const int grid = (int)((warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32));
  // Put in place as the choice ends rather than after it (a call of either
  // measured size 2 us shorter: 20.5 to 18.4 and 49.4 to 47.1).
  cudaLaunchConfig_t copy = {};
  copy.gridDim = dim3(grid);
  copy.blockDim = dim3(kCopyThreads);
  copy.stream = s;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  copy.attrs = early;
  copy.numAttrs = 1;
  return cudaLaunchKernelEx(&copy, kv16_copy_kernel, src, dst, keep,
                            static_cast<const int32_t*>(counts),
                            static_cast<const int32_t*>(kept));
}

}  // namespace oscar
