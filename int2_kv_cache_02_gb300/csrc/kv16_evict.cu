// Eviction by accumulated weight: the kept positions of every (sequence, KV
// head), then the copy of the kept tokens into another cache.
//
// Choice.  The keep_top largest weights between the first and the recent
// tokens, lower positions first among equals.  A weight becomes a 32-bit key
// of the same order; three rounds of counting (11, 11 and 10 bits) find the
// key of the last one kept and how many of its equals are kept.  One more pass
// numbers the kept tokens in order of position.
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

__global__ void __launch_bounds__(kSelThreads)
kv16_select_kernel(const Kv16 c, int max_tok, int first, int recent, int top, int32_t* counts,
                   int32_t* kept) {
  __shared__ int hist[kBins];
  __shared__ int s_scan[2][kSelWarps];
  __shared__ int s_bin, s_need;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x, b = row / c.Hkv, h = row - b * c.Hkv;
  const int keep = first + recent + top;
  int32_t* out = kept + (long long)row * keep;
  const int n = kv16_length(c, b, max_tok);
  if (n < 0 && tid == 0) record_error(c.status, kDevErrBadPaged);
  if (n <= keep) {
    for (int i = tid; i < keep; i += kSelThreads) out[i] = i < n ? i : -1;
    if (tid == 0) counts[row] = n;
    return;
  }
  auto key_at = [&](int j) -> uint32_t {
    const int r = kv16_block_row(c, b, h, j / kPage);
    if (r < 0) {
      record_error(c.status, kDevErrBadPaged);
      return 0u;
    }
    return order_key(c.weight[(long long)r + j % kPage]);
  };
  const int lo = first, hi = n - recent;    // the tokens to choose from
  // the key of the last kept token, found from its top bits down
  uint32_t prefix = 0, mask = 0;
  int need = top;
  if (top > 0) {
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
      const int bins = round == 2 ? 1024 : 2048;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kSelThreads) {
        const uint32_t k = key_at(j);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // the bin in which the count from above reaches `need`: a thread takes
      // two bins, highest first
      const int b0 = kBins - 1 - 2 * tid;
      const int c0 = hist[b0], c1 = hist[b0 - 1];
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
      __syncthreads();
    }
  }
  // number the kept tokens: each warp a run of 32-token pieces
  const int pieces = top > 0 ? (hi - lo + 31) / 32 : 0;
  const int per = (pieces + kSelWarps - 1) / kSelWarps;
  const int p0 = min(pieces, warp * per), p1 = min(pieces, p0 + per);
  int gt = 0, eq = 0;
  for (int p = p0; p < p1; ++p) {
    const int j = lo + p * 32 + lane;
    const uint32_t k = j < hi ? key_at(j) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, j < hi && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, j < hi && k == prefix));
  }
  if (lane == 0) {
    s_scan[0][warp] = gt;
    s_scan[1][warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  for (int w = 0; w < warp; ++w) {
    gt += s_scan[0][w];
    eq += s_scan[1][w];
  }
  const uint32_t below = (1u << lane) - 1;
  for (int p = p0; p < p1; ++p) {
    const int j = lo + p * 32 + lane;
    const uint32_t k = j < hi ? key_at(j) : 0u;
    const uint32_t mg = __ballot_sync(0xffffffffu, j < hi && k > prefix);
    const uint32_t me = __ballot_sync(0xffffffffu, j < hi && k == prefix);
    const int g_here = gt + __popc(mg & below), e_here = eq + __popc(me & below);
    if (((mg >> lane) & 1) || (((me >> lane) & 1) && e_here < need))
      out[first + g_here + min(e_here, need)] = j;
    gt += __popc(mg);
    eq += __popc(me);
  }
  for (int i = tid; i < first; i += kSelThreads) out[i] = i;
  for (int i = tid; i < recent; i += kSelThreads) out[first + top + i] = n - recent + i;
  if (tid == 0) counts[row] = keep;
}

constexpr int kCopyThreads = 128;
constexpr int kCopyTokens = 8;    // tokens of a warp, all in flight

// A warp copies kCopyTokens kept tokens of one row: lanes 0-15 the key's
// 16-byte pieces, lanes 16-31 the value's.
__global__ void __launch_bounds__(kCopyThreads)
kv16_copy_kernel(const Kv16 c, const Kv16 d, int keep, const int32_t* __restrict__ counts,
                 const int32_t* __restrict__ kept) {
  const int lane = threadIdx.x & 31;
  const int per_row = (keep + kCopyTokens - 1) / kCopyTokens;
  const int w = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
  const int row = w / per_row;
  if (row >= c.B * c.Hkv) return;
  const int b = row / c.Hkv, h = row - b * c.Hkv;
  const int i0 = (w - row * per_row) * kCopyTokens;
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
  kv16_select_kernel<<<rows, kSelThreads, 0, s>>>(src, max_tok, keep_first, keep_recent, keep_top,
                                                  counts, kept);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long warps = (long long)rows * ((keep + kCopyTokens - 1) / kCopyTokens);
  const int grid = (int)((warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32));
  kv16_copy_kernel<<<grid, kCopyThreads, 0, s>>>(src, dst, keep, counts, kept);
  return cudaGetLastError();
}

}  // namespace oscar
