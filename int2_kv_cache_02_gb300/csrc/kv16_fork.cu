// Sequences made of others: the parent's whole pages taken over by reference
// (its table entries) or copied, and the page in which its tokens end copied.
// A copy, bound by its bytes for whole sequences (512 B read and 512 B written
// per token and KV head) and, where pages are shared, by one chain of loads
// (parent, length, table, data).
//
// A warp takes the tokens of one (sequence, block, KV head): lanes 0-15 the
// key's 16-byte pieces, lanes 16-31 the value's, eight tokens in flight, and ends:
// the next unit's loads are another warp's, so none waits for these stores.
//
// Measured (GB300): 12 copies of sequences of 7.8K to 16K tokens, 8 heads, with
// weights, 178 us, 6.9 TB/s read and written (floor 182 at the rate of a plain
// copy); 8 samples of an 8190-token prompt by reference 4.7 us, a step of 96 beams 5.6.
#include <algorithm>

#include "kv16.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 8;    // tokens of a warp in flight

struct ForkParams {
  Kv16 src, dst;
  const int32_t* parent;
  int max_tok, blocks;        // blocks of the longest sequence that the call takes
  bool share, same;           // same: src and dst are one cache
};

// The tokens that sequence b of dst gets, or -1 if it stays as it is.
__device__ __forceinline__ int fork_length(const ForkParams& p, int b, int& from, bool report) {
  from = __ldg(p.parent + b);
  if (from < 0 || (p.same && from == b)) return -1;
  bool ok = from < p.src.B;
  if (ok && p.same) {
    // a sequence that is forked from is not one that is written
    const int up = __ldg(p.parent + from);
    ok = up < 0 || up == from;
  }
  int n = -1;
  if (ok) n = kv16_length(p.src, from, p.max_tok);
  if (n > p.dst.cap) n = -1;
  if (n < 0 && report) record_error(p.src.status, kDevErrBadPaged);
  return n;
}

__global__ void __launch_bounds__(kThreads) kv16_fork_kernel(const ForkParams p) {
  const long long gid = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long threads = (long long)gridDim.x * kThreads;
  // lengths and, where pages are shared, table entries
  for (long long e = gid; e < (long long)p.dst.B * p.blocks; e += threads) {
    const int b = (int)(e / p.blocks), j = (int)(e % p.blocks);
    int from;
    const int n = fork_length(p, b, from, j == 0);
    if (n < 0) continue;
    if (j == 0) p.dst.n_tok[b] = n;
    if (p.share && j < n / kPage) {
      const int page = __ldg(p.src.table + (long long)from * p.src.max_blocks + j);
      if ((unsigned)page < (unsigned)p.src.n_pages)
        const_cast<int32_t*>(p.dst.table)[(long long)b * p.dst.max_blocks + j] = page;
      else
        record_error(p.src.status, kDevErrBadPaged);
    }
  }
  const int lane = threadIdx.x & 31, Hkv = p.src.Hkv;
  const int per = p.share ? 1 : p.blocks;     // blocks of a sequence to look at
  const long long units = (long long)p.dst.B * per * Hkv;
  for (long long u = gid >> 5; u < units; u += threads >> 5) {
    const int h = (int)(u % Hkv), b = (int)(u / Hkv / per);
    int j = (int)(u / Hkv % per), from;
    const int n = fork_length(p, b, from, false);
    if (n < 0) continue;
    if (p.share) j = n / kPage;
    const int count = min(n - j * kPage, kPage);
    if (count <= 0) continue;
    const int s0 = kv16_block_row(p.src, from, h, j), d0 = kv16_block_row(p.dst, b, h, j);
    if (s0 < 0 || d0 < 0) {
      if (lane == 0) record_error(p.src.status, kDevErrBadPaged);
      continue;
    }
    if (p.src.k == p.dst.k && s0 == d0) continue;      // the page is the sequence's own already
    const bool is_v = lane >= 16;
    const uint4* s = reinterpret_cast<const uint4*>(is_v ? p.src.v : p.src.k) +
                     (long long)s0 * 16 + (lane & 15);
    uint4* d = reinterpret_cast<uint4*>(is_v ? p.dst.v : p.dst.k) + (long long)d0 * 16 + (lane & 15);
    for (int t0 = 0; t0 < count; t0 += kTokens) {
      uint4 x[kTokens];
#pragma unroll
      for (int i = 0; i < kTokens; ++i)
        if (t0 + i < count) x[i] = __ldcs(s + (t0 + i) * 16);
#pragma unroll
      for (int i = 0; i < kTokens; ++i)
        if (t0 + i < count) d[(t0 + i) * 16] = x[i];
    }
    if (p.dst.weight && lane < count) p.dst.weight[(long long)d0 + lane] = p.src.weight[(long long)s0 + lane];
  }
}

}  // namespace

cudaError_t launch_kv16_fork(const Kv16& src, const Kv16& dst, const int32_t* parent, bool share,
                             bool same, int max_tok, cudaStream_t s) {
  ForkParams p{src, dst, parent, max_tok, 1, share, same};
  p.blocks = std::max(1, (std::min({max_tok, src.cap, dst.cap}) + kPage - 1) / kPage);
  const long long units = (long long)dst.B * (share ? 1 : p.blocks) * src.Hkv;
  const long long ctas = (std::max(units * 32, (long long)dst.B * p.blocks) + kThreads - 1) / kThreads;
  kv16_fork_kernel<<<(int)std::min<long long>(ctas, 1 << 30), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace oscar
