// New tokens into the 16-bit cache: a copy, bound by its bytes (512 B read and
// 512 B written per token and KV head) for prompts and by one chain of loads
// (start, pos0, block table, data) for single tokens.
//
// A warp takes one token: it finds the token's sequence in start[], then its
// place, and copies head after head, lanes 0-15 the key's 16-byte pieces and
// lanes 16-31 the value's, four heads in flight.
//
// Measured (GB300): 34.7K tokens of 8 heads 45 us, 6.3 TB/s read and written
// (floor 42); one token for each of 8 sequences 2.7 us.
#include "kv16.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 4;    // heads of a token in flight

__global__ void __launch_bounds__(kThreads)
kv16_write_kernel(const Kv16 c, const uint16_t* __restrict__ k_new, long long k_stride,
                  const uint16_t* __restrict__ v_new, long long v_stride,
                  const int32_t* __restrict__ start, const int32_t* __restrict__ pos0, int total) {
  const long long gid = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  for (long long b = gid; b < c.B; b += (long long)gridDim.x * kThreads) {
    const long long end = (long long)pos0[b] + start[b + 1] - start[b];
    const bool ok = pos0[b] >= 0 && start[b] >= 0 && start[b + 1] >= start[b] &&
                    start[b + 1] <= total && end <= c.cap;
    if (ok) c.n_tok[b] = (int)end;
    else record_error(c.status, kDevErrBadPaged);
  }
  if ((gid >> 5) >= total) return;
  const int r = (int)(gid >> 5);
  const int b = ragged_sequence(start, c.B, r);
  if (b < 0) return;
  const int s0 = __ldg(start + b), s1 = __ldg(start + b + 1), p0 = __ldg(pos0 + b);
  if (s0 < 0 || s1 > total || p0 < 0 || (long long)p0 + (s1 - s0) > c.cap) return;
  const int at = p0 + r - s0;
  const int row0 = kv16_block_row(c, b, 0, at / kPage);
  if (row0 < 0) {
    if (lane == 0) record_error(c.status, kDevErrBadPaged);
    return;
  }
  const long long head_rows = c.table ? kPage : c.T_cap;   // rows from one head to the next
  const long long dst0 = (long long)row0 + at % kPage;
  const bool is_v = lane >= 16;
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? v_new + r * v_stride
                                                         : k_new + r * k_stride) + (lane & 15);
  uint4* dst = reinterpret_cast<uint4*>(is_v ? c.v : c.k) + dst0 * 16 + (lane & 15);
  for (int h0 = 0; h0 < c.Hkv; h0 += kHeads) {
    uint4 x[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (h0 + i < c.Hkv) x[i] = __ldg(src + (h0 + i) * 16);
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (h0 + i < c.Hkv) dst[(h0 + i) * head_rows * 16] = x[i];
  }
  if (c.weight)
    for (int h = lane; h < c.Hkv; h += 32) c.weight[dst0 + h * head_rows] = 0.0f;
}

}  // namespace

cudaError_t launch_kv16_write(const Kv16& c, const uint16_t* k_new, long long k_stride,
                              const uint16_t* v_new, long long v_stride, const int32_t* start,
                              const int32_t* pos0, int total, cudaStream_t s) {
  const long long threads = (long long)total * 32;
  const int grid = (int)((threads + kThreads - 1) / kThreads);
  kv16_write_kernel<<<grid > 0 ? grid : 1, kThreads, 0, s>>>(c, k_new, k_stride, v_new, v_stride,
                                                             start, pos0, total);
  return cudaGetLastError();
}

}  // namespace oscar
