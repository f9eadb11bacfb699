// Attention weight of stored tokens under a ragged batch of queries.
#include <algorithm>

#include "kv16.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 4;

// A warp per (token, KV head), over the sequence's queries in order.
template <class T>
__global__ void __launch_bounds__(kWarps * 32)
kv16_weight_kernel(const Kv16 c, const Kv16Query q, const float* __restrict__ lse, int n_obs) {
  const int lane = threadIdx.x & 31;
  const int j = blockIdx.x * kWarps + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
  const int n = kv16_length(c, b, q.max_tok);
  if (n < 0) {
    if (lane == 0 && j == 0) record_error(c.status, kDevErrBadPaged);
    return;
  }
  if (j >= n) return;
  const int r1 = q.start ? min(__ldg(q.start + b + 1), q.total) : b + 1;
  int r0 = q.start ? max(0, __ldg(q.start + b)) : b;
  if (r1 - r0 > n) {
    if (lane == 0) record_error(c.status, kDevErrBadPaged);
    return;
  }
  if (n_obs > 0) r0 = max(r0, r1 - n_obs);
  const int row = kv16_block_row(c, b, h, j / kPage);
  if (row < 0) {
    if (lane == 0) record_error(c.status, kDevErrBadPaged);
    return;
  }
  const uint2 kr = reinterpret_cast<const uint2*>(c.k)[((long long)row + j % kPage) * 32 + lane];
  const float2 k0 = T::unpack(kr.x), k1 = T::unpack(kr.y);
  const int g = q.Hq / c.Hkv;
  float w = 0.0f;
  for (int r = r0; r < r1; ++r) {
    if (!kv16_visible(j, n - (r1 - r), q.window, q.n_sink)) continue;
    for (int i = 0; i < g; ++i) {
      const uint2 qr = reinterpret_cast<const uint2*>(q.q + r * q.stride + (h * g + i) * kD)[lane];
      const float2 q0 = T::unpack(qr.x), q1 = T::unpack(qr.y);
      float s = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      w += fast_exp2(s * q.scale_log2 - lse[(long long)r * q.Hq + h * g + i] * kLog2e);
    }
  }
  if (lane == 0) c.weight[(long long)row + j % kPage] += w;
}

}  // namespace

cudaError_t launch_kv16_accumulate(const Kv16& c, const Kv16Query& q, const float* lse, int n_obs,
                                   cudaStream_t s) {
  const dim3 grid((std::min(q.max_tok, c.cap) + kWarps - 1) / kWarps, c.Hkv, c.B);
  if (c.half)
    kv16_weight_kernel<Fp16><<<grid, kWarps * 32, 0, s>>>(c, q, lse, n_obs);
  else
    kv16_weight_kernel<Bf16><<<grid, kWarps * 32, 0, s>>>(c, q, lse, n_obs);
  return cudaGetLastError();
}

}  // namespace oscar
