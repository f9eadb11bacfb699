// Attention of a ragged batch of queries over the 16-bit cache.
#include "kv16.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 4;

// A warp per (query, head).
template <class T>
__global__ void __launch_bounds__(kWarps * 32)
kv16_rows_kernel(const Kv16 c, const Kv16Query q, uint16_t* __restrict__ out,
                 float* __restrict__ lse) {
  const int w = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (w >= q.total * q.Hq) return;
  const int r = w / q.Hq, head = w - r * q.Hq;
  int b = r, at = 0;
  if (q.start) {
    b = ragged_sequence(q.start, c.B, r);
    if (b < 0) return;
  }
  const int n = kv16_length(c, b, q.max_tok);
  at = q.start ? n - (__ldg(q.start + b + 1) - r) : n - 1;
  if (n < 0 || (q.start && at < 0)) {
    if (lane == 0) record_error(c.status, kDevErrBadPaged);
    at = -1;
  }
  const Span sp(at, at, q.window, q.n_sink);
  float m, l, o[4];
  kv16_warp_row<T>(c, q.q + r * q.stride + (long long)head * kD, b, head / (q.Hq / c.Hkv), at, sp,
                   0, sp.blocks, q.window, q.n_sink, q.scale_log2, m, l, o);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const long long row = (long long)r * q.Hq + head;
  reinterpret_cast<uint2*>(out + row * kD)[lane] =
      make_uint2(T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv));
  if (lse && lane == 0) lse[row] = kv16_lse(m, l);
}

}  // namespace

cudaError_t launch_kv16_rows(const Kv16& c, const Kv16Query& q, uint16_t* out, float* lse,
                             cudaStream_t s) {
  const int grid = (q.total * q.Hq + kWarps - 1) / kWarps;
  if (c.half)
    kv16_rows_kernel<Fp16><<<grid, kWarps * 32, 0, s>>>(c, q, out, lse);
  else
    kv16_rows_kernel<Bf16><<<grid, kWarps * 32, 0, s>>>(c, q, out, lse);
  return cudaGetLastError();
}

size_t kv16_attention_ws_bytes(const Kv16&, int, int, int, int, int) { return 0; }

cudaError_t launch_kv16_attention(const Kv16& c, const Kv16Query& q, uint16_t* out, float* lse,
                                  void*, int* launches, cudaStream_t s) {
  *launches = 1;
  return launch_kv16_rows(c, q, out, lse, s);
}

}  // namespace oscar
