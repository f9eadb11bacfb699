// Attention of sequences that share a prefix: a group's whole pages below the
// prefix's end are read from its first sequence's table row, the rest from each
// sequence's own.
#include "kv16_groups.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 4;

// A warp per (query, head): the prefix's blocks, then the sequence's own.
template <class T>
__global__ void __launch_bounds__(kWarps * 32)
kv16_shared_kernel(const Kv16 c, const Kv16Query q, const Kv16Groups g, uint16_t* out, float* lse) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (long long)q.total * q.Hq) return;
  const int r = (int)(row / q.Hq), head = (int)(row % q.Hq), h = head / (q.Hq / c.Hkv);
  const int b = q.start ? ragged_sequence(q.start, c.B, r) : r;
  if (b < 0) return;
  int n = kv16_length(c, b, q.max_tok), back = 1;
  if (q.start) {
    const int s0 = __ldg(q.start + b), s1 = __ldg(q.start + b + 1);
    if (s0 < 0 || s1 > q.total) n = -1;
    back = s1 - r;
    if (n >= 0 && n < s1 - s0 && lane == 0) record_error(c.status, kDevErrBadPaged);
  }
  if (n < 0 && lane == 0) record_error(c.status, kDevErrBadPaged);
  const int at = max(n - back, -1);
  const int i = group_of(g, b);
  Shared s{b, b, 0};
  if (i >= 0) s = shared_of(c, g, i, q.max_tok, lane == 0);
  const Span all(at, at, q.window, q.n_sink);
  const uint16_t* qr = q.q + r * q.stride + (long long)head * kD;
  float m[2], l[2], o[2][4];
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const Span sp = part ? all.from(s.blocks) : all.below(s.blocks);
    kv16_warp_row<T>(c, qr, part ? b : s.lead, h, at, sp, 0, sp.blocks, q.window, q.n_sink,
                     q.scale_log2, 15u, m[part], l[part], o[part]);
  }
  const float M = fmaxf(m[0], m[1]);
  const float a = m[0] == M ? 1.0f : fast_exp2(m[0] - M), z = m[1] == M ? 1.0f : fast_exp2(m[1] - M);
  const float L = a * l[0] + z * l[1], inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
  for (int x = 0; x < 4; ++x) o[0][x] = (a * o[0][x] + z * o[1][x]) * inv;
  reinterpret_cast<uint2*>(out + row * kD)[lane] =
      make_uint2(T::pack(o[0][0], o[0][1]), T::pack(o[0][2], o[0][3]));
  if (lse && lane == 0) lse[row] = kv16_lse(M, L);
}

}  // namespace

size_t kv16_shared_ws_bytes(const Kv16&, int, int, int, int, int, int) { return kDecodeWsHeader; }

cudaError_t launch_kv16_shared(const Kv16& c, const Kv16Query& q, const Kv16Groups& g,
                               uint16_t* out, float* lse, void*, int* launches, cudaStream_t s) {
  const int grid = (int)(((long long)q.total * q.Hq + kWarps - 1) / kWarps);
  if (c.half) kv16_shared_kernel<Fp16><<<grid, kWarps * 32, 0, s>>>(c, q, g, out, lse);
  else kv16_shared_kernel<Bf16><<<grid, kWarps * 32, 0, s>>>(c, q, g, out, lse);
  *launches = 1;
  return cudaGetLastError();
}

}  // namespace oscar
