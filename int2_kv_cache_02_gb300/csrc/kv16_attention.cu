// Attention of a ragged batch of queries over the 16-bit cache: the join of split
// records and the launches (the kernel: kv16_attention.cuh).
#include "kv16_attention.cuh"

namespace oscar {
namespace {

// Joins the splits' records of a (query, head), a warp each; queries that
// belong to no sequence are left alone.
template <class T>
__global__ void __launch_bounds__(128) kv16_join_kernel(const AttnParams p) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)p.q.total * p.q.Hq) return;
  const int b = ragged_sequence(p.q.start, p.c.B, (int)(row / p.q.Hq));
  if (b < 0 || __ldg(p.q.start + b) < 0 || __ldg(p.q.start + b + 1) > p.q.total) return;
  const float* rec = p.part + row * p.splits * kRecFloats;
  float M = -INFINITY, L = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < p.splits; ++s) M = fmaxf(M, rec[s * kRecFloats]);
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(rec + s * kRecFloats);
    const float4 v = *reinterpret_cast<const float4*>(rec + s * kRecFloats + 4 + 4 * lane);
    const float a = M == -INFINITY ? 1.0f : fast_exp2(ml.x - M);
    L += a * ml.y;
    o[0] += a * v.x;
    o[1] += a * v.y;
    o[2] += a * v.z;
    o[3] += a * v.w;
  }
  store_row4<T>(p, row, lane, o, L == 0.0f ? 0.0f : 1.0f / L);
  if (p.lse && lane == 0) p.lse[row] = row_lse<T>(M, L);
}

template <class T>
cudaError_t launch(const AttnParams& p, int* launches, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!kv16_query_map(&mq, p.q, p.c.half, p.g, p.tokens) || !kv16_row_map(&mk, p.c, p.c.k) ||
      !kv16_row_map(&mv, p.c, p.c.v))
    return cudaErrorNotSupported;
  const auto kernel = kv16_attention_kernel<T, kWhole>;
  constexpr int kStages = stages_of(kWhole);
  constexpr int smem = (2 + kStages) * kTileBytes + (int)sizeof(Smem<kWhole>);
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(p.tiles * p.c.Hkv * p.splits, sm_count());
  kernel<<<grid, kThreads, smem, s>>>(mq, mk, mv, p);
  e = cudaGetLastError();
  *launches = 1;
  if (e != cudaSuccess || p.splits == 1) return e;
  const long long rows = (long long)p.q.total * p.q.Hq;
  kv16_join_kernel<T><<<(int)((rows + 3) / 4), 128, 0, s>>>(p);
  *launches = 2;
  return cudaGetLastError();
}

}  // namespace

size_t kv16_attention_ws_bytes(const Kv16& c, int Hq, int total, int max_tok, int window,
                               int n_sink) {
  const int splits = attention_splits(c, Hq, total, max_tok, window, n_sink);
  return splits > 1 ? (size_t)total * Hq * splits * kRecFloats * sizeof(float) : 0;
}

cudaError_t launch_kv16_attention(const Kv16& c, const Kv16Query& q, uint16_t* out, float* lse,
                                  void* ws, int* launches, cudaStream_t s) {
  AttnParams p;
  p.c = c;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.part = static_cast<float*>(ws);
  p.line = SharedParts{};
  p.g = q.Hq / c.Hkv;
  p.tokens = 128 / p.g;
  const long long tiles = attention_tiles(c.B, p.g, q.total);
  p.splits = attention_splits(c, q.Hq, q.total, q.max_tok, q.window, q.n_sink);
  if (tiles * c.Hkv * p.splits > 0x7fffffffLL) return cudaErrorInvalidValue;
  p.tiles = (int)tiles;
  p.wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;
  // a negative scale becomes a negated Q in the product, so that the largest
  // score is always the largest sum; a scale of 0 the smallest number there is,
  // so that a masked -inf stays one (times the largest score it is 5e-7)
  p.negate = q.scale_log2 < 0.0f;
  p.scale = std::max(std::fabs(q.scale_log2), std::numeric_limits<float>::denorm_min());
  return c.half ? launch<Fp16>(p, launches, s) : launch<Bf16>(p, launches, s);
}

}  // namespace oscar
