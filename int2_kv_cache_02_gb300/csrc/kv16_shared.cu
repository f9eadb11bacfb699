// Attention of sequences that share a prefix.  A group's whole pages below the
// prefix's end are worked once for all its sequences, by the tensor-core kernel
// of the prompt attention (kPrefix: rows are the group's queries, so up to 256
// (query, head) rows meet each key and value that is read); what stands behind
// them a sequence at a time, by the decode's kernel for one query each, else by
// the prompt attention's (kOwn).  Softmax parts are joined by their maxima and
// sums: the decode folds the prefix's records into a row that it begins, several
// queries have a kernel of their own for it.
#include "kv16_attention.cuh"

namespace oscar {
namespace {

// A (query, head) row's records joined, a warp each; queries that belong to no
// sequence are left alone.
template <class T>
__global__ void __launch_bounds__(128) kv16_shared_join_kernel(const AttnParams p,
                                                               const SharedParts prefix) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)p.q.total * p.q.Hq) return;
  const int r = (int)(row / p.q.Hq), head = (int)(row - (long long)r * p.q.Hq);
  const int b = ragged_sequence(p.q.start, p.c.B, r);
  if (b < 0 || __ldg(p.q.start + b) < 0 || __ldg(p.q.start + b + 1) > p.q.total) return;
  const int h = head / p.g, i = group_of(p.groups, b);
  const Joint in = joint_of(prefix, p.c, p.q, r, h, i);
  const int own = p.splits, n = own + in.n;
  const float* rec = p.part + row * own * kRecFloats;
  auto record = [&](int j) {
    return j < own ? rec + j * kRecFloats : in.record(j - own) + (head - h * p.g) * kRecFloats;
  };
  float M = -INFINITY, L = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = lane; j < n; j += 32) M = fmaxf(M, __ldcg(record(j)));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const float* e = record(j);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(e));
    const float4 v = __ldcg(reinterpret_cast<const float4*>(e + 4 + 4 * lane));
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

template <class T, int PART>
cudaError_t launch_part(const AttnParams& p, int grid, size_t more, bool early, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!kv16_query_map(&mq, p.q, p.c.half, p.g, p.tokens) || !kv16_row_map(&mk, p.c, p.c.k) ||
      !kv16_row_map(&mv, p.c, p.c.v))
    return cudaErrorNotSupported;
  const auto kernel = kv16_attention_kernel<T, PART>;
  constexpr int kStages = stages_of(PART);
  constexpr int fixed = (2 + kStages) * kTileBytes + (int)sizeof(Smem<kStages>);
  static_assert(fixed + (PART == kPrefix ? (kMaxGroups + 1 + kThreads / 32) * 4 : 0) <= 227 * 1024,
                "shared memory of a CTA");
  const int smem = fixed + (int)more;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = kThreads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, p);
}

// Where the records lie in the workspace, behind what the own parts' kernel has.
struct Layout {
  size_t part, cut, line, bytes;
};
size_t up16(size_t n) { return (n + 15) / 16 * 16; }
Layout layout(size_t own, long long rows, int ctas, int n_groups) {
  Layout x;
  x.part = up16(own);
  x.cut = x.part + (size_t)rows * kRecFloats * sizeof(float);
  x.line = x.cut + (size_t)ctas * 256 * kRecFloats * sizeof(float);
  x.bytes = x.line + (size_t)(n_groups + 1) * sizeof(SharedLine);
  return x;
}

// CTAs of the prefixes' kernel: one per SM, or as many as there can be tiles.
int prefix_grid(const Kv16& c, int Hq, int n_groups, int total, int max_tok) {
  const int two = 2 * (128 / (Hq / c.Hkv));
  const long long rows = (total / two + std::min(n_groups, total)) * (long long)c.Hkv;
  const long long tiles = rows * ((std::min(max_tok, c.cap) + 127) / 128);
  return (int)std::max<long long>(1, std::min<long long>(tiles / kMinTiles + 1, sm_count()));
}

size_t own_bytes(const Kv16& c, int Hq, int total, bool decode, int max_tok, int window, int n_sink) {
  if (decode) return kv16_decode_ws_bytes(c, Hq, max_tok, window, n_sink, false);
  const int splits = attention_splits(c, Hq, total, max_tok, window, n_sink);
  return kDecodeWsHeader + (size_t)total * Hq * splits * kRecFloats * sizeof(float);
}

template <class T>
cudaError_t launch(const AttnParams& prefix, int ctas, const SharedParts& parts, AttnParams own,
                   void* ws, int* launches, cudaStream_t s) {
  cudaError_t e = launch_part<T, kPrefix>(
      prefix, ctas, (size_t)(prefix.groups.n + 1 + kThreads / 32) * sizeof(int), false, s);
  if (e != cudaSuccess) return e;
  *launches = 1;
  if (!own.q.start) {
    int n = 0;
    e = launch_kv16_decode_own(own.c, own.q, parts, own.out, ws, &n, s);
    *launches += n;
    return e;
  }
  e = launch_part<T, kOwn>(own, std::min(own.tiles * own.c.Hkv * own.splits, sm_count()), 0, true, s);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)(((long long)own.q.total * own.q.Hq + 3) / 4);
  cfg.blockDim = 128;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  *launches = 3;
  return cudaLaunchKernelEx(&cfg, kv16_shared_join_kernel<T>, own, parts);
}

}  // namespace

size_t kv16_shared_ws_bytes(const Kv16& c, int Hq, int n_groups, int total, bool decode,
                            int max_tok, int window, int n_sink) {
  return layout(own_bytes(c, Hq, total, decode, max_tok, window, n_sink), (long long)total * Hq,
                prefix_grid(c, Hq, n_groups, total, max_tok), n_groups).bytes;
}

cudaError_t launch_kv16_shared(const Kv16& c, const Kv16Query& q, const Kv16Groups& g,
                               uint16_t* out, float* lse, void* ws, int* launches, cudaStream_t s) {
  const bool decode = !q.start;
  const int ctas = prefix_grid(c, q.Hq, g.n, q.total, q.max_tok);
  const Layout at = layout(own_bytes(c, q.Hq, q.total, decode, q.max_tok, q.window, q.n_sink),
                           (long long)q.total * q.Hq, ctas, g.n);
  uint8_t* base = static_cast<uint8_t*>(ws);
  AttnParams p;
  p.c = c;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.part = reinterpret_cast<float*>(base + at.part);
  p.cut = reinterpret_cast<float*>(base + at.cut);
  p.line = reinterpret_cast<SharedLine*>(base + at.line);
  p.groups = g;
  p.g = q.Hq / c.Hkv;
  p.tokens = 128 / p.g;
  p.tiles = 0;
  p.splits = 1;
  p.negate = q.scale_log2 < 0.0f;
  p.scale = std::max(std::fabs(q.scale_log2), std::numeric_limits<float>::denorm_min());
  p.wide = false;
  const SharedParts parts{g, p.part, p.cut, p.line, ctas, p.tokens, p.g};
  AttnParams own = p;
  own.part = reinterpret_cast<float*>(base + kDecodeWsHeader);
  if (!decode) {
    const long long tiles = attention_tiles(c.B, p.g, q.total);
    own.splits = attention_splits(c, q.Hq, q.total, q.max_tok, q.window, q.n_sink);
    if (tiles * c.Hkv * own.splits > 0x7fffffffLL) return cudaErrorInvalidValue;
    own.tiles = (int)tiles;
  }
  *launches = 0;
  return c.half ? launch<Fp16>(p, ctas, parts, own, ws, launches, s)
                : launch<Bf16>(p, ctas, parts, own, ws, launches, s);
}

}  // namespace oscar
