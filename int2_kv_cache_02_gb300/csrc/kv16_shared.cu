// Attention of sequences that share a prefix.  A group's whole pages below the
// prefix's end are worked once for all its sequences, by the tensor-core kernel
// of the prompt attention (kPrefix: rows are the group's queries, so up to 256
// (query, head) rows meet each key and value that is read); what stands behind
// them a sequence at a time, by a kernel of the decode's kind for one query each
// (kv16_shared_decode.cu), else by the prompt attention's (kOwn).  Both leave
// records, which a third kernel joins by their maxima and sums.
#include "kv16_attention.cuh"

namespace oscar {
namespace {

// What the values that a row sees hold in a channel.
constexpr unsigned kSeenNan = 1, kSeenPlus = 2, kSeenMinus = 4, kOpen = 8;
__device__ __forceinline__ unsigned seen_in(float x) {
  return x != x ? kSeenNan : x == INFINITY ? kSeenPlus : x == -INFINITY ? kSeenMinus : 0u;
}

// Blocks of a chunk are at least a run's length and below two: three runs at most.
constexpr int kBlockRuns = 3;
// A line has less than half as many blocks as CTAs where it has chunks.
constexpr int kMaxCtas = 160;
constexpr int kList = kBlockRuns * (kMaxCtas / 2 + 1);

// The records of both parts of a (query, KV head) joined, by W warps: as many
// warps for a head as there are (up to W heads at a time), each every so-many-th
// record.  Queries that belong to no sequence are left alone.
//
// A record may hold an infinity (a visible one) that its factor of 0 turns into
// NaN.  Where a channel is NaN although the row's sum is a number, what the
// visible values hold there decides, as in the decode.
template <class T, int W>
__global__ void __launch_bounds__(W * 32) kv16_shared_join_kernel(
    const Kv16 c, const Kv16Query q, const SharedParts s, uint16_t* out, float* lse) {
  __shared__ float4 s_o[W][32];
  __shared__ float2 s_ml[W];
  __shared__ int list[kList];
  __shared__ unsigned s_ch[kD];
  __shared__ uint8_t s_nan[kMaxGroup];
  __shared__ int s_open;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = s.g;
  const int r = blockIdx.x / c.Hkv, h = blockIdx.x - r * c.Hkv;
  int b = r, back = 1;
  if (q.start) {
    b = warp_search(q.start, c.B, r);
    const int s0 = __ldg(q.start + b), s1 = __ldg(q.start + b + 1);
    if (s0 < 0 || s0 > r || r >= s1 || s1 > q.total) return;
    back = s1 - r;
  }
  // the sequence's own records
  const long long row = (long long)r * q.Hq + h * g;
  int own = s.splits, w0 = 0;
  if (!q.start) {
    const int f0 = __ldcg(s.own_line + b), f1 = __ldcg(s.own_line + b + 1);
    const int per = run_share(__ldcg(s.own_line + c.B) * c.Hkv, s.workers);
    const int at = f0 * c.Hkv + h * (f1 - f0);
    w0 = at / per;
    own = f1 > f0 ? (at + f1 - f0 - 1) / per - w0 + 1 : 0;
  }
  // the prefix's
  const int i = warp_search(s.groups.group, s.groups.n, b);
  SharedLine line{0, 0, 0, 0};
  if (__ldg(s.groups.group + i) <= b && b < __ldg(s.groups.group + i + 1)) {
    const int4 x = __ldcg(reinterpret_cast<const int4*>(s.line) + i);
    line = SharedLine{x.x, x.y, x.z, x.w};
  }
  int n = own, c0 = 0, blocks = 1, in_chunk = 0;
  const int two = 2 * s.tokens, chunk = r >= line.r0 ? (r - line.r0) / two : line.chunks;
  if (line.tiles > 0 && chunk < line.chunks) {
    const int in = (r - line.r0) % two, w = in >= s.tokens ? 1 : 0;
    in_chunk = w * 128 + (in - w * s.tokens) * g;
    const int per = line_share(__ldcg(&s.line[s.groups.n].first), s.ctas);
    blocks = line_blocks(line.tiles, line.chunks, per);
    const long long base = line.first + (long long)h * line.chunks * line.tiles;
    auto ctas_of = [&](int k, int& from) {
      const int t0 = block_tile(line.tiles, blocks, k), t1 = block_tile(line.tiles, blocks, k + 1);
      const long long at = base + (long long)line.chunks * t0 + (long long)chunk * (t1 - t0);
      from = (int)min(at / per, s.ctas - 1LL);
      return (int)min((at + t1 - t0 - 1) / per, s.ctas - 1LL) - from + 1;
    };
    if (blocks == 1) {
      n += ctas_of(0, c0);
    } else {
      for (int k = tid; k < blocks; k += W * 32) {
        int from;
        const int m = ctas_of(k, from);
        for (int x = 0; x < kBlockRuns; ++x)
          list[k * kBlockRuns + x] = x >= m ? -1 : x > 0 || k > 0 ? (from + x) * 2 + (x == 0) : -2;
      }
      n += blocks * kBlockRuns;
    }
  }
  for (int x = tid; x < kD; x += W * 32) s_ch[x] = 0u;
  if (tid == 0) s_open = 0;
  __syncthreads();
  // record j for head 0 of the group, or nullptr
  auto record = [&](int j) -> const float* {
    if (j < own)
      return (q.start ? s.own + (row * own + j) * kRecFloats
              : j == 0 ? s.own + row * kRecFloats
                       : s.own_cut + (long long)(w0 + j) * g * kRecFloats);
    j -= own;
    const int at = blocks > 1 ? list[j] : j == 0 ? -2 : (c0 + j) * 2;
    return at == -1 ? nullptr
           : at < 0 ? s.part + row * kRecFloats
                    : s.cut + ((long long)at * 256 + in_chunk) * kRecFloats;
  };
  int subs = W;      // warps of a head
  while (subs > 1 && W / subs < g) subs >>= 1;
  const int sub = warp % subs;
  for (int h0 = 0; h0 < g; h0 += W / subs) {
    const int head = h0 + warp / subs;
    float M = -INFINITY, L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (head < g) {
      constexpr int U = 4;       // records in flight
      for (int j0 = sub; j0 < n; j0 += U * subs) {
        float2 ml[U];
        float4 v[U];
        float mx = M;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * subs;
          const float* e = j < n ? record(j) : nullptr;
          ml[u] = make_float2(-INFINITY, 0.0f);
          v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (e) {
            // (own records of several queries: a head's lie behind one another)
            e += (j < own && q.start ? head * own : head) * kRecFloats;
            ml[u] = __ldcg(reinterpret_cast<const float2*>(e));
            v[u] = __ldcg(reinterpret_cast<const float4*>(e + 4) + lane);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) mx = fmaxf(mx, ml[u].x);
        const float f = mx == -INFINITY ? 1.0f : fast_exp2(M - mx);
        M = mx;
        L *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float a = mx == -INFINITY ? 1.0f : fast_exp2(ml[u].x - mx);
          L += a * ml[u].y;
          o.x += a * v[u].x;
          o.y += a * v[u].y;
          o.z += a * v[u].z;
          o.w += a * v[u].w;
        }
      }
    }
    if (subs > 1) {
      s_o[warp][lane] = o;
      if (lane == 0) s_ml[warp] = make_float2(M, L);
      __syncthreads();
      if (sub == 0 && head < g) {
        float mx = M;
        for (int u = 1; u < subs; ++u) mx = fmaxf(mx, s_ml[warp + u].x);
        const float f = mx == -INFINITY ? 1.0f : fast_exp2(M - mx);
        M = mx;
        L *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
        for (int u = 1; u < subs; ++u) {
          const float2 ml = s_ml[warp + u];
          const float4 v = s_o[warp + u][lane];
          const float a = mx == -INFINITY ? 1.0f : fast_exp2(ml.x - mx);
          L += a * ml.y;
          o.x += a * v.x;
          o.y += a * v.y;
          o.z += a * v.z;
          o.w += a * v.w;
        }
      }
      __syncthreads();
    }
    if (sub == 0 && head < g) {
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      reinterpret_cast<uint2*>(out + (row + head) * kD)[lane] =
          make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv));
      if (lse && lane == 0) lse[row + head] = row_lse<T>(M, L);
      if (lane == 0) s_nan[head] = L != L;
      if (L == L) {
        const float x[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (x[k] != x[k]) {
            s_ch[4 * lane + k] = kOpen;
            s_open = 1;
          }
      }
    }
  }
  __syncthreads();
  if (!s_open) return;

  // open channels: what the visible values hold in them
  const int len = kv16_length(c, b, q.max_tok), at = len < 0 ? -1 : max(len - back, -1);
  const int gi = group_of(s.groups, b);
  Shared sh{b, b, 0};
  if (gi >= 0) sh = shared_of(c, s.groups, gi, q.max_tok, false);
  const Span sp(at, at, q.window, q.n_sink);
  for (int x = warp; x < sp.blocks; x += W) {
    const int blk = sp.block(x);
    const int kr = kv16_block_row(c, blk < sh.blocks ? sh.lead : b, h, blk);
    if (kr < 0) continue;
    const unsigned see =
        __ballot_sync(0xffffffffu, kv16_visible(blk * kPage + lane, at, q.window, q.n_sink));
    unsigned f[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
    for (int t = 0; t < kPage; ++t) {
      uint2 v = make_uint2(0u, 0u);
      if ((see >> t) & 1u) v = reinterpret_cast<const uint2*>(c.v)[((long long)kr + t) * 32 + lane];
      const float2 a = T::unpack(v.x), z = T::unpack(v.y);
      f[0] |= seen_in(a.x);
      f[1] |= seen_in(a.y);
      f[2] |= seen_in(z.x);
      f[3] |= seen_in(z.y);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f[k]) atomicOr(&s_ch[4 * lane + k], f[k]);
  }
  __syncthreads();
  for (int x = tid; x < g * 64; x += W * 32) {
    const int head = x >> 6, pair = x & 63;
    if (s_nan[head]) continue;
    uint32_t* d = reinterpret_cast<uint32_t*>(out + (row + head) * kD) + pair;
    float2 v = T::unpack(*d);
    auto settled = [&](float y, unsigned k) {
      return y == y ? y : k == (kOpen | kSeenPlus) ? INFINITY : k == (kOpen | kSeenMinus) ? -INFINITY : y;
    };
    v.x = settled(v.x, s_ch[2 * pair]);
    v.y = settled(v.y, s_ch[2 * pair + 1]);
    *d = T::pack(v.x, v.y);
  }
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

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// CTAs of the prefixes' kernel: one per SM, or as many as there can be tiles.
int prefix_grid(const Kv16& c, int Hq, int n_groups, int total, int max_tok) {
  const int two = 2 * (128 / (Hq / c.Hkv));
  const long long rows = (total / two + std::min(n_groups, total)) * (long long)c.Hkv;
  const long long tiles = rows * ((std::min(max_tok, c.cap) + 127) / 128);
  return (int)std::max<long long>(
      1, std::min<long long>(tiles / kMinTiles + 1, std::min(sm_count(), kMaxCtas)));
}

// The call's plan: grids, splits, and where the records lie in the workspace.
struct Plan {
  SharedParts s;
  size_t bytes;
};
Plan plan(const Kv16& c, int Hq, const Kv16Groups& groups, int total, bool decode, int max_tok,
          int window, int n_sink, uint8_t* ws) {
  Plan x{};
  SharedParts& s = x.s;
  s.groups = groups;
  s.g = Hq / c.Hkv;
  s.tokens = 128 / s.g;
  s.ctas = prefix_grid(c, Hq, groups.n, total, max_tok);
  auto take = [&](size_t n) {
    uint8_t* p = ws + x.bytes;
    x.bytes += up16(n);
    return p;
  };
  const size_t rec = kRecFloats * sizeof(float), rows = (size_t)total * Hq;
  s.part = reinterpret_cast<float*>(take(rows * rec));
  s.cut = reinterpret_cast<float*>(take((size_t)s.ctas * 2 * 256 * rec));
  s.line = reinterpret_cast<SharedLine*>(take((size_t)(groups.n + 1) * sizeof(SharedLine)));
  if (decode) {
    const long long pages = (long long)c.B * c.Hkv * ((std::min(max_tok, c.cap) + kPage - 1) / kPage);
    s.workers = kv16_own_workers(pages, sm_count());
    s.own = reinterpret_cast<float*>(take(rows * rec));
    s.own_cut = reinterpret_cast<float*>(take((size_t)s.workers * s.g * rec));
    s.own_line = reinterpret_cast<int*>(take((size_t)(c.B + 1) * sizeof(int)));
  } else {
    s.splits = attention_splits(c, Hq, total, max_tok, window, n_sink);
    s.own = reinterpret_cast<float*>(take(rows * s.splits * rec));
  }
  return x;
}

template <class T, int W>
cudaError_t launch_join(const Kv16& c, const Kv16Query& q, const SharedParts& s, uint16_t* out,
                        float* lse, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)((long long)q.total * c.Hkv);
  cfg.blockDim = W * 32;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv16_shared_join_kernel<T, W>, c, q, s, out, lse);
}

template <class T>
cudaError_t launch(AttnParams p, const SharedParts& s, uint16_t* out, float* lse, int* launches,
                   cudaStream_t stream) {
  p.part = s.part;
  p.splits = 1;
  cudaError_t e = launch_part<T, kPrefix>(
      p, s.ctas, (size_t)(p.groups.n + 1 + kThreads / 32) * sizeof(int), false, stream);
  if (e != cudaSuccess) return e;
  *launches = 1;
  if (!p.q.start) {
    e = launch_kv16_own(p.c, p.q, s, stream);
  } else {
    p.part = s.own;
    p.splits = s.splits;
    e = launch_part<T, kOwn>(p, std::min(p.tiles * p.c.Hkv * p.splits, sm_count()), 0, true, stream);
  }
  if (e != cudaSuccess) return e;
  *launches = 3;
  return p.q.start ? launch_join<T, 4>(p.c, p.q, s, out, lse, stream)
                   : launch_join<T, 8>(p.c, p.q, s, out, lse, stream);
}

}  // namespace

size_t kv16_shared_ws_bytes(const Kv16& c, int Hq, int n_groups, int total, bool decode,
                            int max_tok, int window, int n_sink) {
  return plan(c, Hq, Kv16Groups{nullptr, nullptr, n_groups}, total, decode, max_tok, window, n_sink,
              nullptr).bytes;
}

cudaError_t launch_kv16_shared(const Kv16& c, const Kv16Query& q, const Kv16Groups& g,
                               uint16_t* out, float* lse, void* ws, int* launches, cudaStream_t s) {
  const Plan x = plan(c, q.Hq, g, q.total, !q.start, q.max_tok, q.window, q.n_sink,
                      static_cast<uint8_t*>(ws));
  AttnParams p;
  p.c = c;
  p.q = q;
  p.out = nullptr;
  p.lse = nullptr;
  p.cut = x.s.cut;
  p.line = x.s.line;
  p.groups = g;
  p.g = x.s.g;
  p.tokens = x.s.tokens;
  p.tiles = 0;
  if (q.start) {
    const long long tiles = attention_tiles(c.B, p.g, q.total);
    if (tiles * c.Hkv * x.s.splits > 0x7fffffffLL) return cudaErrorInvalidValue;
    p.tiles = (int)tiles;
  }
  p.negate = q.scale_log2 < 0.0f;
  p.scale = std::max(std::fabs(q.scale_log2), std::numeric_limits<float>::denorm_min());
  p.wide = false;
  *launches = 0;
  return c.half ? launch<Fp16>(p, x.s, out, lse, launches, s)
                : launch<Bf16>(p, x.s, out, lse, launches, s);
}

}  // namespace oscar
