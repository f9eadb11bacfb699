// Attention of sequences that share a prefix.  A group's whole pages below the
// prefix's end are worked once for all its queries, so that up to 256 (query,
// head) rows meet each key and value that is read; what stands behind them a
// sequence at a time.  Both by the tensor-core kernel of the prompt attention, over
// one line of key tiles that its CTAs share evenly (kLine, kv16_line.h); the
// records that it leaves are joined by their maxima and sums in a second launch,
// which is placed while the first ends.
//
// Probabilities are rounded to the type of V for the product, as in the prompt's
// attention (the decode's own kernel keeps the remainder too: it has tensor time to
// spare where 256 rows a key have not): half a step relative, as the output itself.
// So the two ways of the decode differ in that; what they are off by stands in the header.
//
// What bounds it.  256 rows need 256 flops for each byte of keys and values; the GPU
// has 287 for each byte that HBM delivers (both measured).  A group of fewer rows is
// bound by HBM, of more by the tensor cores; what the sequences have of their own is
// bound by HBM, at g rows for each key.
//
// Measured (GB300, in a graph; in brackets the same by the calls that do not know of
// groups).  Sixteen samples of an 8K prompt, 32/8 heads, 200 to 512 tokens each of
// their own: 25 us [62] (floor 8.3; of the rest 6 pass before the first product, as
// many after the last).  128 requests under four prompts of 10K to 16K, 0.2K to 2K
// tokens each of their own: 158 us [780], 827 MB from HBM (floor 120).  128 requests
// about two documents of 54K and 66K, 32/4 heads, fp16: 148 us [1590] (floor 65; the
// prefixes' 7.5K tiles of two query tiles take 1.65 us each, 0.79 of the measured bf16
// rate, on 108 of the SMs, while the others read what the requests have of their own).
// 48 sequences under four instructions of 4.3K to 6K, a window of 4K and 4 sinks, 24/2
// heads, fp16: 33 us [40] (floor 13; masked tiles of two query tiles take 3 us each).
// 951 tokens of 16 questions behind two instructions of 7.7K and 8.2K: 128 us [181] (floor
// 64, 20 of it the join of 30K rows).  112 drafted tokens of 32 samples of 32K: 84 us
// [685] (floor 31).
//
// Tried, slower: the prefixes in a launch of their own with the decode's kernel for
// the rest, whose CTAs joined a row at a time (236 us for the four prompts), or with
// warps on their own for the rest (157, three launches, and 151 for the documents);
// the two query tiles' results merged in the CTA (3 us an item); tiles called into L2
// four ahead of their copies (185); pages looked up eight tiles ahead (1 to 4 %); a
// round of the softmax before the first scores to fetch its instructions (0.5 to 1 us).
// The two SMs of a pair slow each other down where one has long rows of two query tiles
// and the other many of a single tile of keys (a CTA of the questions 132 us instead of
// 100); the sequences' rows begun with an even CTA, so that no pair has both, cost
// other calls more (1 % on average).
#include "kv16_attention.cuh"

namespace oscar {
namespace {

constexpr int kMaxCtas = 160;      // of the line's kernel

// (bounded: what is not written for a row out of range may hold anything)
__device__ __forceinline__ Runs runs_from(int x, int ctas) {
  const int c0 = min(x & 0xffff, ctas - 1);
  return Runs{c0, min(x >> 16, ctas - c0)};
}

// The records of both parts of a row (query, head) joined by a warp, and queries that
// belong to no sequence left alone.  Few rows (BATCH false): a CTA has rows of one
// query and KV head, a warp each or `subs` of its four warps, each every so-many-th
// record.  Many: a warp has the group's rows of `batch` queries one after another,
// two rows at a time, half its lanes each.
//
// Bound by latency where rows are few: the sequence, its group and its runs are a
// chain of loads, then a record's place is found.  So a warp's lanes find 32 records
// at a time, a lane each, once for the queries that lie in the same rows of the line,
// and eight records are in flight.  Bound by instructions where rows are many (30K
// rows: 28 us by a warp a row, 20 by halves).
constexpr int kJoinWarps = 4, kJoinCtas = 6, kBatchCtas = 5;     // warps of a CTA, CTAs of an SM
template <class T, bool BATCH>
__global__ void __launch_bounds__(kJoinWarps * 32, BATCH ? kBatchCtas : kJoinCtas)
kv16_shared_join_kernel(const __grid_constant__ AttnParams p, int subs, int batch) {
  __shared__ float4 s_o[BATCH ? 1 : kJoinWarps][32];
  __shared__ float2 s_ml[BATCH ? 1 : kJoinWarps];
  const SharedParts& s = p.line;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = p.g, two = 2 * p.tokens;
  int first_r, end_r, h, head0 = 0, sub = 0;
  if constexpr (BATCH) {
    const int x = blockIdx.x / p.c.Hkv;
    h = blockIdx.x - x * p.c.Hkv;
    first_r = (x * kJoinWarps + warp) * batch;
    end_r = min(first_r + batch, p.q.total);
    subs = 1;
  } else {
    const int rows = kJoinWarps / subs, slices = (g + rows - 1) / rows, x = blockIdx.x / slices;
    first_r = x / p.c.Hkv;
    end_r = first_r + 1;
    h = x - first_r * p.c.Hkv;
    head0 = (blockIdx.x - x * slices) * rows + warp / subs;
    sub = warp % subs;
  }
  const int G = s.groups.n;
  // the sequence of query r, and its queries
  int b = -1, seq0 = 0, seq1 = 0;
  auto find = [&](int r) {
    b = r;
    seq0 = r;
    seq1 = r + 1;
    if (!p.q.start) return;
    b = warp_sequence(p.q.start, p.c.B, r);
    if (b < 0) return;
    seq0 = __ldg(p.q.start + b);
    seq1 = __ldg(p.q.start + b + 1);
    if (seq0 < 0 || seq1 > p.q.total) b = -1;
  };
  // A first wave of CTAs waits for the line: it finds its sequence and group meanwhile,
  // from what the call was given (0.5 to 1.5 us of a call), where later ones load
  // what the line has found.
  const bool early = !BATCH && blockIdx.x < kJoinCtas * s.ctas;
  int2 sq = make_int2(-1, 0);
  int4 gr = make_int4(0, 0, 0, 0);
  if (!BATCH) find(first_r);
  if (early && b >= 0) {
    sq.x = warp_sequence(s.groups.group, G, b);
    if (sq.x >= 0) {
      const GroupEntry y = warp_group_entry(p, sq.x);
      sq.y = y.s.blocks;
      gr = make_int4(key_tiles(y.sp.blocks), y.r0, y.r1, 0);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned per = line_share(__ldcg(s.first + G + p.c.B), s.ctas);

  // of the queries [.., same): their sequence, and their rows of the line
  int same = first_r, n = 0;
  Runs own{0, 0}, prefix{0, 0};
  int twice_own = 0, twice = 0;     // two records a run
  int in_own = 0, in_prefix = 0;    // the query's place in its chunks
  int kind = 0;
  int chunks = 1, chunk = 0;
  unsigned at = 0;
  Blocks blocks(0, 1, 0, 1);
  // the lane's record of head 0 in 32-byte steps from the first of all, or none; from a
  // query to the next it moves by `step`, and by `fix` more into a chunk's second tile
  constexpr unsigned kNone = ~0u, kSteps = kPartFloats / 8;
  static_assert((4 * kMaxSharedRows + kMaxCtas * 512LL) * kSteps < kNone, "records' places");
  const unsigned fix = (128 - p.tokens * g) * kSteps;
  unsigned off = kNone, step = 0;
  int in = -1;                      // 0 own, 1 prefix: which chunk the record's place goes by
  auto locate = [&](int j, int r) {
    off = kNone;
    step = 0;
    in = -1;
    const int n_own = own.n << twice_own;
    const bool mine = j < n_own;
    if (j >= n) return;
    if (!mine) j -= n_own;
    const int second = (mine ? twice_own : twice) ? j & 1 : 0;
    j >>= mine ? twice_own : twice;
    Runs x = mine ? own : prefix;
    int k = 0;
    if (!mine && blocks.count > 1) {
      k = j / kBlockRuns;
      j -= k * kBlockRuns;
      const int t0 = blocks.first(k), t1 = blocks.first(k + 1);
      const int p0 = tile_place(t0, kind), len = row_places(t1, kind) - p0;
      x = runs_of(at + (unsigned)chunks * p0 + (unsigned)chunk * len + (k == 0 ? row_cost(kind) : 0),
                  (t1 - t0 - 1) * tile_cost(kind), per, s.ctas);
    }
    if (j >= x.n) return;
    const float* e;
    if (j == 0 && k == 0) {
      e = (mine ? s.own : s.prefix) +
          (((long long)second * p.q.total + r) * p.q.Hq + h * g) * kPartFloats;
      step = p.q.Hq * kSteps;
    } else {
      in = mine ? 0 : 1;
      const int i = mine ? in_own : in_prefix, w = i >= p.tokens ? 1 : 0;
      e = s.cut + ((long long)(x.c0 + j) * 512 + (j == 0 ? 256 : 0) + (second + w) * 128 +
                   (i - w * p.tokens) * g) * kPartFloats;
      step = g * kSteps;
    }
    off = (unsigned)((e - s.prefix) / 8);
  };
#pragma unroll 1
  for (int r = first_r; r < end_r; ++r) {
    if (r < same) {
      // the same rows of the line, the next query
      ++in_own;
      ++in_prefix;
      off += step;
      if ((in == 0 && in_own == p.tokens) || (in == 1 && in_prefix == p.tokens)) off += fix;
    } else {
      same = r + 1;
      if (BATCH) find(r);
      if (b < 0) continue;
      if (!early) sq = __ldcg(s.seq + b);
      const int len = kv16_length(p.c, b, p.q.max_tok), own_chunk = (r - seq0) / two;
      const int row0 = seq0 + own_chunk * two;
      int to = min(seq1, row0 + two);
      in_own = r - row0;
      twice_own = seq1 - row0 <= p.tokens;
      own = prefix = Runs{0, 0};
      // does the chunk's last query stand in or behind the first block of its own?
      if (len - (seq1 - to) - 1 >= sq.y * kPage && len > 0)
        own = runs_from(__ldcg(s.own_runs + (long long)row0 * p.c.Hkv + h), s.ctas);
      blocks = Blocks(0, 1, 0, 1);
      if (sq.x >= 0) {
        if (!early) gr = __ldcg(s.group + sq.x);
        const int tiles = gr.x, rows = gr.z - gr.y;
        chunk = (r - gr.y) / two;
        chunks = (rows + two - 1) / two;
        if (tiles > 0 && r >= gr.y && chunk < chunks) {
          const int p_row0 = gr.y + chunk * two;
          kind = group_kind(p, rows);
          in_prefix = r - p_row0;
          twice = gr.z - p_row0 <= p.tokens;
          to = min(to, p_row0 + two);
          blocks = Blocks(tiles, chunks, kind, per);
          if (blocks.count > 1) {
            at = __ldcg(s.first + sq.x) + (unsigned)chunks * (unsigned)row_places(tiles, kind) * h;
            prefix = Runs{0, blocks.count * kBlockRuns};
          } else {
            prefix = runs_from(__ldcg(s.prefix_runs + (long long)p_row0 * p.c.Hkv + h), s.ctas);
          }
        }
      }
      same = to;
      n = (own.n << twice_own) + (prefix.n << twice);
      locate(sub + lane * subs, r);
    }
    if (b < 0) continue;
    if constexpr (BATCH) {
      const int half = lane >> 4, ch = lane & 15;      // 8 channels a lane
#pragma unroll 1
      for (int pair0 = 0; pair0 < g; pair0 += 2) {
        const int head = min(pair0 + half, g - 1);     // (an odd group's last row twice)
        float M = -INFINITY, L = 0.0f, o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += 32) {
          if (n > 32) locate(j0 + lane, r);
          unsigned have = __ballot_sync(0xffffffffu, off != kNone);
#pragma unroll 1
          while (have) {
            constexpr int U = 5;
            float2 ml[U];
            float4 v[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const unsigned from = __shfl_sync(0xffffffffu, off, __ffs(have) - 1);
              ml[u] = make_float2(-INFINITY, 0.0f);
              v[u][0] = v[u][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (have) {
                const float* e = s.prefix + (size_t)(from + head * kSteps) * 8;
                ml[u] = __ldcg(reinterpret_cast<const float2*>(e));
                v[u][0] = __ldcg(reinterpret_cast<const float4*>(e + kPartHead) + 2 * ch);
                v[u][1] = __ldcg(reinterpret_cast<const float4*>(e + kPartHead) + 2 * ch + 1);
              }
              have &= have - 1;
            }
            float mx = M;
#pragma unroll
            for (int u = 0; u < U; ++u) mx = fmaxf(mx, ml[u].x);
            // (a maximum of -inf has met only sums of 0, or NaN, and outputs of 0)
            const float ms = mx == -INFINITY ? 0.0f : mx, f = fast_exp2(M - ms);
            M = mx;
            L *= f;
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const float a = fast_exp2(ml[u].x - ms);
              L += a * ml[u].y;
              o[0] += a * v[u][0].x;
              o[1] += a * v[u][0].y;
              o[2] += a * v[u][0].z;
              o[3] += a * v[u][0].w;
              o[4] += a * v[u][1].x;
              o[5] += a * v[u][1].y;
              o[6] += a * v[u][1].z;
              o[7] += a * v[u][1].w;
            }
          }
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const long long row = (long long)r * p.q.Hq + h * g + head;
        reinterpret_cast<uint4*>(p.out + row * kD)[ch] =
            make_uint4(T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv),
                       T::pack(o[4] * inv, o[5] * inv), T::pack(o[6] * inv, o[7] * inv));
        if (p.lse && ch == 0) p.lse[row] = row_lse<T>(M, L);
        bool open = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) open |= o[k] != o[k];
        const unsigned bad = __ballot_sync(0xffffffffu, open && L == L);
        if (bad == 0) continue;
        // rows with a channel that is NaN though the sum is not, by the whole warp
        for (int z = 0; z < 2 && pair0 + z < g; ++z) {
          if (!(bad & (z ? 0xffff0000u : 0xffffu))) continue;
          float x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float lo = __shfl_sync(0xffffffffu, o[k], z * 16 + (lane >> 1));
            const float hi = __shfl_sync(0xffffffffu, o[k + 4], z * 16 + (lane >> 1));
            x[k] = lane & 1 ? hi : lo;
          }
          const float i = __shfl_sync(0xffffffffu, inv, z * 16);
          const float4 y = settle<T>(p.c, p.q, s.groups, b, h, seq1 - r, make_float4(x[0], x[1], x[2], x[3]));
          __syncwarp();
          reinterpret_cast<uint2*>(p.out + ((long long)r * p.q.Hq + h * g + pair0 + z) * kD)[lane] =
              make_uint2(T::pack(y.x * i, y.y * i), T::pack(y.z * i, y.w * i));
        }
      }
    } else {
      if (head0 >= g) n = 0;
      float M = -INFINITY, L = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
      for (int j0 = sub; j0 < n; j0 += 32 * subs) {
        if (n > 32 * subs) locate(j0 + lane * subs, r);
        unsigned have = __ballot_sync(0xffffffffu, off != kNone);
#pragma unroll 1
        while (have) {
          constexpr int U = 8;
          float2 ml[U];
          float4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const unsigned from = __shfl_sync(0xffffffffu, off, __ffs(have) - 1);
            ml[u] = make_float2(-INFINITY, 0.0f);
            v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (have) {
              const float* e = s.prefix + (size_t)(from + head0 * kSteps) * 8;
              ml[u] = __ldcg(reinterpret_cast<const float2*>(e));
              v[u] = __ldcg(reinterpret_cast<const float4*>(e + kPartHead) + lane);
            }
            have &= have - 1;
          }
          float mx = M;
#pragma unroll
          for (int u = 0; u < U; ++u) mx = fmaxf(mx, ml[u].x);
          const float ms = mx == -INFINITY ? 0.0f : mx, f = fast_exp2(M - ms);
          M = mx;
          L *= f;
          o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float a = fast_exp2(ml[u].x - ms);
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
        if (sub > 0) return;
        float mx = M;
        for (int u = 1; u < subs; ++u) mx = fmaxf(mx, s_ml[warp + u].x);
        const float ms = mx == -INFINITY ? 0.0f : mx, f = fast_exp2(M - ms);
        M = mx;
        L *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
        for (int u = 1; u < subs; ++u) {
          const float2 ml = s_ml[warp + u];
          const float4 v = s_o[warp + u][lane];
          const float a = fast_exp2(ml.x - ms);
          L += a * ml.y;
          o.x += a * v.x;
          o.y += a * v.y;
          o.z += a * v.z;
          o.w += a * v.w;
        }
      }
      if (head0 >= g) return;
      const bool open = o.x != o.x || o.y != o.y || o.z != o.z || o.w != o.w;
      if (L == L && __any_sync(0xffffffffu, open)) o = settle<T>(p.c, p.q, s.groups, b, h, seq1 - r, o);
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      const long long row = (long long)r * p.q.Hq + h * g + head0;
      reinterpret_cast<uint2*>(p.out + row * kD)[lane] =
          make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv));
      if (p.lse && lane == 0) p.lse[row] = row_lse<T>(M, L);
    }
  }
}

size_t up32(size_t n) { return (n + 31) / 32 * 32; }

// The line's CTAs: one per SM, or as many as there can be runs.
int line_ctas(const Kv16& c, int Hq, int n_groups, int total, int max_tok) {
  const int two = 2 * (128 / (Hq / c.Hkv));
  const long long rows = (2LL * (total / two) + n_groups + std::min(c.B, total)) * c.Hkv;
  const long long places = rows * (row_cost(3) + (std::min(max_tok, c.cap) + 127LL) / 128 * kMostTileCost);
  return (int)std::max<long long>(
      1, std::min<long long>(places / kMinPlaces, std::min(sm_count(), kMaxCtas)));
}

// Where the line and its records lie in the workspace, and how much that takes.
SharedParts layout(const Kv16& c, int Hq, const Kv16Groups& groups, int total, int max_tok,
                   uint8_t* ws, size_t* bytes) {
  SharedParts s;
  s.groups = groups;
  s.g = Hq / c.Hkv;
  s.tokens = 128 / s.g;
  s.ctas = line_ctas(c, Hq, groups.n, total, max_tok);
  // (the caller's workspace is 16-byte aligned)
  uintptr_t at = up32(reinterpret_cast<uintptr_t>(ws));
  auto take = [&](size_t n) {
    void* p = reinterpret_cast<void*>(at);
    at += up32(n);
    return p;
  };
  const size_t rec = kPartFloats * sizeof(float), rows = (size_t)total * Hq;
  s.prefix = static_cast<float*>(take(2 * rows * rec));
  s.own = static_cast<float*>(take(2 * rows * rec));
  s.cut = static_cast<float*>(take((size_t)s.ctas * 512 * rec));
  s.first = static_cast<int*>(take((size_t)(groups.n + c.B + 1) * sizeof(int)));
  s.seq = static_cast<int2*>(take((size_t)c.B * sizeof(int2)));
  s.prefix_runs = static_cast<int*>(take((size_t)total * c.Hkv * sizeof(int)));
  s.own_runs = static_cast<int*>(take((size_t)total * c.Hkv * sizeof(int)));
  s.group = static_cast<int4*>(take((size_t)groups.n * sizeof(int4)));
  *bytes = at - reinterpret_cast<uintptr_t>(ws) + 16;
  return s;
}

template <class T>
cudaError_t launch(const AttnParams& p, int* launches, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!kv16_query_map(&mq, p.q, p.c.half, p.g, p.tokens) || !kv16_row_map(&mk, p.c, p.c.k) ||
      !kv16_row_map(&mv, p.c, p.c.v))
    return cudaErrorNotSupported;
  const auto kernel = kv16_attention_kernel<T, kLine>;
  constexpr int kStages = stages_of(kLine);
  constexpr int fixed = (2 + kStages) * kTileBytes + (int)sizeof(Smem<kLine>);
  constexpr int most = fixed + (kMaxGroups + kMaxDecodeBatch + 1 + kThreads / 32) * (int)sizeof(int);
  static_assert(most <= 227 * 1024, "shared memory of a CTA");
  const int smem = fixed + (p.line.groups.n + p.c.B + 1 + kThreads / 32) * (int)sizeof(int);
  cudaError_t e = allow_shared(kernel, most);
  if (e != cudaSuccess) return e;
  kernel<<<p.line.ctas, kThreads, smem, s>>>(mq, mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a warp or more for a row; where that is far more than a wave and the rows have few
  // records (several queries a sequence), queries of a warp
  const long long rows = (long long)p.q.total * p.q.Hq, sms = sm_count();
  const long long wave = kJoinWarps * kJoinCtas * sms, warps = kJoinWarps * kBatchCtas * sms;
  const bool many = p.q.start && rows > 2 * wave;
  const int batch = many ? (int)std::min<long long>((rows + warps * p.g - 1) / (warps * p.g), 32) : 1;
  int subs = 1;
  while (subs < kJoinWarps && rows * subs * 2 <= wave) subs *= 2;
  const int at_once = kJoinWarps / subs, queries = batch * kJoinWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)(many ? (long long)((p.q.total + queries - 1) / queries) * p.c.Hkv
                                : (long long)p.q.total * p.c.Hkv * ((p.g + at_once - 1) / at_once));
  cfg.blockDim = kJoinWarps * 32;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  *launches = 2;
  return many ? cudaLaunchKernelEx(&cfg, kv16_shared_join_kernel<T, true>, p, 1, batch)
              : cudaLaunchKernelEx(&cfg, kv16_shared_join_kernel<T, false>, p, subs, 1);
}

// Is a CTA for each (sequence, KV head) the quicker way?  A wave of them takes 3.4 us
// and 7.2 for each 1000 tokens of the longest, the line about 15 and 3 for each 100
// rows, the groups' among them.  Measured, that way and by the line (rows + rows of
// groups, tokens; us): 16 + 8 of 533 8.7 and 15.8, 128 + 8 of 1021 11.8 and 18.5, 128 +
// 8 of 2001 19.1 and 19.2, 512 + 8 of 511 24.9 and 25.7, 1024 + 8 of 511 43 and 42, 1024
// + 8 of 131 27 and 37, 1024 + 512 of 321 40 and 63, 1024 + 256 of 1089 73 and 66, 2048
// + 2048 of 309 82 and 159, 4096 + 256 of 577 197 and 159, 8192 + 1024 of 577 392 and
// 374, 16384 + 8192 of 321 601 and 911.
bool short_rows(const Kv16& c, const Kv16Query& q, const Kv16Groups& g) {
  const long long rows = (long long)c.B * c.Hkv, sms = sm_count();
  return !q.start && (rows + sms - 1) / sms * (q.max_tok + 470LL) * 72 <=
                         150000 + 300 * (rows + (long long)g.n * c.Hkv);
}

}  // namespace

size_t kv16_shared_ws_bytes(const Kv16& c, int Hq, int n_groups, int total, int max_tok) {
  size_t n;
  layout(c, Hq, Kv16Groups{nullptr, nullptr, n_groups}, total, max_tok, nullptr, &n);
  return n;
}

cudaError_t launch_kv16_shared(const Kv16& c, const Kv16Query& q, const Kv16Groups& g,
                               uint16_t* out, float* lse, void* ws, unsigned copied, int* launches,
                               cudaStream_t s) {
  size_t n;
  AttnParams p;
  p.c = c;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.part = nullptr;
  p.line = layout(c, q.Hq, g, q.total, q.max_tok, static_cast<uint8_t*>(ws), &n);
  p.line.copied = copied;
  p.g = p.line.g;
  p.tokens = p.line.tokens;
  p.tiles = 0;
  p.splits = 1;
  p.negate = q.scale_log2 < 0.0f;
  p.scale = std::max(std::fabs(q.scale_log2), std::numeric_limits<float>::denorm_min());
  p.wide = false;
  *launches = 0;
  if (short_rows(c, q, g)) {
    *launches = 1;
    return launch_kv16_shared_short(c, q, g, out, copied == kAllItems ? kTcWaitLimit : 0u, s);
  }
  return c.half ? launch<Fp16>(p, launches, s) : launch<Bf16>(p, launches, s);
}

}  // namespace oscar
