// Attention of one query per sequence over the 16-bit cache: a stream over the
// visible keys and values, 512 B per (token, KV head), bound by HBM.
//
// Work split.  The visible pages of all (sequence, KV head) rows stand in one
// line, row after row; every CTA takes an equal run of it, so unequal lengths
// leave no CTA idle and the grid is one wave, whatever the batch.  Where a run
// ends inside a row the CTA leaves a partial record (m, l, o[128] per head);
// the row's last CTA to arrive joins the records in order of CTA, so the bits
// do not depend on the order of arrival.  A row that one CTA holds whole is
// written at once.  A CTA has at most two partial rows: the one it enters in
// the middle (slot 0) and the one it leaves in the middle (slot 1).
//
// Inside a CTA each of 10 warps takes every tenth page of the run, through a
// shared-memory slot of its own: 4 tensor copies (TMA, 128-byte swizzle) per
// page, keys and values in halves of 64 channels, completing on the slot's
// barrier.  While one warp computes, the other nine's pages are on their way
// (160 KB per SM), so a deeper ring per warp gains nothing and more warps do:
// with 4 warps of three slots each a page's chain of mma and softmax (about a
// microsecond) bounded the stream (batch 16 x 64K, 8 heads a group: 349 us; 8
// warps 320, 10 warps 314).  One page (32 tokens) per step is also what the
// block table gives.
//
// Mathematics.  S = Q K^T by mma.sync m16n8k16 with the group's query heads as
// the 16 rows (up to 16 heads in one pass over the keys, the rest padding):
// the tensor work of a page, 96 instructions, is under the time that its 16 KB
// take to arrive, so padding rows cost nothing.  The accumulator layout of S is
// the operand layout of P in O += P V, so probabilities stay in registers.  One
// pass with the running maximum and sum in fp32 (log2 domain); probabilities
// enter the product with V as the sum of two numbers of the cache's type (hi +
// lo, 16 bits of mantissa and more), so the output is rounded once, at the end.
// fp16's smallest number is 2^-24, so there the largest probability stands at
// 2^14, not at 1: the two parts keep 16 bits down to 2^-30 of the largest and
// something of a probability down to 2^-39 (a sink may outweigh every other
// token by more than 2^24, and with a value near 0 leave them the output).
//
// A probability whose second part is 0 or negative turns a visible infinity in V
// into NaN.  A row with a channel that is NaN although its sum is a number is
// therefore looked at again once it is joined: what its visible values hold in
// that channel decides (settle_row).
//
// The accumulated weights need the joined maximum and sum.  So the scores go to
// the workspace (4 bytes per token and query head beside 512 per token and KV
// head) and a second launch turns them into probabilities.
//
// Measured (GB300, copies run at 6.79 TB/s): batch 16 x 64K, 32/4 heads, even
// lengths 314 us, 6.84 TB/s; lengths of 14K to 64K 198 us (floor 191), with
// weights 217 + 21 us; batch 48 x 16K with a window of 4096, 32/8 heads, 130 us
// (floor 118: 129 pages a row leave three rows and their joins to a CTA); one
// head and 1024 tokens 8.4 us, a chain of dependent loads: length, table, page,
// records.
#include <algorithm>

#include "kv16.cuh"
#include "kv16_tma.h"
#include "tc5.cuh"

namespace oscar {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

namespace {

constexpr int NW = 10;                   // warps of a CTA, each with a slot of its own
constexpr int kSlotBytes = 4 * 4096;     // a page: K and V, two halves of 64 channels each
constexpr int kMinPages = NW;            // pages of a CTA's run, if the batch has as many: one a warp
constexpr float kBelow = 14.0f;          // fp16: the maximum in use is 2^14 below the largest
constexpr int kORow = 136;               // floats of a head's output row in shared memory

struct DecodeParams {
  Kv16 c;
  Kv16Query q;
  uint16_t* out;
  unsigned* counters;   // [B * Hkv], zero between calls
  float* part;          // [grid][2][g][kRecFloats]
  float2* stats;        // [B][Hq] (m, 1 / l), accumulate only
  float* scores;        // [pages][g][32] log2-domain scores, accumulate only
  int g;
  unsigned wait_limit;  // polls of a wait for a copy
  bool halves;          // the warps' outputs are joined in two steps
};

// First pages of the sequences in the line of pages (of one KV head): first[0]
// .. first[B].  Called by all threads; ends with a barrier.  Returns first[B].
__device__ int line_up(const Kv16& c, const Kv16Query& q, int* first, int* scan, int threads,
                       bool report) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = threads >> 5;
  int carry = 0;
  for (int b0 = 0; b0 < c.B; b0 += threads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < c.B) {
      n = kv16_length(c, b, q.max_tok);
      if (n < 0) {
        if (report) record_error(c.status, kDevErrBadPaged);
        n = 0;
      }
    }
    int x = Span(n - 1, n - 1, q.window, q.n_sink).blocks;
    const int mine = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int before = carry, total = carry;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    if (b < c.B) first[b] = before + x - mine;
    carry = total;
    __syncthreads();
  }
  if (tid == 0) first[c.B] = carry;
  __syncthreads();
  return carry;
}

// A row of the line: its sequence, head, pages [r0, r1) and span.
struct Row {
  int b, h, r0, r1, at;
  Span sp;
};

__device__ __forceinline__ void find_row(Row& r, int x, const DecodeParams& p, const int* first) {
  const int key = x / p.c.Hkv;     // first[b] <= key < first[b + 1]
  int lo = 0, hi = p.c.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= key) lo = mid; else hi = mid;
  }
  const int pages = first[lo + 1] - first[lo];
  r.b = lo;
  r.h = (x - first[lo] * p.c.Hkv) / pages;
  r.r0 = first[lo] * p.c.Hkv + r.h * pages;
  r.r1 = r.r0 + pages;
  r.at = __ldg(p.c.n_tok + lo) - 1;
  r.sp = Span(r.at, r.at, p.q.window, p.q.n_sink);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <class T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (T::kHalf)
    mma_16816_acc(d, a, b0, b1);
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The row's joined result (M, L, o of channel pair `pair`) to the output.
template <class T>
__device__ __forceinline__ void write_out(const DecodeParams& p, const Row& r, int head, int pair,
                                          float M, float L, float o0, float o1, bool stats) {
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const long long row = (long long)r.b * p.q.Hq + r.h * p.g + head;
  reinterpret_cast<uint32_t*>(p.out + row * kD)[pair] = T::pack(o0 * inv, o1 * inv);
  if (stats && pair == 0) p.stats[row] = make_float2(M, inv);
}

// What the values that a row sees hold in a channel.
constexpr unsigned kSeenNan = 1, kSeenPlus = 2, kSeenMinus = 4, kOpen = 8;
__device__ __forceinline__ unsigned seen_in(float x) {
  return x != x ? kSeenNan : x == INFINITY ? kSeenPlus : x == -INFINITY ? kSeenMinus : 0u;
}

// The open channels (ch[c] & kOpen) of row r's written result, NaN so far, for
// the heads whose sum is a number: infinite where the visible values hold
// infinities of one sign and no NaN.  All threads; leaves ch at zero.  A CTA reads
// the values alone, 16 tokens of every warp in flight, and stops early once every
// open channel has met a NaN or both infinities.
template <class T>
__device__ __noinline__ void settle_row(const DecodeParams& p, Row r, unsigned* ch,
                                        const uint8_t* sum_nan) {
  constexpr int kTokens = 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile unsigned* mine = ch + 4 * lane;
  for (int x = r.r0 + warp; x < r.r1; x += NW) {
    bool undecided = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned c = mine[i];
      undecided |= (c & kOpen) && !(c & kSeenNan) && (c & (kSeenPlus | kSeenMinus)) != (kSeenPlus | kSeenMinus);
    }
    if (!__any_sync(0xffffffffu, undecided)) break;
    const int blk = r.sp.block(x - r.r0), row = kv16_block_row(p.c, r.b, r.h, blk);
    if (row < 0) continue;
    const unsigned see = __ballot_sync(
        0xffffffffu, kv16_visible(blk * kPage + lane, r.at, p.q.window, p.q.n_sink));
    unsigned f[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int t0 = 0; t0 < kPage; t0 += kTokens) {
      uint2 v[kTokens];
#pragma unroll
      for (int u = 0; u < kTokens; ++u) {
        v[u] = make_uint2(0u, 0u);
        if ((see >> (t0 + u)) & 1u)
          v[u] = reinterpret_cast<const uint2*>(p.c.v)[((long long)row + t0 + u) * 32 + lane];
      }
#pragma unroll
      for (int u = 0; u < kTokens; ++u) {
        const float2 a = T::unpack(v[u].x), b = T::unpack(v[u].y);
        f[0] |= seen_in(a.x);
        f[1] |= seen_in(a.y);
        f[2] |= seen_in(b.x);
        f[3] |= seen_in(b.y);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (f[i]) atomicOr(ch + 4 * lane + i, f[i]);
  }
  __syncthreads();
  for (int i = tid; i < p.g * 64; i += NW * 32) {
    const int head = i >> 6, pair = i & 63;
    if (sum_nan[head]) continue;
    uint32_t* o = reinterpret_cast<uint32_t*>(
                      p.out + ((long long)r.b * p.q.Hq + r.h * p.g + head) * kD) + pair;
    float2 v = T::unpack(*o);
    auto settled = [&](float y, unsigned c) {
      c &= kOpen | kSeenNan | kSeenPlus | kSeenMinus;
      return y == y ? y : c == (kOpen | kSeenPlus) ? INFINITY : c == (kOpen | kSeenMinus) ? -INFINITY : y;
    };
    v.x = settled(v.x, ch[2 * pair]);
    v.y = settled(v.y, ch[2 * pair + 1]);
    *o = T::pack(v.x, v.y);
  }
  __syncthreads();
  for (int i = tid; i < kD; i += NW * 32) ch[i] = 0u;
  __syncthreads();
}

template <class T, bool ACC>
__global__ void __launch_bounds__(NW * 32, 1)
kv16_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[NW];
  __shared__ int scan[NW];
  __shared__ float sm_m[NW][kMaxGroup], sm_l[NW][kMaxGroup];
  __shared__ int s_last, s_open;
  __shared__ unsigned s_ch[kD];            // of settle_row
  __shared__ uint8_t s_nan[kMaxGroup];     // heads whose sum is NaN
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;   // swizzle atoms
  uint8_t* slot = smem + warp * kSlotBytes;
  const int parts = p.halves ? NW / 2 : NW;
  float* obuf = reinterpret_cast<float*>(smem + NW * kSlotBytes);   // [parts][g][kORow]
  int* first = reinterpret_cast<int*>(obuf + parts * p.g * kORow);

  if (tid == 0) {
    for (int w = 0; w < NW; ++w) mbar_init(&full[w], 1);
    mbar_fence_init();
    s_open = 0;
  }
  for (int i = tid; i < kD; i += NW * 32) s_ch[i] = 0u;
  const int line = line_up(p.c, p.q, first, scan, NW * 32, blockIdx.x == 0);
  // rows without visible tokens: zeros
  for (int b = blockIdx.x; b < p.c.B; b += gridDim.x)
    if (first[b] == first[b + 1]) {
      uint4* o = reinterpret_cast<uint4*>(p.out + (long long)b * p.q.Hq * kD);
      for (int i = tid; i < p.q.Hq * (kD / 8); i += NW * 32) o[i] = make_uint4(0, 0, 0, 0);
    }

  const int P = line * p.c.Hkv;                     // pages in the line
  if (P == 0) return;
  const int per = max(kMinPages, (P - 1) / (int)gridDim.x + 1);
  const long long x0l = (long long)blockIdx.x * per;
  if (x0l >= P) return;
  const int x0 = (int)x0l, x1 = (int)min((long long)P, x0l + per);

  // the warp's next page to fetch, and the row it is in
  Row nr;
  nr.r0 = nr.r1 = 0;
  auto fetch = [&](int x) {
    if (x >= x1) return;
    if (x < nr.r0 || x >= nr.r1) find_row(nr, x, p, first);
    int row = kv16_block_row(p.c, nr.b, nr.h, nr.sp.block(x - nr.r0));
    if (row < 0) {
      // past the end of the pool: the copy reads zeros
      row = p.c.n_pages * p.c.Hkv * kPage;
      if (lane == 0) record_error(p.c.status, kDevErrBadPaged);
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[warp], kSlotBytes);
      tma_box2(slot, &map_k, 0, row, &full[warp]);
      tma_box2(slot + 4096, &map_k, 64, row, &full[warp]);
      tma_box2(slot + 8192, &map_v, 0, row, &full[warp]);
      tma_box2(slot + 12288, &map_v, 64, row, &full[warp]);
    }
  };
  int x = x0 + warp;                // the warp's next page to work on
  fetch(x);
  unsigned phase = 0;
  // A warp whose copies do not land in time works no further pages, but joins in
  // all that follows: the rows' counters have to come back to zero.
  bool gave_up = false;

  const int hr = lane >> 2, hc = 2 * (lane & 3);    // accumulator row, column
  int seg = x0;
  Row r;
  while (seg < x1) {
    find_row(r, seg, p, first);
    const int seg_end = min(r.r1, x1);
    // the group's queries as A operands: rows are heads, padding rows zero
    uint32_t qa[8][4];
    {
      const uint16_t* q0 = p.q.q + r.b * p.q.stride + (long long)r.h * p.g * kD;
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int head = hr + 8 * (i & 1), ch = 16 * k + hc + 8 * (i >> 1);
          qa[k][i] = head < p.g ? __ldg(reinterpret_cast<const uint32_t*>(q0 + head * kD + ch)) : 0u;
        }
    }
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

    for (; x < seg_end && !gave_up; x += NW) {
      // (one answer for the warp: its lanes may see the barrier differently)
      gave_up = !__all_sync(0xffffffffu, mbar_wait_bounded(&full[warp], phase, p.wait_limit));
      if (gave_up) {
        if (lane == 0) record_error(p.c.status, kDevErrWaitTimeout);
        break;
      }
      const int j0 = r.sp.block(x - r.r0) * kPage;
      const bool whole = j0 + kPage - 1 <= r.at &&
                         (p.q.window == 0 || j0 > r.at - p.q.window || j0 + kPage <= p.q.n_sink);
      if (!whole) {
        // a hidden token's value must not meet its zero probability: clear it
        const int j = j0 + lane;
        if (!kv16_visible(j, r.at, p.q.window, p.q.n_sink)) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            reinterpret_cast<uint4*>(slot + 8192 + (i >> 3) * 4096 + lane * 128)[i & 7] =
                make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      // S: 16 heads x 32 tokens
      float sc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.0f;
      const unsigned sa = smem_u32(slot);
      const int mrow = lane & 7, mid = lane >> 3;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // 8x8 tiles: channels 16k, 16k + 8 of tokens t, t + 8
        const int chunk = 2 * (k & 3) + (mid & 1);
        const unsigned a = sa + (k >> 2) * 4096 + ((mid >> 1) * 8 + mrow) * 128 + ((chunk ^ mrow) << 4);
        uint32_t b0[4], b1[4];
        ldsm4(b0, a);
        ldsm4(b1, a + 16 * 128);
        mma<T>(sc[0], qa[k], b0[0], b0[1]);
        mma<T>(sc[1], qa[k], b0[2], b0[3]);
        mma<T>(sc[2], qa[k], b1[0], b1[1]);
        mma<T>(sc[3], qa[k], b1[2], b1[3]);
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = sc[i][e] * p.q.scale_log2;
          if (!whole && !kv16_visible(j0 + 8 * i + hc + (e & 1), r.at, p.q.window, p.q.n_sink))
            v = -INFINITY;
          sc[i][e] = v;
          mx[e >> 1] = fmaxf(mx[e >> 1], v);
        }
      if constexpr (ACC) {
        float* d = p.scores + ((size_t)x * p.g + hr) * kPage + hc;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (hr < p.g) *reinterpret_cast<float2*>(d + 8 * i) = make_float2(sc[i][0], sc[i][1]);
          if (hr + 8 < p.g)
            *reinterpret_cast<float2*>(d + 8 * kPage + 8 * i) = make_float2(sc[i][2], sc[i][3]);
        }
      }
      bool grew = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        if (T::kHalf) mx[i] -= kBelow;
        grew |= mx[i] > m[i];
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mn = fmaxf(m[i], mx[i]);
          const float a = mn == -INFINITY ? 1.0f : fast_exp2(m[i] - mn);
          m[i] = mn;
          l[i] *= a;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            o[n][2 * i] *= a;
            o[n][2 * i + 1] *= a;
          }
        }
      }
      const float ms[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
      uint32_t pa[2][4], pb[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = fast_exp2(sc[i][0] - ms[0]), p1 = fast_exp2(sc[i][1] - ms[0]);
        const float p2 = fast_exp2(sc[i][2] - ms[1]), p3 = fast_exp2(sc[i][3] - ms[1]);
        l[0] += p0 + p1;
        l[1] += p2 + p3;
        const uint32_t h0 = T::pack(p0, p1), h1 = T::pack(p2, p3);
        const float2 u0 = T::unpack(h0), u1 = T::unpack(h1);
        pa[i >> 1][2 * (i & 1)] = h0;
        pa[i >> 1][2 * (i & 1) + 1] = h1;
        pb[i >> 1][2 * (i & 1)] = T::pack(p0 - u0.x, p1 - u0.y);
        pb[i >> 1][2 * (i & 1) + 1] = T::pack(p2 - u1.x, p3 - u1.y);
      }
      // O += P V: 8x8 tiles, transposed on the way: tokens t, t + 8 of channels c, c + 8
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int chunk = 2 * (n & 3) + (mid >> 1);
        const unsigned a = sa + 8192 + (n >> 2) * 4096 + ((mid & 1) * 8 + mrow) * 128 +
                           ((chunk ^ mrow) << 4);
        uint32_t b0[4], b1[4];
        ldsm4t(b0, a);
        ldsm4t(b1, a + 16 * 128);
        mma<T>(o[2 * n], pa[0], b0[0], b0[1]);
        mma<T>(o[2 * n + 1], pa[0], b0[2], b0[3]);
        mma<T>(o[2 * n], pa[1], b1[0], b1[1]);
        mma<T>(o[2 * n + 1], pa[1], b1[2], b1[3]);
        mma<T>(o[2 * n], pb[0], b0[0], b0[1]);
        mma<T>(o[2 * n + 1], pb[0], b0[2], b0[3]);
        mma<T>(o[2 * n], pb[1], b1[0], b1[1]);
        mma<T>(o[2 * n + 1], pb[1], b1[2], b1[3]);
      }
      // refill the slot once every lane has read it; cleared values first
      // become visible to the copy engine
      if (!whole) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      fetch(x + NW);
      phase ^= 1;
    }

    // join the warps: in one step, or the upper half's results into the lower
    // half's first where the buffer holds half of them
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    auto leave = [&](int part) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int head = hr + 8 * i;
        if (head >= p.g) continue;
        if ((lane & 3) == 0) {
          sm_m[part][head] = m[i];
          sm_l[part][head] = l[i];
        }
        float* d = obuf + (part * p.g + head) * kORow + hc;
#pragma unroll
        for (int n = 0; n < 16; ++n)
          *reinterpret_cast<float2*>(d + 8 * n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
      }
    };
    if (p.halves) {
      if (warp >= NW / 2) leave(warp - NW / 2);
      __syncthreads();
      if (warp < NW / 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int head = hr + 8 * i;
          if (head >= p.g) continue;
          const float m2 = sm_m[warp][head], M = fmaxf(m[i], m2);
          const float a = M == -INFINITY ? 1.0f : fast_exp2(m[i] - M);
          const float a2 = M == -INFINITY ? 1.0f : fast_exp2(m2 - M);
          const float* d = obuf + (warp * p.g + head) * kORow + hc;
          m[i] = M;
          l[i] = a * l[i] + a2 * sm_l[warp][head];
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const float2 v = *reinterpret_cast<const float2*>(d + 8 * n);
            o[n][2 * i] = a * o[n][2 * i] + a2 * v.x;
            o[n][2 * i + 1] = a * o[n][2 * i + 1] + a2 * v.y;
          }
        }
        __syncwarp();    // a warp's own part: read by all lanes, then written
        leave(warp);
      }
    } else {
      leave(warp);
    }
    __syncthreads();
    const bool own_row = seg == r.r0 && seg_end == r.r1;
    const int c0 = r.r0 / per, c1 = (r.r1 - 1) / per;
    // the row's result, and which of its channels are open
    auto result = [&](int head, int pair, float M, float L, float a0, float a1) {
      write_out<T>(p, r, head, pair, M, L, a0, a1, ACC);
      if (pair == 0) s_nan[head] = L != L;
      if (L == L && (a0 != a0 || a1 != a1)) {
        if (a0 != a0) s_ch[2 * pair] = kOpen;
        if (a1 != a1) s_ch[2 * pair + 1] = kOpen;
        s_open = 1;
      }
    };
    float* rec0 = p.part + ((long long)blockIdx.x * 2 + ((int)blockIdx.x == c0 ? 1 : 0)) * p.g * kRecFloats;
    for (int i = tid; i < p.g * 64; i += NW * 32) {
      const int head = i >> 6, pair = i & 63;
      float M = -INFINITY, L = 0.0f, a0 = 0.0f, a1 = 0.0f;
      for (int w = 0; w < parts; ++w) M = fmaxf(M, sm_m[w][head]);
#pragma unroll 5
      for (int w = 0; w < parts; ++w) {
        const float mw = sm_m[w][head];
        const float a = mw == -INFINITY && M == -INFINITY ? 1.0f : fast_exp2(mw - M);
        const float2 v = *reinterpret_cast<const float2*>(obuf + (w * p.g + head) * kORow + 2 * pair);
        L += a * sm_l[w][head];
        a0 += a * v.x;
        a1 += a * v.y;
      }
      if (own_row) {
        result(head, pair, M, L, a0, a1);
      } else {
        float* rec = rec0 + head * kRecFloats;
        if (pair == 0) *reinterpret_cast<float2*>(rec) = make_float2(M, L);
        *reinterpret_cast<float2*>(rec + 4 + 2 * pair) = make_float2(a0, a1);
      }
    }
    __syncthreads();
    if (!own_row) {
      // the row's CTAs are c0 .. c1; the last to arrive joins their records
      if (tid == 0) {
        unsigned prev;
        unsigned* ctr = p.counters + (long long)r.b * p.c.Hkv + r.h;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                     : "=r"(prev) : "l"(ctr) : "memory");
        s_last = prev == (unsigned)(c1 - c0);
        if (s_last) *ctr = 0u;
        if (prev > (unsigned)(c1 - c0)) record_error(p.c.status, kDevErrArrival);
      }
      __syncthreads();
      if (s_last) {
        for (int i = tid; i < p.g * 64; i += NW * 32) {
          const int head = i >> 6, pair = i & 63;
          auto rec = [&](int c) {
            return p.part + (((long long)c * 2 + (c == c0 ? 1 : 0)) * p.g + head) * kRecFloats;
          };
          float M = -INFINITY, L = 0.0f, a0 = 0.0f, a1 = 0.0f;
          for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(rec(c)));
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            const float* d = rec(c);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(d));
            const float2 v = __ldcg(reinterpret_cast<const float2*>(d + 4 + 2 * pair));
            const float a = ml.x == -INFINITY && M == -INFINITY ? 1.0f : fast_exp2(ml.x - M);
            L += a * ml.y;
            a0 += a * v.x;
            a1 += a * v.y;
          }
          result(head, pair, M, L, a0, a1);
        }
        __syncthreads();
      }
    }
    if (s_open) {
      settle_row<T>(p, r, s_ch, s_nan);
      if (tid == 0) s_open = 0;
      __syncthreads();
    }
    seg = seg_end;
  }
  // the copy in flight lands before its memory is given back
  if (gave_up && !mbar_wait_bounded(&full[warp], phase, kDrainLimit) && lane == 0)
    record_error(p.c.status, kDevErrDrainTimeout);
}

constexpr int kWThreads = 256;


// weight[j] += sum over the group's heads of 2^(s_j - m) / l: a warp takes four
// neighbouring pages at a time, eight lanes a page and four tokens a lane.
// The scores are addressed by the page's place in the line alone, so their
// loads do not wait for the row's to be found.
__global__ void __launch_bounds__(kWThreads) kv16_decode_weights_kernel(const DecodeParams p) {
  extern __shared__ int first[];
  __shared__ int scan[kWThreads / 32];
  const int P = line_up(p.c, p.q, first, scan, kWThreads, false) * p.c.Hkv;
  const int lane = threadIdx.x & 31, t0 = 4 * (lane & 7);
  const long long step = (long long)gridDim.x * (kWThreads / 32) * 4;
  long long x = ((long long)blockIdx.x * (kWThreads / 32) + (threadIdx.x >> 5)) * 4 + (lane >> 3);
  Row r;
  r.r0 = r.r1 = 0;
  for (; x < P; x += step) {
    const float* sp = p.scores + (size_t)x * p.g * kPage + t0;
    float4 s[8];
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < p.g) s[h] = __ldcs(reinterpret_cast<const float4*>(sp + h * kPage));
    if (x < r.r0 || x >= r.r1) find_row(r, (int)x, p, first);
    const int j0 = r.sp.block((int)x - r.r0);
    const int row = kv16_block_row(p.c, r.b, r.h, j0);
    if (row < 0) continue;
    const float2* st = p.stats + (long long)r.b * p.q.Hq + r.h * p.g;
    float* wp = p.c.weight + (long long)row + t0;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int h0 = 0; h0 < p.g; h0 += 8) {
      if (h0 > 0) {
#pragma unroll
        for (int h = 0; h < 8; ++h)
          if (h0 + h < p.g) s[h] = __ldcs(reinterpret_cast<const float4*>(sp + (h0 + h) * kPage));
      }
#pragma unroll
      for (int h = 0; h < 8; ++h)
        if (h0 + h < p.g) {
          const float2 ml = st[h0 + h];
          const float v[4] = {s[h].x, s[h].y, s[h].z, s[h].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (v[i] != -INFINITY) sum[i] += fast_exp2(v[i] - ml.x) * ml.y;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (kv16_visible(j0 * kPage + t0 + i, r.at, p.q.window, p.q.n_sink)) wp[i] += sum[i];
  }
}

// Pages that a sequence of at most max_tok tokens can show to its last query.
long long most_pages(int max_tok, int cap, int window, int n_sink) {
  const long long all = (std::min(max_tok, cap) + kPage - 1) / kPage;
  if (window == 0) return all;
  const long long near = ((long long)window + 2 * kPage - 2) / kPage;
  const long long sinks = ((long long)n_sink + kPage - 1) / kPage;
  return std::min(all, near + sinks);
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 152;
  return sms;
}

long long line_pages(const Kv16& c, int max_tok, int window, int n_sink) {
  return (long long)c.B * c.Hkv * most_pages(max_tok, c.cap, window, n_sink);
}

// One CTA per SM, fewer for batches of fewer than kMinPages pages per CTA.
int decode_grid(long long pages) {
  return (int)std::max<long long>(1, std::min<long long>(sm_count(), (pages + kMinPages - 1) / kMinPages));
}

// Dynamic shared memory that a CTA may have beside the static.
constexpr size_t kSmemMost = 227 * 1024 - 2048;
static_assert(NW * kSlotBytes + NW / 2 * kMaxGroup * kORow * 4 + (kMaxDecodeBatch + 1) * 4 + 1024 <=
                  kSmemMost, "the widest group of the largest batch");

size_t part_bytes(int grid, int g) { return (size_t)grid * 2 * g * kRecFloats * sizeof(float); }
size_t stats_bytes(int B, int Hq) { return ((size_t)B * Hq * sizeof(float2) + 15) / 16 * 16; }

template <class T, bool ACC>
cudaError_t launch_main(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeParams& p,
                        int grid, size_t smem, cudaStream_t s) {
  const auto kernel = kv16_decode_kernel<T, ACC>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, NW * 32, smem, s>>>(mk, mv, p);
  return cudaGetLastError();
}

}  // namespace

size_t kv16_decode_ws_bytes(const Kv16& c, int Hq, int max_tok, int window, int n_sink,
                            bool accumulate) {
  const int g = Hq / c.Hkv;
  const long long pages = line_pages(c, max_tok, window, n_sink);
  size_t n = kDecodeWsHeader + part_bytes(decode_grid(pages), g);
  if (accumulate) n += stats_bytes(c.B, Hq) + (size_t)pages * g * kPage * sizeof(float);
  return n;
}

cudaError_t launch_kv16_decode(const Kv16& c, const Kv16Query& q, bool accumulate, uint16_t* out,
                               void* ws, unsigned wait_limit, int* launches, cudaStream_t s) {
  DecodeParams p;
  p.c = c;
  p.q = q;
  p.out = out;
  p.g = q.Hq / c.Hkv;
  p.wait_limit = wait_limit;
  const long long pages = line_pages(c, q.max_tok, q.window, q.n_sink);
  const int grid = decode_grid(pages);
  p.counters = decode_row_counters(ws);
  p.part = decode_partials(ws);
  p.stats = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(p.part) + part_bytes(grid, p.g));
  p.scores = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.stats) + stats_bytes(c.B, q.Hq));
  const size_t lines = (size_t)(c.B + 1) * 4;
  const size_t heads = (size_t)NW * p.g * kORow * 4;
  p.halves = NW * kSlotBytes + heads + lines + 1024 > kSmemMost;
  const size_t smem = NW * kSlotBytes + (p.halves ? heads / 2 : heads) + lines + 1024;
  CUtensorMap mk, mv;
  if (!kv16_row_map(&mk, c, c.k) || !kv16_row_map(&mv, c, c.v)) return cudaErrorNotSupported;
  cudaError_t e =
      c.half ? (accumulate ? launch_main<Fp16, true>(mk, mv, p, grid, smem, s)
                           : launch_main<Fp16, false>(mk, mv, p, grid, smem, s))
             : (accumulate ? launch_main<Bf16, true>(mk, mv, p, grid, smem, s)
                           : launch_main<Bf16, false>(mk, mv, p, grid, smem, s));
  *launches = 1;
  if (e != cudaSuccess || !accumulate) return e;
  e = cudaFuncSetAttribute(kv16_decode_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)lines);
  if (e != cudaSuccess) return e;
  const int wgrid = (int)std::max<long long>(
      1, std::min<long long>((pages + 31) / 32, 8LL * sm_count()));
  kv16_decode_weights_kernel<<<wgrid, kWThreads, lines, s>>>(p);
  *launches = 2;
  return cudaGetLastError();
}

}  // namespace oscar
