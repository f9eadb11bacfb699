// Groups of sequences that share a prefix, as the kernels see them.
#pragma once

#include "kv16.cuh"
#include "kv16_line.h"

namespace oscar {

// What group i shares: the whole blocks [0, blocks) of its first sequence,
// `lead`, for the sequences [lead, end).  A group out of range shares nothing, and a
// group of one has it all as its own (8 prompts of up to 2K tokens behind as
// many, alone in their groups: 423 us, 588 by two rows).
struct Shared {
  int lead, end, blocks;
};
__device__ __forceinline__ Shared shared_of(const Kv16& c, const Kv16Groups& g, int i, int max_tok,
                                            bool report) {
  Shared s{__ldg(g.group + i), __ldg(g.group + i + 1), 0};
  const int n = __ldg(g.prefix + i);
  const bool ok = s.lead >= 0 && s.lead <= s.end && s.end <= c.B && n >= 0 && n <= c.cap &&
                  n <= max_tok;
  if (!ok) {
    if (report) record_error(c.status, kDevErrBadPaged);
    s.end = s.lead;
  } else if (s.end - s.lead > 1) {
    s.blocks = n / kPage;
  }
  return s;
}

// The group of sequence b, or -1.
__device__ __forceinline__ int group_of(const Kv16Groups& g, int b) {
  return ragged_sequence(g.group, g.n, b);
}

// A record of a run: m, l, 6 floats' room, o[128]; every piece that a thread
// writes is a whole 32-byte sector (with 16-byte pieces, of the split records'
// layout, an item of 256 rows took 8 us to write instead of 1).
constexpr int kPartHead = 8, kPartFloats = kPartHead + 128;

// The line and its records in the workspace (32-byte aligned).  A run that has a
// row's first tile leaves its records at the query rows' places, else with the
// CTA: [2][256], 0 for a run that begins inside a block, 1 for one that begins a
// block.  A chunk that fills one query tile only (rows <= 128 / g * g) is worked by
// both, with every other tile of keys each: two records a run, the second in the
// second half.
struct SharedParts {
  Kv16Groups groups;
  float* prefix;            // [2][total][Hq]
  float* own;               // [2][total][Hq]
  float* cut;               // [ctas][2][256]
  int* first;               // [groups + B + 1]: the entries' first places, the line's end
  int4* group;              // [groups]: tiles of a row, first query row, the row behind the last
  int2* seq;                // [B]: a sequence's group or -1, the blocks that are its group's
  // by a chunk's first query row and the KV head: the CTAs that have its tiles (of
  // rows that have any and, prefixes, one block): first | count << 16
  int* prefix_runs;         // [total][Hkv]
  int* own_runs;
  int ctas;
  int tokens, g;            // tokens of a query tile, heads of a group
  unsigned copied;          // items of a CTA that are copied: all but in a self-test
};

// ragged_sequence by a warp: 32 numbers of `start` at a time, not one.
__device__ __forceinline__ int warp_sequence(const int32_t* start, int B, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, at = lo + (lane + 1) * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && __ldg(start + min(at, B)) <= r);
    lo += __popc(le) * step;
    hi = min(hi, lo + step);
  }
  return __ldg(start + lo) <= r && r < __ldg(start + lo + 1) ? lo : -1;
}

// What the values that a row sees hold in a channel.
constexpr unsigned kSeenNan = 1, kSeenPlus = 2, kSeenMinus = 4;
__device__ __forceinline__ unsigned seen_in(float x) {
  return x != x ? kSeenNan : x == INFINITY ? kSeenPlus : x == -INFINITY ? kSeenMinus : 0u;
}

// The channels of a row (4 lane .. 4 lane + 3, relative to its sum) that are NaN
// although the sum is a number: infinite where the visible values hold infinities
// of one sign and no NaN.  A record may hold an infinity that its factor of 0 has
// turned into NaN.  A warp; rare, and as slow as one warp's pass over the values.
template <class T>
__device__ __noinline__ float4 settle(const Kv16& c, const Kv16Query& q, const Kv16Groups& groups,
                                      int b, int h, int back, float4 x) {
  const int lane = threadIdx.x & 31;
  const int len = kv16_length(c, b, q.max_tok), at = len < 0 ? -1 : max(len - back, -1);
  const int i = group_of(groups, b);
  Shared sh{b, b, 0};
  if (i >= 0) sh = shared_of(c, groups, i, q.max_tok, false);
  const Span sp(at, at, q.window, q.n_sink);
  float o[4] = {x.x, x.y, x.z, x.w};
  unsigned f[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int k = 0; k < sp.blocks; ++k) {
    bool undecided = false;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      undecided |= o[u] != o[u] && !(f[u] & kSeenNan) &&
                   (f[u] & (kSeenPlus | kSeenMinus)) != (kSeenPlus | kSeenMinus);
    if (!__any_sync(0xffffffffu, undecided)) break;
    const int blk = sp.block(k);
    const int row = kv16_block_row(c, blk < sh.blocks ? sh.lead : b, h, blk);
    if (row < 0) continue;
    const unsigned see =
        __ballot_sync(0xffffffffu, kv16_visible(blk * kPage + lane, at, q.window, q.n_sink));
#pragma unroll 8
    for (int t = 0; t < kPage; ++t) {
      uint2 v = make_uint2(0u, 0u);
      if ((see >> t) & 1u)
        v = reinterpret_cast<const uint2*>(c.v)[((long long)row + t) * 32 + lane];
      const float2 a = T::unpack(v.x), z = T::unpack(v.y);
      f[0] |= seen_in(a.x);
      f[1] |= seen_in(a.y);
      f[2] |= seen_in(z.x);
      f[3] |= seen_in(z.y);
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (o[u] != o[u] && (f[u] == kSeenPlus || f[u] == kSeenMinus))
      o[u] = f[u] == kSeenPlus ? INFINITY : -INFINITY;
  return make_float4(o[0], o[1], o[2], o[3]);
}

}  // namespace oscar
