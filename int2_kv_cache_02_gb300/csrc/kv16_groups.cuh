// Groups of sequences that share a prefix, as the kernels see them.
#pragma once

#include "kv16.cuh"
#include "kv16_line.h"

namespace oscar {

// What group i shares: the whole blocks [0, blocks) of its first sequence,
// `lead`, for the sequences [lead, end).  A group out of range shares nothing.
struct Shared {
  int lead, end, blocks;
};
__device__ __forceinline__ Shared shared_of(const Kv16& c, const Kv16Groups& g, int i, int max_tok,
                                            bool report) {
  Shared s{__ldg(g.group + i), __ldg(g.group + i + 1), 0};
  const int n = __ldg(g.prefix + i);
  const bool ok = s.lead >= 0 && s.lead <= s.end && s.end <= c.B && n >= 0 && n <= c.cap &&
                  n <= max_tok;
  if (ok) s.blocks = n / kPage;
  else if (report) record_error(c.status, kDevErrBadPaged);
  if (!ok) s.end = s.lead;
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

}  // namespace oscar
