// Groups of sequences that share a prefix, as the kernels see them.
#pragma once

#include "kv16.cuh"

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

// The work of a call stands in one line of key tiles (128 tokens against up to 256
// query rows), and each of `ctas` CTAs takes an equal run of it.  A row of the line
// (the tiles of one chunk of query rows and KV head) begins with kRowCost places
// without a tile, for what it costs to begin and end an item.  Entry i below
// the number of groups is group i's prefix, the others are the sequences' own
// blocks behind it.  An entry has its tiles KV head by KV head:
//  a sequence  chunk of query rows after chunk, each its own tiles (causal: a
//              later chunk has more)
//  a group     block after block of places, and within a block chunk after chunk.
//              A single chunk has one block, the whole row; several have blocks of
//              a run's length or a little more, so that the CTAs that work the
//              same keys for different chunks do so at the same time, and the keys
//              come from HBM once.
constexpr int kRowCost = 3;
constexpr int kMinPlaces = 2;   // of a CTA's run, if the line has as many
__host__ __device__ __forceinline__ int line_share(int places, int ctas) {
  const int per = places / ctas + (places % ctas != 0);
  return per > kMinPlaces ? per : kMinPlaces;
}
// Blocks of a group's row of so many places.
__host__ __device__ __forceinline__ int line_blocks(int places, int chunks, int per) {
  return chunks > 1 && places >= 2 * per ? places / per : 1;
}
// First place of block i of n.
__host__ __device__ __forceinline__ int block_place(int places, int n, int i) {
  return (int)((long long)places * i / n);
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
  int4* group;              // [groups]: places of a row, first query row, the row behind the last
  int ctas;
  int tokens, g;            // tokens of a query tile, heads of a group
};

}  // namespace oscar
