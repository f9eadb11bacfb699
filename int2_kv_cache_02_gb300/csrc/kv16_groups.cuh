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

// What the prefixes' kernel leaves in the workspace for who joins the records.
// All key tiles of 128 tokens stand in one line, and each of `ctas` CTAs takes an
// equal run of it.  Group by group and, in a group, KV head by KV head, a line
// has the tiles of `chunks` query tiles (256 rows each): block after block of
// them, and within a block chunk after chunk.  A single chunk has one block, all
// its tiles; several have blocks of a run's length or a little more, so that the
// CTAs that work the same keys for different chunks do so at the same time, and
// the keys come from HBM once.
struct SharedLine {
  int first;          // place of the group's first tile (the last entry: the line's end)
  int tiles, chunks;  // tiles of a chunk (0: nothing shared), chunks of a head
  int r0;             // the group's first query row
};
constexpr int kMinTiles = 1;    // key tiles of a CTA's run, if the line has as many
__host__ __device__ __forceinline__ int line_share(int tiles, int ctas) {
  const int per = tiles / ctas + (tiles % ctas != 0);
  return per > kMinTiles ? per : kMinTiles;
}
__host__ __device__ __forceinline__ int line_blocks(int tiles, int chunks, int per) {
  return chunks > 1 && tiles >= 2 * per ? tiles / per : 1;
}
// First tile of block i of n.
__host__ __device__ __forceinline__ int block_tile(int tiles, int n, int i) {
  return (int)((long long)tiles * i / n);
}

// Where the records (m, l, o[128], as the decode's) of both parts lie.
struct SharedParts {
  Kv16Groups groups;
  // the prefixes': a chunk's records stand at its rows' own places for the run
  // that has the chunk's first tile, else with the CTA: [2][256], 0 for a run that
  // begins inside a block, 1 for one that begins a block
  float* part;              // [total][Hq]
  float* cut;               // [ctas][2][256]
  SharedLine* line;         // [groups + 1]
  int ctas;
  // the sequences' own: several queries each: [total][Hq][splits]; one query: as
  // above, the first run of pages at the row's place, else with the warp
  float* own;
  float* own_cut;           // [workers][g]
  int* own_line;            // [B + 1]: pages of one KV head before sequence b
  int splits, workers;
  int tokens, g;            // tokens of a query tile, heads of a group
};
constexpr int kMinRun = 2;      // pages of a warp's run, if the line has as many
__host__ __device__ __forceinline__ int run_share(int pages, int workers) {
  const int per = pages / workers + (pages % workers != 0);
  return per > kMinRun ? per : kMinRun;
}

// The last i in [0, n) with a[i] <= x (0 if there is none), by a warp.
__device__ __forceinline__ int warp_search(const int32_t* a, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, at = lo + (lane + 1) * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && __ldg(a + min(at, n - 1)) <= x);
    lo += __popc(le) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace oscar
