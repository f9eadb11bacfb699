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

// The line of key tiles that the prefixes' kernel has cut: group i's tiles stand
// from first on, `tiles` of them for each (KV head, 256 query rows).  Left in the
// workspace for who joins the records; the last entry's first is the line's end.
struct SharedLine {
  int first, tiles;
};
constexpr int kMinTiles = 1;    // key tiles of a CTA's run, if the line has as many
__host__ __device__ __forceinline__ int line_share(int tiles, int ctas) {
  const int per = tiles / ctas + (tiles % ctas != 0);
  return per > kMinTiles ? per : kMinTiles;
}


// The records (m, l, o[128], as the decode's) of the prefixes' kernel.
struct SharedParts {
  Kv16Groups groups;
  const float* part;        // [total][Hq]: of a row's first run of tiles
  const float* cut;         // [ctas][256]: of a run that begins inside a row
  const SharedLine* line;
  int ctas, tokens, g;      // tokens of a query tile, heads of a group
};
// Those of query row r and KV head h, head 0 of its group (head i: i records on).
struct Joint {
  int n;
  const float* first;
  const float* cut;
  __device__ __forceinline__ const float* record(int j) const {
    return j == 0 ? first : cut + (long long)j * 256 * kRecFloats;
  }
};
__device__ __forceinline__ Joint joint_of(const SharedParts& s, const Kv16& c, const Kv16Query& q,
                                          int r, int h, int i) {
  Joint x{0, nullptr, nullptr};
  if (i < 0) return x;
  const int tiles = __ldcg(&s.line[i].tiles);
  if (tiles <= 0) return x;
  int r0 = __ldg(s.groups.group + i), r1 = __ldg(s.groups.group + i + 1);
  if (q.start) r0 = __ldg(q.start + r0), r1 = __ldg(q.start + r1);
  if (r < r0 || r >= r1) return x;
  const int two = 2 * s.tokens, chunks = (r1 - r0 + two - 1) / two;
  const int chunk = (r - r0) / two, in = (r - r0) % two, w = in >= s.tokens ? 1 : 0;
  const long long at = __ldcg(&s.line[i].first) + ((long long)h * chunks + chunk) * tiles;
  const int per = line_share(__ldcg(&s.line[s.groups.n].first), s.ctas);
  const int c0 = (int)(at / per);
  if (c0 >= s.ctas) return x;
  x.n = (int)min((at + tiles - 1) / per, (long long)s.ctas - 1) - c0 + 1;
  x.first = s.part + ((long long)r * q.Hq + h * s.g) * kRecFloats;
  x.cut = s.cut + ((long long)c0 * 256 + w * 128 + (in - w * s.tokens) * s.g) * kRecFloats;
  return x;
}

}  // namespace oscar
