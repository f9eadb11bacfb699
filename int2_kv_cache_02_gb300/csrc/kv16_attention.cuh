// Attention of a ragged batch of queries over the 16-bit cache, on the
// tcgen05 tensor cores: 4 * 128 flops per visible (query, key) pair and head.
//
// Tiles.  A CTA takes up to two tiles of 128 query rows of one (sequence, KV
// head): a row is a (token, head of the group) pair, token-major, so the whole
// group reads each key and value once and a tile spans only 128 / g tokens
// (less masked work on the diagonal and at the edges of a window).  Keys come
// in tiles of four pages = 128 tokens; the pages that any row of the CTA sees
// (the sinks', then the window's) are numbered through, so a tile mixes pages
// from both places and pages outside are never read.
//
// Roles (12 warps, one CTA per SM that walks over the work items): a softmax
// warpgroup per query tile (a thread per row, so maxima and sums need no
// shuffles), a warp that copies (TMA, five stages of 32 KB that hold key and
// value tiles in turn), a warp per query tile that issues its MMAs, a warp that
// finds the items and hands them on.
//   S_w = Q_w K^T   128 x 128 x 128, both operands in shared memory
//   O_w += P_w V    P_w from TMEM, where it takes the place of S_w; V as it
//                   lies (along N)
// TMEM: S_0, S_1, O_0, O_1, 128 columns each.
//
// What the order is made of.  The tensor cores' queue is a few MMAs deep, so a
// warp that waits leaves them idle: two warps issue, and what one waits for
// passes under what the other has issued (one warp for both: 404 us against 399
// for the case below, and no better with more softmax warps).  They take turns,
// a key tile's products at a time, so that one tile's scores come while the
// other's softmax runs (in step with one another: 399 us; in turns: 332).  P
// goes over in two halves of 64 keys, the first product starting under the
// second half's exponentials.  Loads from TMEM are waited for at once: left in
// flight under the exponentials they slow them down (344 us).
//
// Softmax.  One pass, fp32, base 2.  A row's maximum is looked for only where it
// has none yet, and where the probabilities of 64 keys on the old one sum to
// more than kMost: so the loop over scores takes no maximum at all, P stays in
// the range of the type, and O is seldom rescaled.  Probabilities are rounded to
// the type of V for the product (half a step relative, as the output itself);
// the sum is of the unrounded ones.  fp16 has little range below 1 (2^-14 for
// whole steps, 2^-24 in all) and a token may outweigh the others by more, so
// there the largest score gives 2^7: whole steps down to 2^-21 of the largest
// and something down to 2^-32.  What is left below the largest number, 65504, is
// room to grow before O is rescaled: with 2^9 the window case below took 234 us,
// with 2^8 228, with 2^7 or 2^6 215.
//
// Measured (GB300): 8K-token causal prompt, 32/8 heads, bf16: 333 us, 1.65
// PFLOP/s, 0.85 of the measured bf16 burst rate; in a loop of seconds the power
// limit is reached and it takes 363 us (0.89 of the sustained rate).  Four
// sequences of 3K to 4K new tokens, window 1000 and 4 sinks, 32/4 heads, fp16:
// 204 us against 119; each 32-token item spends 9 key tiles on 7.9 tiles' worth
// of visible keys, and its first tile, masks and results (about 7 of 30
// thousand cycles) leave the tensor cores idle.
//
// Hidden values.  A hidden token's probability is exactly 0, but 0 * NaN is
// not: rows past the end of the sequence are cleared in shared memory, and the
// channels of a row that are NaN although its sum is a number are worked again
// by a warp that touches only the tokens the row sees (redo_row).  That may take
// longer than the bounded waits allow, so they do not run out while a warp says
// that it is at it.  A sum that is NaN has met a visible score that is NaN or
// +inf: the whole row is NaN and stays so.  (An 8K prompt, 32/8 heads, 0.36 ms:
// with a NaN in a key the same, in its first value 1.1 ms, in its middle one 10,
// in its last, hidden from the rest of its tile, 21; bf16 with an infinity in the
// first value 71.  Done after the last item instead, in line or out of line, it
// cost every prompt 2 to 5 %: the loop's registers.)
//
// Few tiles over a long cache: the key tiles are split over several CTAs, which
// leave (m, l, o[128]) records that a second kernel joins.
//
// kLine: sequences that share prefixes.  The same kernel over a line of work (see
// kv16_line.h) in which a group's queries meet its shared blocks together and
// each sequence's queries the blocks behind; an item is the piece of a CTA's run
// that lies in one row of the line.  All items leave records.  Rows for one query
// tile only (a decode step's, mostly) are worked by both, every other tile of keys
// each and at their own pace: a tile's chain of product, softmax and product takes
// 2.6 us with its loads, and two chains keep up with HBM (one: 165 us against 151 for
// 128 requests under four prompts).  A wider Item in kWhole's way cost it 0.8 %.
#pragma once

#include <algorithm>
#include <cmath>
#include <limits>

#include "kv16_groups.cuh"
#include "kv16_tma.h"
#include "tc5.cuh"

namespace oscar {
namespace {

constexpr int kSoftmaxWarps = 8;       // a warpgroup per query tile, a thread per row
constexpr int kThreads = kSoftmaxWarps * 32 + 128;
enum Part { kWhole, kLine };
// Floats of a record and before its o.
constexpr int rec_floats(int part) { return part == kWhole ? kRecFloats : kPartFloats; }
constexpr int rec_head(int part) { return part == kWhole ? 4 : kPartHead; }
// (The line's entries take a stage's room.  A ring of five for chunks that fill both
// query tiles and of three a query tile for the others, the table elsewhere, was
// slower, 5 to 15 %: more to count between two products.)
constexpr int stages_of(int part) { return part == kLine ? 4 : 5; }
constexpr int kTileBytes = 32768;      // 128 rows of 128 elements, two halves of 64 columns
constexpr int kHalf = 16384;
constexpr int kKeyPages = 4;           // pages of a key tile
// The maximum in use lies kBelow (log2) under the largest score that it was taken
// from, and a sum of 64 probabilities above kMost asks for a new one.
template <class T>
struct Range {
  static constexpr float kBelow = T::kHalf ? 7.0f : 0.0f;
  static constexpr float kMost = T::kHalf ? 65000.0f : 4096.0f;
};
constexpr uint32_t kO = 256;           // TMEM columns: S_w at 128 w, O_w at 256 + 128 w

struct AttnParams {
  Kv16 c;
  Kv16Query q;
  uint16_t* out;
  float* lse;
  float* part;          // [total * Hq][splits][kRecFloats] if splits > 1
  SharedParts line;     // kLine
  int g, tokens;        // heads of a group, tokens of a query tile
  int tiles;            // upper bound on work items of one KV head and split
  int splits;
  float scale;          // |scale| in the log2 domain
  bool negate;
  bool wide;            // out is 32-byte aligned
};

// Query rows for two tiles; or for one, worked by both, each with these queries and
// its own tiles of keys: those in stages 0 and 1 are query tile 0's, those in 2 and
// 3 tile 1's (first: the one that has the item's first).
constexpr int kPair = -1;
constexpr int kItems = 4;              // work items on their way to the other warps

// A work item as the scheduling warp hands it on.
struct Item {
  int stop;            // no more items
  int b, h, split, n;
  int row0, nrow;      // first row of q, tokens (of one or two tiles)
  int at0;             // position of the first token
  WholeSpan sp;
  int k0, k1;          // key tiles
  int cnt[2];          // of them, for each query tile: k0 .. k0 + cnt - 1
  bool clear;          // the last one's last page is the sequence's and lacks tokens
};

struct LineItem : Item {
  int end;             // the sequence behind a group's last (b is its first), -1: b's own
  int first;           // kPair, or the query tile that has the first tile of keys
  int s0;              // of the span
};
template <int PART>
struct ItemOf {
  using type = Item;
  static __device__ __forceinline__ int end(const Item*) { return -1; }
  static __device__ __forceinline__ int first(const Item*) { return kPair; }
  static __device__ __forceinline__ const WholeSpan& span(const Item* it) { return it->sp; }
};
template <>
struct ItemOf<kLine> {
  using type = LineItem;
  static __device__ __forceinline__ int end(const LineItem* it) { return it->end; }
  static __device__ __forceinline__ int first(const LineItem* it) { return it->first; }
  static __device__ __forceinline__ Span span(const LineItem* it) { return Span(it->sp, it->s0); }
};

template <int PART>
struct Smem {
  static constexpr int STAGES = stages_of(PART);
  uint64_t q_full[2], q_empty[2], full[STAGES], empty[STAGES];
  uint64_t s_full[2], p_full[2][2], h_full[2], o_full[2], turn[2], tail, drain[2];
  uint64_t together;                     // kLine: both query tiles' MMA warps are at an item
  uint64_t i_full[kItems], i_empty[kItems];
  uint32_t tmem;
  int state;           // of the waits
  int met[kSoftmaxWarps];
  typename ItemOf<PART>::type item[kItems];
};
constexpr int kItemReaders = kSoftmaxWarps + 3;   // warps that read an item: all but one

// Work item x.  One KV head's items are numbered through: sequence b's start
// at start[b] / (2 tokens) + b, which leaves room for all of them; those left
// over are empty (false).
__device__ __forceinline__ bool find_item(const AttnParams& p, int x, Item& it) {
  const int two = 2 * p.tokens, per_split = p.tiles * p.c.Hkv;
  it.split = x / per_split;
  const int y = x - it.split * per_split, t = y / p.c.Hkv;
  it.h = y - t * p.c.Hkv;
  int lo = 0, hi = p.c.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (min(max(__ldg(p.q.start + mid), 0), p.q.total) / two + mid <= t) lo = mid; else hi = mid;
  }
  it.b = lo;
  const int r0 = __ldg(p.q.start + lo), r1 = __ldg(p.q.start + lo + 1), nq = r1 - r0;
  const bool report = (threadIdx.x & 31) == 0;
  if (r0 < 0 || r1 > p.q.total || nq < 0) {
    if (report) record_error(p.c.status, kDevErrBadPaged);
    return false;
  }
  const int mine = t - (r0 / two + lo), all = (nq + two - 1) / two;
  if (mine < 0 || mine >= all) return false;
  it.n = kv16_length(p.c, lo, p.q.max_tok);
  if (it.n < nq) {     // a length out of range, or fewer tokens than queries
    if (report) record_error(p.c.status, kDevErrBadPaged);
    it.n = max(it.n, 0);
  }
  const int q0 = (all - 1 - mine) * two;        // the longest rows first
  it.row0 = r0 + q0;
  it.nrow = min(two, nq - q0);
  it.at0 = it.n - nq + q0;
  it.sp = WholeSpan(it.at0, it.at0 + it.nrow - 1, p.q.window, p.q.n_sink);
  const int kt = (it.sp.blocks + kKeyPages - 1) / kKeyPages;
  it.k0 = (int)((long long)kt * it.split / p.splits);
  it.k1 = (int)((long long)kt * (it.split + 1) / p.splits);
  it.cnt[0] = it.k1 - it.k0;
  it.cnt[1] = 0;
  if (it.nrow > p.tokens) {
    // the first tile's keys end before the second's
    it.cnt[1] = it.cnt[0];
    const int blocks = WholeSpan(it.at0, it.at0 + p.tokens - 1, p.q.window, p.q.n_sink).blocks;
    it.cnt[0] = min(it.k1, max(it.k0, (blocks + kKeyPages - 1) / kKeyPages)) - it.k0;
  }
  it.clear = it.k1 > it.k0 && it.k1 == kt && it.n % kPage != 0 &&
             it.sp.block(it.sp.blocks - 1) == (it.n - 1) / kPage;
  return true;
}

__device__ __forceinline__ int key_tiles(int blocks) { return (blocks + kKeyPages - 1) / kKeyPages; }

// The lowest and the highest position of queries, those of sequence b or none.
struct Reach {
  int lo, hi;
};
__device__ __forceinline__ Reach reach_of(const AttnParams& p, int b) {
  const int n = kv16_length(p.c, b, p.q.max_tok);
  const int nq = p.q.start ? __ldg(p.q.start + b + 1) - __ldg(p.q.start + b) : 1;
  return n > 0 && nq > 0 ? Reach{max(n - nq, 0), n - 1} : Reach{0x7fffffff, -1};
}
// Those of sequences [b0, b1).  A warp.
__device__ __forceinline__ Reach warp_reach(const AttnParams& p, int b0, int b1) {
  Reach x{0x7fffffff, -1};
  for (int b = b0 + (threadIdx.x & 31); b < b1; b += 32) {
    const Reach y = reach_of(p, b);
    x = Reach{min(x.lo, y.lo), max(x.hi, y.hi)};
  }
  return Reach{__reduce_min_sync(0xffffffffu, x.lo), __reduce_max_sync(0xffffffffu, x.hi)};
}

// A group's entry of the line: its sequences' queries [r0, r1) against the blocks
// of `sp`.  reach: of its sequences, asked for under a window.
struct GroupEntry {
  Shared s;
  int r0, r1;
  Span sp;
};
template <class F>
__device__ __forceinline__ GroupEntry group_entry(const AttnParams& p, int i, bool report,
                                                  F&& reach) {
  GroupEntry x;
  x.s = shared_of(p.c, p.line.groups, i, p.q.max_tok, report);
  x.r0 = x.s.lead;
  x.r1 = x.s.end;
  if (p.q.start && x.r1 > x.r0) {
    x.r0 = __ldg(p.q.start + x.s.lead);
    x.r1 = __ldg(p.q.start + x.s.end);
    if (x.r0 < 0 || x.r1 > p.q.total || x.r1 < x.r0) {
      if (report) record_error(p.c.status, kDevErrBadPaged);
      x.r0 = x.r1 = 0;
    }
  }
  x.sp.sink_blocks = x.sp.w0 = x.sp.s0 = 0;
  x.sp.blocks = x.r1 > x.r0 ? x.s.blocks : 0;
  if (p.q.window > 0 && x.sp.blocks > 0) {
    const Reach y = reach(x.s);
    x.sp = Span(y.lo, y.hi, p.q.window, p.q.n_sink).below(x.s.blocks);
  }
  return x;
}
__device__ __forceinline__ GroupEntry warp_group_entry(const AttnParams& p, int i) {
  return group_entry(p, i, false, [&](const Shared& s) { return warp_reach(p, s.lead, s.end); });
}

// Kind of a group's rows (kv16_line.h).
__device__ __forceinline__ int group_kind(const AttnParams& p, int rows) {
  return (rows > p.tokens ? 1 : 0) | (p.q.window > 0 ? 2 : 0);
}

// A sequence's own entry: nq queries from row r0 on, the first at position at0,
// against its blocks from `shared` on.
struct OwnEntry {
  int r0, nq, n, at0, group, shared;
  __device__ __forceinline__ Span span(const AttnParams& p, int tok, int count) const {
    return Span(at0 + tok, at0 + tok + count - 1, p.q.window, p.q.n_sink).from(shared);
  }
  // key tiles of chunk i, and the places of its row
  __device__ __forceinline__ int tiles(const AttnParams& p, int i) const {
    const int two = 2 * p.tokens;
    return key_tiles(span(p, i * two, min(two, nq - i * two)).blocks);
  }
  __device__ __forceinline__ int kind(const AttnParams& p, int i) const {
    return nq - i * 2 * p.tokens > p.tokens;
  }
  __device__ __forceinline__ int places(const AttnParams& p, int i) const {
    return row_places(tiles(p, i), kind(p, i));
  }
};
__device__ __forceinline__ OwnEntry own_entry(const AttnParams& p, int b, bool report) {
  OwnEntry x;
  x.r0 = b;
  x.nq = 1;
  x.n = kv16_length(p.c, b, p.q.max_tok);
  bool ok = x.n >= 0;
  if (p.q.start) {
    const int r0 = __ldg(p.q.start + b), r1 = __ldg(p.q.start + b + 1);
    x.r0 = r0;
    x.nq = r1 - r0;
    if (r0 < 0 || r1 > p.q.total || r1 < r0) x.nq = 0, ok = false;
    ok = ok && x.n >= x.nq;            // (fewer tokens than queries)
  }
  if (!ok && report) record_error(p.c.status, kDevErrBadPaged);
  x.n = max(x.n, 0);
  x.at0 = x.n - x.nq;
  x.group = group_of(p.line.groups, b);
  x.shared = x.group < 0 ? 0 : shared_of(p.c, p.line.groups, x.group, p.q.max_tok, false).blocks;
  return x;
}

__device__ __forceinline__ int saturate(long long x) { return (int)min(x, 0x7fffffffLL); }

// The entries' first places, first[0 .. groups + B] (no more than the largest int,
// so that groups that overlap do not wrap around).  All threads of the CTA; ends
// with a barrier.  reach: [groups], room that is free until then.  (Under a window a
// group's span goes by all its sequences, a thread each: 512 of one group 38 us, 54 by
// a thread a group.)
__device__ __forceinline__ void line_up(const AttnParams& p, int* first, int* scan, Reach* reach) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int two = 2 * p.tokens, G = p.line.groups.n, entries = G + p.c.B;
  const bool report = blockIdx.x == 0;
  if (p.q.window > 0) {
    for (int e = tid; e < G; e += kThreads) reach[e] = Reach{0x7fffffff, -1};
    __syncthreads();
    for (int b = tid; b < p.c.B; b += kThreads) {
      const Reach y = reach_of(p, b);
      const int i = y.hi < 0 ? -1 : group_of(p.line.groups, b);
      if (i < 0) continue;
      atomicMin(&reach[i].lo, y.lo);
      atomicMax(&reach[i].hi, y.hi);
    }
    __syncthreads();
  }
  unsigned carry = 0;      // sums of two numbers below 2^31
  auto plus = [](unsigned a, unsigned b) { return min(a + b, 0x7fffffffu); };
  for (int e0 = 0; e0 < entries; e0 += kThreads) {
    const int e = e0 + tid;
    unsigned x = 0;
    if (e < G) {
      const GroupEntry y = group_entry(p, e, report, [&](const Shared&) { return reach[e]; });
      const int tiles = key_tiles(y.sp.blocks), rows = y.r1 - y.r0;
      x = (unsigned)saturate((long long)((rows + two - 1) / two) * p.c.Hkv *
                             row_places(tiles, group_kind(p, rows)));
      if (report) p.line.group[e] = make_int4(tiles, y.r0, y.r1, 0);
    } else if (e < entries) {
      const OwnEntry y = own_entry(p, e - G, report);
      long long n = 0;
      for (int i = 0; i * two < y.nq; ++i) n += y.places(p, i);
      x = (unsigned)saturate(n * p.c.Hkv);
      if (report) p.line.seq[e - G] = make_int2(y.group, y.shared);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x = plus(x, y);
    }
    unsigned before = __shfl_up_sync(0xffffffffu, x, 1);
    if (lane == 0) before = 0;
    if (lane == 31) scan[warp] = (int)x;
    __syncthreads();
    unsigned base = carry;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base = plus(base, (unsigned)scan[w]);
      carry = plus(carry, (unsigned)scan[w]);
    }
    if (e < entries) {
      first[e] = (int)plus(base, before);
      if (report) p.line.first[e] = first[e];
    }
    __syncthreads();
  }
  if (tid == 0) {
    first[entries] = (int)carry;
    if (report) p.line.first[entries] = (int)carry;
  }
  // (copies may land where `reach` was)
  if (p.q.window > 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
}

// The item at place x of the line, as far as x1; its number of places.  share: the
// places of a CTA's run.  A warp.
// (Maxima and minima: whatever the groups and lengths hold by now, what follows
// stays in bounds.)
__device__ __forceinline__ int find_piece(const AttnParams& p, const int* first, int share, int x,
                                          int x1, LineItem& it) {
  const int G = p.line.groups.n, two = 2 * p.tokens, lane = threadIdx.x & 31;
  int lo = 0, hi = G + p.c.B;     // first[i] <= x < first[i + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  const int at = x - first[lo];
  int from, to;                   // places of the row
  int kind;
  int all, tiles0 = 0;            // tiles of the row, of a sequence's first query tile (whose keys end first)
  int* runs;
  it.clear = false;
  if (lo < G) {
    const GroupEntry y = warp_group_entry(p, lo);
    const int rows = y.r1 - y.r0, tiles = max(key_tiles(y.sp.blocks), 1);
    kind = group_kind(p, rows);
    to = row_places(tiles, kind);
    int p0 = 0, chunk = 0;
    all = tiles;
    if (rows <= two) {
      it.h = min(at / to, p.c.Hkv - 1);
      from = at - it.h * to;
    } else {
      const int chunks = (rows + two - 1) / two, places = to;
      const int per_head = chunks * places;       // (no more than the line has: it fits)
      it.h = min(at / per_head, p.c.Hkv - 1);
      const int in_head = at - it.h * per_head, z = min(in_head / chunks, places - 1);
      const Blocks blocks(tiles, chunks, kind, share);
      const int t = whole_tiles(max(z - row_cost(kind), 0), kind);
      const int i = min(t / blocks.least, blocks.count - 1);
      p0 = tile_place(blocks.first(i), kind);
      if (blocks.count > 1) all = 0;
      if (i + 1 < blocks.count) to = tile_place(blocks.first(i + 1), kind);
      const int in = in_head - chunks * p0;
      chunk = min(in / (to - p0), chunks - 1);
      from = p0 + in - chunk * (to - p0);
    }
    it.b = y.s.lead;
    it.end = y.s.end;
    it.n = it.at0 = 0;
    it.row0 = y.r0 + chunk * two;
    it.nrow = min(two, y.r1 - it.row0);
    it.sp = y.sp;
    it.s0 = 0;
    it.split = from <= row_cost(kind) ? 0 : from > p0 ? 1 : 2;  // where the records go
    runs = p.line.prefix_runs;
  } else {
    const OwnEntry y = own_entry(p, lo - G, false);
    int in, chunk = 0;
    if (y.nq <= two) {
      const int places = max(y.places(p, 0), 1);
      it.h = min(at / places, p.c.Hkv - 1);
      in = at - it.h * places;
    } else {
      // the chunk that has place `in` of the head's
      const int chunks = (y.nq + two - 1) / two;
      const int per_head = max((first[lo + 1] - first[lo]) / p.c.Hkv, 1);
      it.h = min(at / per_head, p.c.Hkv - 1);
      in = at - it.h * per_head;
      for (int c0 = 0;; c0 += 32) {
        const int mine = c0 + lane < chunks ? y.places(p, c0 + lane) : 0;
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int z = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += z;
        }
        const unsigned past = __ballot_sync(0xffffffffu, sum > in);
        if (past == 0 && c0 + 32 < chunks) {
          in -= __shfl_sync(0xffffffffu, sum, 31);
          continue;
        }
        const int l = past ? __ffs(past) - 1 : 31;
        chunk = min(c0 + l, chunks - 1);
        in -= __shfl_sync(0xffffffffu, sum - mine, l);
        break;
      }
    }
    it.b = lo - G;
    it.end = -1;
    it.n = y.n;
    it.row0 = y.r0 + chunk * two;
    it.nrow = min(two, y.nq - chunk * two);
    it.at0 = y.at0 + chunk * two;
    const Span sp = y.span(p, chunk * two, it.nrow);
    it.sp = sp;
    it.s0 = sp.s0;
    from = max(in, 0);
    kind = y.kind(p, chunk);
    all = key_tiles(it.sp.blocks);
    to = row_places(all, kind);
    runs = p.line.own_runs;
    tiles0 = key_tiles(y.span(p, chunk * two, min(it.nrow, p.tokens)).blocks);
    it.split = from <= row_cost(kind) ? -1 : 1;
  }
  const int end = (int)min(min((long long)from + (x1 - x), (long long)to),
                           (long long)from + (first[lo + 1] - x));
  it.k0 = tiles_before(from, kind);
  it.k1 = tiles_before(end, kind);
  it.cnt[0] = it.nrow > 0 ? max(it.k1 - it.k0, 0) : 0;
  it.cnt[1] = it.nrow > p.tokens ? it.cnt[0] : 0;
  if (lane == 0 && it.split <= 0 && all > 0 && it.cnt[0] > 0) {
    const int last = x - from + row_cost(kind) + (all - 1) * tile_cost(kind);
    const int n = min(last / share, (int)gridDim.x - 1) - (int)blockIdx.x + 1;
    runs[(long long)it.row0 * p.c.Hkv + it.h] = blockIdx.x | n << 16;
  }
  if (lo >= G && it.cnt[0] > 0) {
    if (it.cnt[1] > 0) it.cnt[0] = min(it.k1, max(it.k0, tiles0)) - it.k0;
    it.clear = end == to && it.n % kPage != 0 &&
               it.sp.block(it.sp.blocks - 1) == (it.n - 1) / kPage;
  }
  return max(end - from, 1);
}

// The record of a row of an item: at the row's place (`second`: of query tile 1,
// where both tiles have these queries), or the CTA's.
__device__ __forceinline__ float* line_record(const AttnParams& p, int split, bool second,
                                              long long row, int cut_row) {
  if (split > 0)
    return p.line.cut + (((long long)blockIdx.x * 2 + split - 1) * 256 + cut_row) * kPartFloats;
  if (second) row += (long long)p.q.total * p.q.Hq;
  return (split == 0 ? p.line.prefix : p.line.own) + row * kPartFloats;
}

// The position of query row r of a group's sequences [b0, b1).
__device__ __forceinline__ int position_of(const AttnParams& p, int b0, int b1, int r) {
  int b = r, back = 1;
  if (p.q.start) {
    int lo = b0, hi = b1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.q.start + mid) <= r) lo = mid; else hi = mid;
    }
    b = lo;
    back = __ldg(p.q.start + lo + 1) - r;
  }
  const int n = kv16_length(p.c, b, p.q.max_tok);
  return n < 0 ? -1 : max(n - back, -1);
}

template <class T>
__device__ __forceinline__ void store_row4(const AttnParams& p, long long row, int lane,
                                           const float (&o)[4], float inv) {
  reinterpret_cast<uint2*>(p.out + row * kD)[lane] =
      make_uint2(T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv));
}

// log(sum exp) of a row: the sum as it is on the largest score, whose logarithm
// is the small one.
template <class T>
__device__ __forceinline__ float row_lse(float m, float l) {
  return kv16_lse(m + Range<T>::kBelow, l * (T::kHalf ? 1.0f / 128.0f : 1.0f));
}

// Is a channel of O (or of the result) one to be worked again?  NaN is, and in
// bf16 an infinity too: sums of probabilities up to kMost times the largest
// values can overflow.  In fp16 they cannot: an infinity there is a visible one.
template <class T>
__device__ __forceinline__ bool is_open(float x) {
  return T::kHalf ? x != x : !(fabsf(x) < INFINITY);
}
// NaN once x was such a channel.
template <class T>
__device__ __forceinline__ float gather_open(float x, float so_far) {
  if constexpr (T::kHalf) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(so_far));
    return y;
  } else {
    return fmaf(x, 0.0f, so_far);
  }
}

// Row `row` of a work item, position `at`, whose results this warp has just
// written: its open channels again, from the tokens alone that it sees.  *met is
// the block in which such a row of this warp has last met its NaN: the others
// most likely meet it there too, so they look there first.
template <class T, int PART, class S>
__device__ __forceinline__ void redo_row(const AttnParams& p, int b, int h, int split, int k0,
                                         int k1, const S& sp, long long row, int at, int* met,
                                         int cut_row, int first_tile, int w) {
  const int lane = threadIdx.x & 31;
  const bool record = PART != kWhole || p.splits > 1;
  float* rec = PART == kLine ? line_record(p, split, first_tile != kPair && w == 1, row, cut_row)
                               : p.part + (row * p.splits + split) * rec_floats(PART);
  uint2* out = reinterpret_cast<uint2*>(p.out + row * kD) + lane;
  float x[4];
  if (record) {
    if (rec[1] != rec[1]) return;            // the sum
    const float4 v = *reinterpret_cast<const float4*>(rec + rec_head(PART) + 4 * lane);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *out;
    const float2 a = T::unpack(v.x), b = T::unpack(v.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  }
  unsigned open = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) open |= is_open<T>(x[i]) ? 1u << i : 0u;
  if (!__any_sync(0xffffffffu, open != 0)) return;
  const long long token = row / p.q.Hq;
  const int head = (int)(row - token * p.q.Hq);
  float m, l, o[4];
  const uint16_t* q = p.q.q + token * p.q.stride + (long long)head * kD;
  if (PART == kLine && first_tile != kPair) {
    // every other tile of keys is this query tile's
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int k = k0 + ((first_tile ^ w) & 1); k < k1; k += 2) {
      const int i = kv16_warp_row<T>(p.c, q, b, h, at, sp, k * kKeyPages,
                                     min((k + 1) * kKeyPages, sp.blocks), p.q.window, p.q.n_sink,
                                     p.q.scale_log2, open, m, l, o);
      const float f = m == -INFINITY || rec[0] == -INFINITY ? 1.0f : fast_exp2(m - rec[0]);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += o[e] * f;
      if (i >= 0) break;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((open >> e) & 1u) rec[rec_head(PART) + 4 * lane + e] = sum[e];
    return;
  }
  const int i0 = k0 * kKeyPages, i1 = min(k1 * kKeyPages, sp.blocks), there = *met;
#pragma unroll 1
  for (int look = there >= i0 && there < i1 ? 0 : 1; look < 2; ++look) {
    const int i = kv16_warp_row<T>(p.c, q, b, h,
                                   at, sp, look ? i0 : there, look ? i1 : there + 1, p.q.window,
                                   p.q.n_sink, p.q.scale_log2, open, m, l, o);
    if (i < 0) continue;
    __syncwarp();
    if (lane == 0) *met = i;
    __syncwarp();
    break;
  }
  // a record's channels stand on the record's maximum
  float f = l == 0.0f ? 0.0f : 1.0f / l;
  if (record) {
    const float m0 = rec[0];
    f = m == -INFINITY || m0 == -INFINITY ? 1.0f : fast_exp2(m - m0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((open >> i) & 1u) x[i] = o[i] * f;
  if (record)
    *reinterpret_cast<float4*>(rec + rec_head(PART) + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *out = make_uint2(T::pack(x[0], x[1]), T::pack(x[2], x[3]));
}

template <class T, int PART>
__global__ void __launch_bounds__(kThreads, 1)
kv16_attention_kernel(const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const AttnParams p) {
  constexpr int kStages = stages_of(PART);
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* sq = smem;                            // two query tiles
  uint8_t* ring = smem + 2 * kTileBytes;
  using It = typename ItemOf<PART>::type;
  auto& sm = *reinterpret_cast<Smem<PART>*>(smem + (2 + kStages) * kTileBytes);
  int* first = reinterpret_cast<int*>(&sm + 1);  // kLine: [groups + B + 1], then a number a warp
  if (smem_u32(smem) & 1023) {                   // the swizzle counts on it
    if (tid == 0) record_error(p.c.status, kDevErrWaitTimeout);
    return;
  }

  int x0 = 0, x1 = 0, share = 0;                 // kLine: the CTA's run of the line
  if constexpr (PART != kWhole) {
    asm volatile("griddepcontrol.launch_dependents;");
    if (tid < 3)
      asm volatile("prefetch.tensormap [%0];" ::"l"(tid == 0 ? &map_q : tid == 1 ? &map_k : &map_v));
  }
  if constexpr (PART == kLine) {
    const int entries = p.line.groups.n + p.c.B;
    line_up(p, first, first + entries + 1, reinterpret_cast<Reach*>(smem));
    const int total = first[entries];
    share = line_share(total, gridDim.x);
    x0 = (int)min((long long)blockIdx.x * share, (long long)total);
    x1 = (int)min((long long)x0 + share, (long long)total);
    if (x0 == x1) return;
  }
  if (warp == kSoftmaxWarps) tc5_alloc(&sm.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 4);
      mbar_init(&sm.p_full[i][1], 4);
      mbar_init(&sm.h_full[i], 1);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.turn[i], 1);
      mbar_init(&sm.drain[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.i_full[i], 1);
      mbar_init(&sm.i_empty[i], kItemReaders);
    }
    mbar_init(&sm.tail, 1);
    mbar_init(&sm.together, 2);
    mbar_fence_init();
    sm.state = 0;
    for (int i = 0; i < kSoftmaxWarps; ++i) sm.met[i] = -1;
  }
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const uint32_t tmem = sm.tmem;
  volatile int* state = &sm.state;
  // an item is read by every warp but the scheduling one, and then given back
  auto take = [&](unsigned n) -> const It* {
    return tc5_wait(&sm.i_full[n % kItems], (n / kItems) & 1, state) ? &sm.item[n % kItems]
                                                                     : nullptr;
  };

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    bool ok = true;
    if (warp == kSoftmaxWarps + 3) {
      // -------------------------------------------------- scheduling: the items
      // x, rounds of the grid in turn forwards and backwards, so that a CTA
      // with the longest of one round gets the shortest of the next
      unsigned n = 0, passed = 0;      // items, tiles of keys
      const int items = p.tiles * p.c.Hkv * p.splits, grid = gridDim.x;
      for (int round = 0; ok; ++round) {
        bool stop;
        It it;
        if constexpr (PART == kLine) {
          stop = x0 >= x1;
          if (!stop) {
            x0 += find_piece(p, first, share, x0, x1, it);
            if (it.cnt[0] <= 0 && it.cnt[1] <= 0) {              // (places without tiles)
              ok = !(*state & 1);
              continue;
            }
            const int nk = it.k1 - it.k0;
            it.first = it.nrow > p.tokens ? kPair : (int)(passed & 1);
            if (it.first != kPair) {
              it.cnt[0] = it.first == 0 ? nk - nk / 2 : nk / 2;
              it.cnt[1] = nk - it.cnt[0];
            }
            passed += nk;
          }
        } else {
          const long long x = (long long)round * grid +
                              ((round & 1) ? grid - 1 - blockIdx.x : blockIdx.x);
          stop = (long long)round * grid >= items;
          if (!stop && (x >= items || !find_item(p, (int)x, it))) continue;
        }
        it.stop = stop;
        if (n >= kItems) ok = tc5_wait(&sm.i_empty[n % kItems], (n / kItems - 1) & 1, state);
        if (!ok) break;
        if (lane == 0) {
          sm.item[n % kItems] = it;
          mbar_arrive(&sm.i_full[n % kItems]);
        }
        __syncwarp();
        ++n;
        if (stop) break;
      }
    } else if (warp == kSoftmaxWarps) {
      // ------------------------------------------------------------ copies
      const int none = p.c.table ? p.c.n_pages * p.c.Hkv * kPage
                                 : p.c.B * p.c.Hkv * p.c.T_cap;      // reads zeros
      const unsigned qbytes = 2 * 64 * 2 * p.g * p.tokens;
      unsigned used = 0, q_used[2] = {0, 0}, tails = 0;
      unsigned kept = ~0u;     // the tile that has come and is not passed on yet
      int kept_page = 0, kept_at = 0;          // kLine: its last page, and the tokens there
      // Clears the rows behind the sequence's last token in the kept tile and passes
      // it on.
      auto pass_on = [&](int page, int tokens) {
        const unsigned st = kept % kStages;
        ok = ok && tc5_wait(&sm.tail, (tails - 1) & 1, state);
        if (!ok) return;
        if (lane >= tokens) {
          uint8_t* r = ring + st * kTileBytes + (page * kPage + lane) * 128;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            reinterpret_cast<uint4*>(r + (i >> 3) * kHalf)[i & 7] = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[st]);
        kept = ~0u;
      };
      // kLine: what may take long is waited for only once the kept tile is passed on,
      // but what is ready is begun before (the kept tile's way here and the next
      // item's first copies overlap)
      auto settled_wait = [&](uint64_t* bar, unsigned parity) -> bool {
        if (PART == kLine && kept != ~0u) {
          if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
          pass_on(kept_page, kept_at);
        }
        return ok && tc5_wait(bar, parity, state);
      };
      for (unsigned ni = 0; ok && (PART != kLine || ni < p.line.copied); ++ni) {
        if (!(ok = settled_wait(&sm.i_full[ni % kItems], (ni / kItems) & 1))) break;
        const It* ip = &sm.item[ni % kItems];
        if (ip->stop) break;
        const It it = *ip;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.i_empty[ni % kItems]);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!ok || it.cnt[w] == 0) continue;
          if (q_used[w] > 0) ok = settled_wait(&sm.q_empty[w], (q_used[w] - 1) & 1);
          if (!ok) continue;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.q_full[w], qbytes);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              tma_box3(sq + w * kTileBytes + i * kHalf, &map_q, 64 * i, it.h * p.g,
                       it.row0 + (ItemOf<PART>::first(&it) == kPair ? w * p.tokens : 0),
                       &sm.q_full[w]);
          }
          __syncwarp();
          ++q_used[w];
        }
        const auto& sp = ItemOf<PART>::span(&it);
        int row = none;
        auto ask = [&](int kv, unsigned st, uint64_t* bar) {
          uint8_t* dst = ring + st * kTileBytes;
          if (lane == 0) mbar_arrive_expect_tx(bar, kTileBytes);
          __syncwarp();
          if (lane < kKeyPages) {          // a lane per page
            tma_box2(dst + lane * 4096, kv ? &map_v : &map_k, 0, row, bar);
            tma_box2(dst + kHalf + lane * 4096, kv ? &map_v : &map_k, 64, row, bar);
          }
          __syncwarp();
        };
        for (int k = it.k0; k < it.k1 && ok; ++k) {
          row = none;
          if (lane < kKeyPages && k * kKeyPages + lane < sp.blocks) {
            row = kv16_block_row(p.c, it.b, it.h, sp.block(k * kKeyPages + lane));
            if (row < 0) {
              record_error(p.c.status, kDevErrBadPaged);
              row = none;
            }
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const unsigned st = used % kStages;
            if (used >= kStages) ok = ok && settled_wait(&sm.empty[st], (used / kStages - 1) & 1);
            if (!ok || (kv == 1 && it.clear && k + 1 == it.k1)) break;
            ask(kv, st, &sm.full[st]);
            ++used;
          }
        }
        if (ok && it.clear) {
          // The rows behind the sequence's last token hold anything.  The value
          // tile that has them, the last one, lands on a barrier of this warp's,
          // which clears them and only then passes the tile on.
          const unsigned st = used % kStages;
          if (PART == kLine && kept != ~0u) pass_on(kept_page, kept_at);
          if (!ok) break;
          ask(1, st, &sm.tail);
          ++tails;
          kept = used++;
          const int last = sp.blocks - 1;
          kept_page = last - (it.k1 - 1) * kKeyPages;
          kept_at = it.n - sp.block(last) * kPage;
          if (PART == kWhole) pass_on(kept_page, kept_at);
        }
      }
      if (PART == kLine && ok && kept != ~0u) pass_on(kept_page, kept_at);
      // what is in flight lands before the memory is given back, whoever gives up
      bool landed = true;
      for (int w = 0; w < 2; ++w)
        if (q_used[w]) landed &= mbar_wait_bounded(&sm.q_full[w], (q_used[w] - 1) & 1, kDrainLimit);
      if (tails) landed &= mbar_wait_bounded(&sm.tail, (tails - 1) & 1, kDrainLimit);
      for (unsigned i = used > kStages ? used - kStages : 0; i < used; ++i)
        if (i != kept)
          landed &= mbar_wait_bounded(&sm.full[i % kStages], (i / kStages) & 1, kDrainLimit);
      if (!landed && lane == 0) record_error(p.c.status, kDevErrDrainTimeout);
    } else {
      // -------------------------------------------------------------- MMAs
      // A warp per query tile: what one waits for passes under what the other
      // has issued (the tensor cores' queue is too short to cover a wait).  They
      // take turns, a key tile's products at a time: so one tile's scores come
      // while the other's softmax runs, and not both at once.
      const int w = warp - kSoftmaxWarps - 1;
      if (elect_one()) {
        const uint32_t id_s = tc5_idesc(T::kHalf, 128, 128, false, p.negate);
        const uint32_t id_o = tc5_idesc(T::kHalf, 128, 128, true, false);
        constexpr uint64_t kAlongK = tc5_desc_base(16, 1024);          // Q, K
        constexpr uint64_t kAlongN = tc5_desc_base(kHalf, 1024);       // V
        const uint64_t dq = tc5_desc(kAlongK, smem_u32(sq + w * kTileBytes));
        const uint32_t ts = tmem + 128 * w, to = tmem + kO + 128 * w;
        const unsigned ring_addr = smem_u32(ring);
        auto qk = [&](unsigned stage) {
          const uint64_t k = tc5_desc(kAlongK, ring_addr + stage * kTileBytes);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const unsigned off = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
            tc5_mma_ss(ts, dq + off, k + off, id_s, i > 0);
          }
          tc5_commit(&sm.s_full[w]);
        };
        unsigned st = 0, ph = 0;         // the next stage: K_0 V_0 K_1 V_1 ...
        auto next = [&] {
          if (++st == kStages) {
            st = 0;
            ph ^= 1;
          }
        };
        unsigned q_used = 0, p_used = 0, turns = 0, meets = 0;
        bool apart = false;
        auto my_turn = [&]() -> bool {
          const unsigned n = turns++;
          if (w == 1) return tc5_wait(&sm.turn[1], n & 1, state);
          return n == 0 || tc5_wait(&sm.turn[0], (n - 1) & 1, state);
        };
        for (unsigned ni = 0; ok; ++ni) {
          const It* ip = take(ni);
          if (!(ok = ip != nullptr) || ip->stop) break;
          const int cnt = ip->cnt[w], nk = ip->k1 - ip->k0;
          const int first_tile = ItemOf<PART>::first(ip);
          mbar_arrive(&sm.i_empty[ni % kItems]);
          if (nk <= 0) continue;
          if (PART == kLine && first_tile != kPair) {
            // A stage is one query tile's: the other passes over it, and they take no
            // turns.  (A warp sees every use of its stages, so a phase is the one that it
            // waits for.)
            apart = true;
            int done = 0;
            for (int j = 0; j < nk && ok; ++j) {
              const unsigned ks = st, kp = ph;
              next();
              const unsigned vs = st, vp = ph;
              next();
              if (((first_tile + j) & 1) != w) continue;
              ok = tc5_wait(&sm.full[ks], kp, state);
              if (ok && done == 0) ok = tc5_wait(&sm.q_full[w], q_used++ & 1, state);
              if (!ok) break;
              tc5_fence_after();
              qk(ks);
              if (done + 1 == cnt) tc5_commit(&sm.q_empty[w]);
              tc5_commit(&sm.empty[ks]);
              tc5_commit(&sm.empty[ks]);
              ok = tc5_wait(&sm.full[vs], vp, state);
              if (ok) ok = tc5_wait(&sm.p_full[w][0], p_used & 1, state);
              if (!ok) break;
              const uint64_t v = tc5_desc(kAlongN, ring_addr + vs * kTileBytes);
              tc5_fence_after();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                tc5_mma_ts(to, ts + 8 * i, v + i * (2048 >> 4), id_o, done > 0 || i > 0);
              tc5_commit(&sm.h_full[w]);
              ok = tc5_wait(&sm.p_full[w][1], p_used++ & 1, state);
              if (!ok) break;
              tc5_fence_after();
#pragma unroll
              for (int i = 4; i < 8; ++i)
                tc5_mma_ts(to, ts + 32 + 8 * i, v + i * (2048 >> 4), id_o, true);
              if (++done == cnt) tc5_commit(&sm.o_full[w]);
              tc5_commit(&sm.empty[vs]);
              tc5_commit(&sm.empty[vs]);
            }
            continue;
          }
          if (PART == kLine && apart) {
            // from here on both use all stages: neither may be a use ahead of the other
            mbar_arrive(&sm.together);
            ok = tc5_wait(&sm.together, meets++ & 1, state);
            if (!ok) break;
            apart = false;
          }
          // a stage that this tile has no use for is given back as it comes
          ok = tc5_wait(&sm.full[st], ph, state);
          if (ok && cnt > 0) ok = tc5_wait(&sm.q_full[w], q_used++ & 1, state);
          if (ok) ok = my_turn();
          if (!ok) break;
          if (cnt > 0) {
            tc5_fence_after();
            qk(st);
            if (cnt == 1) tc5_commit(&sm.q_empty[w]);
            tc5_commit(&sm.empty[st]);
          } else {
            mbar_arrive(&sm.empty[st]);
          }
          mbar_arrive(&sm.turn[w ^ 1]);
          next();
          for (int j = 0; j < nk && ok; ++j) {
            const unsigned vs = st, vp = ph;
            next();
            const bool more = j + 1 < nk;
            ok = tc5_wait(&sm.full[vs], vp, state);
            if (ok && more) ok = tc5_wait(&sm.full[st], ph, state);
            if (ok && j < cnt) ok = tc5_wait(&sm.p_full[w][0], p_used & 1, state);
            if (ok) ok = my_turn();
            if (!ok) break;
            if (j < cnt) {
              // P comes in halves of 64 keys
              const uint64_t v = tc5_desc(kAlongN, ring_addr + vs * kTileBytes);
              tc5_fence_after();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                tc5_mma_ts(to, ts + 8 * i, v + i * (2048 >> 4), id_o, j > 0 || i > 0);
              tc5_commit(&sm.h_full[w]);
              ok = tc5_wait(&sm.p_full[w][1], p_used++ & 1, state);
              if (!ok) break;
              tc5_fence_after();
#pragma unroll
              for (int i = 4; i < 8; ++i)
                tc5_mma_ts(to, ts + 32 + 8 * i, v + i * (2048 >> 4), id_o, true);
              if (j + 1 < cnt) qk(st);
              else tc5_commit(&sm.o_full[w]);
              mbar_arrive(&sm.turn[w ^ 1]);
              tc5_commit(&sm.empty[vs]);
              if (j + 2 == cnt) tc5_commit(&sm.q_empty[w]);
            } else {
              mbar_arrive(&sm.turn[w ^ 1]);
              mbar_arrive(&sm.empty[vs]);
            }
            if (more) {
              if (j + 1 < cnt) tc5_commit(&sm.empty[st]);
              else mbar_arrive(&sm.empty[st]);
              next();
            }
          }
        }
        // the last commits' arrivals land before the CTA ends
        tc5_commit(&sm.drain[w]);
        if (!mbar_wait_bounded(&sm.drain[w], 0, kTcWaitLimit))
          record_error(p.c.status, kDevErrDrainTimeout);
      }
      __syncwarp();
    }
    if ((*state & 1) && lane == 0) record_error(p.c.status, kDevErrWaitTimeout);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // -------------------------------------------------------------- softmax
    const int w = warp >> 2, r = tid & 127;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp & 3) << 21);
    const uint32_t s_addr = lane_addr + 128 * w, o_addr = lane_addr + kO + 128 * w;
    const int tok = r / p.g, head = r - tok * p.g;
    const float2 sc2 = make_float2(p.scale, p.scale);
    unsigned s_used = 0, o_used = 0;
    bool ok = true;
    for (unsigned ni = 0; ok; ++ni) {
      const It* ip = take(ni);
      if (!(ok = ip != nullptr) || ip->stop) break;
      const int first_tile = ItemOf<PART>::first(ip);
      const bool pair = first_tile == kPair;
      const int shift = pair ? w * p.tokens : 0;
      const int ntok = min(p.tokens, ip->nrow - shift), my_n = ip->cnt[w];
      const int b = ip->b, h = ip->h, split = ip->split, k0 = ip->k0, k1 = ip->k1;
      const int seq_end = ItemOf<PART>::end(ip);
      const int at_first = ip->at0 + shift, row_first = ip->row0 + shift;
      const auto sp = ItemOf<PART>::span(ip);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.i_empty[ni % kItems]);
      if (ntok <= 0) continue;
      // the thread's row; rows past the tile's end work like its last token
      const bool valid = tok < ntok;
      const int at =                                          // (-1: before the first token)
          PART == kLine && seq_end >= 0
              ? position_of(p, b, seq_end, row_first + min(tok, ntok - 1))
              : max(at_first + min(tok, ntok - 1), -1);
      // key tiles [in0, in1), counted from k0, whose pages the warp's rows all see
      int in0, in1;
      {
        const int at_min = PART == kLine ? __reduce_min_sync(0xffffffffu, at)
                                         : __shfl_sync(0xffffffffu, at, 0);
        const int at_max = PART == kLine ? __reduce_max_sync(0xffffffffu, at)
                                         : __shfl_sync(0xffffffffu, at, 31);
        const int first = p.q.window == 0 ? 0 : max(at_max - p.q.window + kPage, 0) / kPage;
        const int v0 = sp.sink_blocks + max(first - sp.w0, 0);
        int v1 = sp.sink_blocks + (at_min + 1) / kPage - sp.w0;            // behind the last
        if (PART == kLine) v1 = min(v1, sp.blocks);
        in0 = (v0 + kKeyPages - 1) / kKeyPages - k0;
        in1 = max(v1, 0) / kKeyPages - k0;
      }
      // page v of the span: scores of the tokens that the row does not see to -inf.
      // It sees the columns [0, up); of them [from, ..) in the window, [0, sink) sinks.
      auto hide = [&](float* s, int v) {
        const int base = sp.block(v) * kPage;
        const int up = v >= sp.blocks || at < base ? 0 : min(at - base + 1, 32);
        const int from = p.q.window == 0 ? 0 : max(at - p.q.window + 1, 0) - base;
        const int sink = p.q.n_sink <= base ? 0 : min(p.q.n_sink - base, 32);
        const uint32_t below_up = up >= 32 ? 0xffffffffu : (1u << up) - 1;
        const uint32_t near = from <= 0 ? 0xffffffffu : from >= 32 ? 0u : 0xffffffffu << from;
        const uint32_t first = sink >= 32 ? 0xffffffffu : (1u << sink) - 1;
        const uint32_t see = below_up & (near | first);
        if (__all_sync(0xffffffffu, see == 0xffffffffu)) return;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!((see >> e) & 1u)) s[e] = -INFINITY;
      };
      // 64 scores to probabilities on the maximum in use, packed in place; their sum
      float m = -INFINITY, l = 0.0f;
      auto weigh = [&](uint32_t* sr) -> float {
        float* s = reinterpret_cast<float*>(sr);
        const float ms = m == -INFINITY ? 0.0f : m;
        const float2 m2 = make_float2(-ms, -ms);
        float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          float2 x = fma2(make_float2(s[e], s[e + 1]), sc2, m2);
          float2 y = fma2(make_float2(s[e + 2], s[e + 3]), sc2, m2);
          x = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
          sum0 = add2(sum0, x);
          sum1 = add2(sum1, y);
          sr[e / 2] = T::pack(x.x, x.y);
          sr[e / 2 + 1] = T::pack(y.x, y.y);
        }
        return (sum0.x + sum0.y) + (sum1.x + sum1.y);
      };
      for (int j = 0; j < my_n; ++j) {
        ok = tc5_wait(&sm.s_full[w], s_used & 1, state);
        if (!ok) break;
        tc5_fence_after();
        const int t = pair ? j : ((first_tile ^ w) & 1) + 2 * j;      // key tile of the item
        const bool inside = t >= in0 && t < in1;
        uint32_t sr[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tc5_ld32(sr + 32 * i, s_addr + 32 * i);
        tc5_wait_ld();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t* x = sr + 64 * i;
          const int v = (k0 + t) * kKeyPages + 2 * i;
          auto mask = [&] {
            if (inside) return;
            hide(reinterpret_cast<float*>(x), v);
            hide(reinterpret_cast<float*>(x) + 32, v + 1);
          };
          // the maximum of these scores where a row has none or outgrew it, and
          // l and O on it
          auto raise = [&] {
            const float* s = reinterpret_cast<const float*>(x);
            float mx0 = fmaxf(s[0], s[1]), mx1 = fmaxf(s[2], s[3]);
#pragma unroll
            for (int e = 4; e < 64; e += 4) {
              mx0 = fmaxf(mx0, fmaxf(s[e], s[e + 1]));
              mx1 = fmaxf(mx1, fmaxf(s[e + 2], s[e + 3]));
            }
            const float mx = fmaxf(mx0, mx1) * p.scale - Range<T>::kBelow;
            const bool grow = mx > m;         // true where m is -inf and mx is not
            const bool worked = valid && grow && m != -INFINITY;    // (else l and O are 0)
            const float a = worked ? fast_exp2(m - mx) : 1.0f;
            if (grow) m = mx;
            if (!__any_sync(0xffffffffu, worked)) return;
            l *= a;
            // S of this tile is there, so the products of the tiles before it are
            // complete; that of the first half may be under way
            if (i == 1) {
              ok = tc5_wait(&sm.h_full[w], s_used & 1, state);
              if (!ok) return;
              tc5_fence_after();
            }
            if (j > 0 || i == 1) {
#pragma unroll 1
              for (int k = 0; k < 4; ++k) {
                uint32_t o[32];
                tc5_ld32(o, o_addr + 32 * k);
                tc5_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                tc5_st32(o_addr + 32 * k, o);
              }
            }
          };
          mask();
          // (rows past the tile's end have no say: they hold the next sequence's
          // queries, or what was in shared memory)
          if (__any_sync(0xffffffffu, valid && m == -INFINITY)) raise();
          float sum = weigh(x);
          if (__any_sync(0xffffffffu, valid && sum > Range<T>::kMost)) {
            tc5_ld32(x, s_addr + 64 * i);
            tc5_ld32(x + 32, s_addr + 64 * i + 32);
            tc5_wait_ld();
            mask();
            raise();
            sum = weigh(x);
          }
          if (!ok) break;
          l += sum;
          tc5_st32(s_addr + 64 * i, x);
          tc5_wait_st();
          tc5_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[w][i]);
        }
        if (!ok) break;
        ++s_used;
      }

      // ------------------------------------------------------------ results
      if (PART == kLine && !pair && my_n == 0) {
        // the other query tile had the only tile of keys: nothing seen, outputs 0
        if (valid) {
          float* none = line_record(p, split, w == 1,
                                    (long long)(row_first + tok) * p.q.Hq + h * p.g + head, w * 128 + r);
          const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
          *reinterpret_cast<float2*>(none) = make_float2(-INFINITY, 0.0f);
#pragma unroll 1
          for (int e = 0; e < kD; e += 8) st_global32(none + kPartHead + e, zero);
        }
        continue;
      }
      if (ok && my_n > 0) ok = tc5_wait(&sm.o_full[w], o_used++ & 1, state);
      if (!ok) break;
      tc5_fence_after();
      const long long row = (long long)(row_first + tok) * p.q.Hq + h * p.g + head;
      const bool record = PART != kWhole || p.splits > 1;
      const float inv = record ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
      float odd = 0.0f, odd1 = 0.0f, odd2 = 0.0f, odd3 = 0.0f;   // NaN: a channel is open
      const int cut_row = w * 128;
      float* rec = PART == kLine ? line_record(p, split, !pair && w == 1, row, cut_row + r)
                                   : p.part + (row * p.splits + split) * rec_floats(PART);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[32];
        if (my_n > 0) {
          tc5_ld32(o, o_addr + 32 * i);
          tc5_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          odd = gather_open<T>(__uint_as_float(o[e]), odd);
          odd1 = gather_open<T>(__uint_as_float(o[e + 1]), odd1);
          odd2 = gather_open<T>(__uint_as_float(o[e + 2]), odd2);
          odd3 = gather_open<T>(__uint_as_float(o[e + 3]), odd3);
        }
        if (record) {
          if constexpr (PART == kWhole) {
            if (valid)
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<uint4*>(rec + 4 + 32 * i + e) =
                    make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else {
            if (valid)
#pragma unroll
              for (int e = 0; e < 32; e += 8) st_global32(rec + kPartHead + 32 * i + e, o + e);
          }
        } else {
          uint32_t v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = T::pack(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          if (valid) {
            uint32_t* d = reinterpret_cast<uint32_t*>(p.out + row * kD) + 16 * i;
            if (p.wide) {
              st_global32(d, v);
              st_global32(d + 8, v + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<uint4*>(d + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
          }
        }
      }
      tc5_fence_before();       // O has been read: the next item's products may follow
      odd += odd1 + odd2 + odd3;
      if (valid) {
        if (record) *reinterpret_cast<float2*>(rec) = make_float2(m, l);
        else if (p.lse) p.lse[row] = row_lse<T>(m, l);
      }
      // rows with open channels, by the whole warp; the other warps' waits do not
      // run out meanwhile
      __syncwarp();
      unsigned bad = __ballot_sync(0xffffffffu, valid && odd != odd && l == l);
      if (bad) {
        if (lane == 0) atomicAdd(&sm.state, kTcBusy);
        for (; bad; bad &= bad - 1) {
          const int src = __ffs(bad) - 1;
          redo_row<T, PART>(p, b, h, split, k0, k1, sp, __shfl_sync(0xffffffffu, row, src),
                            __shfl_sync(0xffffffffu, at, src), &sm.met[warp],
                            cut_row + (warp & 3) * 32 + src, first_tile, w);
        }
        if (lane == 0) atomicAdd(&sm.state, -kTcBusy);
      }
    }
    if (!ok && lane == 0) record_error(p.c.status, kDevErrWaitTimeout);
    tc5_fence_before();
  }
  __syncthreads();
  if (warp == kSoftmaxWarps) {
    tc5_fence_after();
    tc5_dealloc(tmem, 512);
  }
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 152;
  return sms;
}

// Upper bound on the work items of one KV head: every sequence's last may be partial.
long long attention_tiles(int B, int g, int total) {
  const int two = 2 * (128 / g);
  return (long long)total / two + B;
}

// Splits of the key tiles: so many that the CTAs fill the SMs about once, each
// with at least four key tiles.
int attention_splits(const Kv16& c, int Hq, int total, int max_tok, int window, int n_sink) {
  const int g = Hq / c.Hkv, two = 2 * (128 / g);
  const int sms = sm_count();
  const long long ctas = ((total + two - 1) / two + std::min(c.B, total) - 1LL) * c.Hkv;
  long long keys = std::min(max_tok, c.cap);
  if (window > 0) keys = std::min<long long>(keys, (long long)window + two + n_sink + 3 * kPage);
  const long long by_keys = keys / (4 * 128);
  return (int)std::max<long long>(1, std::min<long long>({sms / std::max(1LL, ctas), by_keys, 64}));
}

}  // namespace
}  // namespace oscar
