// The line of work of the attention over shared prefixes, in whole numbers only:
// the kernels use it, and it also compiles as plain C++.
#pragma once

#include "kv16_span.h"

#ifdef __CUDACC__
#define KV16_CONST __host__ __device__ constexpr
#else
#define KV16_CONST constexpr
#endif

namespace oscar {

// The work of a call stands in one line, and each of `ctas` CTAs takes an equal run
// of it.  A row of the line is one chunk of up to 256 query rows and one KV head
// against its tiles of 128 keys: some places for what it costs to begin and end an
// item, then some a tile, by what they took on the GPU (in 0.14 us).  Entry i below
// the number of groups is group i's prefix, the others are the sequences' own blocks
// behind it.  An entry has its rows KV head by KV head:
//  a sequence  chunk after chunk, each its own tiles (causal: a later chunk has
//              more)
//  a group     block after block of tiles, and within a block chunk after chunk.
//              A single chunk has one block, the whole row; several have blocks of
//              a run's length, so that the CTAs that work the same keys for
//              different chunks do so at the same time, and the keys come from HBM
//              once.
// A tile is the run's that has its first place.
// The kind of a row has bit 0 if its chunk fills both query tiles, and bit 1 if it is a
// group's under a window: its sequences' windows begin at different tokens, so its
// tiles are masked row by row, which takes longer.  The costs are by the CTAs' ends in
// seven calls of 26 to 160 us (with 20 and 56 for the rows, 8 and 11 for the tiles, 16
// and 22 masked, CTAs ended up to 30 us apart: 128 requests about two documents 155 us
// instead of 148, drafts of 32 samples 90 instead of 84; 36 other calls of 26 to 1180
// us took 1.2 % longer on average).
constexpr int kRow = 28, kPairRow = 48;
constexpr int kTile = 10, kPairTile = 13, kMaskedTile = 16, kMaskedPairTile = 22;
KV16_CONST int row_cost(int kind) { return kind & 1 ? kPairRow : kRow; }
KV16_CONST int tile_cost(int kind) {
  return kind & 2 ? (kind & 1 ? kMaskedPairTile : kMaskedTile) : kind & 1 ? kPairTile : kTile;
}
// Whole tiles in so many places (the divisors are constants: quick).
KV16_CONST int whole_tiles(int x, int kind) {
  return kind & 2 ? (kind & 1 ? x / kMaskedPairTile : x / kMaskedTile)
                  : (kind & 1 ? x / kPairTile : x / kTile);
}
constexpr int kMostTileCost = tile_cost(3);
constexpr int kMinPlaces = kMostTileCost;   // of a CTA's run: any within a row has a tile
KV16_BOTH int line_share(int places, int ctas) {
  const int per = places / ctas + (places % ctas != 0);
  return per > kMinPlaces ? per : kMinPlaces;
}
// The blocks of a group's rows of so many tiles: `count` of `least` tiles each, as
// long as a run or a little longer; the last has what is left too.
struct Blocks {
  int count, least, tiles;
  KV16_BOTH Blocks(int tiles, int chunks, int kind, int per)
      : count(1), least(tiles), tiles(tiles) {
    const int run = whole_tiles(per + tile_cost(kind) - 1, kind);
    if (chunks > 1 && tiles >= 2 * run) count = tiles / run, least = run;
  }
  KV16_BOTH int first(int i) const { return i < count ? i * least : tiles; }
};
// Place in its row where tile t begins (those of tile 0 with the row's own).
KV16_BOTH int tile_place(int t, int kind) {
  return t == 0 ? 0 : row_cost(kind) + t * tile_cost(kind);
}
// Tiles that begin before place x of a row.
KV16_BOTH int tiles_before(int x, int kind) {
  x -= row_cost(kind);
  return x <= 0 ? 0 : whole_tiles(x + tile_cost(kind) - 1, kind);
}
// Places of a row of so many tiles.
KV16_BOTH int row_places(int tiles, int kind) {
  return tiles > 0 ? row_cost(kind) + tiles * tile_cost(kind) : 0;
}

// The CTAs [c0, c0 + n) that have tiles of a block whose first tile is at place `at`
// of the line and whose last is `more` places on.
struct Runs {
  int c0, n;
};
KV16_BOTH Runs runs_of(unsigned at, unsigned more, unsigned per, int ctas) {
  const int c0 = std::min((int)(at / per), ctas - 1);
  return Runs{c0, std::min((int)((at + more) / per), ctas - 1) - c0 + 1};
}
// A block is no shorter than a run and shorter than two: three runs at most.
constexpr int kBlockRuns = 3;

}  // namespace oscar
