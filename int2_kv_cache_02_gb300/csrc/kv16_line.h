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
// item, then some a tile, by what they took on the GPU (in 0.14 us; `pair`: a chunk
// that fills both query tiles).  Entry i below the number of groups is group i's
// prefix, the others are the sequences' own blocks behind it.  An entry has its
// rows KV head by KV head:
//  a sequence  chunk after chunk, each its own tiles (causal: a later chunk has
//              more)
//  a group     block after block of tiles, and within a block chunk after chunk.
//              A single chunk has one block, the whole row; several have blocks of
//              a run's length, so that the CTAs that work the same keys for
//              different chunks do so at the same time, and the keys come from HBM
//              once.
// A tile is the run's that has its first place.
KV16_CONST int row_cost(bool pair) { return pair ? 56 : 20; }
KV16_CONST int tile_cost(bool pair) { return pair ? 11 : 8; }
constexpr int kMinPlaces = 12;   // of a CTA's run: any within a row has a tile
KV16_BOTH int line_share(int places, int ctas) {
  const int per = places / ctas + (places % ctas != 0);
  return per > kMinPlaces ? per : kMinPlaces;
}
// The blocks of a group's rows of so many tiles: `count` of `least` tiles each, as
// long as a run or a little longer; the last has what is left too.
struct Blocks {
  int count, least, tiles;
  KV16_BOTH Blocks(int tiles, int chunks, bool pair, int per)
      : count(1), least(tiles), tiles(tiles) {
    const int run = (per + tile_cost(pair) - 1) / tile_cost(pair);
    if (chunks > 1 && tiles >= 2 * run) count = tiles / run, least = run;
  }
  KV16_BOTH int first(int i) const { return i < count ? i * least : tiles; }
};
// Place in its row where tile t begins (those of tile 0 with the row's own).
KV16_BOTH int tile_place(int t, bool pair) {
  return t == 0 ? 0 : row_cost(pair) + t * tile_cost(pair);
}
// Tiles that begin before place x of a row.
KV16_BOTH int tiles_before(int x, bool pair) {
  x -= row_cost(pair);
  return x <= 0 ? 0 : pair ? (x + tile_cost(true) - 1) / tile_cost(true)
                           : (x + tile_cost(false) - 1) / tile_cost(false);
}
// Places of a row of so many tiles.
KV16_BOTH int row_places(int tiles, bool pair) {
  return tiles > 0 ? row_cost(pair) + tiles * tile_cost(pair) : 0;
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
