// Which tokens of the 16-bit cache a query sees, in whole numbers only: the
// kernels use it, and it also compiles as plain C++.
#pragma once

#include <algorithm>

#include "../../include/oscar.h"

#ifdef __CUDACC__
#define KV16_BOTH __host__ __device__ __forceinline__
#else
#define KV16_BOTH inline
#endif

namespace oscar {

constexpr int kPage = OSCAR_GROUP;   // tokens of one page

// The tokens that queries at positions [first, last] of one sequence can see:
// whole blocks, the sinks' (sink_blocks of them from block 0) and then the
// window's (from block w0), numbered 0 .. blocks - 1.  Positions below 0 (a
// sequence of fewer tokens than queries) see nothing; windows go up to 2^31 - 1.
// (The constructor without arguments is there for the prompt attention's work items:
// where they have none, copies of an item cost it 2.5 %.)
struct WholeSpan {
  int sink_blocks, w0, blocks;
  KV16_BOTH WholeSpan() {}
  KV16_BOTH WholeSpan(int first, int last, int window, int n_sink) {
    if (last < 0) {
      sink_blocks = w0 = blocks = 0;
      return;
    }
    const int lo = window > 0 ? std::max(0, std::max(first, 0) - window + 1) : 0;
    const int end = (last + kPage) / kPage;    // blocks up to the last position
    w0 = lo / kPage;
    sink_blocks =
        std::min((int)(((long long)std::min(n_sink, last + 1) + kPage - 1) / kPage), w0);
    blocks = sink_blocks + end - w0;
  }
  KV16_BOTH int block(int i) const { return i < sink_blocks ? i : w0 + i - sink_blocks; }
};

// The same or a part of them, in which the sinks' blocks begin with s0.  (Without s0
// a part from among the sinks on had the hidden blocks behind them too: 16 sequences
// of 32K tokens, window 128, 100 sinks, a shared prefix of 64, 346 us instead of 18.)
struct Span : WholeSpan {
  int s0;
  KV16_BOTH Span() {}
  KV16_BOTH Span(const WholeSpan& s, int s0) : WholeSpan(s), s0(s0) {}
  KV16_BOTH Span(int first, int last, int window, int n_sink)
      : WholeSpan(first, last, window, n_sink), s0(0) {}
  KV16_BOTH int block(int i) const { return WholeSpan::block(i) + (i < sink_blocks ? s0 : 0); }

  // Of these blocks (all of them), those below n.
  KV16_BOTH Span below(int n) const {
    Span s;
    s.s0 = 0;
    s.sink_blocks = std::min(sink_blocks, n);
    s.w0 = w0;
    s.blocks = s.sink_blocks + std::max(0, std::min(w0 + blocks - sink_blocks, n) - w0);
    return s;
  }
  // Those from n on.
  KV16_BOTH Span from(int n) const {
    Span s;
    s.s0 = std::min(n, sink_blocks);
    s.sink_blocks = sink_blocks - s.s0;
    s.w0 = std::max(w0, n);
    s.blocks = s.sink_blocks + std::max(0, w0 + blocks - sink_blocks - s.w0);
    return s;
  }
};

KV16_BOTH bool kv16_visible(int j, int at, int window, int n_sink) {
  return j <= at && (window == 0 || j > at - window || j < n_sink);
}

}  // namespace oscar
