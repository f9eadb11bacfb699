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
struct Span {
  int sink_blocks, w0, blocks;
  KV16_BOTH Span() {}
  KV16_BOTH Span(int first, int last, int window, int n_sink) {
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

KV16_BOTH bool kv16_visible(int j, int at, int window, int n_sink) {
  return j <= at && (window == 0 || j > at - window || j < n_sink);
}

}  // namespace oscar
