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

}  // namespace oscar
