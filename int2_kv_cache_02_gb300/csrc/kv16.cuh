// The 16-bit key/value cache (oscar_kv16_cache) as the kernels see it, and
// the device helpers that its operators share.
#pragma once

#include "common.cuh"
#include "kv16_span.h"
#include "launch.h"

namespace oscar {

// bf16 and fp16 as the element type of keys, values, queries and outputs.
struct Bf16 {
  static constexpr bool kHalf = false;
  static __device__ __forceinline__ float2 unpack(uint32_t u) { return bf16_pair(u); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};
struct Fp16 {
  static constexpr bool kHalf = true;
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(u32_as_half2(u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    return half2_as_u32(__floats2half2_rn(lo, hi));
  }
};

// Row number (in units of 128 elements) of the first token of a logical block
// of (b, h); -1 where the table names a page outside the pool.
__device__ __forceinline__ int kv16_block_row(const Kv16& c, int b, int h, int block) {
  if (!c.table) return (b * c.Hkv + h) * c.T_cap + block * kPage;
  const int page = __ldg(c.table + (long long)b * c.max_blocks + block);
  return (unsigned)page < (unsigned)c.n_pages ? (page * c.Hkv + h) * kPage : -1;
}

// A sequence's length, or -1 if it is outside [0, min(capacity, max_tok)].
__device__ __forceinline__ int kv16_length(const Kv16& c, int b, int max_tok) {
  const int n = c.n_tok[b];
  return n >= 0 && n <= c.cap && n <= max_tok ? n : -1;
}

// The sequence of row r of a ragged batch: the last b with start[b] <= r, or
// -1 if r is in no sequence's range.
__device__ __forceinline__ int ragged_sequence(const int32_t* start, int B, int r) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(start + mid) <= r) lo = mid; else hi = mid;
  }
  return __ldg(start + lo) <= r && r < __ldg(start + lo + 1) ? lo : -1;
}

// One query against the blocks [i0, i1) of a span, worked by a warp: the
// running maximum m (log2 domain) and sum l, and the unnormalised output of
// channels 4 lane .. 4 lane + 3.  fp32 throughout; a token that the query
// does not see is not touched, whatever its key and value hold.  Ends early,
// with m and l not complete, once every channel that `open` (a bit for each of
// the lane's four) asks for is NaN: nothing changes it any more.  The block that
// it ended with, or -1.
constexpr int kRowTokens = 8;    // tokens whose loads are in flight together
template <class T, class S>
__device__ __forceinline__ int kv16_warp_row(const Kv16& c, const uint16_t* q, int b, int h,
                                             int at, const S& sp, int i0, int i1, int window,
                                             int n_sink, float scale_log2, unsigned open,
                                             float& m, float& l, float (&o)[4]) {
  const int lane = threadIdx.x & 31;
  const uint2 qr = reinterpret_cast<const uint2*>(q)[lane];
  const float2 q0 = T::unpack(qr.x), q1 = T::unpack(qr.y);
  m = -INFINITY;
  l = 0.0f;
  o[0] = o[1] = o[2] = o[3] = 0.0f;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const int blk = sp.block(i), row = kv16_block_row(c, b, h, blk);
    if (row < 0) {
      if (lane == 0) record_error(c.status, kDevErrBadPaged);
      continue;
    }
    const unsigned see =
        __ballot_sync(0xffffffffu, kv16_visible(blk * kPage + lane, at, window, n_sink));
#pragma unroll 1
    for (int t0 = 0; t0 < kPage; t0 += kRowTokens) {
      const unsigned here = see >> t0;
      if ((here & ((1u << kRowTokens) - 1)) == 0) continue;
      uint2 kr[kRowTokens], vr[kRowTokens];
#pragma unroll
      for (int u = 0; u < kRowTokens; ++u) {
        const long long e = ((long long)row + t0 + u) * 32 + lane;
        kr[u] = vr[u] = make_uint2(0u, 0u);
        if ((here >> u) & 1u) {
          kr[u] = reinterpret_cast<const uint2*>(c.k)[e];
          vr[u] = reinterpret_cast<const uint2*>(c.v)[e];
        }
      }
      float s[kRowTokens], mn = m;
#pragma unroll
      for (int u = 0; u < kRowTokens; ++u) {
        const float2 k0 = T::unpack(kr[u].x), k1 = T::unpack(kr[u].y);
        s[u] = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1)
#pragma unroll
        for (int u = 0; u < kRowTokens; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], x);
#pragma unroll
      for (int u = 0; u < kRowTokens; ++u) {
        s[u] = (here >> u) & 1u ? s[u] * scale_log2 : -INFINITY;
        mn = fmaxf(mn, s[u]);
      }
      // a maximum of -inf has met only scores of -inf: they weigh nothing
      const float a = mn == -INFINITY ? 1.0f : fast_exp2(m - mn);
      m = mn;
      l *= a;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] *= a;
#pragma unroll
      for (int u = 0; u < kRowTokens; ++u) {
        const float p = s[u] == -INFINITY ? 0.0f : fast_exp2(s[u] - mn);
        const float2 v0 = T::unpack(vr[u].x), v1 = T::unpack(vr[u].y);
        l += p;
        o[0] += p * v0.x;
        o[1] += p * v0.y;
        o[2] += p * v1.x;
        o[3] += p * v1.y;
      }
    }
    bool settled = true;
#pragma unroll
    for (int x = 0; x < 4; ++x) settled &= !((open >> x) & 1u) || o[x] != o[x];
    if (__all_sync(0xffffffffu, settled)) return i;
  }
  return -1;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// log(sum exp) from a maximum in the log2 domain and a sum relative to it.
__device__ __forceinline__ float kv16_lse(float m, float l) {
  return l > 0.0f ? (m + __log2f(l)) * kLn2 : (l == 0.0f ? -INFINITY : l);
}

}  // namespace oscar
