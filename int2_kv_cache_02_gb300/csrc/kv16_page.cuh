// A page of the 16-bit cache against the group's queries, by a warp with
// mma.sync: what the decode's kernels do with each page.
#pragma once

#include "kv16.cuh"

namespace oscar {

constexpr int kSlotBytes = 4 * 4096;     // a page: K and V, two halves of 64 channels each
constexpr float kBelow = 14.0f;          // fp16: the maximum in use is 2^14 below the largest

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <class T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (T::kHalf)
    mma_16816_acc(d, a, b0, b1);
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The group's queries as A operands: rows are heads, padding rows zero.
__device__ __forceinline__ void page_queries(uint32_t (&qa)[8][4], const uint16_t* q, int g) {
  const int lane = threadIdx.x & 31, hr = lane >> 2, hc = 2 * (lane & 3);
#pragma unroll
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int head = hr + 8 * (i & 1), ch = 16 * k + hc + 8 * (i >> 1);
      qa[k][i] = head < g ? __ldg(reinterpret_cast<const uint32_t*>(q + head * kD + ch)) : 0u;
    }
}

// The page in `slot` (its first token j0; 128-byte swizzle, in shared memory)
// against the query at position `at`: scores, the running maximum m (log2
// domain) and sum l (a lane's share of it), o += P V.  Thread layout of the
// accumulators: rows lane / 4 and + 8, columns 2 (lane % 4) of each 8.
// on_scores gets the masked scores.  Clears the values of hidden tokens in the
// slot, and then returns false: the whole page is not visible.
template <class T, class F>
__device__ __forceinline__ bool page_step(uint8_t* slot, int j0, int at, int window, int n_sink,
                                          float scale_log2, const uint32_t (&qa)[8][4],
                                          float (&o)[16][4], float (&m)[2], float (&l)[2],
                                          F&& on_scores) {
  const int lane = threadIdx.x & 31, hc = 2 * (lane & 3);
  const bool whole = j0 + kPage - 1 <= at &&
                     (window == 0 || j0 > at - window || j0 + kPage <= n_sink);
  if (!whole) {
    // a hidden token's value must not meet its zero probability: clear it
    const int j = j0 + lane;
    if (!kv16_visible(j, at, window, n_sink)) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        reinterpret_cast<uint4*>(slot + 8192 + (i >> 3) * 4096 + lane * 128)[i & 7] =
            make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
  }
  // S: 16 heads x 32 tokens
  float sc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.0f;
  const unsigned sa = smem_u32(slot);
  const int mrow = lane & 7, mid = lane >> 3;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // 8x8 tiles: channels 16k, 16k + 8 of tokens t, t + 8
    const int chunk = 2 * (k & 3) + (mid & 1);
    const unsigned a = sa + (k >> 2) * 4096 + ((mid >> 1) * 8 + mrow) * 128 + ((chunk ^ mrow) << 4);
    uint32_t b0[4], b1[4];
    ldsm4(b0, a);
    ldsm4(b1, a + 16 * 128);
    mma<T>(sc[0], qa[k], b0[0], b0[1]);
    mma<T>(sc[1], qa[k], b0[2], b0[3]);
    mma<T>(sc[2], qa[k], b1[0], b1[1]);
    mma<T>(sc[3], qa[k], b1[2], b1[3]);
  }
  float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = sc[i][e] * scale_log2;
      if (!whole && !kv16_visible(j0 + 8 * i + hc + (e & 1), at, window, n_sink))
        v = -INFINITY;
      sc[i][e] = v;
      mx[e >> 1] = fmaxf(mx[e >> 1], v);
    }
  on_scores(sc);
  bool grew = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
    mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
    if (T::kHalf) mx[i] -= kBelow;
    grew |= mx[i] > m[i];
  }
  if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mn = fmaxf(m[i], mx[i]);
      const float a = mn == -INFINITY ? 1.0f : fast_exp2(m[i] - mn);
      m[i] = mn;
      l[i] *= a;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        o[n][2 * i] *= a;
        o[n][2 * i + 1] *= a;
      }
    }
  }
  const float ms[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
  uint32_t pa[2][4], pb[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p0 = fast_exp2(sc[i][0] - ms[0]), p1 = fast_exp2(sc[i][1] - ms[0]);
    const float p2 = fast_exp2(sc[i][2] - ms[1]), p3 = fast_exp2(sc[i][3] - ms[1]);
    l[0] += p0 + p1;
    l[1] += p2 + p3;
    const uint32_t h0 = T::pack(p0, p1), h1 = T::pack(p2, p3);
    const float2 u0 = T::unpack(h0), u1 = T::unpack(h1);
    pa[i >> 1][2 * (i & 1)] = h0;
    pa[i >> 1][2 * (i & 1) + 1] = h1;
    pb[i >> 1][2 * (i & 1)] = T::pack(p0 - u0.x, p1 - u0.y);
    pb[i >> 1][2 * (i & 1) + 1] = T::pack(p2 - u1.x, p3 - u1.y);
  }
  // O += P V: 8x8 tiles, transposed on the way: tokens t, t + 8 of channels c, c + 8
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int chunk = 2 * (n & 3) + (mid >> 1);
    const unsigned a = sa + 8192 + (n >> 2) * 4096 + ((mid & 1) * 8 + mrow) * 128 +
                       ((chunk ^ mrow) << 4);
    uint32_t b0[4], b1[4];
    ldsm4t(b0, a);
    ldsm4t(b1, a + 16 * 128);
    mma<T>(o[2 * n], pa[0], b0[0], b0[1]);
    mma<T>(o[2 * n + 1], pa[0], b0[2], b0[3]);
    mma<T>(o[2 * n], pa[1], b1[0], b1[1]);
    mma<T>(o[2 * n + 1], pa[1], b1[2], b1[3]);
    mma<T>(o[2 * n], pb[0], b0[0], b0[1]);
    mma<T>(o[2 * n + 1], pb[0], b0[2], b0[3]);
    mma<T>(o[2 * n], pb[1], b1[0], b1[1]);
    mma<T>(o[2 * n + 1], pb[1], b1[2], b1[3]);
  }
  return whole;
}

}  // namespace oscar
