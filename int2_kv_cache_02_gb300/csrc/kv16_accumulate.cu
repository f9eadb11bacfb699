// Attention weight of stored tokens under a ragged batch of queries, on the
// tcgen05 tensor cores: weight[j] += sum over rows i of 2^(scale s_ij - lse_i),
// a row being a (query, head of the group) pair.  The log of the sum is known,
// so nothing is kept per row and the value side is not read: 2 * 128 flops and
// one exponential per visible pair and head.
//
// Tiles.  S^T = K Q^T with 128 keys as the rows of a tile: a thread owns a key
// and adds up its row of S^T, so the column sum of the probabilities needs no
// exchange between threads and has one order.  A work item is 256 keys (two
// tiles, a warpgroup each) of one (sequence, KV head): its keys stay in shared
// memory while the query tiles (128 rows, token-major as in kv16_attention)
// that see any of them stream by, each used twice, 32 KB per 1024 tensor
// cycles.  With 128 keys per item the query tiles alone would take all of an
// SM's 64 B per cycle from L2.
//
// Fewer work items than two for every SM: 128 keys each, whose query tiles the
// two warpgroups take by turns.  One CTA per SM walks over the items, the
// next one's keys on their way while it works.  Fewer items than SMs: their
// query tiles are cut over a cluster's CTAs, which hand their sums to the first
// through distributed shared memory, added in order of rank.
//
// Roles (12 warps): two warpgroups that sum, one warp that copies, one that
// issues the MMAs, two that lay out the query rows' lse.  TMEM: two buffers of
// S^T for each warpgroup.
//
// Measured (GB300): the last 128 queries of four 7K to 16K-token sequences, 32/8
// heads, 65 us (floor 27); all queries of two prompts of 4K tokens, 32/4
// heads, 129 us (floor 68).  Bound by the summing warps: 525 cycles of
// exponentials per tile of S^T on each quarter of an SM, 950 with the waits, the
// loads from TMEM and those of lse, against 512 of the tensor cores.  Four
// warpgroups with a buffer each were slower (148 us), as was fetching the next
// tile's scores under the sums of this one (178 us).
#include <algorithm>
#include <type_traits>

#include "kv16.cuh"
#include "kv16_tma.h"
#include "tc5.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 384;
constexpr int kTileBytes = 32768, kHalf = 16384;
constexpr int kQStages = 3, kKBufs = 2, kLseSlots = 2;
constexpr int kItemKeys = 256;     // at most

struct AccParams {
  Kv16 c;
  Kv16Query q;
  const float* lse;
  int n_obs, g, tokens;
  int keys;         // keys of a work item: 256 or 128
  int items;        // key blocks * B * Hkv
  int cluster;      // CTAs that share an item
};

struct Smem {
  uint64_t k_full[kKBufs], k_empty[kKBufs], q_full[kQStages], q_empty[kQStages];
  uint64_t s_full[2][2], s_empty[2][2], l_full[2][kLseSlots], l_empty[2][kLseSlots], c_full, c_empty, drain;
  uint32_t tmem;
  int state;           // of the waits
  alignas(16) float lse[2][kLseSlots][128];   // per warpgroup; at the end: the CTA's sums
  float part[128];                         // one warpgroup's sums of a lone key tile
};
static_assert(2 * kLseSlots * 128 >= kItemKeys, "room for the sums");

// A work item as every role sees it; t1 <= t0: nothing to do.
struct Item {
  int b, h, key0, n;
  int r0, at_first;   // first row of the sequence's queries, its position
  int ia, ib;         // its queries that may see a key of the item
  int t0, t1;         // this CTA's query tiles of them
  int halves;         // key tiles that hold tokens: a warpgroup each, or one for both,
                      // which take its query tiles by turns
};

__device__ __forceinline__ Item find_item(const AccParams& p, int x, int rank, bool report) {
  Item it;
  it.t0 = it.t1 = 0;
  it.halves = 0;
  if (x >= p.items) return it;
  const int rows = p.c.B * p.c.Hkv;
  const int kb = x / rows, row = x - kb * rows;     // the first keys have the most queries
  it.b = row / p.c.Hkv;
  it.h = row - it.b * p.c.Hkv;
  it.key0 = kb * p.keys;
  const int n = __ldg(p.c.n_tok + it.b);
  const int r0 = __ldg(p.q.start + it.b), r1 = __ldg(p.q.start + it.b + 1), nq = r1 - r0;
  it.n = n;
  it.r0 = r0;
  if (n < 0 || n > p.c.cap || n > p.q.max_tok || r0 < 0 || r1 > p.q.total || nq < 0 || nq > n) {
    if (report && kb == 0) record_error(p.c.status, kDevErrBadPaged);
    return it;
  }
  if (it.key0 >= n) return it;
  it.at_first = n - nq;
  it.ia = max(max(0, it.key0 - it.at_first), p.n_obs > 0 ? nq - p.n_obs : 0);
  it.ib = nq;
  const int last = min(it.key0 + p.keys, n) - 1;
  if (p.q.window > 0 && it.key0 >= p.q.n_sink)
    it.ib = (int)min((long long)nq, (long long)last + p.q.window - it.at_first);
  if (it.ib <= it.ia) return it;
  const int nt = (it.ib - it.ia + p.tokens - 1) / p.tokens;
  it.t0 = (int)((long long)nt * rank / p.cluster);
  it.t1 = (int)((long long)nt * (rank + 1) / p.cluster);
  it.halves = p.keys == 256 && n - it.key0 > 128 ? 2 : 1;
  return it;
}

template <class T>
__global__ void __launch_bounds__(kThreads, 1)
kv16_accumulate_kernel(const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k, const AccParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % p.cluster, first = blockIdx.x / p.cluster;
  // item of a round, or -1: rounds in turn forwards and backwards, so that a CTA
  // with the longest of one round gets the shortest of the next
  const int step = gridDim.x / p.cluster;
  auto item_of = [&](int round) -> int {
    if ((long long)round * step >= p.items) return -1;
    const long long x = (long long)round * step + ((round & 1) ? step - 1 - first : first);
    return x < p.items ? (int)x : p.items;
  };
  Smem& sm = *reinterpret_cast<Smem*>(smem + (kKBufs * 2 + kQStages) * kTileBytes);
  uint8_t* kbuf = smem;                                    // [kKBufs][2] key tiles
  uint8_t* qring = smem + kKBufs * 2 * kTileBytes;         // [kQStages] query tiles

  if (smem_u32(smem) & 1023) {                             // the swizzle counts on it
    if (tid == 0) record_error(p.c.status, kDevErrWaitTimeout);
    return;
  }

  if (warp == 8) tc5_alloc(&sm.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < kKBufs; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
    }
    for (int w = 0; w < 2; ++w)
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.s_full[w][i], 1);
        mbar_init(&sm.s_empty[w][i], 4);
      }
    for (int w = 0; w < 2; ++w)
      for (int i = 0; i < kLseSlots; ++i) {
        mbar_init(&sm.l_full[w][i], 1);
        mbar_init(&sm.l_empty[w][i], 4);
      }
    mbar_init(&sm.c_full, 4);
    mbar_init(&sm.c_empty, 4);
    mbar_init(&sm.drain, 1);
    mbar_fence_init();
    sm.state = 0;
  }
  float sum = 0.0f;      // of the thread's key
  // query rows that no copy fills (groups that do not divide 128) hold zeros
  const int pad = 128 - p.g * p.tokens;
  for (int i = tid; i < kQStages * 2 * pad * 8; i += kThreads) {
    const int tile = i / (pad * 8), rest = i - tile * pad * 8;
    reinterpret_cast<uint4*>(qring + tile * kHalf + (p.g * p.tokens) * 128)[rest] =
        make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const uint32_t tmem = sm.tmem;
  volatile int* state = &sm.state;
  bool ok = true;

  if (warp == 8) {
    // -------------------------------------------------------------- copies
    const int none = p.c.table ? p.c.n_pages * p.c.Hkv * kPage
                               : p.c.B * p.c.Hkv * p.c.T_cap;        // reads zeros
    int uk = 0, uq = 0;
    for (int round = 0; ok && item_of(round) >= 0; ++round) {
      const Item it = find_item(p, item_of(round), rank, rank == 0 && lane == 0);
      if (it.t1 <= it.t0) continue;
      int row = none;
      if (lane < 8) {
        const int blk = it.key0 / kPage + lane;
        if (blk * kPage < it.n) {
          row = kv16_block_row(p.c, it.b, it.h, blk);
          if (row < 0) {
            record_error(p.c.status, kDevErrBadPaged);
            row = none;
          }
        }
      }
      const int kb = uk % kKBufs;
      if (uk >= kKBufs) ok = tc5_wait(&sm.k_empty[kb], (uk / kKBufs - 1) & 1, state);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[kb], it.halves * kTileBytes);
      __syncwarp();
      if (lane < 4 * it.halves) {          // a lane per page
        uint8_t* dst = kbuf + (kb * 2 + lane / 4) * kTileBytes + (lane & 3) * 4096;
        tma_box2(dst, &map_k, 0, row, &sm.k_full[kb]);
        tma_box2(dst + kHalf, &map_k, 64, row, &sm.k_full[kb]);
      }
      __syncwarp();
      ++uk;
      for (int t = it.t0; t < it.t1; ++t) {
        const int st = uq % kQStages;
        if (uq >= kQStages) ok = tc5_wait(&sm.q_empty[st], (uq / kQStages - 1) & 1, state);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full[st], 2 * 64 * 2 * p.g * p.tokens);
          uint8_t* dst = qring + st * kTileBytes;
          tma_box3(dst, &map_q, 0, it.h * p.g, it.r0 + it.ia + t * p.tokens, &sm.q_full[st]);
          tma_box3(dst + kHalf, &map_q, 64, it.h * p.g, it.r0 + it.ia + t * p.tokens, &sm.q_full[st]);
        }
        __syncwarp();
        ++uq;
      }
    }
    if (!ok && lane == 0) record_error(p.c.status, kDevErrWaitTimeout);
    // what is in flight lands before the memory is given back, whoever gives up
    for (int i = max(0, uk - kKBufs); i < uk; ++i)
      if (!mbar_wait_bounded(&sm.k_full[i % kKBufs], (i / kKBufs) & 1, kDrainLimit) && lane == 0)
        record_error(p.c.status, kDevErrDrainTimeout);
    for (int i = max(0, uq - kQStages); i < uq; ++i)
      if (!mbar_wait_bounded(&sm.q_full[i % kQStages], (i / kQStages) & 1, kDrainLimit) && lane == 0)
        record_error(p.c.status, kDevErrDrainTimeout);
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMAs
    if (elect_one()) {
      const uint32_t idesc = tc5_idesc(T::kHalf, 128, 128, false, false);
      constexpr uint64_t kBase = tc5_desc_base(16, 1024);
      const uint64_t dk = tc5_desc(kBase, smem_u32(kbuf)), dq = tc5_desc(kBase, smem_u32(qring));
      unsigned kb = 0, kp = 0, st = 0, sp = 0, us[2] = {0, 0};
      for (int round = 0; ok && item_of(round) >= 0; ++round) {
        const Item it = find_item(p, item_of(round), rank, false);
        if (it.t1 <= it.t0) continue;
        ok = tc5_wait(&sm.k_full[kb], kp, state);
        for (int t = it.t0; t < it.t1 && ok; ++t) {
          ok = tc5_wait(&sm.q_full[st], sp, state);
          const uint64_t q = dq + st * (kTileBytes >> 4);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (!ok || (it.halves == 1 && ((t - it.t0) & 1) != w)) continue;
            const unsigned buf = us[w] & 1;
            if (us[w] >= 2) ok = tc5_wait(&sm.s_empty[w][buf], (us[w] / 2 - 1) & 1, state);
            if (!ok) continue;
            tc5_fence_after();
            const uint64_t k = dk + (kb * 2 + (it.halves == 2 ? w : 0)) * (kTileBytes >> 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const unsigned off = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
              tc5_mma_ss(tmem + 256 * w + 128 * buf, k + off, q + off, idesc, i > 0);
            }
            tc5_commit(&sm.s_full[w][buf]);
            ++us[w];
          }
          if (ok) tc5_commit(&sm.q_empty[st]);
          if (++st == kQStages) {
            st = 0;
            sp ^= 1;
          }
        }
        if (ok) tc5_commit(&sm.k_empty[kb]);
        if (++kb == kKBufs) {
          kb = 0;
          kp ^= 1;
        }
      }
      // the last commits' arrivals land before the CTA ends
      if (!ok) record_error(p.c.status, kDevErrWaitTimeout);
      tc5_commit(&sm.drain);
      if (!mbar_wait_bounded(&sm.drain, 0, kTcWaitLimit))
        record_error(p.c.status, kDevErrDrainTimeout);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ------------------------------ lse of the rows, a warp for each warpgroup
    const int w = warp - 10;
    int tok[4], col[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = lane + 32 * k;
      tok[k] = r / p.g;
      col[k] = r - tok[k] * p.g;
    }
    unsigned ul = 0;
    for (int round = 0; ok && item_of(round) >= 0; ++round) {
      const Item it = find_item(p, item_of(round), rank, false);
      const int by = it.halves == 1 ? 2 : 1;
      float v[4], next[4];
      auto load = [&](int t, float (&x)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int q = it.ia + t * p.tokens + tok[k];
          x[k] = tok[k] < p.tokens && q < it.ib
                     ? -kLog2e * __ldg(p.lse + (long long)(it.r0 + q) * p.q.Hq + it.h * p.g + col[k])
                     : -INFINITY;
        }
      };
      int t = it.t0 + (by == 2 ? w : 0);
      if (t < it.t1) load(t, v);
      for (; t < it.t1; t += by) {
        if (t + by < it.t1) load(t + by, next);      // on its way while this one waits
        const unsigned slot = ul % kLseSlots;
        if (ul >= kLseSlots) ok = tc5_wait(&sm.l_empty[w][slot], (ul / kLseSlots - 1) & 1, state);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sm.lse[w][slot][lane + 32 * k] = v[k];
          v[k] = next[k];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.l_full[w][slot]);
        ++ul;
      }
    }
    if (!ok && lane == 0) record_error(p.c.status, kDevErrWaitTimeout);
  } else {
    // ---------------------------------------------------------------- sums
    const int w = warp >> 2;
    const uint32_t s_base = tmem + ((uint32_t)(warp & 3) << 21) + 256 * w;
    const float2 sc = make_float2(p.q.scale_log2, p.q.scale_log2);
    unsigned ul = 0, us = 0, lone = 0;
    for (int round = 0; ok && item_of(round) >= 0; ++round) {
      const Item it = find_item(p, item_of(round), rank, false);
      if (it.t1 <= it.t0) continue;
      const int tile0 = it.key0 + (it.halves == 2 ? 128 * w : 0), j = tile0 + (tid & 127);
      float2 a0 = make_float2(0.0f, 0.0f), a1 = a0;
      const int by = it.halves == 1 ? 2 : 1;
      for (int t = it.t0 + (by == 2 ? w : 0); t < it.t1; t += by) {
        const unsigned slot = ul % kLseSlots, buf = us & 1;
        ok = tc5_wait(&sm.l_full[w][slot], (ul / kLseSlots) & 1, state) &&
             tc5_wait(&sm.s_full[w][buf], (us / 2) & 1, state);
        if (!ok) break;
        tc5_fence_after();
        // the tokens [lo, hi) of the tile that see the thread's key: rows are
        // token-major, so they are columns [lo g, hi g)
        const int q_lo = it.ia + t * p.tokens, ntok = min(p.tokens, it.ib - q_lo);
        const int at = it.at_first + q_lo;
        const int lo = max(0, j - at);
        int hi = ntok;
        if (p.q.window > 0 && j >= p.q.n_sink)
          hi = (int)min((long long)hi, max(0LL, (long long)j + p.q.window - at));
        const bool whole = __all_sync(0xffffffffu, lo == 0 && hi == p.tokens);
        const int clo = min(lo, 128) * p.g;
        const unsigned cn = max(hi - lo, 0) * p.g;
        const float* ls = sm.lse[w][slot];
        const uint32_t sa = s_base + 128 * buf;
        // 64 columns; tiles that every row of sees every key take the short way
        auto add = [&](auto all, const uint32_t* s, int c0) {
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const float4 z = *reinterpret_cast<const float4*>(ls + c0 + e);
            float2 u = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc,
                            make_float2(z.x, z.y));
            float2 v = fma2(make_float2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), sc,
                            make_float2(z.z, z.w));
            u = make_float2(fast_exp2(u.x), fast_exp2(u.y));
            v = make_float2(fast_exp2(v.x), fast_exp2(v.y));
            if constexpr (!decltype(all)::value) {
              const int c = c0 + e - clo;
              u.x = (unsigned)c < cn ? u.x : 0.0f;
              u.y = (unsigned)(c + 1) < cn ? u.y : 0.0f;
              v.x = (unsigned)(c + 2) < cn ? v.x : 0.0f;
              v.y = (unsigned)(c + 3) < cn ? v.y : 0.0f;
            }
            a0 = add2(a0, u);
            a1 = add2(a1, v);
          }
        };
        auto tile = [&](auto all) {
          // all columns at once: loads left in flight under the sums slow them down
          uint32_t x[128];
#pragma unroll
          for (int i = 0; i < 4; ++i) tc5_ld32(x + 32 * i, sa + 32 * i);
          tc5_wait_ld();
          tc5_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.s_empty[w][buf]);
          add(all, x, 0);
          add(all, x + 64, 64);
        };
        if (whole) tile(std::true_type());
        else tile(std::false_type());
        ++us;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.l_empty[w][slot]);
        ++ul;
      }
      sum = (a0.x + a0.y) + (a1.x + a1.y);
      if (p.cluster > 1 || !ok) continue;
      if (it.halves == 1) {
        // both warpgroups have a part: the second hands its over
        if (w == 1) {
          if (lone > 0) ok = tc5_wait(&sm.c_empty, (lone - 1) & 1, state);
          if (!ok) break;
          sm.part[tid & 127] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.c_full);
        } else {
          ok = tc5_wait(&sm.c_full, lone & 1, state);
          if (!ok) break;
          sum += sm.part[tid];
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.c_empty);
        }
        ++lone;
        if (w == 1) continue;
      }
      if (j < it.n) {
        const int row = kv16_block_row(p.c, it.b, it.h, j / kPage);
        if (row >= 0) p.c.weight[(long long)row + j % kPage] += sum;
      }
    }
    if (!ok && lane == 0) record_error(p.c.status, kDevErrWaitTimeout);
    tc5_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tc5_fence_after();
    tc5_dealloc(tmem, 512);
  }
  if (p.cluster > 1) {
    // one item per cluster: its sums in order of rank
    float* sums = sm.lse[0][0];
    if (tid < kItemKeys) sums[tid] = sum;
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && tid < kItemKeys && first < p.items) {
      const Item it = find_item(p, first, 0, false);
      const int j = it.key0 + tid;
      if (it.halves > 0 && j < it.n && tid < p.keys) {
        float all = 0.0f;
        for (int r = 0; r < p.cluster; ++r)
          for (int i = tid; i < kItemKeys; i += it.halves == 2 ? kItemKeys : 128) {
            unsigned far;
            float v;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(far) : "r"(smem_u32(sums + i)), "r"(r));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(far) : "memory");
            all += v;
          }
        const int row = kv16_block_row(p.c, it.b, it.h, j / kPage);
        if (row >= 0) p.c.weight[(long long)row + j % kPage] += all;
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <class T>
cudaError_t launch(AccParams p, cudaStream_t s) {
  CUtensorMap mq, mk;
  if (!kv16_query_map(&mq, p.q, p.c.half, p.g, p.tokens) || !kv16_row_map(&mk, p.c, p.c.k))
    return cudaErrorNotSupported;
  int dev = 0, sms = 152;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // items of 256 keys where there are two for every SM, else of 128; where even
  // those are fewer than the SMs, clusters share them, at four query tiles or
  // more for every CTA
  const long long rows = p.n_obs > 0 ? std::min<long long>(p.q.total, (long long)p.n_obs * p.c.B)
                                     : p.q.total;
  const long long tiles = std::max(1LL, rows / p.c.B / p.tokens);
  const int most = std::min(p.q.max_tok, p.c.cap);
  auto items = [&](int keys) { return ((long long)most + keys - 1) / keys * p.c.B * p.c.Hkv; };
  p.keys = items(256) >= 2 * sms ? 256 : 128;
  if (items(p.keys) > 0x3fffffffLL) return cudaErrorInvalidValue;
  p.items = (int)items(p.keys);
  p.cluster = 1;
  while (p.cluster < 8 && (long long)p.items * p.cluster < sms && tiles >= 8 * p.cluster)
    p.cluster *= 2;
  const auto kernel = kv16_accumulate_kernel<T>;
  constexpr int smem = (kKBufs * 2 + kQStages) * kTileBytes + (int)sizeof(Smem);
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.cluster > 1 ? p.items * p.cluster : std::min(p.items, sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, mq, mk, p);
}

}  // namespace

cudaError_t launch_kv16_accumulate(const Kv16& c, const Kv16Query& q, const float* lse, int n_obs,
                                   cudaStream_t s) {
  AccParams p;
  p.c = c;
  p.q = q;
  p.lse = lse;
  p.n_obs = n_obs;
  p.g = q.Hq / c.Hkv;
  p.tokens = 128 / p.g;
  return c.half ? launch<Fp16>(p, s) : launch<Bf16>(p, s);
}

}  // namespace oscar
