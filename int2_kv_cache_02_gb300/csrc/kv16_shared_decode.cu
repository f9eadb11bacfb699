// The decode's own part under shared prefixes: one query per sequence against
// the pages behind its group's shared blocks, a stream bound by HBM.
//
// The pages of all (sequence, KV head) rows stand in one line, row after row, and
// every warp takes an equal run of it, through a slot of shared memory of its own
// (a page: four tensor copies), as in the decode's kernel.  But here a warp is on
// its own: it leaves a record (m, l, o[128] per head) for each row of its run and
// no row is joined in this kernel, since the prefix's records come to it anyway.
// Own parts are short (tens of pages): joined by the CTA a row at a time, the
// barriers and the wait for the prefix's records took 14 us a row and CTA.
#include <algorithm>

#include "kv16_groups.cuh"
#include "kv16_page.cuh"
#include "kv16_tma.h"
#include "tc5.cuh"

namespace oscar {
namespace {

constexpr int NW = 10;     // warps of a CTA, each with a slot of its own

struct OwnParams {
  Kv16 c;
  Kv16Query q;
  SharedParts s;
};

// A row of the line: its sequence, head, pages [r0, r1) and span.
struct Row {
  int b, h, r0, r1, at;
  Span sp;
};

__device__ __forceinline__ int own_blocks(const OwnParams& p, int b, int n, bool report, Span& sp) {
  const int i = group_of(p.s.groups, b);
  const int shared = i < 0 ? 0 : shared_of(p.c, p.s.groups, i, p.q.max_tok, report).blocks;
  sp = Span(n - 1, n - 1, p.q.window, p.q.n_sink).from(shared);
  return sp.blocks;
}

template <class T>
__global__ void __launch_bounds__(NW * 32, 1)
kv16_own_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                const __grid_constant__ OwnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[NW];
  __shared__ int scan[NW];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, Hkv = p.c.Hkv, g = p.s.g;
  asm volatile("griddepcontrol.launch_dependents;");
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;   // swizzle atoms
  uint8_t* slot = smem + warp * kSlotBytes;
  int* first = reinterpret_cast<int*>(smem + NW * kSlotBytes);              // [B + 1]

  if (tid == 0) {
    for (int w = 0; w < NW; ++w) mbar_init(&full[w], 1);
    mbar_fence_init();
  }
  // first pages of the sequences in the line (of one KV head)
  int carry = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += NW * 32) {
    const int b = b0 + tid;
    int x = 0;
    if (b < p.c.B) {
      const int n = kv16_length(p.c, b, p.q.max_tok);
      if (n < 0 && blockIdx.x == 0) record_error(p.c.status, kDevErrBadPaged);
      Span sp;
      x = own_blocks(p, b, max(n, 0), false, sp);
    }
    const int mine = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += scan[w];
      carry += scan[w];
    }
    if (b < p.c.B) first[b] = before + x - mine;
    __syncthreads();
  }
  if (tid == 0) first[p.c.B] = carry;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.c.B; b += NW * 32) p.s.own_line[b] = first[b];

  const int P = carry * Hkv, per = run_share(P, p.s.workers);
  const int worker = warp * gridDim.x + blockIdx.x;
  const int x0 = (int)min((long long)worker * per, (long long)P);
  const int x1 = (int)min((long long)x0 + per, (long long)P);

  auto find_row = [&](Row& r, int x) {
    const int key = x / Hkv;     // first[b] <= key < first[b + 1]
    int lo = 0, hi = p.c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= key) lo = mid; else hi = mid;
    }
    const int pages = first[lo + 1] - first[lo];
    r.b = lo;
    r.h = (x - first[lo] * Hkv) / pages;
    r.r0 = first[lo] * Hkv + r.h * pages;
    r.r1 = r.r0 + pages;
    const int n = max(kv16_length(p.c, lo, p.q.max_tok), 0);
    r.at = n - 1;
    own_blocks(p, lo, n, false, r.sp);
  };
  // where page x lies; pages out of range read zeros
  Row nr;
  nr.r0 = nr.r1 = 0;
  auto place = [&](int x) -> int {
    if (x >= x1) return 0;
    if (x < nr.r0 || x >= nr.r1) find_row(nr, x);
    const int row = kv16_block_row(p.c, nr.b, nr.h, nr.sp.block(x - nr.r0));
    if (row >= 0) return row;
    if (lane == 0) record_error(p.c.status, kDevErrBadPaged);
    return p.c.n_pages * Hkv * kPage;
  };
  auto fetch = [&](int x, int row) {
    if (x >= x1 || lane != 0) return;
    mbar_arrive_expect_tx(&full[warp], kSlotBytes);
    tma_box2(slot, &map_k, 0, row, &full[warp]);
    tma_box2(slot + 4096, &map_k, 64, row, &full[warp]);
    tma_box2(slot + 8192, &map_v, 0, row, &full[warp]);
    tma_box2(slot + 12288, &map_v, 64, row, &full[warp]);
  };
  fetch(x0, place(x0));
  unsigned phase = 0;
  bool gave_up = false;
  const int hr = lane >> 2, hc = 2 * (lane & 3);    // accumulator row, column
  for (int x = x0; x < x1;) {
    const Row r = nr;            // (of page x)
    const int seg = x, end = min(r.r1, x1);
    uint32_t qa[8][4];
    page_queries(qa, p.q.q + r.b * p.q.stride + (long long)r.h * g * kD, g);
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    for (; x < end; ++x) {
      const int next = place(x + 1);       // (its loads pass under the wait)
      if (gave_up) continue;
      gave_up = !__all_sync(0xffffffffu, mbar_wait_bounded(&full[warp], phase, kTcWaitLimit));
      if (gave_up) {
        if (lane == 0) record_error(p.c.status, kDevErrWaitTimeout);
        continue;
      }
      const bool whole = page_step<T>(slot, r.sp.block(x - r.r0) * kPage, r.at, p.q.window,
                                      p.q.n_sink, p.q.scale_log2, qa, o, m, l,
                                      [](const float (&)[4][4]) {});
      // refill the slot once every lane has read it; cleared values first
      // become visible to the copy engine
      if (!whole) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      fetch(x + 1, next);
      phase ^= 1;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int head = hr + 8 * i;
      if (head >= g) continue;
      float* rec = seg == r.r0
                       ? p.s.own + ((long long)r.b * p.q.Hq + r.h * g + head) * kRecFloats
                       : p.s.own_cut + ((long long)worker * g + head) * kRecFloats;
      if ((lane & 3) == 0) *reinterpret_cast<float2*>(rec) = make_float2(m[i], l[i]);
#pragma unroll
      for (int n = 0; n < 16; ++n)
        *reinterpret_cast<float2*>(rec + 4 + hc + 8 * n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
    }
  }
  // the copy in flight lands before its memory is given back
  if (gave_up && !mbar_wait_bounded(&full[warp], phase, kDrainLimit) && lane == 0)
    record_error(p.c.status, kDevErrDrainTimeout);
  // (complete only once the prefixes' kernel is, so that who follows has both)
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class T>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const OwnParams& p, cudaStream_t s) {
  const size_t smem = NW * kSlotBytes + (size_t)(p.c.B + 1) * 4 + 1024;
  static_assert(NW * kSlotBytes + (kMaxDecodeBatch + 1) * 4 + 1024 <= 227 * 1024 - 1024, "shared memory");
  const auto kernel = kv16_own_kernel<T>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.s.workers / NW;
  cfg.blockDim = NW * 32;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute early[1];      // starts as the prefixes' kernel ends
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, mk, mv, p);
}

}  // namespace

int kv16_own_workers(long long pages, int sms) {
  return NW * (int)std::max<long long>(1, std::min<long long>(sms, pages / kMinRun + 1));
}

cudaError_t launch_kv16_own(const Kv16& c, const Kv16Query& q, const SharedParts& parts,
                            cudaStream_t s) {
  const OwnParams p{c, q, parts};
  CUtensorMap mk, mv;
  if (!kv16_row_map(&mk, c, c.k) || !kv16_row_map(&mv, c, c.v)) return cudaErrorNotSupported;
  return c.half ? launch<Fp16>(mk, mv, p, s) : launch<Bf16>(mk, mv, p, s);
}

}  // namespace oscar
