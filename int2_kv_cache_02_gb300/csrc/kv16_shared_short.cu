// The decode under shared prefixes where there is little to share: few rows
// (sequence, KV head) of few pages, which a CTA each works by itself, prefix and
// own pages alike.  Latency bounds it: length and group, table, page, and the join
// of the CTA's warps; the line of key tiles (kv16_shared.cu) has two launches and
// records between them.  Measured (GB300): 16 rows of 533 tokens 8.7 us (line 15.8),
// 128 rows of 1021 tokens 11.8 us (18.5); with all a warp's pages one after another
// 7.2 us for each 1000 tokens, so long rows are the line's, which cuts them up.
//
// A warp takes every eighth page, through a slot of shared memory of its own; what
// it does with a page is the decode's (kv16_page.cuh).
#include "kv16_groups.cuh"
#include "kv16_page.cuh"
#include "kv16_tma.h"
#include "tc5.cuh"

namespace oscar {
namespace {

constexpr int NW = 8;
constexpr int kORow = 136;       // floats of a head's output row in shared memory

struct ShortParams {
  Kv16 c;
  Kv16Query q;
  Kv16Groups groups;
  uint16_t* out;
  int g;
  unsigned wait_limit;
};

template <class T>
__global__ void __launch_bounds__(NW * 32, 1)
kv16_shared_short_kernel(const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ ShortParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[NW];
  __shared__ float sm_m[NW][kMaxGroup], sm_l[NW][kMaxGroup];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = p.g;
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;   // swizzle atoms
  uint8_t* slot = smem + warp * kSlotBytes;
  float* obuf = reinterpret_cast<float*>(smem + NW * kSlotBytes);           // [NW][g][kORow]
  const int b = blockIdx.x / p.c.Hkv, h = blockIdx.x - b * p.c.Hkv;
  if (lane == 0) {
    mbar_init(&full[warp], 1);
    mbar_fence_init();
  }
  __syncwarp();
  if (blockIdx.x == 0)
    for (int i = tid; i < p.groups.n; i += NW * 32) shared_of(p.c, p.groups, i, p.q.max_tok, true);
  const int n = kv16_length(p.c, b, p.q.max_tok), at = max(n, 0) - 1;
  if (n < 0 && h == 0 && tid == 0) record_error(p.c.status, kDevErrBadPaged);
  const int i = warp_sequence(p.groups.group, p.groups.n, b);
  Shared sh{b, b, 0};
  if (i >= 0) sh = shared_of(p.c, p.groups, i, p.q.max_tok, false);
  const Span sp(at, at, p.q.window, p.q.n_sink);

  // where page x of the span lies; pages out of range read zeros
  auto place = [&](int x) -> int {
    if (x >= sp.blocks) return 0;
    const int blk = sp.block(x), row = kv16_block_row(p.c, blk < sh.blocks ? sh.lead : b, h, blk);
    if (row >= 0) return row;
    if (lane == 0) record_error(p.c.status, kDevErrBadPaged);
    return p.c.n_pages * p.c.Hkv * kPage;
  };
  auto fetch = [&](int x, int row) {
    if (x >= sp.blocks || lane != 0) return;
    mbar_arrive_expect_tx(&full[warp], kSlotBytes);
    tma_box2(slot, &map_k, 0, row, &full[warp]);
    tma_box2(slot + 4096, &map_k, 64, row, &full[warp]);
    tma_box2(slot + 8192, &map_v, 0, row, &full[warp]);
    tma_box2(slot + 12288, &map_v, 64, row, &full[warp]);
  };
  fetch(warp, place(warp));
  uint32_t qa[8][4];
  page_queries(qa, p.q.q + b * p.q.stride + (long long)h * g * kD, g);
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.0f;
  unsigned phase = 0;
  bool gave_up = false;
  for (int x = warp; x < sp.blocks; x += NW) {
    const int next = place(x + NW);        // (its load passes under the wait)
    gave_up = !__all_sync(0xffffffffu, mbar_wait_bounded(&full[warp], phase, p.wait_limit));
    if (gave_up) {
      if (lane == 0) record_error(p.c.status, kDevErrWaitTimeout);
      break;
    }
    const bool whole = page_step<T>(slot, sp.block(x) * kPage, at, p.q.window, p.q.n_sink,
                                    p.q.scale_log2, qa, o, m, l, [](const float (&)[4][4]) {});
    // refill the slot once every lane has read it; cleared values first become
    // visible to the copy engine
    if (!whole) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    fetch(x + NW, next);
    phase ^= 1;
  }
  // the warps' parts
  const int hr = lane >> 2, hc = 2 * (lane & 3);    // accumulator row, column
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
    const int head = hr + 8 * k;
    if (head >= g) continue;
    if ((lane & 3) == 0) sm_m[warp][head] = m[k], sm_l[warp][head] = l[k];
    float* d = obuf + (warp * g + head) * kORow + hc;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      *reinterpret_cast<float2*>(d + 8 * e) = make_float2(o[e][2 * k], o[e][2 * k + 1]);
  }
  __syncthreads();
  for (int head = warp; head < g; head += NW) {
    float M = -INFINITY, L = 0.0f;
    for (int w = 0; w < NW; ++w) M = fmaxf(M, sm_m[w][head]);
    const float ms = M == -INFINITY ? 0.0f : M;
    float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float a = fast_exp2(sm_m[w][head] - ms);
      const float4 v = reinterpret_cast<const float4*>(obuf + (w * g + head) * kORow)[lane];
      L += a * sm_l[w][head];
      r.x += a * v.x;
      r.y += a * v.y;
      r.z += a * v.z;
      r.w += a * v.w;
    }
    const bool open = r.x != r.x || r.y != r.y || r.z != r.z || r.w != r.w;
    if (L == L && __any_sync(0xffffffffu, open)) r = settle<T>(p.c, p.q, p.groups, b, h, 1, r);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const long long row = (long long)b * p.q.Hq + h * g + head;
    reinterpret_cast<uint2*>(p.out + row * kD)[lane] =
        make_uint2(T::pack(r.x * inv, r.y * inv), T::pack(r.z * inv, r.w * inv));
  }
  // the copy in flight lands before its memory is given back
  if (gave_up && !mbar_wait_bounded(&full[warp], phase, kDrainLimit) && lane == 0)
    record_error(p.c.status, kDevErrDrainTimeout);
}

template <class T>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const ShortParams& p,
                   cudaStream_t s) {
  constexpr int fixed = 1024 + NW * kSlotBytes, head = NW * kORow * (int)sizeof(float);
  static_assert(fixed + kMaxGroup * head <= 226 * 1024, "shared memory");
  const int smem = fixed + p.g * head;
  const auto kernel = kv16_shared_short_kernel<T>;
  const cudaError_t e = allow_shared(kernel, fixed + kMaxGroup * head);
  if (e != cudaSuccess) return e;
  kernel<<<p.c.B * p.c.Hkv, NW * 32, smem, s>>>(mk, mv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv16_shared_short(const Kv16& c, const Kv16Query& q, const Kv16Groups& groups,
                                     uint16_t* out, unsigned wait_limit, cudaStream_t s) {
  const ShortParams p{c, q, groups, out, q.Hq / c.Hkv, wait_limit};
  CUtensorMap mk, mv;
  if (!kv16_row_map(&mk, c, c.k) || !kv16_row_map(&mv, c, c.v)) return cudaErrorNotSupported;
  return c.half ? launch<Fp16>(mk, mv, p, s) : launch<Bf16>(mk, mv, p, s);
}

}  // namespace oscar
