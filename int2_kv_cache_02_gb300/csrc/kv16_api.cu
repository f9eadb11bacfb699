// C ABI of the 16-bit cache (include/oscar.h): argument checks and dispatch.
#include <algorithm>
#include <cmath>

#include "kv16.cuh"
#include "kv16_line.h"
#include "launch.h"

namespace {

using namespace oscar;

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
inline oscar_status from_cuda(cudaError_t e) { return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA; }

constexpr long long kMaxTokens = 0x7fffffffLL - 128;

long long capacity(const oscar_kv16_cache* c) {
  return c->block_table ? (long long)c->max_blocks * kPage : c->T_cap;
}

oscar_status check(const oscar_kv16_cache* c) {
  if (!c || c->B <= 0 || c->Hkv <= 0 || !c->k || !c->v || !c->n_tok) return OSCAR_ERR_INVALID_ARG;
  if (c->dtype != OSCAR_KV16_BF16 && c->dtype != OSCAR_KV16_FP16) return OSCAR_ERR_INVALID_ARG;
  if (c->block_table ? c->max_blocks <= 0 || c->n_pages <= 0 : c->T_cap <= 0)
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->weight, 16) ||
      !aligned(c->block_table, 4) || !aligned(c->n_tok, 4))
    return OSCAR_ERR_ALIGNMENT;
  // the kernels number table entries, rows and tokens in 32 bits (a block may
  // reach 31 rows past the end of a contiguous cache)
  const long long slabs = (long long)(c->block_table ? c->n_pages : c->B) * c->Hkv;
  const long long per_slab = c->block_table ? kPage : c->T_cap;
  if (slabs > kMaxTokens / per_slab || capacity(c) > kMaxTokens ||
      (c->block_table && (long long)c->B * c->max_blocks > 0x7fffffffLL))
    return OSCAR_ERR_UNSUPPORTED;
  return OSCAR_OK;
}

// Rows of 128 elements of k (and of v) of a checked cache.
size_t cache_rows(const oscar_kv16_cache* c) {
  return c->block_table ? (size_t)c->n_pages * c->Hkv * kPage : (size_t)c->B * c->Hkv * c->T_cap;
}

Kv16 view(const oscar_kv16_cache* c) {
  Kv16 v;
  v.k = c->k;
  v.v = c->v;
  v.weight = c->weight;
  v.table = c->block_table;
  v.n_tok = c->n_tok;
  v.status = nullptr;
  v.B = c->B;
  v.Hkv = c->Hkv;
  v.max_blocks = c->max_blocks;
  v.n_pages = c->n_pages;
  v.T_cap = c->T_cap;
  v.cap = (int)capacity(c);
  v.half = c->dtype == OSCAR_KV16_FP16;
  return v;
}

// Rows of a [rows][heads][128] tensor: dense or further apart, in 16-byte steps.
bool stride_ok(long long stride, int heads) {
  return stride >= (long long)heads * kD && stride % 8 == 0 && stride < (1LL << 32);
}

bool heads_ok(int Hq, int Hkv) { return Hq > 0 && Hq % Hkv == 0 && Hq / Hkv <= kMaxGroup; }

bool window_ok(float scale, int max_tok, int window, int n_sink) {
  return std::isfinite(scale) && max_tok >= 0 && window >= 0 && n_sink >= 0;
}

Kv16Query query(const uint16_t* q, long long stride, const int32_t* start, int total, int Hq,
                float scale, int max_tok, int window, int n_sink) {
  return Kv16Query{q, stride, start, total, Hq, max_tok, window, n_sink, scale * kLog2e};
}

struct Range {
  const char* p;
  size_t n;
};
bool overlap(Range a, Range b) {
  return a.p && b.p && a.n && b.n && a.p < b.p + b.n && b.p < a.p + a.n;
}

// Does [n bytes at p] share memory with the queries?  (Rows whose result is not
// finite read their query again after results are written.)
bool in_queries(const void* p, size_t n, const uint16_t* q, long long stride, int rows, int Hq) {
  return overlap({static_cast<const char*>(p), n},
                 {reinterpret_cast<const char*>(q),
                  ((size_t)(rows - 1) * (size_t)stride + (size_t)Hq * kD) * sizeof(uint16_t)});
}

// The decode's pages are numbered in 32 bits over all rows.
bool decode_size_ok(const oscar_kv16_cache* c, int max_tok) {
  const long long blocks = (std::min<long long>(max_tok, capacity(c)) + kPage - 1) / kPage;
  const long long rows = (long long)c->B * c->Hkv;
  return c->B <= kMaxDecodeBatch && rows <= kMaxDecodeRows && rows * blocks <= kMaxTokens;
}

// The places of the line (kv16_line.h: rows are the groups' and the sequences'
// chunks of 256 query rows) are numbered in 32 bits.
bool shared_size_ok(const oscar_kv16_cache* c, int Hq, int n_groups, int total, int max_tok) {
  const long long two = 2 * (128 / (Hq / c->Hkv));
  const long long rows = (2 * (total / two) + n_groups + c->B) * c->Hkv;
  const long long places =
      kMostTileCost * ((std::min<long long>(max_tok, capacity(c)) + 127) / 128) + row_cost(3);
  return c->B <= kMaxDecodeBatch && n_groups <= kMaxGroups && (long long)total * Hq <= kMaxSharedRows &&
         rows <= kMaxTokens && rows * places <= kMaxTokens;
}

// -1 if the three counts are no valid budget.
long long keep_of(int keep_first, int keep_recent, int keep_top) {
  if (keep_first < 0 || keep_recent < 0 || keep_top < 0) return -1;
  const long long keep = (long long)keep_first + keep_recent + keep_top;
  return keep >= 1 && keep <= kMaxTokens ? keep : -1;
}

// The rows' counts, then the kept positions (where the caller takes none).
size_t evict_ws_bytes(const oscar_kv16_cache* src, long long keep) {
  return (size_t)((long long)src->B * src->Hkv) * (size_t)(keep + 4) * sizeof(int32_t);
}

size_t table_bytes(long long B, long long max_blocks) { return (size_t)(B * max_blocks) * sizeof(int32_t); }

// The memory of a cache: keys, values, weights, lengths, table.
struct Extent {
  Range r[5];
};
Extent extent(const oscar_kv16_cache* c) {
  const size_t rows = cache_rows(c);
  auto at = [](const void* p, size_t n) { return Range{static_cast<const char*>(p), n}; };
  return Extent{{at(c->k, rows * kD * 2), at(c->v, rows * kD * 2), at(c->weight, rows * 4),
                 at(c->n_tok, (size_t)c->B * 4),
                 at(c->block_table, c->block_table ? table_bytes(c->B, c->max_blocks) : 0)}};
}

// Are the pages of a and b the same memory, page for page?
bool same_pool(const oscar_kv16_cache* a, const oscar_kv16_cache* b) {
  return a->block_table && b->block_table && a->k == b->k && a->v == b->v &&
         a->n_pages == b->n_pages && (a->weight == b->weight || !b->weight);
}

// May a call copy tokens from src to dst?  They are of one kind, and their
// keys, values and weights lie apart or are one pool's.
oscar_status copy_ok(const oscar_kv16_cache* src, const oscar_kv16_cache* dst) {
  if (src->Hkv != dst->Hkv || src->dtype != dst->dtype || (dst->weight && !src->weight))
    return OSCAR_ERR_INVALID_ARG;
  if (same_pool(src, dst)) return OSCAR_OK;
  const Extent a = extent(src), b = extent(dst);
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 3; ++j)
      if (overlap(a.r[i], b.r[j])) return OSCAR_ERR_INVALID_ARG;
  return OSCAR_OK;
}

bool groups_ok(const int32_t* group, const int32_t* prefix, int n) {
  return n >= 1 && group && prefix;
}

oscar_status shared(const oscar_kv16_cache* c, const uint16_t* q, long long q_stride,
                    const int32_t* start, int total, int Hq, const int32_t* group,
                    const int32_t* prefix, int n_groups, float softmax_scale, int max_tok,
                    int window, int n_sink, uint16_t* out, float* lse, void* workspace,
                    size_t ws_bytes, unsigned copied, void* stream) {
  if (total < 0 || !groups_ok(group, prefix, n_groups) ||
      !window_ok(softmax_scale, max_tok, window, n_sink))
    return OSCAR_ERR_INVALID_ARG;
  if (!heads_ok(Hq, c->Hkv)) return OSCAR_ERR_UNSUPPORTED;
  if ((total > 0 && (!q || !out)) || !stride_ok(q_stride, Hq)) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(start, 4) ||
      !aligned(group, 4) || !aligned(prefix, 4))
    return OSCAR_ERR_ALIGNMENT;
  if (!shared_size_ok(c, Hq, n_groups, total, max_tok)) return OSCAR_ERR_UNSUPPORTED;
  if (total == 0) return OSCAR_OK;
  Kv16 v = view(c);
  if (!workspace || ws_bytes < kv16_shared_ws_bytes(v, Hq, n_groups, total, max_tok))
    return OSCAR_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return OSCAR_ERR_ALIGNMENT;
  const size_t heads = (size_t)total * Hq;
  if (in_queries(out, heads * kD * sizeof(uint16_t), q, q_stride, total, Hq) ||
      in_queries(lse, heads * sizeof(float), q, q_stride, total, Hq))
    return OSCAR_ERR_INVALID_ARG;
  v.status = device_status_word();
  if (!v.status) return OSCAR_ERR_CUDA;
  int launches = 0;
  const cudaError_t e = launch_kv16_shared(
      v, query(q, q_stride, start, total, Hq, softmax_scale, max_tok, window, n_sink),
      Kv16Groups{group, prefix, n_groups}, out, lse, workspace, copied, &launches,
      as_stream(stream));
  count_launches(launches);
  return from_cuda(e);
}

oscar_status shared_decode(const oscar_kv16_cache* c, const uint16_t* q, long long q_stride,
                           int Hq, const int32_t* group, const int32_t* prefix, int n_groups,
                           float softmax_scale, int max_tok, int window, int n_sink, uint16_t* out,
                           void* workspace, size_t ws_bytes, unsigned copied, void* stream) {
  const oscar_status st = check(c);
  if (st != OSCAR_OK) return st;
  if (max_tok >= 0 && !decode_size_ok(c, max_tok)) return OSCAR_ERR_UNSUPPORTED;
  return shared(c, q, q_stride, nullptr, c->B, Hq, group, prefix, n_groups, softmax_scale, max_tok,
                window, n_sink, out, nullptr, workspace, ws_bytes, copied, stream);
}

oscar_status decode(const oscar_kv16_cache* c, const uint16_t* q, long long q_stride, int Hq,
                    float softmax_scale, int max_tok, int window, int n_sink, int accumulate,
                    uint16_t* out, void* workspace, size_t ws_bytes, unsigned wait_limit,
                    void* stream) {
  oscar_status st = check(c);
  if (st != OSCAR_OK) return st;
  if (!q || !out || !window_ok(softmax_scale, max_tok, window, n_sink) ||
      (accumulate != 0 && accumulate != 1) || (accumulate && !c->weight))
    return OSCAR_ERR_INVALID_ARG;
  if (!heads_ok(Hq, c->Hkv)) return OSCAR_ERR_UNSUPPORTED;
  if (!stride_ok(q_stride, Hq)) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16)) return OSCAR_ERR_ALIGNMENT;
  if (!decode_size_ok(c, max_tok)) return OSCAR_ERR_UNSUPPORTED;
  Kv16 v = view(c);
  if (!workspace ||
      ws_bytes < kv16_decode_ws_bytes(v, Hq, max_tok, window, n_sink, accumulate != 0))
    return OSCAR_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return OSCAR_ERR_ALIGNMENT;
  if (in_queries(out, (size_t)c->B * Hq * kD * sizeof(uint16_t), q, q_stride, c->B, Hq))
    return OSCAR_ERR_INVALID_ARG;
  v.status = device_status_word();
  if (!v.status) return OSCAR_ERR_CUDA;
  int launches = 0;
  const cudaError_t e = launch_kv16_decode(
      v, query(q, q_stride, nullptr, c->B, Hq, softmax_scale, max_tok, window, n_sink),
      accumulate != 0, out, workspace, wait_limit, &launches, as_stream(stream));
  count_launches(launches);
  return from_cuda(e);
}

}  // namespace

extern "C" {

oscar_status oscar_kv16_write(const oscar_kv16_cache* c, const uint16_t* k_new,
                              long long k_stride, const uint16_t* v_new, long long v_stride,
                              const int32_t* start, const int32_t* pos0, int total, void* stream) {
  oscar_status st = check(c);
  if (st != OSCAR_OK) return st;
  if (!start || !pos0 || total < 0 || (total > 0 && (!k_new || !v_new)) ||
      !stride_ok(k_stride, c->Hkv) || !stride_ok(v_stride, c->Hkv))
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(start, 4) || !aligned(pos0, 4))
    return OSCAR_ERR_ALIGNMENT;
  const size_t nb = (size_t)c->B * sizeof(int32_t);
  const Range lengths{reinterpret_cast<const char*>(c->n_tok), nb};
  if (overlap(lengths, {reinterpret_cast<const char*>(pos0), nb}) ||
      overlap(lengths, {reinterpret_cast<const char*>(start), nb + sizeof(int32_t)}))
    return OSCAR_ERR_INVALID_ARG;
  if (total > kMaxTokens) return OSCAR_ERR_UNSUPPORTED;
  Kv16 v = view(c);
  v.status = device_status_word();
  if (!v.status) return OSCAR_ERR_CUDA;
  const cudaError_t e = launch_kv16_write(v, k_new, k_stride, v_new, v_stride, start, pos0, total,
                                          as_stream(stream));
  count_launches(1);
  return from_cuda(e);
}

size_t oscar_kv16_attention_workspace_bytes(const oscar_kv16_cache* c, int Hq, int total,
                                            int max_tok, int window, int n_sink) {
  if (check(c) != OSCAR_OK || !heads_ok(Hq, c->Hkv) || total <= 0 ||
      !window_ok(0.0f, max_tok, window, n_sink) || (long long)total * Hq > kMaxTokens)
    return 0;
  return kv16_attention_ws_bytes(view(c), Hq, total, max_tok, window, n_sink);
}

oscar_status oscar_kv16_attention(const oscar_kv16_cache* c, const uint16_t* q,
                                  long long q_stride, const int32_t* start, int total, int Hq,
                                  float softmax_scale, int max_tok, int window, int n_sink,
                                  uint16_t* out, float* lse, void* workspace, size_t ws_bytes,
                                  void* stream) {
  oscar_status st = check(c);
  if (st != OSCAR_OK) return st;
  if (!start || total < 0 || !window_ok(softmax_scale, max_tok, window, n_sink))
    return OSCAR_ERR_INVALID_ARG;
  if (!heads_ok(Hq, c->Hkv)) return OSCAR_ERR_UNSUPPORTED;
  if ((total > 0 && (!q || !out)) || !stride_ok(q_stride, Hq)) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(start, 4))
    return OSCAR_ERR_ALIGNMENT;
  if ((long long)total * Hq > kMaxTokens) return OSCAR_ERR_UNSUPPORTED;
  if (total == 0) return OSCAR_OK;
  Kv16 v = view(c);
  const size_t need = kv16_attention_ws_bytes(v, Hq, total, max_tok, window, n_sink);
  if (need && (!workspace || ws_bytes < need)) return OSCAR_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return OSCAR_ERR_ALIGNMENT;
  const size_t heads = (size_t)total * Hq;
  if (in_queries(out, heads * kD * sizeof(uint16_t), q, q_stride, total, Hq) ||
      in_queries(lse, heads * sizeof(float), q, q_stride, total, Hq))
    return OSCAR_ERR_INVALID_ARG;
  v.status = device_status_word();
  if (!v.status) return OSCAR_ERR_CUDA;
  int launches = 0;
  const cudaError_t e = launch_kv16_attention(
      v, query(q, q_stride, start, total, Hq, softmax_scale, max_tok, window, n_sink), out, lse,
      workspace, &launches, as_stream(stream));
  count_launches(launches);
  return from_cuda(e);
}

size_t oscar_kv16_decode_workspace_bytes(const oscar_kv16_cache* c, int Hq, int max_tok,
                                         int window, int n_sink, int accumulate) {
  if (check(c) != OSCAR_OK || !heads_ok(Hq, c->Hkv) ||
      !window_ok(0.0f, max_tok, window, n_sink) || !decode_size_ok(c, max_tok))
    return 0;
  return kv16_decode_ws_bytes(view(c), Hq, max_tok, window, n_sink, accumulate != 0);
}

oscar_status oscar_kv16_decode_attention(const oscar_kv16_cache* c, const uint16_t* q,
                                         long long q_stride, int Hq, float softmax_scale,
                                         int max_tok, int window, int n_sink, int accumulate,
                                         uint16_t* out, void* workspace, size_t ws_bytes,
                                         void* stream) {
  return decode(c, q, q_stride, Hq, softmax_scale, max_tok, window, n_sink, accumulate, out,
                workspace, ws_bytes, kTcWaitLimit, stream);
}

oscar_status oscar_selftest_kv16_decode_timeout(const oscar_kv16_cache* c, const uint16_t* q,
                                                int Hq, int max_tok, uint16_t* out,
                                                void* workspace, size_t ws_bytes, void* stream) {
  return decode(c, q, (long long)Hq * kD, Hq, 1.0f, max_tok, 0, 0, 0, out, workspace, ws_bytes, 0,
                stream);
}

oscar_status oscar_kv16_accumulate(const oscar_kv16_cache* c, const uint16_t* q,
                                   long long q_stride, const float* lse, const int32_t* start,
                                   int total, int Hq, float softmax_scale, int max_tok,
                                   int window, int n_sink, int n_obs, void* stream) {
  oscar_status st = check(c);
  if (st != OSCAR_OK) return st;
  if (!start || total < 0 || n_obs < 0 || !c->weight ||
      !window_ok(softmax_scale, max_tok, window, n_sink))
    return OSCAR_ERR_INVALID_ARG;
  if (!heads_ok(Hq, c->Hkv)) return OSCAR_ERR_UNSUPPORTED;
  if ((total > 0 && (!q || !lse)) || !stride_ok(q_stride, Hq)) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(lse, 4) || !aligned(start, 4)) return OSCAR_ERR_ALIGNMENT;
  if ((long long)total * Hq > kMaxTokens) return OSCAR_ERR_UNSUPPORTED;
  if (total == 0 || max_tok == 0) return OSCAR_OK;
  Kv16 v = view(c);
  v.status = device_status_word();
  if (!v.status) return OSCAR_ERR_CUDA;
  const cudaError_t e = launch_kv16_accumulate(
      v, query(q, q_stride, start, total, Hq, softmax_scale, max_tok, window, n_sink), lse, n_obs,
      as_stream(stream));
  count_launches(1);
  return from_cuda(e);
}

size_t oscar_kv16_evict_workspace_bytes(const oscar_kv16_cache* src, int max_tok, int keep_first,
                                        int keep_recent, int keep_top) {
  const long long keep = keep_of(keep_first, keep_recent, keep_top);
  if (check(src) != OSCAR_OK || keep < 0 || max_tok < 0) return 0;
  return evict_ws_bytes(src, keep);
}

oscar_status oscar_kv16_evict(const oscar_kv16_cache* src, const oscar_kv16_cache* dst,
                              int max_tok, int keep_first, int keep_recent, int keep_top,
                              int32_t* kept, void* workspace, size_t ws_bytes, void* stream) {
  oscar_status st = check(src);
  if (st == OSCAR_OK) st = check(dst);
  if (st != OSCAR_OK) return st;
  const long long keep = keep_of(keep_first, keep_recent, keep_top);
  if (keep < 0 || max_tok < 0 || !src->weight || src->B != dst->B || src->Hkv != dst->Hkv ||
      src->dtype != dst->dtype)
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(kept, 4)) return OSCAR_ERR_ALIGNMENT;
  auto kv = [](const oscar_kv16_cache* c, const void* p) {
    return Range{static_cast<const char*>(p), cache_rows(c) * kD * 2};
  };
  auto w = [](const oscar_kv16_cache* c) {
    return Range{reinterpret_cast<const char*>(c->weight), cache_rows(c) * 4};
  };
  auto n = [](const oscar_kv16_cache* c) {
    return Range{reinterpret_cast<const char*>(c->n_tok), (size_t)c->B * 4};
  };
  const Range from[] = {kv(src, src->k), kv(src, src->v), w(src), n(src)};
  const Range to[] = {kv(dst, dst->k), kv(dst, dst->v), w(dst), n(dst)};
  for (const Range& a : from)
    for (const Range& b : to)
      if (overlap(a, b)) return OSCAR_ERR_INVALID_ARG;
  if (keep > capacity(dst)) return OSCAR_ERR_CAPACITY;
  if ((long long)src->B * src->Hkv > kMaxTokens / keep) return OSCAR_ERR_UNSUPPORTED;
  Kv16 s = view(src), d = view(dst);
  if (!workspace || ws_bytes < evict_ws_bytes(src, keep)) return OSCAR_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return OSCAR_ERR_ALIGNMENT;
  s.status = d.status = device_status_word();
  if (!s.status) return OSCAR_ERR_CUDA;
  const cudaError_t e = launch_kv16_evict(s, d, max_tok, keep_first, keep_recent, keep_top, kept,
                                          workspace, as_stream(stream));
  count_launches(2);
  return from_cuda(e);
}

size_t oscar_kv16_shared_decode_workspace_bytes(const oscar_kv16_cache* c, int Hq, int n_groups,
                                                int max_tok, int window, int n_sink) {
  if (check(c) != OSCAR_OK || !heads_ok(Hq, c->Hkv) || n_groups < 1 ||
      !window_ok(0.0f, max_tok, window, n_sink) ||
      !shared_size_ok(c, Hq, n_groups, c->B, max_tok) || !decode_size_ok(c, max_tok))
    return 0;
  return kv16_shared_ws_bytes(view(c), Hq, n_groups, c->B, max_tok);
}

oscar_status oscar_kv16_shared_decode_attention(const oscar_kv16_cache* c, const uint16_t* q,
                                                long long q_stride, int Hq, const int32_t* group,
                                                const int32_t* prefix, int n_groups,
                                                float softmax_scale, int max_tok, int window,
                                                int n_sink, uint16_t* out, void* workspace,
                                                size_t ws_bytes, void* stream) {
  return shared_decode(c, q, q_stride, Hq, group, prefix, n_groups, softmax_scale, max_tok, window,
                       n_sink, out, workspace, ws_bytes, kAllItems, stream);
}

oscar_status oscar_selftest_kv16_shared_timeout(const oscar_kv16_cache* c, const uint16_t* q,
                                                int Hq, const int32_t* group, const int32_t* prefix,
                                                int n_groups, int max_tok, int items, uint16_t* out,
                                                void* workspace, size_t ws_bytes, void* stream) {
  if (items < 0) return OSCAR_ERR_INVALID_ARG;
  return shared_decode(c, q, (long long)Hq * kD, Hq, group, prefix, n_groups, 1.0f, max_tok, 0, 0,
                       out, workspace, ws_bytes, (unsigned)items, stream);
}

size_t oscar_kv16_shared_attention_workspace_bytes(const oscar_kv16_cache* c, int Hq, int n_groups,
                                                   int total, int max_tok, int window, int n_sink) {
  if (check(c) != OSCAR_OK || !heads_ok(Hq, c->Hkv) || n_groups < 1 || total <= 0 ||
      !window_ok(0.0f, max_tok, window, n_sink) || !shared_size_ok(c, Hq, n_groups, total, max_tok))
    return 0;
  return kv16_shared_ws_bytes(view(c), Hq, n_groups, total, max_tok);
}

oscar_status oscar_kv16_shared_attention(const oscar_kv16_cache* c, const uint16_t* q,
                                         long long q_stride, const int32_t* start, int total,
                                         int Hq, const int32_t* group, const int32_t* prefix,
                                         int n_groups, float softmax_scale, int max_tok,
                                         int window, int n_sink, uint16_t* out, float* lse,
                                         void* workspace, size_t ws_bytes, void* stream) {
  const oscar_status st = check(c);
  if (st != OSCAR_OK) return st;
  if (!start) return OSCAR_ERR_INVALID_ARG;
  return shared(c, q, q_stride, start, total, Hq, group, prefix, n_groups, softmax_scale, max_tok,
                window, n_sink, out, lse, workspace, ws_bytes, kAllItems, stream);
}

oscar_status oscar_kv16_fork(const oscar_kv16_cache* src, const oscar_kv16_cache* dst,
                             const int32_t* parent, int share, int max_tok, void* stream) {
  oscar_status st = check(src);
  if (st == OSCAR_OK) st = check(dst);
  if (st != OSCAR_OK) return st;
  if (!parent || (share != 0 && share != 1) || max_tok < 0) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(parent, 4)) return OSCAR_ERR_ALIGNMENT;
  st = copy_ok(src, dst);
  if (st != OSCAR_OK) return st;
  if (share && !same_pool(src, dst)) return OSCAR_ERR_INVALID_ARG;
  // one cache, or lengths and tables apart from each other's and from all that is read
  const bool same = same_pool(src, dst) && src->n_tok == dst->n_tok &&
                    src->block_table == dst->block_table && src->B == dst->B &&
                    src->max_blocks == dst->max_blocks;
  const Extent a = extent(src), b = extent(dst);
  const Range par{reinterpret_cast<const char*>(parent), (size_t)dst->B * sizeof(int32_t)};
  if (!same)
    for (int i = 3; i < 5; ++i)
      for (int j = 3; j < 5; ++j)
        if (overlap(a.r[i], b.r[j])) return OSCAR_ERR_INVALID_ARG;
  for (int j = 0; j < 5; ++j)
    if (overlap(par, b.r[j])) return OSCAR_ERR_INVALID_ARG;
  Kv16 s = view(src), d = view(dst);
  s.status = d.status = device_status_word();
  if (!s.status) return OSCAR_ERR_CUDA;
  const cudaError_t e = launch_kv16_fork(s, d, parent, share != 0, same, max_tok, as_stream(stream));
  count_launches(1);
  return from_cuda(e);
}

oscar_status oscar_kv16_copy_pages(const oscar_kv16_cache* src, const oscar_kv16_cache* dst,
                                   const int32_t* pairs, const int32_t* n_pairs, int max_pairs,
                                   void* stream) {
  oscar_status st = check(src);
  if (st == OSCAR_OK) st = check(dst);
  if (st != OSCAR_OK) return st;
  if (!src->block_table || !dst->block_table || max_pairs < 0 || !n_pairs ||
      (max_pairs > 0 && !pairs))
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(pairs, 8) || !aligned(n_pairs, 4)) return OSCAR_ERR_ALIGNMENT;
  st = copy_ok(src, dst);
  if (st != OSCAR_OK || max_pairs == 0) return st;
  if (max_pairs > kMaxTokens / src->Hkv) return OSCAR_ERR_UNSUPPORTED;
  Kv16 s = view(src), d = view(dst);
  s.status = d.status = device_status_word();
  if (!s.status) return OSCAR_ERR_CUDA;
  const cudaError_t e = launch_kv16_copy_pages(s, d, pairs, n_pairs, max_pairs, as_stream(stream));
  count_launches(1);
  return from_cuda(e);
}

size_t oscar_page_compact_workspace_bytes(int B, int max_blocks, int n_pages) {
  if (B <= 0 || max_blocks <= 0 || n_pages <= 0 || n_pages > kMaxPages) return 0;
  return page_compact_ws_bytes(n_pages);
}

oscar_status oscar_page_compact(const int32_t* block_table, int32_t* new_table, int B,
                                int max_blocks, int n_pages, int32_t* moves, int32_t* counts,
                                void* workspace, size_t ws_bytes, void* stream) {
  if (!block_table || !new_table || B <= 0 || max_blocks <= 0 || n_pages <= 0 || !counts ||
      (n_pages > 1 && !moves))
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(new_table, 4) || !aligned(moves, 8) ||
      !aligned(counts, 4))
    return OSCAR_ERR_ALIGNMENT;
  const long long entries = (long long)B * max_blocks;
  if (entries > kMaxTokens || n_pages > kMaxPages) return OSCAR_ERR_UNSUPPORTED;
  const size_t tb = table_bytes(B, max_blocks);
  const Range out[] = {{reinterpret_cast<const char*>(new_table), tb},
                       {reinterpret_cast<const char*>(moves), (size_t)(n_pages / 2) * 8},
                       {reinterpret_cast<const char*>(counts), 8}};
  const Range in{reinterpret_cast<const char*>(block_table), tb};
  for (int i = 0; i < 3; ++i) {
    if (overlap(in, out[i]) && !(i == 0 && block_table == new_table)) return OSCAR_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return OSCAR_ERR_INVALID_ARG;
  }
  if (!workspace || ws_bytes < page_compact_ws_bytes(n_pages)) return OSCAR_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return OSCAR_ERR_ALIGNMENT;
  unsigned* status = device_status_word();
  if (!status) return OSCAR_ERR_CUDA;
  const cudaError_t e = launch_page_compact(block_table, new_table, entries, n_pages, moves, counts,
                                            workspace, status, as_stream(stream));
  count_launches(1);
  return from_cuda(e);
}

}  // extern "C"
