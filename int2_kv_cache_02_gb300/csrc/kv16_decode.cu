// Attention of one query per sequence over the 16-bit cache.
#include "kv16.cuh"

namespace oscar {

cudaError_t launch_kv16_rows(const Kv16& c, const Kv16Query& q, uint16_t* out, float* lse,
                             cudaStream_t s);

size_t kv16_decode_ws_bytes(const Kv16& c, int Hq, int, int, int, bool) {
  return kDecodeWsHeader + (size_t)c.B * Hq * sizeof(float);
}

cudaError_t launch_kv16_decode(const Kv16& c, const Kv16Query& q, bool accumulate, uint16_t* out,
                               void* ws, int* launches, cudaStream_t s) {
  float* lse = decode_partials(ws);
  *launches = accumulate ? 2 : 1;
  cudaError_t e = launch_kv16_rows(c, q, out, lse, s);
  if (e == cudaSuccess && accumulate) e = launch_kv16_accumulate(c, q, lse, 1, s);
  return e;
}

}  // namespace oscar
