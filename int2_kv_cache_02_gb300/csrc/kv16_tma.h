// Tensor maps over the 16-bit tensors of the kv16 operators (host side).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "launch.h"

namespace oscar {

// cuTensorMapEncodeTiled, looked up once through the runtime (the library does
// not link the driver); nullptr if the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Has `encode` written its map?  The encoder asks for a context, and a
// host thread that has made no runtime call of its own has none: it gets the current
// device's.
template <class F>
bool tensor_map_encoded(F&& encode) {
  if (encode() == CUDA_SUCCESS) return true;
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess &&
         encode() == CUDA_SUCCESS;
}

// k or v of a cache as rows of 128 elements, fetched 64 columns x 32 rows (one
// page's half) at a time with the 128-byte swizzle; rows past the end read 0.
inline bool kv16_row_map(CUtensorMap* m, const Kv16& c, const uint16_t* base) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t rows = c.table ? (cuuint64_t)c.n_pages * c.Hkv * OSCAR_GROUP
                                  : (cuuint64_t)c.B * c.Hkv * c.T_cap;
  const cuuint64_t dims[2] = {OSCAR_HEAD_DIM, rows};
  const cuuint64_t strides[1] = {OSCAR_HEAD_DIM * 2};
  const cuuint32_t box[2] = {64, OSCAR_GROUP}, step[2] = {1, 1};
  return tensor_map_encoded([&] {
    return enc(m, c.half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<uint16_t*>(base), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

// The queries as [total][Hq][128], fetched 64 columns x g heads x `tokens` rows
// at a time with the 128-byte swizzle; rows past the end read 0.
inline bool kv16_query_map(CUtensorMap* m, const Kv16Query& q, bool half, int g, int tokens) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {OSCAR_HEAD_DIM, (cuuint64_t)q.Hq, (cuuint64_t)q.total};
  const cuuint64_t strides[2] = {OSCAR_HEAD_DIM * 2, (cuuint64_t)q.stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)tokens}, step[3] = {1, 1, 1};
  return tensor_map_encoded([&] {
    return enc(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<uint16_t*>(q.q), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

}  // namespace oscar
