// Host-side checks that the entry points of the microscaled operators share.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace moe {
namespace mx {

constexpr int kMaxE = 1024;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1024;  // a tile past the last row stays an int
constexpr int64_t kMaxDim = (int64_t)1 << 24;

inline int dtype_size(int dt) { return dt == MOE_F32 ? 4 : (dt == MOE_F16 || dt == MOE_BF16) ? 2 : 0; }
inline bool aligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline bool dim_ok(int64_t v) { return v >= 1 && v < kMaxDim; }

// rows x [N or I] products: row and tile numbers are 32-bit ints in the kernels
inline int check_product_shape(int64_t rows, int64_t E, int64_t N, int64_t K) {
  if (rows < 0 || rows >= kMaxRows || E < 1 || E > kMaxE || !dim_ok(N) || !dim_ok(K))
    return MOE_ERR_SHAPE;
  if (E * N >= kMaxRows) return MOE_ERR_SHAPE;
  if (((rows + 127) / 128 + E) * ((N + 127) / 128) >= kMaxRows) return MOE_ERR_SHAPE;
  return MOE_OK;
}
// The alignment of one operand in blocks; null pointers are MOE_ERR_NULL.
inline int check_operand(const uint8_t* codes, const uint8_t* scales) {
  if (!codes || !scales) return MOE_ERR_NULL;
  return aligned(codes, 16) && aligned(scales, 4) ? MOE_OK : MOE_ERR_ALIGN;
}
inline int check_ws(const void* ws, size_t have, size_t need) {
  return ws && aligned(ws, 256) && have >= need ? MOE_OK : MOE_ERR_WORKSPACE;
}

}  // namespace mx
}  // namespace moe
