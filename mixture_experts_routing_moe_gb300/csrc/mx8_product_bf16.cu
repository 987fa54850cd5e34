// The 8-bit product with results in bf16 (see mx8_gemm.cu).
#include "mx_gemm.cuh"

namespace moe {

cudaError_t launch_mx8_product_bf16(MxRows a, int64_t rows, MxRows b, const int32_t* offsets, int E, int N,
                                  int K, void* out, unsigned* status, bool zero_status,
                                  cudaStream_t s) {
  return launch_product<Fmt8, __nv_bfloat16>(a, rows, b, offsets, E, N, K, out, status, zero_status, s);
}

}  // namespace moe
