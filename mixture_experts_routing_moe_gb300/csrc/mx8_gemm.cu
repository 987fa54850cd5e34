// The grouped products of microscaled 8-bit rows: instances of mx_gemm.cuh (those of the product's types
// in files of their own, which compile side by side).
#include "mx_gemm.cuh"

namespace moe {

#define MX8_PRODUCT(name)                                                                       \
  cudaError_t name(MxRows a, int64_t rows, MxRows b, const int32_t* offsets, int E, int N, int K, \
                   void* out, unsigned* status, bool zero_status, cudaStream_t s)
MX8_PRODUCT(launch_mx8_product_f32);
MX8_PRODUCT(launch_mx8_product_f16);
MX8_PRODUCT(launch_mx8_product_bf16);

cudaError_t launch_mx8_product(MxRows a, int64_t rows, MxRows b, const int32_t* offsets, int E,
                               int N, int K, void* out, int odt, unsigned* status,
                               bool zero_status, cudaStream_t s) {
  const auto fn = odt == MOE_F32   ? launch_mx8_product_f32
                  : odt == MOE_F16 ? launch_mx8_product_f16
                                   : launch_mx8_product_bf16;
  return fn(a, rows, b, offsets, E, N, K, out, status, zero_status, s);
}

cudaError_t launch_mx8_gate_up(MxRows a, int64_t rows, MxRows gate, MxRows up,
                               const int32_t* offsets, int E, int I, int H, uint8_t* codes,
                               uint8_t* scales, unsigned* status, bool zero_status,
                               cudaStream_t s) {
  return launch_gate_up<Fmt8>(a, rows, gate, up, offsets, E, I, H, codes, scales, status, zero_status,
                              s);
}

}  // namespace moe
