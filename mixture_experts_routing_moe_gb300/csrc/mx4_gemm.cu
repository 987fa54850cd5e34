// The grouped products of microscaled 4-bit rows: instances of mx_gemm.cuh.
#include "mx_gemm.cuh"

namespace moe {

cudaError_t launch_mx4_product(MxRows a, int64_t rows, MxRows b, const int32_t* offsets, int E,
                               int N, int K, void* out, int odt, unsigned* status,
                               bool zero_status, cudaStream_t s) {
  const auto fn = odt == MOE_F32   ? launch_product<Fmt4, float>
                  : odt == MOE_F16 ? launch_product<Fmt4, __half>
                                   : launch_product<Fmt4, __nv_bfloat16>;
  return fn(a, rows, b, offsets, E, N, K, out, status, zero_status, s);
}

cudaError_t launch_mx4_gate_up(MxRows a, int64_t rows, MxRows gate, MxRows up,
                               const int32_t* offsets, int E, int I, int H, uint8_t* codes,
                               uint8_t* scales, unsigned* status, cudaStream_t s) {
  return launch_gate_up<Fmt4>(a, rows, gate, up, offsets, E, I, H, codes, scales, status, false, s);
}

}  // namespace moe
