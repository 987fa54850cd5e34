// The grouped products of microscaled 8-bit rows: instances of mx_gemm.cuh.
#include "mx_gemm.cuh"

namespace moe {

cudaError_t launch_mx8_product(MxRows a, int64_t rows, MxRows b, const int32_t* offsets, int E,
                               int N, int K, void* out, int odt, unsigned* status,
                               bool zero_status, cudaStream_t s) {
  return launch_product<Fmt8>(a, rows, b, offsets, E, N, K, out, odt, status, zero_status, s);
}

cudaError_t launch_mx8_gate_up(MxRows a, int64_t rows, MxRows gate, MxRows up,
                               const int32_t* offsets, int E, int I, int H, uint8_t* codes,
                               uint8_t* scales, unsigned* status, bool zero_status, cudaStream_t s) {
  return launch_gate_up<Fmt8>(a, rows, gate, up, offsets, E, I, H, codes, scales, status,
                              zero_status, s);
}

}  // namespace moe
