// Arguments of the norm's launchers (validated by the entry points in norm_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct NormArgs {
  const void* x;
  const void* residual;  // may be null
  const void* weight;
  bool w32;              // the weight is FP32 (else of the rows' type)
  int64_t T, H, ldx, ldr, lds, ldy;
  float eps;
  void* sum;             // may be null, as y, codes (with scales) and rstd
  void* y;
  uint8_t* codes;
  uint8_t* scales;
  float* rstd;
};
cudaError_t launch_rms_norm(const NormArgs& a, int dt, cudaStream_t s);

struct NormGradArgs {
  const void* dy;
  const void* s;         // the rows that were normalised
  const void* weight;
  bool w32;
  const float* rstd;
  const void* dsum;      // may be null
  int64_t T, H, lddy, lds, ldds, lddx;
  void* dx;              // may be null, as dweight
  float* dweight;
  float* part_dw;        // rms_norm_backward_scratch_bytes() bytes, with dweight
};
size_t rms_norm_backward_scratch_bytes(int64_t T, int64_t H);
cudaError_t launch_rms_norm_backward(const NormGradArgs& a, int dt, cudaStream_t s);

}  // namespace moe
