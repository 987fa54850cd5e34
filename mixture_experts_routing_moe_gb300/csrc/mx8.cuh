// Microscaled 8-bit (MXFP8) blocks on the device: sizes, a block's scale, codes and values.
#pragma once

#include "../../include/moe_mx8.h"
#include "mx4.cuh"

namespace moe {
namespace mx8 {

using mx4::blocks_of;
using mx4::inv_scale;
using mx4::scale_pitch;
using mx4::scale_value;
__host__ __device__ inline int64_t code_pitch(int64_t K) { return blocks_of(K) * 32; }

// Scale byte of a block whose largest magnitude has the bits `amax` (sign clear): the least power of
// two that leaves it at most 448 = 1.75 * 2^8.  With amax = 2^p m, 1 <= m < 2, that is 2^(p - 8), or
// 2^(p - 7) for m > 1.75, which the addition carries into the exponent field.  Byte p + 119 or p + 120;
// clamped to 0 below, and infinities and NaN (field 255) get 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t f = (amax + 0x1FFFFFu) >> 23;
  return amax >= 0x7F800000u ? 255u : (f < 8u ? 0u : f - 8u);
}

// Four scaled values to four e4m3 codes, the first in the lowest byte (round to nearest even; the scale
// leaves none above 448).
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
  uint32_t r;
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h0, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h1, %4, %3;\n\t"
      "mov.b32 %0, {h0, h1};\n\t}"
      : "=r"(r)
      : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv));
  return r;
}
// The same of two register pairs, scaled with the packed multiplication.
__device__ __forceinline__ uint32_t codes4(const unsigned long long* v, unsigned long long inv) {
  uint32_t r;
  asm("{\n\t.reg .b64 a, b;\n\t.reg .f32 f0, f1, f2, f3;\n\t.reg .b16 h0, h1;\n\t"
      "mul.rn.f32x2 a, %1, %3;\n\t"
      "mul.rn.f32x2 b, %2, %3;\n\t"
      "mov.b64 {f0, f1}, a;\n\t"
      "mov.b64 {f2, f3}, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h0, f1, f0;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h1, f3, f2;\n\t"
      "mov.b32 %0, {h0, h1};\n\t}"
      : "=r"(r)
      : "l"(v[0]), "l"(v[1]), "l"(inv));
  return r;
}
// Four codes to four values.
__device__ __forceinline__ void values4(uint32_t c, float s, float* v) {
  uint32_t h[2];
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "mov.b32 {h0, h1}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h0;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h1;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

}  // namespace mx8

// ---- launchers (arguments are validated by the entry points in mx8_api.cu) ----
cudaError_t launch_mx8_quantize(const void* x, int xdt, int64_t rows, int64_t K, int64_t ldx,
                                uint8_t* codes, uint8_t* scales, cudaStream_t s);
cudaError_t launch_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                  int64_t K, void* out, int odt, int64_t ldo, cudaStream_t s);
// As launch_mx4_product() and launch_mx4_gate_up(); zero_status: the launch zeroes *status.
cudaError_t launch_mx8_product(MxRows a, int64_t rows, MxRows b, const int32_t* offsets, int E,
                               int N, int K, void* out, int odt, unsigned* status,
                               bool zero_status, cudaStream_t s);
cudaError_t launch_mx8_gate_up(MxRows a, int64_t rows, MxRows gate, MxRows up,
                               const int32_t* offsets, int E, int I, int H, uint8_t* codes,
                               uint8_t* scales, unsigned* status, bool zero_status,
                               cudaStream_t s);


}  // namespace moe
