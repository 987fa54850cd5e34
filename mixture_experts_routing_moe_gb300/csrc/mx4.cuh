// Microscaled 4-bit (MXFP4) blocks on the device: sizes, a block's scale, codes and values.
#pragma once

#include "../../include/moe_mx4.h"
#include "common.cuh"

namespace moe {
namespace mx4 {

__host__ __device__ inline int64_t blocks_of(int64_t K) { return (K + 31) / 32; }
__host__ __device__ inline int64_t code_pitch(int64_t K) { return blocks_of(K) * 16; }
__host__ __device__ inline int64_t scale_pitch(int64_t K) { return (blocks_of(K) + 3) / 4 * 4; }

// Scale byte of a block whose largest magnitude has the bits `amax` (sign clear): with
// amax = 2^p m, 1 <= m < 2, the scale is 2^(p - 2), byte p + 125, which is the exponent field
// less two; subnormals and tiny values clamp to byte 0, and infinities and NaN (field 255) keep
// 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t f = amax >> 23;
  return f == 255u ? 255u : (f < 2u ? 0u : f - 2u);
}
// 2^-(scale), exact: byte b in [0, 252] gives exponent field 254 - b in [2, 254].  For byte 255
// it is 0, which makes the codes of finite values zero (those of NaN are cleared by the caller).
__device__ __forceinline__ float inv_scale(uint32_t b) {
  return __uint_as_float(b == 255u ? 0u : (254u - b) << 23);
}
// 2^(b - 127); byte 0 is the subnormal 2^-127, 255 a NaN.
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : (b == 255u ? 0x7FC00000u : b << 23));
}

// Eight scaled values to four bytes of codes, the first value in the lowest nibble (round to
// nearest even, saturating).
__device__ __forceinline__ uint32_t codes8(const float* v, float inv) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv), "f"(v[4] * inv),
        "f"(v[5] * inv), "f"(v[6] * inv), "f"(v[7] * inv));
  return r;
}
// Four bytes of codes to eight values.
__device__ __forceinline__ void values8(uint32_t c, float s, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

}  // namespace mx4

// ---- launchers (arguments are validated by the entry points in mx4_api.cu) ----
// status, when not null, is zeroed by the launch (the first of its entry point).
cudaError_t launch_mx4_quantize(const void* x, int xdt, int64_t rows, int64_t K, int64_t ldx,
                                uint8_t* codes, uint8_t* scales, unsigned* status, cudaStream_t s);
cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                  int64_t K, void* out, int odt, int64_t ldo, cudaStream_t s);
// One row operand of a product.
struct Mx4Rows {
  const uint8_t* codes;
  const uint8_t* scales;
};
// out = A B^T by groups; zero_status: this launch zeroes *status (it is the first of the call).
cudaError_t launch_mx4_product(Mx4Rows a, int64_t rows, Mx4Rows b, const int32_t* offsets, int E,
                               int N, int K, void* out, int odt, unsigned* status,
                               bool zero_status, cudaStream_t s);
// codes / scales of silu(A gate^T) * (A up^T), rows of I values.
cudaError_t launch_mx4_gate_up(Mx4Rows a, int64_t rows, Mx4Rows gate, Mx4Rows up,
                               const int32_t* offsets, int E, int I, int H, uint8_t* codes,
                               uint8_t* scales, unsigned* status, cudaStream_t s);


// The whole layer for a few tokens.  ws holds tokens_layout().total bytes; its first `zeroed` bytes
// are cleared by the first launch.
struct Mx4TokensLayout {
  size_t ready, done, zeroed;      // counters behind the header
  size_t logits, xq, xs, aq, as, y, total;
};
Mx4TokensLayout mx4_tokens_layout(int64_t T, int64_t E, int64_t H, int64_t I, int k);
struct Mx4TokensArgs {
  const void* x;
  const void* router;
  int dt, T, E, H, I, k, renorm;
  Mx4Rows gate, up, down;
  void* out;
  uint32_t* idx;  // may be null
  float* w;       // may be null
  uint8_t* ws;
};
cudaError_t launch_mx4_tokens(const Mx4TokensArgs& a, cudaStream_t s);
constexpr int kMx4TokensMaxT = 64, kMx4TokensMaxK = 32, kMx4TokensMaxSlots = 1024;

}  // namespace moe
