// moe_mx4_quantize / moe_mx4_dequantize: rows to microscaled 4-bit blocks and back.
//
// A block's scale is a power of two taken from the exponent field of its largest magnitude, so
// scaling is exact and the only rounding is the conversion to e2m1.  Both kernels are bound by
// memory: 2 or 4 bytes a value against 17/32 of a byte.  A lane owns eight consecutive values
// (16 or 32 bytes in, four bytes of codes out), four lanes a block; the block's maximum is two
// shuffles.  A group of L lanes (L = 32, or a smaller power of two for narrow rows) walks one
// row; wide rows are split over several warps so that a few rows still fill the GPU.
#include "launch.h"
#include "mx4.cuh"

namespace moe {
namespace {
using namespace mx4;

constexpr int kThreads = 256;

// How rows are laid over warps: L lanes a row, U units of 8 values a lane in flight, `splits`
// pieces a row.
struct RowPlan {
  int L;
  int splits;
  int units;        // units of 8 values in a row (4 a block)
  int64_t tasks;    // row pieces
};

RowPlan plan_rows(int64_t rows, int64_t K, int U) {
  RowPlan p;
  p.units = (int)blocks_of(K) * 4;
  p.L = 4;
  while (p.L < 32 && p.L < p.units) p.L *= 2;
  const int steps = (p.units + p.L * U - 1) / (p.L * U);
  p.splits = steps;
  // enough pieces to fill 152 SMs x 2048 threads twice; wider rows stay whole beyond that
  while (p.splits > 1 && rows * p.splits * p.L > (int64_t)152 * 2048 * 8) p.splits = (p.splits + 1) / 2;
  p.tasks = rows * p.splits;
  return p;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c0, int K, float* v) {
  if (VEC && c0 + 8 <= K) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
      Vec16<T> q;
      q.u = ld_nc_v4(row + c0 + i * N);
      q.to_float(v + i * N);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + i < K ? Dt<T>::to_f(__ldg(row + c0 + i)) : 0.f;
  }
}

template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(kThreads)
    moe_mx4_quantize_kernel(const T* __restrict__ x, int64_t rows, int K, int64_t ldx,
                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int L,
                            int splits, int units, unsigned* status) {
  if (status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  const int lane = threadIdx.x & 31, gl = lane & (L - 1);
  const int64_t task = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
  const bool ok = task < rows * splits;
  const int64_t r = ok ? task / splits : 0;
  const int piece = ok ? (int)(task - r * splits) : 0;
  const int steps = (units + L * U - 1) / (L * U);
  const T* row = x + r * ldx;
  uint8_t* crow = codes + r * (int64_t)(units * 4);
  uint8_t* srow = scales + r * (int64_t)((units / 4 + 3) / 4 * 4);
  for (int st = piece; st < steps; st += splits) {
    float v[U][8];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int unit = (st * U + j) * L + gl;
      if (ok && unit < units) load8<T, VEC>(row, unit * 8, K, v[j]);
      else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int unit = (st * U + j) * L + gl;
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const uint32_t b = scale_byte(top);
      const uint32_t c = b == 255u ? 0u : codes8(v[j], inv_scale(b));
      if (ok && unit < units) {
        *reinterpret_cast<uint32_t*>(crow + unit * 4) = c;
        if ((unit & 3) == 0) srow[unit >> 2] = (uint8_t)b;
        // the bytes past the last block of the row
        if (unit == units - 1)
          for (int q = units >> 2; q & 3; ++q) srow[q] = 0;
      }
    }
  }
}

template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(kThreads)
    moe_mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                              const uint8_t* __restrict__ scales, int64_t rows, int K,
                              T* __restrict__ out, int64_t ldo, int L, int splits, int units) {
  const int lane = threadIdx.x & 31, gl = lane & (L - 1);
  const int64_t task = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
  if (task >= rows * splits) return;
  const int64_t r = task / splits;
  const int piece = (int)(task - r * splits);
  const int steps = (units + L * U - 1) / (L * U);
  T* row = out + r * ldo;
  const uint8_t* crow = codes + r * (int64_t)(units * 4);
  const uint8_t* srow = scales + r * (int64_t)((units / 4 + 3) / 4 * 4);
  for (int st = piece; st < steps; st += splits) {
    uint32_t c[U], b[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int unit = (st * U + j) * L + gl;
      c[j] = unit < units ? __ldg(reinterpret_cast<const uint32_t*>(crow + unit * 4)) : 0u;
      b[j] = unit < units ? __ldg(srow + (unit >> 2)) : 0u;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int unit = (st * U + j) * L + gl, c0 = unit * 8;
      float v[8];
      values8(c[j], scale_value(b[j]), v);
      if (unit >= units) continue;
      if (VEC && c0 + 8 <= K) {
        constexpr int N = Vec16<T>::N;
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
          Vec16<T> q;
          q.from_float(v + i * N);
          st_v4(row + c0 + i * N, q.u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + i < K) row[c0 + i] = Dt<T>::from_f(v[i]);
      }
    }
  }
}

bool vec_rows(const void* p, int64_t ld, int size) {
  return ((uintptr_t)p & 15u) == 0 && (ld * size) % 16 == 0;
}
unsigned grid_of(const RowPlan& p) {
  return (unsigned)((p.tasks * p.L + kThreads - 1) / kThreads);
}

template <typename T>
cudaError_t quantize_t(const T* x, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                       uint8_t* scales, unsigned* status, cudaStream_t s) {
  constexpr int U = 4;
  const RowPlan p = plan_rows(rows, K, U);
  if (vec_rows(x, ldx, sizeof(T)))
    moe_mx4_quantize_kernel<T, true, U><<<grid_of(p), kThreads, 0, s>>>(
        x, rows, (int)K, ldx, codes, scales, p.L, p.splits, p.units, status);
  else
    moe_mx4_quantize_kernel<T, false, U><<<grid_of(p), kThreads, 0, s>>>(
        x, rows, (int)K, ldx, codes, scales, p.L, p.splits, p.units, status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                         T* out, int64_t ldo, cudaStream_t s) {
  constexpr int U = 4;
  const RowPlan p = plan_rows(rows, K, U);
  if (vec_rows(out, ldo, sizeof(T)))
    moe_mx4_dequantize_kernel<T, true, U><<<grid_of(p), kThreads, 0, s>>>(
        codes, scales, rows, (int)K, out, ldo, p.L, p.splits, p.units);
  else
    moe_mx4_dequantize_kernel<T, false, U><<<grid_of(p), kThreads, 0, s>>>(
        codes, scales, rows, (int)K, out, ldo, p.L, p.splits, p.units);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* x, int xdt, int64_t rows, int64_t K, int64_t ldx,
                                uint8_t* codes, uint8_t* scales, unsigned* status,
                                cudaStream_t s) {
  switch (xdt) {
    case MOE_F32: return quantize_t((const float*)x, rows, K, ldx, codes, scales, status, s);
    case MOE_F16: return quantize_t((const __half*)x, rows, K, ldx, codes, scales, status, s);
    case MOE_BF16:
      return quantize_t((const __nv_bfloat16*)x, rows, K, ldx, codes, scales, status, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                  int64_t K, void* out, int odt, int64_t ldo, cudaStream_t s) {
  switch (odt) {
    case MOE_F32: return dequantize_t(codes, scales, rows, K, (float*)out, ldo, s);
    case MOE_F16: return dequantize_t(codes, scales, rows, K, (__half*)out, ldo, s);
    case MOE_BF16: return dequantize_t(codes, scales, rows, K, (__nv_bfloat16*)out, ldo, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
