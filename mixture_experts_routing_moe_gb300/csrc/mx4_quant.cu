// moe_mx4_quantize / moe_mx4_dequantize: rows to microscaled 4-bit blocks and back.
//
// A block's scale is a power of two taken from the exponent field of its largest magnitude, so
// scaling is exact and the only rounding is the conversion to e2m1.  Both kernels are bound by
// memory: 2 or 4 bytes a value against 17/32 of a byte.  A lane owns units of eight consecutive
// values (16 or 32 bytes in, four bytes of codes out), four lanes a block; the block's maximum is
// two shuffles.  A group of L lanes (32, or a smaller power of two for narrow rows) takes U * L
// units of one row, U of them in flight; values wait in their storage type (16 registers for four
// units of 16 bits), which leaves room for 2048 threads an SM: with them widened on arrival,
// 1024 threads fitted and 16384 x 7168 bf16 took 100 us to quantise under the profiler.
// Rows that are not 16-byte aligned are read and written one element a lane, consecutive lanes
// consecutive elements, and turned around in shared memory.
#include "launch.h"
#include "mx4.cuh"

namespace moe {
namespace {
using namespace mx4;

constexpr int kThreads = 256, U = 4;

// Eight values of a unit in their storage type.
template <typename T>
union Unit {
  static constexpr int V = sizeof(T) / 2;  // 16-byte vectors
  uint4 u[V];
  T e[8];
};
// The bits of the largest |value| (as a float; NaN and infinities have an exponent field of 255).
__device__ __forceinline__ uint32_t top_bits(const Unit<float>& q) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(q.e[i]) & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ uint32_t top_bits16(const uint4& u) {
  const uint32_t a = __vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu);
  const uint32_t b = __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu);
  const uint32_t c = __vmaxu2(a, b);
  return max(c & 0xFFFFu, c >> 16);
}
__device__ __forceinline__ uint32_t top_bits(const Unit<__nv_bfloat16>& q) {
  return top_bits16(q.u[0]) << 16;
}
__device__ __forceinline__ uint32_t top_bits(const Unit<__half>& q) {
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top_bits16(q.u[0]))));
}

// Group g of L lanes: row g of the grid's x extent, piece blockIdx.y of the row.
struct Place {
  int64_t row;
  int gl, unit0;  // lane of the group, first unit of the piece
  bool ok;
};
__device__ __forceinline__ Place place(int64_t rows, int L) {
  Place p;
  p.row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
  p.gl = threadIdx.x & (L - 1);
  p.unit0 = (int)blockIdx.y * L * U;
  p.ok = p.row < rows;
  return p;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    moe_mx4_quantize_kernel(const T* __restrict__ x, int64_t rows, int K, int64_t ldx,
                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int L,
                            int units, unsigned* status) {
  __shared__ __align__(16) T turn[VEC ? 1 : kThreads / 32][VEC ? 8 : 256];
  if (status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  const Place p = place(rows, L);
  const T* row = x + (p.ok ? p.row : 0) * ldx;
  Unit<T> q[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u0 = p.unit0 + j * L;  // the group's first unit of this step
    if (VEC) {
      const int c0 = (u0 + p.gl) * 8;
#pragma unroll
      for (int i = 0; i < Unit<T>::V; ++i) q[j].u[i] = make_uint4(0, 0, 0, 0);
      if (p.ok && c0 + 8 <= K) {
#pragma unroll
        for (int i = 0; i < Unit<T>::V; ++i) q[j].u[i] = ld_nc_v4(row + c0 + i * (16 / sizeof(T)));
      } else if (p.ok && c0 < K) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + i < K) q[j].e[i] = __ldg(row + c0 + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = u0 * 8 + i * L + p.gl;
        q[j].e[i] = p.ok && c < K ? __ldg(row + c) : Dt<T>::from_f(0.f);
      }
    }
  }
  uint8_t* crow = codes + p.row * (int64_t)(units * 4);
  uint8_t* srow = scales + p.row * (int64_t)((units / 4 + 3) / 4 * 4);
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (!VEC) {
      T* t = turn[threadIdx.x >> 5] + (threadIdx.x & 31 & ~(L - 1)) * 8;  // the group's part
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i * L + p.gl] = q[j].e[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < Unit<T>::V; ++i)
        q[j].u[i] = *reinterpret_cast<const uint4*>(t + p.gl * 8 + i * (16 / sizeof(T)));
      __syncwarp();
    }
    const int unit = p.unit0 + j * L + p.gl;
    uint32_t top = top_bits(q[j]);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t b = scale_byte(top);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Dt<T>::to_f(q[j].e[i]);
    const uint32_t c = b == 255u ? 0u : codes8(v, inv_scale(b));
    if (p.ok && unit < units) {
      *reinterpret_cast<uint32_t*>(crow + unit * 4) = c;
      if ((unit & 3) == 0) srow[unit >> 2] = (uint8_t)b;
      // the bytes past the last block of the row
      if (unit == units - 1)
        for (int z = units >> 2; z & 3; ++z) srow[z] = 0;
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    moe_mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                              const uint8_t* __restrict__ scales, int64_t rows, int K,
                              T* __restrict__ out, int64_t ldo, int L, int units) {
  __shared__ __align__(16) T turn[VEC ? 1 : kThreads / 32][VEC ? 8 : 256];
  const Place p = place(rows, L);
  T* row = out + p.row * ldo;
  const uint8_t* crow = codes + p.row * (int64_t)(units * 4);
  const uint8_t* srow = scales + p.row * (int64_t)((units / 4 + 3) / 4 * 4);
  uint32_t c[U], b[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int unit = p.unit0 + j * L + p.gl;
    const bool in = p.ok && unit < units;
    c[j] = in ? __ldg(reinterpret_cast<const uint32_t*>(crow + unit * 4)) : 0u;
    b[j] = in ? __ldg(srow + (unit >> 2)) : 0u;
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u0 = p.unit0 + j * L, c0 = (u0 + p.gl) * 8;
    float v[8];
    values8(c[j], scale_value(b[j]), v);
    Unit<T> q;
#pragma unroll
    for (int i = 0; i < 8; ++i) q.e[i] = Dt<T>::from_f(v[i]);
    if (VEC) {
      if (p.ok && c0 + 8 <= K) {
#pragma unroll
        for (int i = 0; i < Unit<T>::V; ++i) st_v4(row + c0 + i * (16 / sizeof(T)), q.u[i]);
      } else if (p.ok) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + i < K) row[c0 + i] = q.e[i];
      }
    } else {
      T* t = turn[threadIdx.x >> 5] + (threadIdx.x & 31 & ~(L - 1)) * 8;
#pragma unroll
      for (int i = 0; i < Unit<T>::V; ++i)
        *reinterpret_cast<uint4*>(t + p.gl * 8 + i * (16 / sizeof(T))) = q.u[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = u0 * 8 + i * L + p.gl;
        if (p.ok && e < K) row[e] = t[i * L + p.gl];
      }
      __syncwarp();
    }
  }
}

struct RowPlan {
  int L, units;  // lanes of a group; units of 8 values in a row (4 a block)
  dim3 grid;
};
RowPlan plan_rows(int64_t rows, int64_t K) {
  RowPlan p;
  p.units = (int)blocks_of(K) * 4;
  p.L = 4;
  while (p.L < 32 && p.L < p.units) p.L *= 2;
  p.grid = dim3((unsigned)((rows * p.L + kThreads - 1) / kThreads),
                (unsigned)((p.units + p.L * U - 1) / (p.L * U)));
  return p;
}

bool vec_rows(const void* p, int64_t ld, int size) {
  return ((uintptr_t)p & 15u) == 0 && (ld * size) % 16 == 0;
}

template <typename T>
cudaError_t quantize_t(const T* x, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                       uint8_t* scales, unsigned* status, cudaStream_t s) {
  const RowPlan p = plan_rows(rows, K);
  const auto kern = vec_rows(x, ldx, sizeof(T)) ? moe_mx4_quantize_kernel<T, true>
                                                : moe_mx4_quantize_kernel<T, false>;
  kern<<<p.grid, kThreads, 0, s>>>(x, rows, (int)K, ldx, codes, scales, p.L, p.units, status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                         T* out, int64_t ldo, cudaStream_t s) {
  const RowPlan p = plan_rows(rows, K);
  const auto kern = vec_rows(out, ldo, sizeof(T)) ? moe_mx4_dequantize_kernel<T, true>
                                                  : moe_mx4_dequantize_kernel<T, false>;
  kern<<<p.grid, kThreads, 0, s>>>(codes, scales, rows, (int)K, out, ldo, p.L, p.units);
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
