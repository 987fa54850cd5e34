// The residual stream's sum and its root-mean-square norm (moe_rms_norm), and the norm's gradient
// (moe_rms_norm_backward).
//
//   s = round(x + residual);  r = (mean(s^2) + eps)^(-1/2);  n = s r;  y = n w
//   dx = ds + r (dy w - n mean(dy w n));  dw = sum over rows of dy n
//
// Both are bound by memory: one read of each input, one write of each output.  A row belongs to W
// consecutive warps of a block (a block holds G rows when rows are short).  A lane owns units of
// eight values, U of them, which wait in registers between the row's sum and its use, so nothing is
// read twice; rows too long for that take kernels that read them again.  Aligned rows: a unit is
// eight consecutive values (16 or 32 bytes), four lanes a block of 32.  Other rows: value i of a
// warp's units is the 32-value block i, a value a lane, so accesses stay coalesced and a block's
// maximum is one warp reduction.  Sums of squares, means and dw are FP32.
#include "launch.h"
#include "mx8.cuh"
#include "norm.cuh"

namespace moe {
namespace {

// Units of a lane: 16 registers an input.
template <typename T>
constexpr int kUnits = sizeof(T) == 4 ? 2 : 4;

template <typename T>
union Unit {
  static constexpr int V = sizeof(T) / 2;
  uint4 u[V];
  T e[8];
};

// Plain loads: outputs may be the inputs themselves.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// Column of value i of a lane's unit, where the warp's 32 units start at unit u0.
template <bool VEC>
__device__ __forceinline__ int column(int u0, int lane, int i) {
  return VEC ? (u0 + lane) * 8 + i : u0 * 8 + i * 32 + lane;
}
// A lane's unit of a row of H values (zeros past it).
template <typename T, bool VEC>
__device__ __forceinline__ Unit<T> load_unit(const T* row, int u0, int lane, int H) {
  Unit<T> q;
  if (VEC && column<VEC>(u0, lane, 8) <= H) {
#pragma unroll
    for (int i = 0; i < Unit<T>::V; ++i)
      q.u[i] = ld_v4(row + column<VEC>(u0, lane, 0) + i * (16 / sizeof(T)));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(u0, lane, i);
      q.e[i] = c < H ? row[c] : Dt<T>::from_f(0.f);
    }
  }
  return q;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* row, const Unit<T>& q, int u0, int lane, int H) {
  if (VEC && column<VEC>(u0, lane, 8) <= H) {
#pragma unroll
    for (int i = 0; i < Unit<T>::V; ++i)
      st_v4(row + column<VEC>(u0, lane, 0) + i * (16 / sizeof(T)), q.u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(u0, lane, i);
      if (c < H) row[c] = q.e[i];
    }
  }
}
template <typename T>
__device__ __forceinline__ void widen(const Unit<T>& q, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = Dt<T>::to_f(q.e[i]);
}
template <typename T>
__device__ __forceinline__ Unit<T> narrow(const float* v) {
  Unit<T> q;
#pragma unroll
  for (int i = 0; i < 8; ++i) q.e[i] = Dt<T>::from_f(v[i]);
  return q;
}
// Eight weights, held in T or in FP32.
template <typename T, bool VEC>
__device__ __forceinline__ void load_weight(const void* w, bool w32, int u0, int lane, int H,
                                            float* v) {
  if (w32) widen(load_unit<float, VEC>((const float*)w, u0, lane, H), v);
  else widen(load_unit<T, VEC>((const T*)w, u0, lane, H), v);
}

// Where a thread works: row `t` of the grid, its warp of the row, and the row's slot of the block.
struct Place {
  int lane, w, g;
  int64_t t;
  bool ok;
};
__device__ __forceinline__ Place place(int W, int64_t T) {
  Place p;
  const int warp = threadIdx.x >> 5;
  p.lane = threadIdx.x & 31;
  p.g = warp / W;
  p.w = warp - p.g * W;
  p.t = (int64_t)blockIdx.x * (blockDim.x / (32 * W)) + p.g;
  p.ok = p.t < T;
  return p;
}
// The sum of v over a row's W warps, in a fixed order (every thread of the block calls it; `part` has
// a float for each warp).
__device__ __forceinline__ float row_sum(float v, int W, const Place& p, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (W == 1) return v;
  __syncthreads();  // the last sum's parts have been read
  if (p.lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < W; ++i) v += part[p.g * W + i];
  return v;
}

// y, and its blocks, of a lane's unit of normalised values.  (Every lane of the warp calls it.)
template <typename T, bool VEC>
__device__ __forceinline__ void finish_unit(const NormArgs& a, int64_t t, bool ok, int u0, int lane,
                                            int blocks, const float* h, float r) {
  const int H = (int)a.H;
  float w[8], v[8];
  load_weight<T, VEC>(a.weight, a.w32, u0, lane, H, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = h[i] * r * w[i];
  if (a.y && ok) store_unit<T, VEC>((T*)a.y + t * a.ldy, narrow<T>(v), u0, lane, H);
  if (!a.codes) return;
  uint8_t* crow = a.codes + t * ((int64_t)blocks * 32);
  uint8_t* srow = a.scales + t * (int64_t)((blocks + 3) / 4 * 4);
  auto put_scale = [&](int blk, uint32_t b) {
    srow[blk] = (uint8_t)b;
    if (blk == blocks - 1)  // the bytes past the last block of the row
      for (int z = blocks; z & 3; ++z) srow[z] = 0;
  };
  // (values past H are zero: their weights are)
  if (VEC) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (column<VEC>(u0, lane, i) >= H) v[i] = 0.f;
      top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t b = mx8::scale_byte(top);
    const float inv = mx8::inv_scale(b);
    uint2 c = make_uint2(mx8::codes4(v, inv), mx8::codes4(v + 4, inv));
    if (b == 255u) c = make_uint2(0u, 0u);
    const int unit = u0 + lane;
    if (ok && unit < blocks * 4) {
      *reinterpret_cast<uint2*>(crow + unit * 8) = c;
      if ((unit & 3) == 0) put_scale(unit >> 2, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(u0, lane, i), blk = u0 / 4 + i;
      float x[4] = {c < H ? v[i] : 0.f, 0.f, 0.f, 0.f};
      const uint32_t b = mx8::scale_byte(
          __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x[0]) & 0x7FFFFFFFu));
      const uint32_t code = b == 255u ? 0u : mx8::codes4(x, mx8::inv_scale(b));
      if (ok && blk < blocks) {
        crow[c] = (uint8_t)code;
        if (lane == 0) put_scale(blk, b);
      }
    }
  }
}

template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(1024)
    moe_rms_norm_kernel(const __grid_constant__ NormArgs a, int W, int blocks) {
  __shared__ float part[32];
  const Place p = place(W, a.T);
  const int H = (int)a.H;
  const int64_t t = p.ok ? p.t : 0;
  const T* x = (const T*)a.x + t * a.ldx;
  const T* res = a.residual ? (const T*)a.residual + t * a.ldr : nullptr;
  Unit<T> q[U];
#pragma unroll
  for (int j = 0; j < U; ++j) q[j] = load_unit<T, VEC>(x, (j * W + p.w) * 32, p.lane, H);
  if (res) {
    Unit<T> q2[U];
#pragma unroll
    for (int j = 0; j < U; ++j) q2[j] = load_unit<T, VEC>(res, (j * W + p.w) * 32, p.lane, H);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float v[8], v2[8];
      widen(q[j], v);
      widen(q2[j], v2);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += v2[i];
      q[j] = narrow<T>(v);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    float v[8];
    widen(q[j], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
  }
  ss = row_sum(ss, W, p, part);
  const float r = 1.f / sqrtf(ss / (float)H + a.eps);
  if (a.rstd && p.ok && p.w == 0 && p.lane == 0) a.rstd[t] = r;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u0 = (j * W + p.w) * 32;
    if (a.sum && p.ok) store_unit<T, VEC>((T*)a.sum + t * a.lds, q[j], u0, p.lane, H);
    float v[8];
    widen(q[j], v);
    finish_unit<T, VEC>(a, t, p.ok, u0, p.lane, blocks, v, r);
  }
}

// Rows that a block's registers do not hold: a block a row, which it reads twice.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024)
    moe_rms_norm_long(const __grid_constant__ NormArgs a, int blocks) {
  __shared__ float part[32];
  const Place p = place(32, a.T);
  const int H = (int)a.H, steps = (blocks * 4 + 1023) / 1024;
  const T* x = (const T*)a.x + p.t * a.ldx;
  const T* res = a.residual ? (const T*)a.residual + p.t * a.ldr : nullptr;
  T* sum = a.sum ? (T*)a.sum + p.t * a.lds : nullptr;
  auto value = [&](int u0) {
    Unit<T> q = load_unit<T, VEC>(x, u0, p.lane, H);
    if (!res) return q;
    float v[8], v2[8];
    widen(q, v);
    widen(load_unit<T, VEC>(res, u0, p.lane, H), v2);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += v2[i];
    return narrow<T>(v);
  };
  float ss = 0.f;
  for (int j = 0; j < steps; ++j) {
    const int u0 = (j * 32 + p.w) * 32;
    const Unit<T> q = value(u0);
    if (sum) store_unit<T, VEC>(sum, q, u0, p.lane, H);
    float v[8], s = 0.f;
    widen(q, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
    ss += s;
  }
  ss = row_sum(ss, 32, p, part);
  const float r = 1.f / sqrtf(ss / (float)H + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[p.t] = r;
  for (int j = 0; j < steps; ++j) {
    const int u0 = (j * 32 + p.w) * 32;
    // a lane reads what it wrote itself (the sum may lie where x or the residual was)
    const Unit<T> q = sum ? load_unit<T, VEC>(sum, u0, p.lane, H) : value(u0);
    float v[8];
    widen(q, v);
    finish_unit<T, VEC>(a, p.t, true, u0, p.lane, blocks, v, r);
  }
}

// -------------------------------------------------------------------------------- backward
// Row groups walk the rows g, g + groups, ...; each keeps its columns' share of dw in registers and
// leaves it in part_dw[group]; moe_column_sum adds the groups in order, so dw repeats bit for bit.
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(512)
    moe_rms_norm_backward_kernel(const __grid_constant__ NormGradArgs a, int W, int groups) {
  __shared__ float part[16];
  const int H = (int)a.H;
  const Place p = place(W, groups);
  float dw[U][8];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  // (the block's groups take their turns together; one without a row left works on row 0 for nothing)
  const int64_t first = (int64_t)blockIdx.x * (blockDim.x / (32 * W));
  for (int64_t t0 = first; t0 < a.T; t0 += groups) {
    const bool ok = p.ok && t0 + p.g < a.T;
    const int64_t t = ok ? t0 + p.g : 0;
    Unit<T> qd[U], qs[U], qa[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u0 = (j * W + p.w) * 32;
      qd[j] = load_unit<T, VEC>((const T*)a.dy + t * a.lddy, u0, p.lane, H);
      qs[j] = load_unit<T, VEC>((const T*)a.s + t * a.lds, u0, p.lane, H);
      if (a.dsum) qa[j] = load_unit<T, VEC>((const T*)a.dsum + t * a.ldds, u0, p.lane, H);
    }
    const float r = a.rstd[t];
    float along = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float d[8], s[8], w[8];
      widen(qd[j], d);
      widen(qs[j], s);
      load_weight<T, VEC>(a.weight, a.w32, (j * W + p.w) * 32, p.lane, H, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = s[i] * r;
        if (ok) dw[j][i] = fmaf(d[i], n, dw[j][i]);
        along = fmaf(d[i] * w[i], n, along);
      }
    }
    if (!a.dx) continue;
    along = row_sum(along, W, p, part) / (float)H;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u0 = (j * W + p.w) * 32;
      float d[8], s[8], w[8], v[8];
      widen(qd[j], d);
      widen(qs[j], s);
      load_weight<T, VEC>(a.weight, a.w32, u0, p.lane, H, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r * (d[i] * w[i] - s[i] * r * along);
      if (a.dsum) {
        float e[8];
        widen(qa[j], e);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += e[i];
      }
      if (ok) store_unit<T, VEC>((T*)a.dx + t * a.lddx, narrow<T>(v), u0, p.lane, H);
    }
  }
  if (!a.dweight || !p.ok) return;
  float* mine = a.part_dw + p.t * (int64_t)a.H;
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>((j * W + p.w) * 32, p.lane, i);
      if (c < H) mine[c] = dw[j][i];
    }
}

// Longer rows: dx by a block a row that reads its row twice; dw's shares by blocks of 256 columns and
// a run of rows.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024)
    moe_rms_norm_backward_long(const __grid_constant__ NormGradArgs a) {
  __shared__ float part[32];
  const Place p = place(32, a.T);
  const int H = (int)a.H, steps = (int)((a.H + 8191) / 8192);
  const T* dy = (const T*)a.dy + p.t * a.lddy;
  const T* s = (const T*)a.s + p.t * a.lds;
  const float r = a.rstd[p.t];
  float along = 0.f;
  for (int j = 0; j < steps; ++j) {
    const int u0 = (j * 32 + p.w) * 32;
    float d[8], h[8], w[8], sum = 0.f;
    widen(load_unit<T, VEC>(dy, u0, p.lane, H), d);
    widen(load_unit<T, VEC>(s, u0, p.lane, H), h);
    load_weight<T, VEC>(a.weight, a.w32, u0, p.lane, H, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(d[i] * w[i], h[i] * r, sum);
    along += sum;
  }
  along = row_sum(along, 32, p, part) / (float)H;
  for (int j = 0; j < steps; ++j) {
    const int u0 = (j * 32 + p.w) * 32;
    float d[8], h[8], w[8], v[8];
    widen(load_unit<T, VEC>(dy, u0, p.lane, H), d);
    widen(load_unit<T, VEC>(s, u0, p.lane, H), h);
    load_weight<T, VEC>(a.weight, a.w32, u0, p.lane, H, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r * (d[i] * w[i] - h[i] * r * along);
    if (a.dsum) {
      float e[8];
      widen(load_unit<T, VEC>((const T*)a.dsum + p.t * a.ldds, u0, p.lane, H), e);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += e[i];
    }
    store_unit<T, VEC>((T*)a.dx + p.t * a.lddx, narrow<T>(v), u0, p.lane, H);
  }
}
template <typename T>
__global__ void __launch_bounds__(256)
    moe_rms_norm_weight_long(const __grid_constant__ NormGradArgs a, int groups) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float dw = 0.f;
  for (int64_t t = blockIdx.y; t < a.T; t += groups)
    dw = fmaf(Dt<T>::to_f(((const T*)a.dy)[t * a.lddy + c]),
              Dt<T>::to_f(((const T*)a.s)[t * a.lds + c]) * a.rstd[t], dw);
  a.part_dw[blockIdx.y * a.H + c] = dw;
}

// out[c] = sum over groups of part[group][c], in a fixed order: a block takes 32 columns, its warps
// every eighth group each.
__global__ void __launch_bounds__(256)
    moe_column_sum(const float* __restrict__ part, int groups, int64_t H, float* __restrict__ out) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int g = warp; g < groups; g += 8) v += part[g * H + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < H) {
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    out[c] = v;
  }
}

bool rows_aligned(const void* p, int64_t ld, size_t size) {
  return !p || (((uintptr_t)p & 15u) == 0 && (ld * (int64_t)size) % 16 == 0);
}

template <typename T, bool VEC, int U>
cudaError_t norm_u(const NormArgs& a, int blocks, int W, cudaStream_t s) {
  const int G = W >= 8 ? 1 : 8 / W;
  moe_rms_norm_kernel<T, VEC, U>
      <<<(unsigned)((a.T + G - 1) / G), 32 * W * G, 0, s>>>(a, W, blocks);
  return cudaGetLastError();
}
template <typename T, bool VEC>
cudaError_t norm_v(const NormArgs& a, cudaStream_t s) {
  const int64_t blocks = mx8::blocks_of(a.H), warps = (blocks + 7) / 8;  // warps at a unit a lane
  constexpr int U = kUnits<T>;
  if (warps > 32 * U) {
    moe_rms_norm_long<T, VEC><<<(unsigned)a.T, 1024, 0, s>>>(a, (int)blocks);
    return cudaGetLastError();
  }
  // Few rows: a unit a lane, for latency.  Many: U, for bytes in flight with fewer threads.
  if (warps <= 32 && a.T * warps <= 152 * 16) return norm_u<T, VEC, 1>(a, (int)blocks, (int)warps, s);
  return norm_u<T, VEC, U>(a, (int)blocks, (int)((warps + U - 1) / U), s);
}
template <typename T>
cudaError_t norm_t(const NormArgs& a, cudaStream_t s) {
  const bool vec = rows_aligned(a.x, a.ldx, sizeof(T)) && rows_aligned(a.residual, a.ldr, sizeof(T)) &&
                   rows_aligned(a.sum, a.lds, sizeof(T)) && rows_aligned(a.y, a.ldy, sizeof(T)) &&
                   rows_aligned(a.weight, 0, 4);
  return vec ? norm_v<T, true>(a, s) : norm_v<T, false>(a, s);
}

// W warps a row and the number of row groups whose shares of dw the workspace holds.
struct GradPlan {
  int W, G, groups;
  bool stays;  // a row fits its warps' registers
};
GradPlan grad_plan(int64_t T, int64_t H, int U) {
  GradPlan p;
  const int64_t warps = (H + 255) / 256;  // at a unit a lane
  p.stays = warps <= 16 * U;
  p.W = p.stays ? (int)((warps + U - 1) / U) : 1;
  p.G = p.W >= 8 ? 1 : 8 / p.W;
  // two blocks an SM of 256 threads (or one of up to 512)
  const int64_t most = p.stays ? (int64_t)152 * (p.W > 8 ? 1 : 2) * p.G : 64;
  const int64_t even = (T + p.G - 1) / p.G * p.G;
  p.groups = (int)(even < most ? even : most);
  return p;
}

template <typename T, bool VEC>
cudaError_t grad_v(const NormGradArgs& a, cudaStream_t s) {
  const GradPlan p = grad_plan(a.T, a.H, kUnits<T>);
  if (p.stays) {
    moe_rms_norm_backward_kernel<T, VEC, kUnits<T>>
        <<<(unsigned)(p.groups / p.G), 32 * p.W * p.G, 0, s>>>(a, p.W, p.groups);
  } else {
    if (a.dweight)  // first: dx may lie where dy was
      moe_rms_norm_weight_long<T>
          <<<dim3((unsigned)((a.H + 255) / 256), (unsigned)p.groups), 256, 0, s>>>(a, p.groups);
    if (a.dx) moe_rms_norm_backward_long<T, VEC><<<(unsigned)a.T, 1024, 0, s>>>(a);
  }
  if (a.dweight)
    moe_column_sum<<<(unsigned)((a.H + 31) / 32), 256, 0, s>>>(a.part_dw, p.groups, a.H, a.dweight);
  return cudaGetLastError();
}
template <typename T>
cudaError_t grad_t(const NormGradArgs& a, cudaStream_t s) {
  const bool vec = rows_aligned(a.dy, a.lddy, sizeof(T)) && rows_aligned(a.s, a.lds, sizeof(T)) &&
                   rows_aligned(a.dsum, a.ldds, sizeof(T)) && rows_aligned(a.dx, a.lddx, sizeof(T)) &&
                   rows_aligned(a.weight, 0, 4);
  return vec ? grad_v<T, true>(a, s) : grad_v<T, false>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int dt, cudaStream_t s) {
  switch (dt) {
    case MOE_F32: return norm_t<float>(a, s);
    case MOE_F16: return norm_t<__half>(a, s);
    case MOE_BF16: return norm_t<__nv_bfloat16>(a, s);
  }
  return cudaErrorInvalidValue;
}

size_t rms_norm_backward_scratch_bytes(int64_t T, int64_t H, int dt) {
  return T < 1 ? 0 : (size_t)grad_plan(T, H, dt == MOE_F32 ? kUnits<float> : kUnits<__half>).groups *
                         H * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const NormGradArgs& a, int dt, cudaStream_t s) {
  switch (dt) {
    case MOE_F32: return grad_t<float>(a, s);
    case MOE_F16: return grad_t<__half>(a, s);
    case MOE_BF16: return grad_t<__nv_bfloat16>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
