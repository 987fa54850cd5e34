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
//
// Measured: 16384 x 7168 bf16, sum, y and blocks 170 us, 6.2 TB/s of what it has to move (0.91 of a
// copy's rate); the gradient at 16384 x 4096 with ds 87 us and the sum of dw's shares 3, 6.0 TB/s.
// A row a block, without the next one's loads in flight, took 183 and 133.
#include "launch.h"
#include "mx8.cuh"
#include "norm.cuh"

namespace moe {
namespace {

// Units of a lane: 16 registers an input.
template <typename T>
constexpr int kUnits = sizeof(T) == 4 ? 2 : 4;

// Eight values, as words: a union with elements of 16 bits is taken apart into them where a full and a
// partial unit's paths meet, and every word put together again.
template <typename T>
struct Unit {
  static constexpr int V = sizeof(T) / 2, WORDS = 4 * V;  // 16-byte vectors, 32-bit words
  uint32_t w[WORDS];
};
template <typename T>
__device__ __forceinline__ void put_vec(Unit<T>& q, int i, const uint4& v) {
  q.w[4 * i] = v.x, q.w[4 * i + 1] = v.y, q.w[4 * i + 2] = v.z, q.w[4 * i + 3] = v.w;
}
// One element of a row (0 past it), as bits; READ_ONLY: no one writes the row.
template <typename T, bool READ_ONLY>
__device__ __forceinline__ uint32_t element(const T* row, int c, int H) {
  if (c >= H) return 0u;
  if constexpr (sizeof(T) == 4) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + c;
    return READ_ONLY ? __ldg(p) : *p;
  } else {
    const unsigned short* p = reinterpret_cast<const unsigned short*>(row) + c;
    return READ_ONLY ? __ldg(p) : *p;
  }
}

// Rows are read once and leave L1 to the weights; not through the read-only path, as outputs may be
// the inputs themselves.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
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
template <typename T, bool VEC, bool READ_ONLY>
__device__ __forceinline__ void load_elements(const T* row, int u0, int lane, int H, Unit<T>& q) {
  constexpr int PER = 8 / Unit<T>::WORDS;  // elements of a word
#pragma unroll
  for (int i = 0; i < Unit<T>::WORDS; ++i) {
    q.w[i] = element<T, READ_ONLY>(row, column<VEC>(u0, lane, PER * i), H);
    if (PER == 2)
      q.w[i] |= element<T, READ_ONLY>(row, column<VEC>(u0, lane, PER * i + 1), H) << 16;
  }
}
// A lane's unit of a row of H values (zeros past it).
template <typename T, bool VEC>
__device__ __forceinline__ Unit<T> load_unit(const T* row, int u0, int lane, int H) {
  Unit<T> q;
  if (VEC && column<VEC>(u0, lane, 8) <= H) {
#pragma unroll
    for (int i = 0; i < Unit<T>::V; ++i)
      put_vec(q, i, ld_v4(row + column<VEC>(u0, lane, 0) + i * (16 / sizeof(T))));
  } else {
    load_elements<T, VEC, false>(row, u0, lane, H, q);
  }
  return q;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* row, const Unit<T>& q, int u0, int lane, int H) {
  if (VEC && column<VEC>(u0, lane, 8) <= H) {
#pragma unroll
    for (int i = 0; i < Unit<T>::V; ++i)
      st_v4(row + column<VEC>(u0, lane, 0) + i * (16 / sizeof(T)),
            make_uint4(q.w[4 * i], q.w[4 * i + 1], q.w[4 * i + 2], q.w[4 * i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(u0, lane, i);
      if (c >= H) continue;
      if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(row)[c] = q.w[i];
      else reinterpret_cast<unsigned short*>(row)[c] = (unsigned short)(q.w[i / 2] >> (i % 2 * 16));
    }
  }
}
// Two FP32 values in a register pair, for the packed instructions: the kernels are nearly as much bound
// by the issue of instructions as by memory (16384 x 7168 bf16 with residual and blocks: 44 a value and
// 205 us with elements of 16 bits, one FP32 value an instruction and the weight read behind the sum; 30
// and 170 us so).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(f2 v) {
  const float2 f = unpack(v);
  return f.x + f.y;
}

// The values of a unit in FP32, and back (rounded once).
__device__ __forceinline__ void widen(const Unit<float>& q, f2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pack(__uint_as_float(q.w[2 * i]), __uint_as_float(q.w[2 * i + 1]));
}
__device__ __forceinline__ void widen(const Unit<__half>& q, f2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(q.w[i]));
    v[i] = pack(lo, hi);
  }
}
__device__ __forceinline__ void widen(const Unit<__nv_bfloat16>& q, f2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pack(__uint_as_float(q.w[i] << 16), __uint_as_float(q.w[i] & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ Unit<T> narrow(const f2* v) {
  Unit<T> q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack(v[i]);
    if constexpr (sizeof(T) == 4) {
      q.w[2 * i] = __float_as_uint(f.x);
      q.w[2 * i + 1] = __float_as_uint(f.y);
    } else if constexpr (Dt<T>::code == MOE_F16) {
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(q.w[i]) : "f"(f.y), "f"(f.x));
    } else {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(q.w[i]) : "f"(f.y), "f"(f.x));
    }
  }
  return q;
}
// s = round(x + residual)
template <typename T>
__device__ __forceinline__ Unit<T> add_units(const Unit<T>& x, const Unit<T>& res) {
  f2 a[4], b[4];
  widen(x, a);
  widen(res, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = add2(a[i], b[i]);
  return narrow<T>(a);
}
// A lane's unit of the weight (zeros past it).
template <typename TW, bool VEC>
__device__ __forceinline__ Unit<TW> load_weight(const void* weight, int u0, int lane, int H) {
  const TW* w = (const TW*)weight;
  Unit<TW> q;
  if (VEC && column<VEC>(u0, lane, 8) <= H) {
#pragma unroll
    for (int i = 0; i < Unit<TW>::V; ++i)
      put_vec(q, i, __ldg(reinterpret_cast<const uint4*>(w + column<VEC>(u0, lane, 0)) + i));
  } else {
    load_elements<TW, VEC, true>(w, u0, lane, H, q);
  }
  return q;
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
// The sum of v over a row's W warps, in a fixed order (every thread of the row calls it: a row has a barrier
// of its own; `part` has a float for each warp, whose last values every thread of the row has read before
// another barrier).
__device__ __forceinline__ float row_sum(float v, int W, const Place& p, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (W == 1) return v;
  if (p.lane == 0) part[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(p.g + 1), "r"(32 * W) : "memory");
  v = 0.f;
  for (int i = 0; i < W; ++i) v += part[p.g * W + i];
  return v;
}

// 1 / sqrt(m) to half a unit in FP32: one step of Newton's method from the approximation, its residual
// 1 - m r^2 taken exactly (fused).  (1 / sqrtf(m) is off by up to one and a half.)
__device__ __forceinline__ float rsqrt_exact(float m) {
  const float r = rsqrtf(m), t = m * r;
  const float e = fmaf(-t, r, 1.f) - fmaf(m, r, -t) * r;
  return r > 0.f && r < INFINITY ? fmaf(0.5f * r, e, r) : r;
}
// The sum of a unit's squares, as a tree.
__device__ __forceinline__ f2 squares(const f2* v) {
  return add2(fma2(v[1], v[1], mul2(v[0], v[0])), fma2(v[3], v[3], mul2(v[2], v[2])));
}
// A mean (with eps) below 2^-100 may have squares that FP32 loses.  Such a row is summed and normalised
// again times 2^100: the square of its smallest number is then 2^-98, the sum of 2^24 squares at most
// 2^124.  Only calls with an eps below 2^-100 can meet one, and take kernels that look (LIFTS): the few
// registers that it takes cost 6 % (16384 x 7168 bf16 with blocks), in f32 5 to 20 %.
constexpr float kTiny = 0x1p-100f, kLift = 0x1p100f;
__device__ __forceinline__ void lift_unit(f2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], pack(kLift, kLift));
}
// The larger of m and two magnitudes; a NaN stays one.
__device__ __forceinline__ float max_abs(float m, f2 v) {
  const float2 f = unpack(v);
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(f.x)), "f"(fabsf(f.y)));
  return m;
}

// y, and its blocks, of a lane's unit of normalised values.  (Every lane of the warp calls it.)
template <typename T, typename TW, bool VEC>
__device__ __forceinline__ void finish_unit(const NormArgs& a, int64_t t, int u0, int lane, int blocks,
                                            const f2* h, const Unit<TW>& w, float r) {
  const int H = (int)a.H;
  f2 v[4];
  widen(w, v);
  const f2 r2 = pack(r, r), minus = pack(-r, -r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // h r w with one rounding (h r and what its rounding left, both times w): a value next to a border
    // between codes is moved by a step of the code.  (An infinite w may meet a remainder of zero: NaN.
    // To look for one cost 7 %, 16384 x 7168 bf16 with blocks.)
    const f2 left = fma2(h[i], r2, mul2(h[i], minus));
    v[i] = fma2(mul2(h[i], r2), v[i], mul2(left, v[i]));
  }
  if (a.y) store_unit<T, VEC>((T*)a.y + t * a.ldy, narrow<T>(v), u0, lane, H);
  if (!a.codes) return;
  uint8_t* crow = a.codes + t * ((int64_t)blocks * 32);
  uint8_t* srow = a.scales + t * (int64_t)((blocks + 3) / 4 * 4);
  auto put_scale = [&](int blk, uint32_t b) {
    srow[blk] = (uint8_t)b;
    if (blk == blocks - 1)  // the bytes past the last block of the row
      for (int z = blocks; z & 3; ++z) srow[z] = 0;
  };
  if (VEC) {
    if (column<VEC>(u0, lane, 8) > H) {  // values past H are zeros, whatever r is
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack(v[i]);
        v[i] = pack(column<VEC>(u0, lane, 2 * i) < H ? f.x : 0.f,
                    column<VEC>(u0, lane, 2 * i + 1) < H ? f.y : 0.f);
      }
    }
    float m = max_abs(max_abs(max_abs(max_abs(0.f, v[0]), v[1]), v[2]), v[3]);
    uint32_t top = __float_as_uint(m);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t b = mx8::scale_byte(top);
    const float inv = mx8::inv_scale(b);
    uint2 c = make_uint2(mx8::codes4(v, pack(inv, inv)), mx8::codes4(v + 2, pack(inv, inv)));
    if (b == 255u) c = make_uint2(0u, 0u);
    const int unit = u0 + lane;
    if (unit < blocks * 4) {
      *reinterpret_cast<uint2*>(crow + unit * 8) = c;
      if ((unit & 3) == 0) put_scale(unit >> 2, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(u0, lane, i), blk = u0 / 4 + i;
      const float2 f = unpack(v[i / 2]);
      float x[4] = {c < H ? (i & 1 ? f.y : f.x) : 0.f, 0.f, 0.f, 0.f};
      const uint32_t b = mx8::scale_byte(
          __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x[0]) & 0x7FFFFFFFu));
      const uint32_t code = b == 255u ? 0u : mx8::codes4(x, mx8::inv_scale(b));
      if (blk < blocks) {
        crow[c] = (uint8_t)code;
        if (lane == 0) put_scale(blk, b);
      }
    }
  }
}

// Blocks of 256 threads on an SM: two leave registers for two rows of 16 bits.
template <typename T>
constexpr int kNormBlocks = sizeof(T) == 4 ? 4 : 2;

// A lane's units of a row of x and of the residual.
template <typename T, bool VEC, int U>
__device__ __forceinline__ void load_rows(const NormArgs& a, int64_t t, int W, const Place& p,
                                          Unit<T>* x, Unit<T>* res) {
  const int H = (int)a.H;
#pragma unroll
  for (int j = 0; j < U; ++j)
    x[j] = load_unit<T, VEC>((const T*)a.x + t * a.ldx, (j * W + p.w) * 32, p.lane, H);
  if (!a.residual) return;
#pragma unroll
  for (int j = 0; j < U; ++j)
    res[j] = load_unit<T, VEC>((const T*)a.residual + t * a.ldr, (j * W + p.w) * 32, p.lane, H);
}

// Row groups walk the rows g, g + groups, ..., a row ahead with their loads where registers allow it;
// the weight stays in registers.  THREADS: the most that a block has; BLOCKS of them an SM.  LIFTS: kTiny.
template <typename T, typename TW, bool VEC, bool LIFTS, int U, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS)
    moe_rms_norm_kernel(const __grid_constant__ NormArgs a, int W, int64_t groups, int blocks) {
  __shared__ float part[LIFTS ? 3 : 2][32];
  constexpr bool AHEAD = U > 1 && sizeof(T) == 2 && THREADS <= 512;
  const int H = (int)a.H;
  const Place p = place(W, groups);
  Unit<TW> w[U];
  Unit<T> q[U], q2[U], n[U], n2[U];
  if (AHEAD && p.t < a.T) load_rows<T, VEC, U>(a, p.t, W, p, n, n2);
#pragma unroll
  for (int j = 0; j < U; ++j) w[j] = load_weight<TW, VEC>(a.weight, (j * W + p.w) * 32, p.lane, H);
  int turn = 0;
  // (the block's groups take their turns together; one without a row left only joins the sum)
  for (int64_t t0 = p.t - p.g; t0 < a.T; t0 += groups, turn ^= 1) {
    const int64_t t = t0 + p.g;
    const bool ok = t < a.T;
    if (AHEAD) {
#pragma unroll
      for (int j = 0; j < U; ++j) q[j] = n[j], q2[j] = n2[j];
      if (t + groups < a.T) load_rows<T, VEC, U>(a, t + groups, W, p, n, n2);
    } else if (ok) {
      load_rows<T, VEC, U>(a, t, W, p, q, q2);
    }
    f2 parts = 0;
    if (ok) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (a.residual) q[j] = add_units(q[j], q2[j]);
        if (a.sum) store_unit<T, VEC>((T*)a.sum + t * a.lds, q[j], (j * W + p.w) * 32, p.lane, H);
        f2 v[4];
        widen(q[j], v);
        parts = add2(parts, squares(v));
      }
    }
    float mean = row_sum(sum2(parts), W, p, part[turn]) / (float)H + a.eps;
    if (!ok) continue;
    const bool lifted = LIFTS && mean < kTiny;
    if (lifted) {
      parts = 0;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        f2 v[4];
        widen(q[j], v);
        lift_unit(v);
        parts = add2(parts, squares(v));
      }
      mean = row_sum(sum2(parts), W, p, part[2]) / (float)H + a.eps * kLift * kLift;
    }
    const float r = rsqrt_exact(mean);
    if (a.rstd && p.w == 0 && p.lane == 0) a.rstd[t] = lifted ? r * kLift : r;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      f2 v[4];
      widen(q[j], v);
      if (lifted) lift_unit(v);
      finish_unit<T, TW, VEC>(a, t, (j * W + p.w) * 32, p.lane, blocks, v, w[j], r);
    }
  }
}

// Rows that a block's registers do not hold: a block a row, which it reads twice.
template <typename T, typename TW, bool VEC, bool LIFTS>
__global__ void __launch_bounds__(1024)
    moe_rms_norm_long(const __grid_constant__ NormArgs a, int blocks) {
  __shared__ float part[LIFTS ? 2 : 1][32];
  const Place p = place(32, a.T);
  const int H = (int)a.H, steps = (blocks * 4 + 1023) / 1024;
  const T* x = (const T*)a.x + p.t * a.ldx;
  const T* res = a.residual ? (const T*)a.residual + p.t * a.ldr : nullptr;
  T* sum = a.sum ? (T*)a.sum + p.t * a.lds : nullptr;
  auto value = [&](int u0) {
    const Unit<T> q = load_unit<T, VEC>(x, u0, p.lane, H);
    return res ? add_units(q, load_unit<T, VEC>(res, u0, p.lane, H)) : q;
  };
  f2 parts = 0;
  for (int j = 0; j < steps; ++j) {
    const int u0 = (j * 32 + p.w) * 32;
    const Unit<T> q = value(u0);
    if (sum) store_unit<T, VEC>(sum, q, u0, p.lane, H);
    f2 v[4];
    widen(q, v);
    parts = add2(parts, squares(v));
  }
  // a lane reads what it wrote itself (the sum may lie where x or the residual was)
  auto again = [&](int u0) { return sum ? load_unit<T, VEC>(sum, u0, p.lane, H) : value(u0); };
  float mean = row_sum(sum2(parts), 32, p, part[0]) / (float)H + a.eps;
  const bool lifted = LIFTS && mean < kTiny;
  if (lifted) {
    parts = 0;
    for (int j = 0; j < steps; ++j) {
      f2 v[4];
      widen(again((j * 32 + p.w) * 32), v);
      lift_unit(v);
      parts = add2(parts, squares(v));
    }
    mean = row_sum(sum2(parts), 32, p, part[LIFTS]) / (float)H + a.eps * kLift * kLift;
  }
  const float r = rsqrt_exact(mean);
  if (a.rstd && threadIdx.x == 0) a.rstd[p.t] = lifted ? r * kLift : r;
  for (int j = 0; j < steps; ++j) {
    const int u0 = (j * 32 + p.w) * 32;
    f2 v[4];
    widen(again(u0), v);
    if (lifted) lift_unit(v);
    finish_unit<T, TW, VEC>(a, p.t, u0, p.lane, blocks, v,
                            load_weight<TW, VEC>(a.weight, u0, p.lane, H), r);
  }
}

// -------------------------------------------------------------------------------- backward
constexpr int kGradBlocks = 2;  // of 256 threads, on an SM
// One unit's terms: n = s r and dn = dy w; what they add to the mean's sum, and to dw.
__device__ __forceinline__ f2 grad_terms(const f2* d, const f2* s, const f2* w, f2 r, f2 along, f2* dw) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 n = mul2(s[i], r);
    if (dw) dw[i] = fma2(d[i], n, dw[i]);
    along = fma2(mul2(d[i], w[i]), n, along);
  }
  return along;
}
// r (dy w - n mean) + ds of a unit; back: -r times the mean.
template <typename T>
__device__ __forceinline__ Unit<T> grad_unit(const f2* d, const f2* s, const f2* w, f2 r, f2 back,
                                             const f2* ds) {
  f2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = mul2(r, fma2(s[i], back, mul2(d[i], w[i])));
    if (ds) v[i] = add2(v[i], ds[i]);
  }
  return narrow<T>(v);
}

// A lane's units of a row's dy, s and ds.
template <typename T, int U>
struct GradRow {
  Unit<T> d[U], s[U], e[U];
  float r;
};
template <typename T, bool VEC, int U>
__device__ __forceinline__ void load_row(const NormGradArgs& a, int64_t t, int W, const Place& p,
                                         GradRow<T, U>& q) {
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u0 = (j * W + p.w) * 32, H = (int)a.H;
    q.d[j] = load_unit<T, VEC>((const T*)a.dy + t * a.lddy, u0, p.lane, H);
    q.s[j] = load_unit<T, VEC>((const T*)a.s + t * a.lds, u0, p.lane, H);
    if (a.dsum) q.e[j] = load_unit<T, VEC>((const T*)a.dsum + t * a.ldds, u0, p.lane, H);
  }
  q.r = __ldg(a.rstd + t);
}

// Row groups walk the rows g, g + groups, ..., a row ahead with their loads; each keeps its columns'
// share of dw in registers and leaves it in part_dw[group]; moe_column_sum adds the groups in order,
// so dw repeats bit for bit.
template <typename T, typename TW, bool VEC, int U, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? kGradBlocks : 1)
    moe_rms_norm_backward_kernel(const __grid_constant__ NormGradArgs a, int W, int groups) {
  __shared__ float part[2][16];
  const int H = (int)a.H;
  const Place p = place(W, groups);
  f2 dw[U][4];
  Unit<TW> qw[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = 0;
    qw[j] = load_weight<TW, VEC>(a.weight, (j * W + p.w) * 32, p.lane, H);
  }
  // (the block's groups take their turns together; one without a row left only joins the sum)
  constexpr bool AHEAD = sizeof(T) == 2;  // (two rows of FP32 would spill)
  GradRow<T, U> q, next;
  if (AHEAD && p.t < a.T) load_row<T, VEC, U>(a, p.t, W, p, next);
  int turn = 0;
  for (int64_t t0 = p.t - p.g; t0 < a.T; t0 += groups, turn ^= 1) {
    const int64_t t = t0 + p.g;
    if (AHEAD) {
      q = next;
      if (t + groups < a.T) load_row<T, VEC, U>(a, t + groups, W, p, next);
    } else if (t < a.T) {
      load_row<T, VEC, U>(a, t, W, p, q);
    }
    const f2 r2 = pack(q.r, q.r);
    f2 sum = 0;
    if (t < a.T) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        f2 d[4], s[4], w[4];
        widen(q.d[j], d);
        widen(q.s[j], s);
        widen(qw[j], w);
        sum = grad_terms(d, s, w, r2, sum, dw[j]);
      }
    }
    if (!a.dx) continue;
    const float along = row_sum(sum2(sum), W, p, part[turn]) / (float)H;
    if (t >= a.T) continue;
    const f2 back = pack(-q.r * along, -q.r * along);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      f2 d[4], s[4], w[4], e[4];
      widen(q.d[j], d);
      widen(q.s[j], s);
      widen(qw[j], w);
      if (a.dsum) widen(q.e[j], e);
      store_unit<T, VEC>((T*)a.dx + t * a.lddx,
                         grad_unit<T>(d, s, w, r2, back, a.dsum ? e : nullptr),
                         (j * W + p.w) * 32, p.lane, H);
    }
  }
  if (!a.dweight) return;
  float* mine = a.part_dw + p.t * (int64_t)a.H;
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack(dw[j][i]);
      const int c = column<VEC>((j * W + p.w) * 32, p.lane, 2 * i);
      const int c1 = column<VEC>((j * W + p.w) * 32, p.lane, 2 * i + 1);
      if (c < H) mine[c] = f.x;
      if (c1 < H) mine[c1] = f.y;
    }
}

// Longer rows: dx by a block a row that reads its row twice; dw's shares by blocks of 256 columns and
// a run of rows.
template <typename T, typename TW, bool VEC>
__global__ void __launch_bounds__(1024)
    moe_rms_norm_backward_long(const __grid_constant__ NormGradArgs a) {
  __shared__ float part[32];
  const Place p = place(32, a.T);
  const int H = (int)a.H, steps = (int)((a.H + 8191) / 8192);
  const T* dy = (const T*)a.dy + p.t * a.lddy;
  const T* s = (const T*)a.s + p.t * a.lds;
  const float r = a.rstd[p.t];
  f2 sum = 0;
  for (int j = 0; j < steps; ++j) {
    const int u0 = (j * 32 + p.w) * 32;
    f2 d[4], h[4], w[4];
    widen(load_unit<T, VEC>(dy, u0, p.lane, H), d);
    widen(load_unit<T, VEC>(s, u0, p.lane, H), h);
    widen(load_weight<TW, VEC>(a.weight, u0, p.lane, H), w);
    sum = add2(sum, grad_terms(d, h, w, pack(r, r), 0, nullptr));
  }
  const float along = row_sum(sum2(sum), 32, p, part) / (float)H;
  const f2 back = pack(-r * along, -r * along);
  for (int j = 0; j < steps; ++j) {
    const int u0 = (j * 32 + p.w) * 32;
    f2 d[4], h[4], w[4], e[4];
    widen(load_unit<T, VEC>(dy, u0, p.lane, H), d);
    widen(load_unit<T, VEC>(s, u0, p.lane, H), h);
    widen(load_weight<TW, VEC>(a.weight, u0, p.lane, H), w);
    if (a.dsum) widen(load_unit<T, VEC>((const T*)a.dsum + p.t * a.ldds, u0, p.lane, H), e);
    store_unit<T, VEC>((T*)a.dx + p.t * a.lddx,
                       grad_unit<T>(d, h, w, pack(r, r), back, a.dsum ? e : nullptr), u0, p.lane, H);
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
// every 32nd group each.
__global__ void __launch_bounds__(1024)
    moe_column_sum(const float* __restrict__ part, int groups, int64_t H, float* __restrict__ out) {
  __shared__ float s[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int g = warp; g < groups; g += 32) v += part[g * H + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < H) {
#pragma unroll 8
    for (int i = 1; i < 32; ++i) v += s[i][lane];
    out[c] = v;
  }
}

bool rows_aligned(const void* p, int64_t ld, size_t size) {
  return !p || (((uintptr_t)p & 15u) == 0 && (ld * (int64_t)size) % 16 == 0);
}

template <typename T, typename TW, bool VEC, bool LIFTS>
cudaError_t norm_l(const NormArgs& a, cudaStream_t s) {
  constexpr int U = kUnits<T>;
  const int64_t blocks = mx8::blocks_of(a.H), warps = (blocks + 7) / 8;  // warps at a unit a lane
  if (warps > 32 * U) {
    moe_rms_norm_long<T, TW, VEC, LIFTS><<<(unsigned)a.T, 1024, 0, s>>>(a, (int)blocks);
    return cudaGetLastError();
  }
  // Few rows: a unit a lane, for latency.  Many: U, for bytes in flight with fewer threads.  (In bf16 with
  // blocks, few / many: 1 x 2048 2.8 / 3.8 us, 608 x 2048 4.2 / 4.5, 1216 x 2048 6.6 / 5.4; 152 x 7168
  // 4.1 / 4.6, 304 x 7168 7.0 / 5.3.)
  const bool few = warps <= 32 && a.T * warps <= 152 * 32;
  const int W = few ? (int)warps : (int)((warps + U - 1) / U), G = W >= 8 ? 1 : 8 / W;
  const auto kern = few       ? moe_rms_norm_kernel<T, TW, VEC, LIFTS, 1, 1024, 1>
                    : W <= 8  ? moe_rms_norm_kernel<T, TW, VEC, LIFTS, U, 256, kNormBlocks<T>>
                    : W <= 16 ? moe_rms_norm_kernel<T, TW, VEC, LIFTS, U, 512, 1>
                              : moe_rms_norm_kernel<T, TW, VEC, LIFTS, U, 1024, 1>;
  const int64_t all = (a.T + G - 1) / G, most = W <= 8 ? 152 * kNormBlocks<T> : 152;
  const int64_t grid = few || all < most ? all : most;
  kern<<<(unsigned)grid, 32 * W * G, 0, s>>>(a, W, grid * G, (int)blocks);
  return cudaGetLastError();
}
template <typename T, typename TW, bool VEC>
cudaError_t norm_v(const NormArgs& a, cudaStream_t s) {
  if constexpr (Dt<T>::code != MOE_F16)  // (FP32 holds f16's squares)
    if (a.eps < kTiny) return norm_l<T, TW, VEC, true>(a, s);
  return norm_l<T, TW, VEC, false>(a, s);
}
template <typename T>
cudaError_t norm_t(const NormArgs& a, cudaStream_t s) {
  const bool vec = rows_aligned(a.x, a.ldx, sizeof(T)) && rows_aligned(a.residual, a.ldr, sizeof(T)) &&
                   rows_aligned(a.sum, a.lds, sizeof(T)) && rows_aligned(a.y, a.ldy, sizeof(T)) &&
                   rows_aligned(a.weight, 0, 4);
  if (a.w32) return vec ? norm_v<T, float, true>(a, s) : norm_v<T, float, false>(a, s);
  return vec ? norm_v<T, T, true>(a, s) : norm_v<T, T, false>(a, s);
}

// U units a lane and W warps a row; the number of row groups whose shares of dw the workspace holds.
struct GradPlan {
  int U, W, G, groups;  // U = 0: a row does not fit its warps' registers
};
GradPlan grad_plan(int64_t T, int64_t H) {
  GradPlan p;
  const int64_t warps = (H + 255) / 256;  // at a unit a lane
  p.U = warps <= 32 ? 2 : 0;  // two of them, and those of the next row, leave two blocks an SM
  p.W = p.U ? (int)((warps + p.U - 1) / p.U) : 1;
  p.G = p.W >= 8 ? 1 : 8 / p.W;
  const int64_t most = p.U ? (int64_t)152 * (p.W > 8 ? 1 : kGradBlocks) * p.G : 64;
  const int64_t even = (T + p.G - 1) / p.G * p.G;
  p.groups = (int)(even < most ? even : most);
  return p;
}

template <typename T, typename TW, bool VEC>
cudaError_t grad_v(const NormGradArgs& a, cudaStream_t s) {
  const GradPlan p = grad_plan(a.T, a.H);
  if (p.U) {
    auto kern = p.W <= 8 ? moe_rms_norm_backward_kernel<T, TW, VEC, 2, 256>
                         : moe_rms_norm_backward_kernel<T, TW, VEC, 2, 512>;
    kern<<<(unsigned)(p.groups / p.G), 32 * p.W * p.G, 0, s>>>(a, p.W, p.groups);
  } else {
    if (a.dweight)  // first: dx may lie where dy was
      moe_rms_norm_weight_long<T>
          <<<dim3((unsigned)((a.H + 255) / 256), (unsigned)p.groups), 256, 0, s>>>(a, p.groups);
    if (a.dx) moe_rms_norm_backward_long<T, TW, VEC><<<(unsigned)a.T, 1024, 0, s>>>(a);
  }
  if (a.dweight)
    moe_column_sum<<<(unsigned)((a.H + 31) / 32), 1024, 0, s>>>(a.part_dw, p.groups, a.H, a.dweight);
  return cudaGetLastError();
}
template <typename T>
cudaError_t grad_t(const NormGradArgs& a, cudaStream_t s) {
  const bool vec = rows_aligned(a.dy, a.lddy, sizeof(T)) && rows_aligned(a.s, a.lds, sizeof(T)) &&
                   rows_aligned(a.dsum, a.ldds, sizeof(T)) && rows_aligned(a.dx, a.lddx, sizeof(T)) &&
                   rows_aligned(a.weight, 0, 4);
  if (a.w32) return vec ? grad_v<T, float, true>(a, s) : grad_v<T, float, false>(a, s);
  return vec ? grad_v<T, T, true>(a, s) : grad_v<T, T, false>(a, s);
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

size_t rms_norm_backward_scratch_bytes(int64_t T, int64_t H) {
  return T < 1 ? 0 : (size_t)grad_plan(T, H).groups * H * sizeof(float);
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
