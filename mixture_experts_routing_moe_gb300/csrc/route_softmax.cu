// Group-limited softmax routing (moe_route_softmax_grouped).
//
// p = softmax(logits) over all E experts; c = p + bias (the bias steers the selection only).  The E
// experts form G contiguous groups; a group scores its largest c, or the sum of its two largest.
// The SG best groups are kept, then the top_k experts inside them by c; ties go to the lower id.
// w = p of the chosen, divided by their sum when renormalising, times scale.
//
// The selection is the one that float64 arithmetic makes.  A warp owns a row, a lane `per`
// consecutive experts, and it is decided in FP32 first:
//   without a bias, experts (and groups by their largest) are ranked by their logits, which is the
//   exact softmax's ranking; sums of two are compared as exp(l1 - max) + exp(l2 - max);
//   with one, c is FP32, off by at most err = kappa p_max + 2^-23 max|c|: an exponential is off by
//   2^-22 (ex2.approx) and by 1.8e-7 d for d = max - l (three roundings of the exponent), which
//   weighs at most 1.25e-6 in a sum of 1024 terms (sum p d <= ln E), and that sum by another
//   (C + 5) 2^-24.
// Where a margin that the choice rests on is within twice the bound (the last kept group against the
// best other one, each chosen expert against the next, unless the two have the same logit and bias),
// or a score is not finite, the warp decides the row again in float64.
//
// What bounds it is the issue of instructions: some 600 a row of 256 experts.  Chosen experts come
// from k rounds of a warp maximum over the lanes' best keys (redux), where the lane that gave the
// maximum looks for its next best.
#include "common.cuh"
#include "launch.h"
#include "route_sigmoid_core.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxGroups = 128;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct SoftmaxRoute {
  const void* logits;
  const float* bias;  // may be null
  int64_t T;
  int E, k, G, SG, two, renorm;
  int per;    // consecutive experts of a lane, per * 32 >= E
  int lanes;  // lanes of a group (a power of two), or 0 where groups are not whole lanes
  float scale;
  uint32_t* idx;
  void* w;
};

// Larger floats give larger keys, never 0; -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key >> 31) ? (key & 0x7FFFFFFFu) : ~key);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// exp(x - m), off by 2^-22 and by 1.8e-7 (m - x)
__device__ __forceinline__ float exp_below(float x, float m) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((x - m) * 1.44269504f));
  return e;
}

// Score of a group whose two largest are b1 >= b2.
template <typename F>
__device__ __forceinline__ F group_score(F b1, F b2, int two) {
  return two && b1 < (F)INFINITY ? b1 + b2 : b1;
}

template <typename T>
__device__ __forceinline__ void write_slot(const SoftmaxRoute& a, int64_t row, int r, int id,
                                           float w) {
  a.idx[row * a.k + r] = (uint32_t)id;
  reinterpret_cast<T*>(a.w)[row * a.k + r] = Dt<T>::from_f(w);
}

// l: the logits of this lane's slots (lane, lane + 32); returns the largest of all slots.
template <typename T>
__device__ __forceinline__ float largest_chosen(const SoftmaxRoute& a, const T* src,
                                                const int* mine, float* l) {
  const int lane = threadIdx.x & 31;
  uint32_t key = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] = lane + 32 * h < a.k ? Dt<T>::to_f(src[mine[h]]) : -INFINITY;
    key = max(key, key_of(l[h]));
  }
  return value_of(__reduce_max_sync(kAll, key));
}

// The row's decision in float64.  cs: scratch of E + kMaxGroups doubles.
template <typename T>
__device__ __noinline__ void route_row_f64(const SoftmaxRoute& a, int64_t row, float m, double* cs) {
  const int lane = threadIdx.x & 31, gs = a.E / a.G;
  const T* src = reinterpret_cast<const T*>(a.logits) + row * a.E;
  double* score = cs + a.E;
  double z = 0.0;
  for (int e = lane; e < a.E; e += 32) {
    cs[e] = exp((double)Dt<T>::to_f(src[e]) - (double)m);
    z += cs[e];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
  bool nan = false;
  if (a.bias)
    for (int e = lane; e < a.E; e += 32) {
      cs[e] = cs[e] / z + (double)a.bias[e];
      nan |= cs[e] != cs[e];
    }
  // (without a bias the exponentials rank groups as the probabilities do)
  if (__any_sync(kAll, nan)) {
    for (int r = lane; r < a.k; r += 32) write_slot<T>(a, row, r, r, __int_as_float(0x7FC00000));
    return;
  }
  __syncwarp();
  for (int g = lane; g < a.G; g += 32) {
    double b1 = -INFINITY, b2 = -INFINITY;
    for (int j = 0; j < gs; ++j) {
      const double v = cs[g * gs + j];
      if (v > b1) {
        b2 = b1;
        b1 = v;
      } else if (v > b2) {
        b2 = v;
      }
    }
    score[g] = group_score(b1, b2, a.two);
  }
  __syncwarp();
  unsigned kept[kMaxGroups / 32] = {};
#pragma unroll
  for (int q = 0; q < kMaxGroups / 32; ++q) {
    const int g = q * 32 + lane;
    int rank = 0;
    if (g < a.G)
      for (int h = 0; h < a.G; ++h)
        rank += score[h] > score[g] || (score[h] == score[g] && h < g);
    kept[q] = __ballot_sync(kAll, g < a.G && rank < a.SG);
  }
  // k rounds of a warp maximum over the experts that are kept and not taken yet
  unsigned open = 0;  // of this lane's experts lane, lane + 32, ...
  for (int i = 0; lane + 32 * i < a.E; ++i) {
    const int g = (lane + 32 * i) / gs;
    unsigned word = 0;
#pragma unroll
    for (int q = 0; q < kMaxGroups / 32; ++q) word = g / 32 == q ? kept[q] : word;
    if ((word >> (g & 31)) & 1u) open |= 1u << i;
  }
  int mine[2] = {0, 0};
  for (int r = 0; r < a.k; ++r) {
    double bv = -INFINITY;
    int bi = 0x7FFFFFFF;
    for (int i = 0; lane + 32 * i < a.E; ++i) {
      const int e = lane + 32 * i;
      const double v = a.bias ? cs[e] : (double)Dt<T>::to_f(src[e]);
      if (((open >> i) & 1u) && (bi == 0x7FFFFFFF || v > bv)) {
        bv = v;
        bi = e;
      }
    }
    warp_argmax(bv, bi);
    if ((bi & 31) == lane) open &= ~(1u << (bi >> 5));
    if (r == lane) mine[0] = bi;
    if (r == lane + 32) mine[1] = bi;
  }
  // renormalised weights do not depend on m: the largest chosen logit keeps them from vanishing
  float l[2];
  const float largest = largest_chosen<T>(a, src, mine, l);
  if (a.renorm) m = largest;
  double sel = 0.0, w[2] = {0.0, 0.0};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (lane + 32 * h < a.k) {
      w[h] = exp((double)l[h] - (double)m);
      sel += w[h];
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sel += __shfl_xor_sync(kAll, sel, o);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (lane + 32 * h < a.k)
      write_slot<T>(a, row, lane + 32 * h, mine[h],
                    (float)(w[h] / (a.renorm ? sel : z) * (double)a.scale));
}

// C: registers for a lane's experts, at least a.per
template <typename T, int C>
__global__ void __launch_bounds__(kWarps * 32)
    moe_route_softmax_kernel(const __grid_constant__ SoftmaxRoute a, int vec) {
  extern __shared__ double soft_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  if (row >= a.T) return;  // whole warps leave
  double* cs = soft_smem + (size_t)warp * (a.E + kMaxGroups);
  const T* src = reinterpret_cast<const T*>(a.logits) + row * a.E;
  const int e0 = lane * a.per, n = max(0, min(a.per, a.E - e0));  // this lane's experts
  float x[C];
  if (vec) {  // per == C, whole 16-byte vectors
    constexpr int PER = 16 / (int)sizeof(T);
#pragma unroll
    for (int v = 0; v < (C + PER - 1) / PER; ++v) {
      Vec16<T> q;
      q.u = make_uint4(0, 0, 0, 0);
      if (n > 0) q.u = ld_nc_v4(src + e0 + v * PER);
#pragma unroll
      for (int i = 0; i < PER && v * PER + i < C; ++i)
        x[v * PER + i] = n > 0 ? Dt<T>::to_f(q.e[i]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = i < n ? Dt<T>::to_f(src[e0 + i]) : -INFINITY;
  }
  float m = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    m = fmaxf(m, x[i]);
    bad |= !(x[i] < INFINITY);  // NaN or +inf
  }
  const uint32_t mk = __reduce_max_sync(kAll, key_of(m));
  m = value_of(mk);
  if (__any_sync(kAll, bad) || m == -INFINITY) {
    for (int r = lane; r < a.k; r += 32) write_slot<T>(a, row, r, r, __int_as_float(0x7FC00000));
    return;
  }
  // c: what ranks the experts; -inf past them
  float z = 0.f, c[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    c[i] = exp_below(x[i], m);
    z += c[i];
  }
  z = warp_sum(z);
  float err = 0.f;
  bool sure = true;
  if (a.bias) {
    const float inv = 1.f / z;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float b = i < n ? __ldg(a.bias + e0 + i) : 0.f;
      c[i] = fmaf(c[i], inv, b);
      if (i < n) top = fmaxf(top, fabsf(c[i]));
      sure &= fabsf(c[i]) < INFINITY;
    }
    top = value_of(__reduce_max_sync(kAll, key_of(top)));
    err = (2.5e-6f + 6.5e-8f * C) * inv + 1.2e-7f * top;
    sure = __all_sync(kAll, sure);
  }
  // keep: whether this lane's experts are in a kept group (bit i: expert i)
  unsigned keep = n > 0 ? (n < 32 ? (1u << n) - 1u : ~0u) : 0u;
  const bool by_logit = !a.bias && !a.two;  // groups too
  if (sure && a.SG < a.G) {
    float* score = reinterpret_cast<float*>(cs);  // [G], the two scores at the border, then c [E]
    const int gs = a.E / a.G;
    if (a.lanes) {  // a group is a.lanes whole lanes
      float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float v = i < n ? (by_logit ? x[i] : c[i]) : -INFINITY;
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
      for (int o = 1; o < a.lanes; o <<= 1) {
        const float o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
      if (n > 0 && (lane & (a.lanes - 1)) == 0) score[lane / a.lanes] = group_score(b1, b2, a.two);
    } else {
      float* sc = score + kMaxGroups + 2;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i < n) sc[e0 + i] = by_logit ? x[i] : c[i];
      __syncwarp();
      for (int g = lane; g < a.G; g += 32) {
        float b1 = -INFINITY, b2 = -INFINITY;
        for (int j = 0; j < gs; ++j) {
          const float v = sc[g * gs + j];
          b2 = fmaxf(b2, fminf(b1, v));
          b1 = fmaxf(b1, v);
        }
        score[g] = group_score(b1, b2, a.two);
      }
    }
    __syncwarp();
    unsigned kept[kMaxGroups / 32] = {};
#pragma unroll
    for (int q = 0; q < kMaxGroups / 32; ++q) {
      if (q * 32 >= a.G) break;
      const int g = q * 32 + lane;
      const float mine = g < a.G ? score[g] : 0.f;
      int rank = 0;
      for (int h = 0; h < a.G; ++h) {
        const float v = score[h];
        rank += v > mine || (v == mine && h < g);
      }
      if (g < a.G && rank >= a.SG - 1 && rank <= a.SG) score[kMaxGroups + rank - a.SG + 1] = mine;
      kept[q] = __ballot_sync(kAll, g < a.G && rank < a.SG);
    }
    __syncwarp();
    if (!by_logit) {
      const float in = score[kMaxGroups], out = score[kMaxGroups + 1];
      // sums of two exponentials: 4e-7 of the sum and 2 * 0.37 * 1.8e-7 (d e^-d <= 0.37)
      const float bound = a.bias ? (a.two ? 2.f * err + 1.2e-7f * fabsf(in) : err)
                                 : 4e-7f * in + 1.4e-7f;
      sure = in - out > 2.f * bound;
    }
    unsigned word = 0, of_kept = 0;
    int was = -1;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (i < n) {
        const int g = (e0 + i) / gs;
        if (g != was) {
          was = g;
#pragma unroll
          for (int q = 0; q < kMaxGroups / 32; ++q) word = g / 32 == q ? kept[q] : word;
        }
        of_kept |= ((word >> (g & 31)) & 1u) << i;
      }
    }
    keep = of_kept;
  }
  // k rounds (and one more for the margin): the lanes' best keys, their maximum, the lowest lane
  uint32_t key[C];
#pragma unroll
  for (int i = 0; i < C; ++i) key[i] = (keep >> i) & 1u ? key_of(a.bias ? c[i] : x[i]) : 0u;
  auto best_of = [&]() {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) b = max(b, key[i]);
    return b;
  };
  uint32_t best = best_of();
  const int rounds = a.k + (a.bias && a.k < a.SG * (a.E / a.G) ? 1 : 0);
  int mine[2] = {0, 0}, last = 0;
  float before = 0.f;
  for (int r = 0; r < rounds && sure; ++r) {
    const uint32_t top = __reduce_max_sync(kAll, best);
    const int from = __ffs(__ballot_sync(kAll, best == top)) - 1;
    int id = 0;
    if (lane == from) {
      int at = 0;
#pragma unroll
      for (int i = C - 1; i >= 0; --i) at = key[i] == top ? i : at;
#pragma unroll
      for (int i = 0; i < C; ++i) key[i] = i == at ? 0u : key[i];
      best = best_of();
      id = e0 + at;
    }
    id = __shfl_sync(kAll, id, from);
    if (a.bias) {
      const float v = value_of(top);
      if (r > 0 && !(before - v > 2.f * err))  // then only equal inputs are sure: the lower id is first
        sure = Dt<T>::to_f(src[id]) == Dt<T>::to_f(src[last]) && a.bias[id] == a.bias[last];
      before = v;
      last = id;
    }
    if (r == lane && r < a.k) mine[0] = id;
    if (r == lane + 32 && r < a.k) mine[1] = id;
  }
  if (!sure) {
    __syncwarp();
    route_row_f64<T>(a, row, m, cs);
    return;
  }
  float w[2] = {0.f, 0.f}, l[2];
  const float largest = largest_chosen<T>(a, src, mine, l);
  if (a.renorm) m = largest;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (lane + 32 * h < a.k) w[h] = expf(l[h] - m);
  const float by = a.renorm ? warp_sum(w[0] + w[1]) : z;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (lane + 32 * h < a.k) write_slot<T>(a, row, lane + 32 * h, mine[h], w[h] / by * a.scale);
}

template <typename T, int C>
cudaError_t launch_c(const SoftmaxRoute& a, cudaStream_t s) {
  const size_t smem = kWarps * (size_t)(a.E + kMaxGroups) * sizeof(double);
  const int vec = a.per == C && a.E % C == 0 && C * sizeof(T) % 16 == 0 &&
                  ((uintptr_t)a.logits & 15u) == 0 && a.E * sizeof(T) % 16 == 0;
  moe_route_softmax_kernel<T, C>
      <<<(unsigned)((a.T + kWarps - 1) / kWarps), kWarps * 32, smem, s>>>(a, vec);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_t(const SoftmaxRoute& a, cudaStream_t s) {
  if (a.per <= 4) return launch_c<T, 4>(a, s);
  if (a.per <= 8) return launch_c<T, 8>(a, s);
  if (a.per <= 16) return launch_c<T, 16>(a, s);
  return launch_c<T, 32>(a, s);
}

}  // namespace

cudaError_t launch_route_softmax_grouped(const void* logits, int ldt, const float* bias, int64_t T,
                                         int E, int k, int G, int SG, int top_two, int renorm,
                                         float scale, uint32_t* idx, void* w, cudaStream_t s) {
  SoftmaxRoute a{};
  a.logits = logits;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.k = k;
  a.G = G;
  a.SG = SG;
  a.two = top_two;
  a.renorm = renorm;
  a.scale = scale;
  a.idx = idx;
  a.w = w;
  // Experts of a lane: the fewest that make a group a power of two of whole lanes, as the groups'
  // scores then take a few shuffles instead of a walk through shared memory; else the fewest.
  const int gs = E / G, least = (E + 31) / 32;
  a.per = least;
  for (int per = least; per <= 32 && per <= gs; ++per)
    if (gs % per == 0 && ((gs / per) & (gs / per - 1)) == 0) {
      a.per = per;
      a.lanes = gs / per;
      break;
    }
  switch (ldt) {
    case MOE_F32: return launch_t<float>(a, s);
    case MOE_F16: return launch_t<__half>(a, s);
    case MOE_BF16: return launch_t<__nv_bfloat16>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
