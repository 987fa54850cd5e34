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
// best other one, each chosen expert against the next, unless the two have the same logit and bias,
// and the last one against the first that is not tied with it so), or a score is not finite, the warp
// decides the row again in float64.
//
// What bounds it is the issue of integer and FP32 instructions: some 1050 a row of 256 experts with
// eight groups and a bias, 18 us for 16384 rows, and the last rows that float64 decides (28 us
// together; 65536 rows 79).  These are of logits of spread 2, where 32 of the 16384 rows go there; a zero
// bias and spreads of 6 and 8 send 8 and 26 % (43 and 79 us), and one bias of -inf all (200).  With k
// rounds of a warp maximum, each of which sent the lane that gave it looking for its next best, a row
// took 1800 (57 us, 25 of them 32 rows in float64).  So the choice is made among few: the rounds run over
// the lanes' best alone, which bounds the last choice from below, the experts above that bound (mostly a
// dozen) go to shared memory, one for each lane, and each counts those before it.  The float64 form keeps
// a lane's scores in registers, so that its exponentials overlap, and ranks them as 64-bit integers.
#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxGroups = 128;
constexpr unsigned kAll = 0xFFFFFFFFu;

// 64-bit words of a warp's scratch: a key an expert and a group; whole 16-byte vectors.
__host__ __device__ constexpr int scratch_words(int E) { return (E + 1) / 2 * 2 + kMaxGroups; }

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

// Order-preserving map of a double that is not NaN to 64 bits (-0 counts as +0), never 0.
__device__ __forceinline__ unsigned long long key64_of(double v) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double value64_of(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}
// The largest of the lanes' keys.
__device__ __forceinline__ unsigned long long warp_max64(unsigned long long k) {
  const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (unsigned long long)hi << 32 | lo;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) { return warp_max64(k); }

// b1, b2: the two largest of a lane's keys so far; takes another one.
template <typename K>
__device__ __forceinline__ void take_two(K& b1, K& b2, K k) {
  b2 = max(b2, min(b1, k));
  b1 = max(b1, k);
}

// Which of a lane's n experts (from e0 on) are in a kept group, as bits.  key: their scores' keys, which
// value and key_of_value turn into scores and back.  VEC: n is C or 0.  scratch: E keys and kMaxGroups
// more.  in, out: the keys of the scores of the last kept group and of the best other one.
template <int C, bool VEC, typename K, typename ToValue, typename ToKey>
__device__ __forceinline__ unsigned kept_experts(const SoftmaxRoute& a, const K* key, int e0, int n,
                                                 K* scratch, ToValue value, ToKey key_of_value,
                                                 K* in, K* out) {
  const int lane = threadIdx.x & 31, gs = a.E / a.G;
  auto score_key = [&](K b1, K b2) { return key_of_value(group_score(value(b1), value(b2), a.two)); };
  if (a.lanes) {  // a group is a.lanes whole lanes: each of them has its score
    K b1 = 0, b2 = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) take_two(b1, b2, (VEC ? n > 0 : i < n) ? key[i] : (K)0);
    for (int o = 1; o < a.lanes; o <<= 1) {
      const K o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
      b2 = max(max(b2, o2), min(b1, o1));
      b1 = max(b1, o1);
    }
    const int mine = lane / a.lanes;
    const K sc = n > 0 ? score_key(b1, b2) : (K)0;
    int rank = 0;
    for (int h = 0; h < a.G; ++h) {
      const K v = __shfl_sync(kAll, sc, h * a.lanes);
      rank += h < mine ? v >= sc : v > sc;
    }
    const bool kept = n > 0 && rank < a.SG;
    *in = ~warp_max(n > 0 && kept ? ~sc : (K)0);
    *out = warp_max(kept ? (K)0 : sc);
    return kept ? (n < 32 ? (1u << n) - 1u : ~0u) : 0u;
  }
  K* score = scratch + a.E;
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i < n) scratch[e0 + i] = key[i];
  __syncwarp();
  for (int g = lane; g < a.G; g += 32) {
    K b1 = 0, b2 = 0;
    for (int j = 0; j < gs; ++j) take_two(b1, b2, scratch[g * gs + j]);
    score[g] = score_key(b1, b2);
  }
  __syncwarp();
  unsigned kept[kMaxGroups / 32] = {};
  K last = 0, best = 0;  // of this lane's: the complement of the least kept, the best other
#pragma unroll
  for (int q = 0; q < kMaxGroups / 32; ++q) {
    const int g = q * 32 + lane;
    if (q * 32 < a.G) {
      const K sc = g < a.G ? score[g] : (K)0;
      int rank = 0;
      for (int h = 0; h < a.G; ++h) rank += h < g ? score[h] >= sc : score[h] > sc;
      const bool keep = g < a.G && rank < a.SG;
      kept[q] = __ballot_sync(kAll, keep);
      if (keep) last = max(last, ~sc);
      else best = max(best, sc);
    }
  }
  *in = ~warp_max(last);
  *out = warp_max(best);
  unsigned bits = 0;
  int g = e0 / gs, left = gs - (e0 - g * gs);  // the expert's group, and how many of it are left
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i < n) {
      unsigned word = 0;
#pragma unroll
      for (int q = 0; q < kMaxGroups / 32; ++q) word = g / 32 == q ? kept[q] : word;
      bits |= ((word >> (g & 31)) & 1u) << i;
      if (--left == 0) {
        left = gs;
        ++g;
      }
    }
  return bits;
}

// The next best of the lanes' keys: its key, and its expert's id in every lane; its owner takes it out.
template <int C, typename K>
__device__ __forceinline__ int take_best(K* key, K& best, int e0, K* top) {
  *top = warp_max(best);
  const int from = __ffs(__ballot_sync(kAll, best == *top)) - 1;  // the lowest lane: the lowest id
  int id = 0;
  if ((int)(threadIdx.x & 31) == from) {
    int at = 0;
#pragma unroll
    for (int i = C - 1; i >= 0; --i) at = key[i] == *top ? i : at;
    best = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      key[i] = i == at ? (K)0 : key[i];
      best = max(best, key[i]);
    }
    id = e0 + at;
  }
  return __shfl_sync(kAll, id, from);
}

// The row's choice in float64 (m: its largest logit, a number): the experts of this lane's slots, lane
// and lane + 32, as two halves; all ones where a bias is NaN.
template <typename T, int C>
__device__ __noinline__ unsigned long long choose_f64(const SoftmaxRoute& a, int64_t row, float m,
                                                      unsigned long long* scratch) {
  typedef unsigned long long K;
  const int lane = threadIdx.x & 31, e0 = lane * a.per, n = max(0, min(a.per, a.E - e0));
  const T* src = reinterpret_cast<const T*>(a.logits) + row * a.E;
  double c[C], z = 0.0;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    c[i] = i < n ? exp((double)Dt<T>::to_f(src[e0 + i]) - (double)m) : 0.0;
    z += c[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
  const double inv = 1.0 / z;
  bool nan = false;
  K key[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (a.bias && i < n) c[i] = fma(c[i], inv, (double)a.bias[e0 + i]);
    nan |= c[i] != c[i];
    key[i] = i < n ? key64_of(c[i]) : 0ull;
  }
  if (__any_sync(kAll, nan)) return ~0ull;
  unsigned keep = n > 0 ? (n < 32 ? (1u << n) - 1u : ~0u) : 0u;
  if (a.SG < a.G) {
    K in, out;
    keep = kept_experts<C, false>(a, key, e0, n, scratch, value64_of, key64_of, &in, &out);
  }
  K best = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    // (without a bias the logits rank the experts, the exponentials only pairs of them)
    if (!a.bias && i < n) key[i] = key_of(Dt<T>::to_f(src[e0 + i]));
    if (!((keep >> i) & 1u)) key[i] = 0;
    best = max(best, key[i]);
  }
  unsigned long long mine = 0;
  for (int r = 0; r < a.k; ++r) {
    K top;
    const unsigned id = take_best<C>(key, best, e0, &top);
    if (r == lane) mine |= id;
    if (r == lane + 32) mine |= (unsigned long long)id << 32;
  }
  return mine;
}

// N values from p on, which is 16-byte aligned.
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  constexpr int PER = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < N / PER; ++i) {
    Vec16<T> q;
    q.u = ld_nc_v4(p + i * PER);
    q.to_float(v + i * PER);
  }
}

// C: registers for a lane's experts, at least a.per; VEC: a.per == C, in 16-byte vectors
template <typename T, int C, bool VEC>
__global__ void __launch_bounds__(kWarps * 32)
    moe_route_softmax_kernel(const __grid_constant__ SoftmaxRoute a) {
  extern __shared__ __align__(16) unsigned long long soft_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  if (row >= a.T) return;  // whole warps leave
  unsigned long long* scratch = soft_smem + (size_t)warp * scratch_words(a.E);
  const T* src = reinterpret_cast<const T*>(a.logits) + row * a.E;
  const int e0 = lane * a.per, n = max(0, min(a.per, a.E - e0));  // this lane's experts
  auto in = [&](int i) { return VEC ? n > 0 : i < n; };
  float x[C], c[C];
#pragma unroll
  for (int i = 0; i < C; ++i) x[i] = -INFINITY;
  if (VEC) {
    if (n > 0) load_vec<T, C>(src + e0, x);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) x[i] = Dt<T>::to_f(src[e0 + i]);
  }
  float m = x[0];
#pragma unroll
  for (int i = 1; i < C; ++i) m = fmaxf(m, x[i]);
  m = value_of(warp_max(key_of(m)));
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    c[i] = exp_below(x[i], m);
    z += c[i];
  }
  z = warp_sum(z);
  if (!(z < INFINITY)) {  // a NaN, a +inf or only -inf: NaN
    for (int r = lane; r < a.k; r += 32) write_slot<T>(a, row, r, r, __int_as_float(0x7FC00000));
    return;
  }
  float err = 0.f;
  bool sure = true;
  uint32_t key[C];  // of what ranks the experts
  if (a.bias) {
    const float inv = 1.f / z;
    float b[C];
    if (VEC) {
#pragma unroll
      for (int i = 0; i < C; ++i) b[i] = 0.f;
      if (n > 0) load_vec<float, C>(a.bias + e0, b);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) b[i] = in(i) ? __ldg(a.bias + e0 + i) : 0.f;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      c[i] = fmaf(c[i], inv, b[i]);
      top = max(top, __float_as_uint(c[i]) & 0x7FFFFFFFu);
      key[i] = key_of(c[i]);
    }
    top = warp_max(top);
    sure = top < 0x7F800000u;
    err = (2.5e-6f + 6.5e-8f * C) * inv + 1.2e-7f * __uint_as_float(top);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) key[i] = key_of(x[i]);
  }
  unsigned keep = n > 0 ? (n < 32 ? (1u << n) - 1u : ~0u) : 0u;
  if (sure && a.SG < a.G) {
    uint32_t last, other;
    uint32_t* floats = reinterpret_cast<uint32_t*>(scratch);
    if (a.bias || !a.two) {
      keep = kept_experts<C, VEC>(a, key, e0, n, floats, value_of, key_of, &last, &other);
    } else {
      uint32_t ekey[C];
#pragma unroll
      for (int i = 0; i < C; ++i) ekey[i] = __float_as_uint(c[i]) | 0x80000000u;  // (not negative)
      keep = kept_experts<C, VEC>(a, ekey, e0, n, floats, value_of, key_of, &last, &other);
    }
    if (a.bias || a.two) {
      // sums of two exponentials: 4e-7 of the sum and 2 * 0.37 * 1.8e-7 (d e^-d <= 0.37)
      const float vi = value_of(last), vo = value_of(other);
      const float bound = a.bias ? (a.two ? 2.f * err + 1.2e-7f * fabsf(vi) : err)
                                 : 4e-7f * vi + 1.4e-7f;
      sure = vi - vo > 2.f * bound;
    }
  }
  uint32_t best = 0;
  if (VEC && a.lanes) {  // a lane's experts are kept together
#pragma unroll
    for (int i = 0; i < C; ++i) best = max(best, key[i]);
    best = keep ? best : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) best = max(best, (keep >> i) & 1u ? key[i] : 0u);
  }
  // one expert more than is chosen, for the last one's margin
  const bool more = a.bias && a.k < a.SG * (a.E / a.G);
  const int rounds = a.k + (more ? 1 : 0);
  auto tied = [&](int i, int j) {  // the same inputs: the lower id, which is first, is sure to be so
    return Dt<T>::to_f(src[i]) == Dt<T>::to_f(src[j]) && a.bias[i] == a.bias[j];
  };
  int mine[2] = {0, 0}, count = 33;
  uint32_t least = 1u;
  if (sure && rounds <= 32) {
    // `rounds` lanes have an expert at or above the bound, so the last choice is at or above it too
    // (or, where fewer lanes have experts, their two best do)
    uint32_t b = best, second = 0;
    if (rounds > __popc(__ballot_sync(kAll, best != 0u))) {
      b = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) take_two(b, second, (keep >> i) & 1u ? key[i] : 0u);
    }
    for (int r = 0; r < rounds; ++r) {
      const uint32_t top = warp_max(b);
      if (top == 0u) break;  // every kept expert
      least = r == rounds - 1 ? top : 1u;
      if (b == top) {
        b = second;
        second = 0;
      }
    }
    unsigned above = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) above |= key[i] >= least ? 1u << i : 0u;
    above &= keep;
    const int have = __popc(above);
    int before = have;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, before, o);
      if (lane >= o) before += v;
    }
    count = __shfl_sync(kAll, before, 31);
    if (count <= 32) {
      // an expert a lane, in the order of their ids; each counts the keys above its own, and those as
      // large of lower ids
      uint32_t* keys = reinterpret_cast<uint32_t*>(scratch);
      uint32_t* ids = keys + 32;
      before -= have;
      __syncwarp();
      keys[lane] = 0u;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < C; ++i)
        if ((above >> i) & 1u) {
          keys[before] = key[i];
          ids[before++] = e0 + i;
        }
      __syncwarp();
      const uint32_t own = keys[lane], id = ids[lane];
      int rank = 0;
      for (int j = 0; j < count; j += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(keys + j);
        rank += v.x + (j < lane) > own;  // (keys are at most 0xFF800000)
        rank += v.y + (j + 1 < lane) > own;
        rank += v.z + (j + 2 < lane) > own;
        rank += v.w + (j + 3 < lane) > own;
      }
      __syncwarp();
      if (lane < count) {
        keys[rank] = own;
        ids[rank] = id;
      }
      __syncwarp();
      mine[0] = lane < count ? (int)ids[lane] : 0;
      if (a.bias) {
        const float v = value_of(keys[lane]), vn = __shfl_down_sync(kAll, v, 1);
        const bool clear = lane < count - 1 && v - vn > 2.f * err;
        const unsigned clears = __ballot_sync(kAll, clear);
        const unsigned chosen = (1u << (a.k - 1)) - 1u;  // pairs among the chosen
        if (more ? (clears & (chosen << 1 | 1u)) != (chosen << 1 | 1u) : (clears & chosen) != chosen) {
          const int next = __shfl_down_sync(kAll, mine[0], 1);
          const unsigned ties =
              __ballot_sync(kAll, lane < count - 1 && !clear && tied(mine[0], next));
          sure = ((clears | ties) & chosen) == chosen;
          if (more) {
            // the last one against the rest: those tied with it, and then a clear margin
            const int end = __ffs(~(ties >> (a.k - 1))) - 1 + a.k - 1;
            sure = sure && ((clears >> end) & 1u || (end == count - 1 && least == 1u));
          }
        }
      }
    }
  }
  if (sure && count > 32) {  // many slots, or many alike: a round each
    best = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      key[i] = (keep >> i) & 1u ? key[i] : 0u;
      best = max(best, key[i]);
    }
    float last_v = 0.f;
    int last = 0;
    const int all = a.SG * (a.E / a.G), end = more ? all : a.k;
    for (int r = 0; r < end && sure; ++r) {
      uint32_t top;
      const int id = take_best<C>(key, best, e0, &top);
      if (a.bias) {
        const float v = value_of(top);
        const bool clear = r > 0 && last_v - v > 2.f * err;
        if (clear && r >= a.k) break;  // (those tied with the last chosen one have been passed)
        sure = r == 0 || clear || tied(id, last);
        last_v = v;
        last = id;
      }
      if (r == lane && r < a.k) mine[0] = id;
      if (r == lane + 32 && r < a.k) mine[1] = id;
    }
  }
  if (!sure) {
    __syncwarp();
    const unsigned long long chosen = choose_f64<T, C>(a, row, m, scratch);
    if (chosen == ~0ull) {
      for (int r = lane; r < a.k; r += 32) write_slot<T>(a, row, r, r, __int_as_float(0x7FC00000));
      return;
    }
    mine[0] = (int)(uint32_t)chosen;
    mine[1] = (int)(chosen >> 32);
  }
  // Weights.  Renormalised ones do not depend on m: the largest chosen logit keeps them from vanishing.
  // The others divide by the fast pass's sum: with its exponentials they are as far off 64 bits as those of
  // an FP32 softmax (at most 4.5e-7 for logits of spread 2), which the rounding of l - m and the sum decide.
  float l[2] = {-INFINITY, -INFINITY}, w[2] = {0.f, 0.f};
  if (lane < a.k) l[0] = Dt<T>::to_f(src[mine[0]]);
  if (lane + 32 < a.k) l[1] = Dt<T>::to_f(src[mine[1]]);
  if (a.renorm) m = value_of(max(warp_max(key_of(l[0])), a.k > 32 ? warp_max(key_of(l[1])) : 0u));
  w[0] = expf(l[0] - m);
  if (a.k > 32) w[1] = expf(l[1] - m);
  const float by = a.renorm ? warp_sum((lane < a.k ? w[0] : 0.f) + (lane + 32 < a.k ? w[1] : 0.f)) : z;
  if (lane < a.k) write_slot<T>(a, row, lane, mine[0], w[0] / by * a.scale);
  if (lane + 32 < a.k) write_slot<T>(a, row, lane + 32, mine[1], w[1] / by * a.scale);
}

template <typename T, int C>
cudaError_t launch_c(const SoftmaxRoute& a, cudaStream_t s) {
  const size_t smem = kWarps * (size_t)scratch_words(a.E) * sizeof(unsigned long long);
  const bool vec = a.per == C && a.E % C == 0 && C * sizeof(T) % 16 == 0 &&
                   a.E * sizeof(T) % 16 == 0 && (((uintptr_t)a.logits | (uintptr_t)a.bias) & 15u) == 0;
  const auto kern = vec ? moe_route_softmax_kernel<T, C, true> : moe_route_softmax_kernel<T, C, false>;
  kern<<<(unsigned)((a.T + kWarps - 1) / kWarps), kWarps * 32, smem, s>>>(a);
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
  // scores then take a few shuffles instead of a walk through shared memory, if that takes no more than
  // twice the registers; else the fewest.  Few lanes with many experts each are slower than the walk, as
  // the fast choice runs out of candidates (16384 rows, k = 8, bias, lanes / walk: 248 experts in 8 groups,
  // 31 a lane for 8, 112 / 36 us; 72 in 8, 9 for 3, 63 / 25; 60 in one, 15 for 2, 59 / 16).  At twice the
  // registers neither is better everywhere (56 in 8 groups, k = 6 27.4 / 22.6 us, one row 3.2 / 3.8; 500 in
  // 20 75.8 / 78.6, one row 5.2 / 6.3).
  const int gs = E / G, least = (E + 31) / 32;
  auto registers = [](int n) { return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32; };  // see launch_t()
  a.per = least;
  for (int per = least; per <= 32 && per <= gs && registers(per) <= 2 * registers(least); ++per)
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
