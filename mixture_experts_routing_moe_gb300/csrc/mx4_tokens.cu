// A whole MoE layer for a few tokens with microscaled 4-bit expert weights, in two launches: the
// router logits; then top-k, gate/up, SwiGLU, down and combine in a cooperative one.
//
//   logits[t, e] = x[t] . router[e];  idx, w as moe_route (softmax over all experts, ties to the
//   lower id);  a = round16(silu(x gate_e^T) * (x up_e^T));  out[t] = sum_j w[t, j] (a_j down_e^T)
//
// The layer reads each active expert's weights once, 17/32 of a byte a weight, and that is its
// floor, so nothing may be spent on the weights but the copy.  The tensor cores decode them:
// tcgen05.mma kind::mxf4 multiplies the packed codes (M = 128 weight rows) by e2m1 tokens and
// applies the block scales of both.  Each block of 32 token values is the sum of eight e2m1 terms,
// each with a scale 2^-3 of the one before (a value scaled to at most 4 is within 1/2 of a code, so a
// term takes three bits off).  What eight leave is at most 2^-23 of the block's largest value, as
// much as one rounding of an FP32 sum that holds that value, and nothing where the value's bits end
// above that: bf16 values down to 2^-15 of the largest are exact, f16 values down to 2^-12.  (Five
// terms, 2^-14, lost the 16 bits of values beside one a few hundred times as large, which activations
// do have.)  The terms are separate columns (N) of the MMA, and the epilogue adds them up.  N is
// small, so they cost no time: a 256-deep slice of 128 weight rows keeps the tensor pipe about 300
// cycles and the memory about 700.
// (Two e4m3 terms under kind::mxf8f6f4 are exact for bf16, but the weights then widen to a byte in
// shared memory: the TMA unit handles rows of 64 packed bytes, and half as many bytes are in
// flight.  The layer of 256 experts took 1.08 ms that way.)
//
// Steps.
//   0  (first launch) terms of x (xq, xs), router logits, counters cleared.
// The second launch has one CTA per SM, all resident; hand-overs between CTAs go through counters
// in global memory.
//   1  every CTA selects the top-k of all tokens for itself (the same arithmetic everywhere) and
//      lists the active experts' tokens in shared memory, expert by expert.
//   2  units of work: (expert, 64 columns of a) for gate/up, then (expert, 128 columns of the
//      output, part of K) for down, dealt to the CTAs in turn.  Warp roles as in the grouped
//      products: weight codes (TMA), token terms (TMA), raw scales, scales, MMA, epilogue, in slices
//      of K = 256.  The gate/up epilogue writes a as terms (aq, as; rows in the order of the lists)
//      and another warp counts the unit on its expert; a down unit's weights are loaded ahead, its
//      tokens once that count is full.  The weight loads never wait for anything but a free slot,
//      from the first unit to the last.
//   3  the down epilogue writes y (FP32, one row a slot and part); once every CTA has counted its
//      last unit, all of them add parts and slots up in order and write out.  (Letting whoever
//      finished an output tile's last unit add it up put several such sums, 20 to 70 us each, on
//      the CTAs that were late already: 775 to 1045 us for the layer of 256 experts.)
// Waits are bounded; on expiry the status word records the timeout and every role leaves.
#include "launch.h"
#include "mx4.cuh"
#include "mx4_mma.cuh"
#include "route_core.cuh"
#include "tiles.cuh"

namespace moe {
namespace {
using namespace tc;
using namespace mx4;

constexpr int kThreads = 416, kWarps = kThreads / 32;
constexpr int P = 8;               // terms of a token value
constexpr int kG = 24;             // tokens of a unit
constexpr int kMaxN = 192;         // columns of a unit
static_assert(kG * P <= kMaxN, "columns of a group");
constexpr int kA = 128 * 128;      // bytes of a slice's weights (128 rows, 256 deep)
constexpr int kMaxStages = 10;
constexpr int kBox = 16;           // rows of token terms a TMA box
constexpr int kBarBytes = 512;
constexpr int kRaw = 3;            // raw scale slots (four slices each) of weights and of tokens
// two accumulators, then the scales of two slices: 2 x 4 columns for A, 2 x 8 for B
constexpr uint32_t kTmemCols = 512, kScaleCol = 2 * kMaxN;
static_assert(kScaleCol + 2 * 24 <= kTmemCols, "tensor memory");
constexpr int kPer = 32 / P;              // tokens that the epilogue takes at a time
constexpr int kExchange = kPer * 64 * 4;  // their gate or up columns on the way between warps

struct TokensParams {
  const void* x;
  const void* router;
  int T, E, H, I, k, renorm;
  const uint8_t *gs, *us, *ds;
  int scales_vec;
  float* logits;
  uint8_t *xq, *xs, *aq, *as;
  float* y;
  unsigned *status, *ready, *done;
  size_t zeroed;  // words of counters behind `status`
  void* out;
  uint32_t* idx;
  float* w;
  int splits;        // parts of K a down unit is cut into
  int stages, ncap;  // ring: slices, columns of its token tiles
  int ncap_raw;      // ncap rounded up to 32
};

// The second launch may start once all CTAs of the first one run (start_next): it sets up its
// barriers and tensor memory and waits for the first to end (wait_previous) before it reads what
// that wrote (single token 24.3 -> 23.4 us of device time; between the launches of the experts the
// same gave nothing).
__device__ __forceinline__ void start_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ unsigned ld_acquire_u32(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ bool wait_count(const unsigned* c, unsigned want, volatile int* abort_f,
                                           unsigned* status) {
  const long long t0 = clock64();
  while (ld_acquire_u32(c) < want) {
    if (*abort_f) return false;
    if (clock64() - t0 > kWaitLimit) {
      *abort_f = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
    __nanosleep(20);
  }
  return true;
}
// A role's place in the ring.
struct RingPos {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int n, int stages) {
    stage += n;
    while (stage >= stages) {
      stage -= stages;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ void back(int stages) {
    if (stage == 0) {
      stage = stages;
      phase ^= 1u;
    }
    --stage;
  }
};
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// A warp writes one block of 32 values (one a lane) as P e2m1 terms: term p's 16 bytes at
// q + p * pitch, its scale byte at sc + p * sc_pitch.  With the largest magnitude in
// [2^n, 2^(n + 1)) the first scale is 2^(n - 1), so scaled values stay under 4; a remainder is at
// most 1/2 and is scaled up by 8 for the next term.
__device__ __forceinline__ void write_terms(float v, uint8_t* q, int64_t pitch, uint8_t* sc,
                                            int64_t sc_pitch, int lane) {
  const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
  const int f = (int)(top >> 23);
  const bool bad = f == 255;
  const int b0 = max(min(f, 254) - 1, 3 * (P - 1));
  float r = bad ? 0.f : v * __uint_as_float((uint32_t)(254 - b0) << 23);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t c, back;
    asm("{\n\t.reg .b8 b, z;\n\tmov.b32 {z, z, z, z}, 0;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %3;\n\t"
        "mov.b32 %0, {b, z, z, z};\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
        : "=r"(c), "=r"(back)
        : "f"(0.f), "f"(r));
    const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, c, 1);
    if ((lane & 1) == 0) q[p * pitch + (lane >> 1)] = (uint8_t)(c | (next << 4));
    if (lane == 0) sc[p * sc_pitch] = (uint8_t)(bad ? 255 : b0 - 3 * p);
    r = (r - __low2float(*reinterpret_cast<const __half2*>(&back))) * 8.f;
  }
}

// One warp selects the top-k of a row of FP32 logits: ids and weights of slots 0 .. k - 1.  Lane l
// holds experts l, l + 32, ...; keys order as route_core.cuh's, ties to the lower id.
template <int C>
__device__ __forceinline__ void select_row(const float* row, int E, int k, int renorm, int lane,
                                           uint16_t* ids, float* ws) {
  uint32_t key[C];
  float m = -INFINITY;
  uint32_t flags = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = c * 32 + lane;
    key[c] = 0;
    if (e < E) {
      const float v = __ldcg(row + e);
      if (v != v || v == INFINITY) flags |= 1u;
      if (v != -INFINITY) flags |= 2u;
      m = fmaxf(m, v);
      key[c] = monotone_bits(v == 0.f ? 0.f : v);  // both zeros take +0's key
    }
  }
  flags = __reduce_or_sync(0xFFFFFFFFu, flags);
  m = group_max<32>(m);
  if ((flags & 1u) || !(flags & 2u)) {
    if (lane < k) {
      ids[lane] = (uint16_t)lane;
      ws[lane] = __int_as_float(0x7FC00000);
    }
    return;
  }
  float s = 0.f, sel = 0.f, mine = 0.f;
  if (!renorm) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * 32 + lane < E) s += expf(from_monotone_bits(key[c]) - m);
    s = group_sum<32>(s);
  }
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int c = 1; c < C; ++c)
      if (key[c] > best) best = key[c], at = c;
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const uint32_t id =
        __reduce_min_sync(0xFFFFFFFFu, best == top ? (uint32_t)(at * 32 + lane) : 0xFFFFu);
    const float ex = expf(from_monotone_bits(top) - m);
    sel += ex;
    if (lane == j) {
      ids[j] = (uint16_t)id;
      mine = ex;
    }
    if ((id & 31u) == (uint32_t)lane) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c == (int)(id >> 5)) key[c] = 0;
    }
  }
  if (lane < k) ws[lane] = mine / (renorm ? sel : s);
}

// Step 0: CTAs below logit_ctas compute the logits of kEB experts and kTB tokens, its warps an
// eighth of H each; the others write the terms of x, a block of 32 values a warp.  CTA 0 clears
// the counters.
constexpr int kEB = 4, kTB = 8, kFirstWarps = 8;
template <typename T>
__global__ void __launch_bounds__(kFirstWarps * 32)
    moe_mx4_tokens_first(const TokensParams p, int logit_ctas) {
  start_next();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (size_t i = threadIdx.x; i < p.zeroed; i += kFirstWarps * 32) p.status[i] = 0;
  const T* x = (const T*)p.x;
  if ((int)blockIdx.x >= logit_ctas) {
    const int hb = p.H / 32, b = ((int)blockIdx.x - logit_ctas) * kFirstWarps + warp;
    if (b >= p.T * hb) return;
    const int t = b / hb, c = b - t * hb;
    const float v = Dt<T>::to_f(x[(int64_t)t * p.H + c * 32 + lane]);
    write_terms(v, p.xq + (int64_t)t * P * (p.H / 2) + c * 16, p.H / 2,
                p.xs + (int64_t)t * P * hb + c, hb, lane);
    return;
  }
  __shared__ float red[kFirstWarps][kEB * kTB];
  const int eb = (p.E + kEB - 1) / kEB;
  const int e0 = blockIdx.x % eb * kEB, t0 = blockIdx.x / eb * kTB;
  const T* router = (const T*)p.router;
  const T *r[kEB], *xt[kTB];
#pragma unroll
  for (int i = 0; i < kEB; ++i) r[i] = router + (int64_t)min(e0 + i, p.E - 1) * p.H;
#pragma unroll
  for (int i = 0; i < kTB; ++i) xt[i] = x + (int64_t)min(t0 + i, p.T - 1) * p.H;
  const int nt = min(kTB, p.T - t0);
  float acc[kEB][kTB] = {};
  for (int v = threadIdx.x; v < p.H / 8; v += kFirstWarps * 32) {
    Vec16<T> a[kEB], q[kTB];
#pragma unroll
    for (int i = 0; i < kEB; ++i) a[i].u = ld_nc_v4(r[i] + v * 8);
#pragma unroll
    for (int i = 0; i < kTB; ++i)
      if (i < nt) q[i].u = ld_nc_v4(xt[i] + v * 8);
#pragma unroll
    for (int i = 0; i < kTB; ++i) {
      if (i >= nt) continue;
      float xf[8];
      q[i].to_float(xf);
#pragma unroll
      for (int j = 0; j < kEB; ++j) {
#pragma unroll
        for (int z = 0; z < 8; ++z) acc[j][i] = fmaf(xf[z], Dt<T>::to_f(a[j].e[z]), acc[j][i]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kEB; ++j)
#pragma unroll
    for (int i = 0; i < kTB; ++i) {
      if (i >= nt) continue;
      const float s = group_sum<32>(acc[j][i]);
      if (lane == 0) red[warp][j * kTB + i] = s;
    }
  __syncthreads();
  const int j = threadIdx.x / kTB, i = threadIdx.x % kTB;
  if (j < kEB && e0 + j < p.E && i < nt) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kFirstWarps; ++w) s += red[w][threadIdx.x];
    p.logits[(int64_t)(t0 + i) * p.E + e0 + j] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    moe_mx4_tokens(const __grid_constant__ CUtensorMap mapG, const __grid_constant__ CUtensorMap mapU,
                   const __grid_constant__ CUtensorMap mapD,
                   const __grid_constant__ CUtensorMap mapX,
                   const __grid_constant__ CUtensorMap mapA, const TokensParams p) {
  extern __shared__ uint8_t mx4_smem_raw[];
  const uint32_t raw = smem_u32(mx4_smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int stage_bytes = kA + p.ncap * 128;
  const int b_chunks = p.ncap > 128 ? 2 : 1;  // scale chunks of 128-deep token terms
  const int sf_bytes = (2 + 2 * b_chunks) * kScaleChunk;
  uint8_t* at = mx4_smem_raw + (base - raw) + p.stages * stage_bytes;
  const uint32_t sf_base = smem_u32(at);  // a stage's scales: two chunks of A, then those of B
  at += p.stages * sf_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(at);
  at += kBarBytes;
  const uint32_t rawa_base = smem_u32(at), rawb_base = rawa_base + kRaw * 128 * 32;
  at += kRaw * (128 + p.ncap_raw) * 32;
  float* exchange = reinterpret_cast<float*>(at);
  at += kExchange;
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(at);  // tokens of an expert
  at += p.E * 8;
  int* start = reinterpret_cast<int*>(at);  // first entry of an expert's tokens in `list`
  at += (p.E + 1) * 4;
  int* act = reinterpret_cast<int*>(at);  // expert | group << 16 of each group of tokens
  const int R = p.T * p.k;
  at += R * 4;  // a group has one slot at least
  float* sel_w = reinterpret_cast<float*>(at);
  at += R * 4;
  uint16_t* sel_id = reinterpret_cast<uint16_t*>(at);
  uint16_t* list = sel_id + R;  // slots t * k + j, expert by expert, by token

  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * kMaxStages + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kMaxStages + 4);
  // raw scales: full, then empty 8 bytes on
  auto rawa_bar = [&](int s) { return bar0 + 8u * (2 * kMaxStages + 5 + 2 * s); };
  auto rawb_bar = [&](int s) { return rawa_bar(kRaw + s); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 5 + 4 * kRaw);
  volatile int* abort_f = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* active_s = reinterpret_cast<int*>(tmem_slot + 2);
  volatile int* written = reinterpret_cast<volatile int*>(tmem_slot + 3);  // gate/up units
  const bool out_vec = ((uintptr_t)p.out & 7u) == 0;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 4);  // weights, tokens, weight scales, token scales
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    mbar_init(drain_bar, 1);
    for (int s = 0; s < 2 * kRaw; ++s) {
      mbar_init(rawa_bar(s), 32);
      mbar_init(rawa_bar(s) + 8, 1);
    }
    *abort_f = 0;
    *active_s = 0;
    *written = 0;
    fence_mbar_init();
    tma_prefetch(&mapG);
    tma_prefetch(&mapU);
    tma_prefetch(&mapD);
    tma_prefetch(&mapX);
    tma_prefetch(&mapA);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  for (int e = threadIdx.x; e < p.E; e += kThreads) mask[e] = 0;

  wait_previous();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // ------------------------------------------------ 1. top-k, lists of the experts' tokens
  for (int t = warp; t < p.T; t += kWarps) {
    const float* row = p.logits + (int64_t)t * p.E;
    uint16_t* ids = sel_id + t * p.k;
    float* ws = sel_w + t * p.k;
    if (p.E <= 128) select_row<4>(row, p.E, p.k, p.renorm, lane, ids, ws);
    else if (p.E <= 256) select_row<8>(row, p.E, p.k, p.renorm, lane, ids, ws);
    else select_row<32>(row, p.E, p.k, p.renorm, lane, ids, ws);
    __syncwarp();
    if (lane < p.k) {
      atomicOr(mask + ids[lane], 1ull << t);
      if (blockIdx.x == 0) {
        if (p.idx) p.idx[t * p.k + lane] = ids[lane];
        if (p.w) p.w[t * p.k + lane] = ws[lane];
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0, n_act = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < p.E ? __popcll(mask[e]) : 0, g = (n + kG - 1) / kG;
      int s = n, sg = g;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, s, o), yg = __shfl_up_sync(0xFFFFFFFFu, sg, o);
        if (lane >= o) s += y, sg += yg;
      }
      if (e < p.E) start[e] = carry + s - n;
      for (int i = 0; i < g; ++i) act[n_act + sg - g + i] = e | i << 16;
      carry += __shfl_sync(0xFFFFFFFFu, s, 31);
      n_act += __shfl_sync(0xFFFFFFFFu, sg, 31);
    }
    if (lane == 0) start[p.E] = carry, *active_s = n_act;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < R; s += kThreads) {
    const int e = sel_id[s], t = s / p.k;
    list[start[e] + __popcll(mask[e] & ((1ull << t) - 1))] = (uint16_t)s;
  }
  __syncthreads();

  // ------------------------------------------------ 2. units
  const int NI = p.I / 64, NH = p.H / 128;
  const int active = *active_s;
  const int n1 = active * NI, per_down = NH * p.splits, total = n1 + active * per_down;
  struct Unit {
    bool down;
    int e, ai;        // expert, place in `act`
    int tile, split;  // column tile, part of K
    int first, n;     // its tokens: list[first .. first + n)
    int k0, k1;       // 256-deep slices
    int cols;         // columns in use
  };
  auto unit_of = [&](int u) {
    Unit r;
    r.down = u >= n1;
    const int v = r.down ? u - n1 : u, per = r.down ? per_down : NI;
    r.ai = v / per;
    const int w = v - r.ai * per;
    r.tile = r.down ? w / p.splits : w;
    r.split = r.down ? w - r.tile * p.splits : 0;
    const int a = act[r.ai];
    r.e = a & 0xFFFF;
    r.first = start[r.e] + (a >> 16) * kG;
    r.n = min(start[r.e + 1] - r.first, kG);
    const int slices = ((r.down ? p.I : p.H) + 255) / 256;
    const int pairs = (slices + 1) / 2;  // parts begin at even slices, 16 bytes of scales
    r.k0 = r.down ? 2 * (pairs * r.split / p.splits) : 0;
    r.k1 = r.down ? min(slices, 2 * (pairs * (r.split + 1) / p.splits)) : slices;
    r.cols = r.n * P;
    return r;
  };

  // a down unit's tokens: its group's gate/up units have all been counted (every lane calls)
  auto unit_ready = [&](int ai) {
    bool ok = true;
    if (lane == 0) ok = wait_count(p.ready + ai, NI, abort_f, p.status);
    ok = __all_sync(0xFFFFFFFFu, ok);
    __syncwarp();  // orders lane 0's acquire before the other lanes' loads (a vote orders nothing)
    fence_proxy_async_all();
    return ok;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- weight codes
    int stage = 0;
    uint32_t phase = 0;
    bool stop = false;
    const uint64_t pol = policy_evict_normal();
    for (int u = blockIdx.x; u < total && !stop; u += gridDim.x) {
      const Unit r = unit_of(u);
      const int row = r.down ? r.e * p.H + r.tile * 128 : r.e * p.I + r.tile * 64;
      for (int k = r.k0; k < r.k1; ++k) {
        if (!__all_sync(0xFFFFFFFFu,
                        wait_bounded(empty_bar(stage), phase ^ 1u, abort_f, p.status))) {
          stop = true;
          break;
        }
        const uint32_t sa = base + stage * stage_bytes, fb = full_bar(stage);
        if (elect_one()) {
          mbar_expect_tx(fb, kA);
          if (r.down) {
            tma_load_2d(sa, &mapD, fb, k * 128, row, pol);
          } else {
            tma_load_2d(sa, &mapG, fb, k * 128, row, pol);
            tma_load_2d(sa + kA / 2, &mapU, fb, k * 128, row, pol);
          }
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool stop = false;
    for (int u = blockIdx.x; u < total && !stop; u += gridDim.x) {
      const Unit r = unit_of(u);
      const uint32_t idesc = make_idesc_mxf4(128, (r.cols + 15) / 16 * 16, 0);
      if (!__all_sync(0xFFFFFFFFu,
                      wait_bounded(tempty_bar(acc), acc_phase ^ 1u, abort_f, p.status)))
        break;
      tc_fence_after();
      const uint32_t d = tmem + acc * kMaxN;
      for (int k = r.k0; k < r.k1; ++k) {
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(full_bar(stage), phase, abort_f, p.status))) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t sa = base + stage * stage_bytes;
        const uint32_t sf = sf_base + stage * sf_bytes, sfb = sf + 2 * kScaleChunk;
        const uint32_t cols = tmem + kScaleCol + (stage & 1) * 24;
        const uint64_t da = make_sdesc(sa), db = make_sdesc(sa + kA);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_cp_scale(cols + c * 12, make_sdesc_scale(sf + c * kScaleChunk));
            tmem_cp_scale(cols + c * 12 + 4, make_sdesc_scale(sfb + c * b_chunks * kScaleChunk));
            if (b_chunks == 2)
              tmem_cp_scale(cols + c * 12 + 8, make_sdesc_scale(sfb + (2 * c + 1) * kScaleChunk));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t ca = cols + (i >> 1) * 12;
            umma_mxf4(d, da + 2u * i, db + 2u * i,
                      (i & 1) ? idesc | (2u << 4) | (2u << 29) : idesc, ca, ca + 4,
                      k != r.k0 || i != 0);
          }
          umma_commit(empty_bar(stage));
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (stop) break;
      if (elect_one()) umma_commit(tfull_bar(acc));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (elect_one()) umma_commit(drain_bar);  // arrives once every MMA issued above has completed
    wait_drain(drain_bar, 0);
  } else if (warp == 2 || warp == 3) {
    // ---------------------------------------------------------------- token terms
    // the two warps take the slices in turn: what one does for a slice (a wait, the barrier, the
    // loads) is a chain of some 600 cycles
    const int mine = warp - 2;
    RingPos at;
    int armed = 0, turn = 0;
    bool stop = false;
    const uint64_t pol = policy_evict_normal();
    for (int u = blockIdx.x; u < total && !stop; u += gridDim.x) {
      const Unit r = unit_of(u);
      if (r.down && !unit_ready(r.ai)) {
        stop = true;
        break;
      }
      // A group's rows of aq are contiguous: boxes of 16.  Its tokens' rows of xq are not: a box
      // each.  (Multiplying all T tokens of x, contiguous too, by every expert that takes many of
      // them was slower throughout: 7 tokens, 8 wide experts 150 us against 124, 32 tokens 4 of 8
      // 96 against 94, 32 tokens 4 of 32 172 against 160.)
      const int boxes = r.down ? (r.cols + kBox - 1) / kBox : r.n;
      const int bytes = r.down ? kBox * 128 : P * 128;  // of a box
      // first rows of boxes lane and lane + 32 (at most kG boxes)
      int box_row[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int i = lane + 32 * z;
        box_row[z] = r.down ? r.first * P + i * kBox
                     : i < r.n ? (int)list[r.first + i] / p.k * P : 0;
      }
      const CUtensorMap* m = r.down ? &mapA : &mapX;
      for (int k = r.k0; k < r.k1; ++k, turn ^= 1) {
        // Each warp waits only for the slots of the slices it takes, by parity.  A slice c needs
        // slice c - S to be consumed (S >= 3 slots); the parity cannot be taken for that of
        // c - 2 S, since the warp's last wait was for c - 2, later than c - S.  (It must not wait
        // for the other's slots: those move on without it, and a parity would come round again.)
        if (turn != mine) {
          at.step(1, p.stages);
          continue;
        }
        if (!__all_sync(0xFFFFFFFFu,
                        wait_bounded(empty_bar(at.stage), at.phase ^ 1u, abort_f, p.status))) {
          stop = true;
          break;
        }
        const uint32_t sb = base + at.stage * stage_bytes + kA, fb = full_bar(at.stage);
        if (elect_one()) mbar_expect_tx(fb, boxes * bytes);
        __syncwarp();
        for (int i = 0; i < boxes; ++i) {
          const int row = __shfl_sync(0xFFFFFFFFu, i < 32 ? box_row[0] : box_row[1], i & 31);
          if (elect_one()) tma_load_2d(sb + i * bytes, m, fb, k * 128, row, pol);
        }
        ++armed;
        at.step(1, p.stages);
      }
    }
    if (stop) {  // let copies still in flight land
      const long long until = clock64() + kWaitLimit;
      for (int i = 0; i < p.stages && armed > 0; ++i) {
        at.back(p.stages);
        wait_until(full_bar(at.stage), at.phase, until);
      }
    }
  } else if (warp == 6 || warp == 7) {
    // ---------------------------------------------------------------- raw scales
    // warp 6: the unit's 128 weight rows; warp 7: its columns' token terms; four slices (32 bytes
    // of a row) at a time.  Lane l copies rows l, l + 32, ...
    constexpr int J = kMaxN / 32;
    const bool tokens = warp == 7;
    RingPos at;
    bool stop = false;
    for (int u = blockIdx.x; u < total && !stop; u += gridDim.x) {
      const Unit r = unit_of(u);
      if (tokens && r.down && !unit_ready(r.ai)) break;
      const int pitch = (r.down ? p.I : p.H) / 32, end = min(r.k1 * 8, pitch);
      const bool vec = (pitch & 15) == 0 && (tokens || p.scales_vec);
      const int lanes_j = tokens ? (r.cols + 31) / 32 : 4;
      const uint8_t* src[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        src[j] = nullptr;
        const int c = 32 * j + lane;
        if (tokens && c < r.cols) {
          const int i = c / P, term = c - i * P;
          const int row = r.down ? (r.first + i) * P + term
                                 : (int)list[r.first + i] / p.k * P + term;
          src[j] = (r.down ? p.as : p.xs) + (int64_t)row * pitch;
        } else if (!tokens && j < 4) {
          src[j] = r.down ? p.ds + ((int64_t)r.e * p.H + r.tile * 128 + c) * pitch
                          : (j < 2 ? p.gs : p.us) +
                                ((int64_t)r.e * p.I + r.tile * 64 + (c & 63)) * pitch;
        }
      }
      for (int k = r.k0; k < r.k1; k += 4) {
        const uint32_t rb = tokens ? rawb_bar(at.stage) : rawa_bar(at.stage);
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(rb + 8, at.phase ^ 1u, abort_f, p.status))) {
          stop = true;
          break;
        }
        const uint32_t slot = tokens ? rawb_base + at.stage * (p.ncap_raw * 32)
                                     : rawa_base + at.stage * (128 * 32);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j >= lanes_j || !src[j]) continue;
          const int row = 32 * j + lane;
          if (vec) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              cp_async16_or_zero(slot + raw_offset(row, h), src[j] + k * 8 + h * 16,
                                 k * 8 + h * 16 < end);
          } else {
            // (four bytes cannot be copied past L1, which may hold a line of `as` from before it
            // was written: loads past it, then stores)
#pragma unroll
            for (int w = 0; w < 8; ++w)
              st_shared_u32(slot + raw_offset(row, w >> 2) + (w & 3) * 4,
                            k * 8 + w * 4 < end ? ld_cg_u32(src[j] + k * 8 + w * 4) : 0u);
          }
        }
        if (vec) cp_async_arrive(rb);
        else mbar_arrive(rb);
        at.step(1, kRaw);
      }
    }
    cp_async_wait_all();  // nothing is on its way when the CTA leaves
  } else if (warp == 4 || warp == 5) {
    // ---------------------------------------------------------------- scales
    // raw rows to the chunks of each slice: warp 4 the weights', warp 5 the tokens'
    constexpr int J = kMaxN / 32;
    const bool tokens = warp == 5;
    RingPos at, raw_at;
    bool stop = false;
    for (int u = blockIdx.x; u < total && !stop; u += gridDim.x) {
      const Unit r = unit_of(u);
      for (int k = r.k0; k < r.k1 && !stop; k += 4) {
        const uint32_t rb = tokens ? rawb_bar(raw_at.stage) : rawa_bar(raw_at.stage);
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(rb, raw_at.phase, abort_f, p.status))) {
          stop = true;
          break;
        }
        const uint32_t slot = tokens ? rawb_base + raw_at.stage * (p.ncap_raw * 32)
                                     : rawa_base + raw_at.stage * (128 * 32);
        uint32_t now[J][8];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 v = make_uint4(0, 0, 0, 0);
            // (rows past the unit's columns hold old bytes: scales of columns that nobody reads)
            if (tokens ? 32 * j < r.cols : j < 4)
              v = ld_shared_v4(slot + raw_offset(32 * j + lane, h));
            now[j][4 * h] = v.x, now[j][4 * h + 1] = v.y;
            now[j][4 * h + 2] = v.z, now[j][4 * h + 3] = v.w;
          }
        __syncwarp();
        if (elect_one()) mbar_arrive(rb + 8);
        raw_at.step(1, kRaw);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (k + i >= r.k1 || stop) continue;
          if (!__all_sync(0xFFFFFFFFu,
                          wait_bounded(empty_bar(at.stage), at.phase ^ 1u, abort_f, p.status))) {
            stop = true;
            continue;
          }
          const uint32_t sf =
              sf_base + at.stage * sf_bytes + (tokens ? 2 * kScaleChunk : 0) + lane * 16;
          const uint32_t half = tokens ? b_chunks * kScaleChunk : kScaleChunk;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int w = 2 * i + h;
            st_shared_v4(sf + h * half, now[0][w], now[1][w], now[2][w], now[3][w]);
            if (tokens && b_chunks == 2)
              st_shared_v4(sf + h * half + kScaleChunk, now[4][w], now[5][w], 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) mbar_arrive(full_bar(at.stage));
          at.step(1, p.stages);
        }
      }
    }
  } else if (warp == 12) {
    // ---------------------------------------------------------------- counts of gate/up units
    // The fence before a count reaches other SMs takes a thousand cycles or more, which the
    // epilogue does not have to spare (wide experts: 160 us with it there).
    int seen = 0;
    for (int u = blockIdx.x; u < n1; u += gridDim.x) {
      const long long t0 = clock64();
      bool ok = true;
      while (*written <= seen) {
        if (*abort_f || clock64() - t0 > kWaitLimit) {
          ok = false;  // (the epilogue's own wait has recorded a timeout, or will)
          break;
        }
        __nanosleep(20);
      }
      // Lanes may see the abort and the last unit's word in different order: they leave together, as
      // the election below waits for all of them.
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      ++seen;
      __syncwarp();
      __threadfence();          // the epilogue's writes, which its barrier ordered before the word
      fence_proxy_async_all();  // aq is read by TMA
      if (elect_one()) atomicAdd(p.ready + unit_of(u).ai, 1u);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- epilogue
    constexpr int PER = kPer;
    const int q = warp & 3;
    int acc = 0, count = 0;
    uint32_t acc_phase = 0;
    auto any_of_epilogue = [&](bool v) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
          "barrier.cta.red.or.pred b, 1, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
          : "=r"(r)
          : "r"((uint32_t)v)
          : "memory");
      return r != 0;
    };
    auto sync_epilogue = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
      const Unit r = unit_of(u);
      // the four warps give up together, as the barriers below need all of them
      if (any_of_epilogue(!wait_bounded(tfull_bar(acc), acc_phase, abort_f, p.status))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + acc * kMaxN;
      for (int i0 = 0; i0 < r.n; i0 += PER) {
        uint32_t v[32];
        tmem_ld32(taddr + i0 * P, v);
        tmem_wait_ld();
        float s[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          s[i] = 0.f;
#pragma unroll
          for (int term = P - 1; term >= 0; --term) s[i] += __uint_as_float(v[i * P + term]);
        }
        if (r.down) {
          float* y = p.y + (int64_t)r.split * R * p.H + r.tile * 128 + q * 32 + lane;
#pragma unroll
          for (int i = 0; i < PER; ++i)
            if (i0 + i < r.n) y[(int64_t)list[r.first + i0 + i] * p.H] = s[i];
        } else {
          // Quarters 0 and 1 hold 64 gate rows, 2 and 3 the same up rows: the first two take the
          // even tokens, the other two the odd ones, and each hands over what it does not need.
          const int odd = q >> 1, part = (q & 1) * 32;
#pragma unroll
          for (int i = 0; i < PER; ++i)
            if ((i & 1) != odd) exchange[i * 64 + part + lane] = s[i];
          sync_epilogue();
          const int ib = p.I / 32, col = r.tile * 64 + part;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            if ((i & 1) != odd || i0 + i >= r.n) continue;
            const int pos = r.first + i0 + i;
            const float other = exchange[i * 64 + part + lane];
            const float g = odd ? other : s[i], up = odd ? s[i] : other;
            const float a = Dt<T>::to_f(Dt<T>::from_f(g / (1.f + expf(-g)) * up));
            write_terms(a, p.aq + (int64_t)pos * P * (p.I / 2) + col / 2, p.I / 2,
                        p.as + (int64_t)pos * P * ib + col / 32, ib, lane);
          }
          sync_epilogue();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
      if (!r.down && threadIdx.x == 8 * 32) {  // behind the last barrier above
        __threadfence_block();
        *written = ++count;
      }
    }
    // 3. every CTA's y is written: the sums over slots, four columns a thread
    __threadfence();
    sync_epilogue();
    bool ok = true;
    if (threadIdx.x == 8 * 32) {
      atomicAdd(p.done, 1u);
      ok = wait_count(p.done, gridDim.x, abort_f, p.status);
    }
    if (!any_of_epilogue(!ok)) {
      __threadfence();
      const int quads = p.H / 4, threads = gridDim.x * 128;
      const int64_t split = (int64_t)R * p.H;
      for (int i = blockIdx.x * 128 + (int)threadIdx.x - 8 * 32; i < p.T * quads; i += threads) {
        const int t = i / quads, h = (i - t * quads) * 4;
        const float* y = p.y + (int64_t)t * p.k * p.H + h;
        const float* w = sel_w + t * p.k;
        float s[4] = {};
#pragma unroll 8
        for (int j = 0; j < p.k; ++j) {
          float4 v = __ldcg(reinterpret_cast<const float4*>(y + (int64_t)j * p.H));
          for (int z = 1; z < p.splits; ++z) {
            const float4 q =
                __ldcg(reinterpret_cast<const float4*>(y + z * split + (int64_t)j * p.H));
            v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
          }
          s[0] = fmaf(w[j], v.x, s[0]), s[1] = fmaf(w[j], v.y, s[1]);
          s[2] = fmaf(w[j], v.z, s[2]), s[3] = fmaf(w[j], v.w, s[3]);
        }
        T* out = (T*)p.out + (int64_t)t * p.H + h;
        if (out_vec) {
          union {
            uint2 u;
            T e[4];
          } o;
#pragma unroll
          for (int c = 0; c < 4; ++c) o.e[c] = Dt<T>::from_f(s[c]);
          *reinterpret_cast<uint2*>(out) = o.u;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) out[c] = Dt<T>::from_f(s[c]);
        }
      }
    }
  }

  settle_after_abort(abort_f);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Bytes of shared memory beside the ring.
size_t fixed_smem(int E, int R, int ncap_raw) {
  return 1024 + kBarBytes + kRaw * (128 + (size_t)ncap_raw) * 32 + kExchange + (size_t)E * 12 + 4 +
         (size_t)R * 12;
}

// Parts of K that a down unit is cut into: enough units for four to a CTA (a CTA's last unit is
// then a quarter of its share), of at least four slices each.
int down_splits(int64_t T, int64_t E, int64_t H, int64_t I, int k) {
  const int64_t slots = T * k, units = (E < slots ? E : slots) * (H / 128);
  int64_t s = units > 0 ? (4 * 152 + units - 1) / units : 1;
  if (s > I / 1024) s = I / 1024;
  return (int)(s < 1 ? 1 : s > 8 ? 8 : s);
}

template <typename T>
cudaError_t launch_t(const Mx4TokensArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0, most = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess)
    err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err == cudaSuccess)
    err = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (err != cudaSuccess) return err;
  const Mx4TokensLayout l = mx4_tokens_layout(a.T, a.E, a.H, a.I, a.k);
  TokensParams p{};
  p.x = a.x;
  p.router = a.router;
  p.T = a.T;
  p.E = a.E;
  p.H = a.H;
  p.I = a.I;
  p.k = a.k;
  p.renorm = a.renorm;
  p.gs = a.gate.scales;
  p.us = a.up.scales;
  p.ds = a.down.scales;
  p.scales_vec = (((uintptr_t)p.gs | (uintptr_t)p.us | (uintptr_t)p.ds) & 15u) == 0;
  p.status = (unsigned*)a.ws;
  p.ready = (unsigned*)(a.ws + l.ready);
  p.done = (unsigned*)(a.ws + l.done);
  p.logits = (float*)(a.ws + l.logits);
  p.xq = a.ws + l.xq;
  p.xs = a.ws + l.xs;
  p.aq = a.ws + l.aq;
  p.as = a.ws + l.as;
  p.y = (float*)(a.ws + l.y);
  p.zeroed = l.zeroed / 4;
  p.out = a.out;
  p.idx = a.idx;
  p.w = a.w;
  p.splits = down_splits(a.T, a.E, a.H, a.I, a.k);
  const int R = a.T * a.k;
  // the ring: as many slices as fit, each with room for the columns of the largest unit
  p.ncap = ((a.T < kG ? a.T : kG) * P + kBox - 1) / kBox * kBox;
  p.ncap_raw = (p.ncap + 31) / 32 * 32;
  const size_t fixed = fixed_smem(a.E, R, p.ncap_raw);
  const size_t stage = kA + (size_t)p.ncap * 128 + (p.ncap > 128 ? 6 : 4) * kScaleChunk;
  p.stages = (int)(((size_t)most - fixed) / stage);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  if (p.stages < 3) return cudaErrorInvalidConfiguration;  // (the token warps take turns)
  const size_t smem = fixed + (size_t)p.stages * stage;

  CUtensorMap mg, mu, md, mx, ma;
  if (!make_map_bytes(&mg, a.gate.codes, a.H / 2, (int64_t)a.E * a.I, 64) ||
      !make_map_bytes(&mu, a.up.codes, a.H / 2, (int64_t)a.E * a.I, 64) ||
      !make_map_bytes(&md, a.down.codes, a.I / 2, (int64_t)a.E * a.H, 128) ||
      !make_map_bytes(&mx, p.xq, a.H / 2, (int64_t)a.T * P, P) ||
      !make_map_bytes(&ma, p.aq, a.I / 2, (int64_t)R * P, kBox))
    return cudaErrorInvalidValue;
  auto kern = moe_mx4_tokens<T>;
  // the same limit in every call: another thread's, of another size, may come before the launch
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (err != cudaSuccess) return err;
  const int logit_ctas = (a.E + kEB - 1) / kEB * ((a.T + kTB - 1) / kTB);
  const int64_t blocks = (int64_t)a.T * (a.H / 32);
  const int split_ctas = (int)((blocks + kFirstWarps - 1) / kFirstWarps);
  moe_mx4_tokens_first<T><<<logit_ctas + split_ctas, kFirstWarps * 32, 0, s>>>(p, logit_ctas);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, mg, mu, md, mx, ma, p);
}

}  // namespace

Mx4TokensLayout mx4_tokens_layout(int64_t T, int64_t E, int64_t H, int64_t I, int k) {
  const int64_t R = T * k;
  Mx4TokensLayout l;
  size_t off = kWsHeader;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  l.ready = take((size_t)R * 4);
  l.done = take(4);
  l.zeroed = off;
  l.logits = take((size_t)T * E * 4);
  l.xq = take((size_t)T * P * (H / 2));
  l.xs = take((size_t)T * P * (H / 32));
  l.aq = take((size_t)R * P * (I / 2));
  l.as = take((size_t)R * P * (I / 32));
  l.y = take((size_t)R * H * 4 * down_splits(T, E, H, I, k));
  l.total = off;
  return l;
}

cudaError_t launch_mx4_tokens(const Mx4TokensArgs& a, cudaStream_t s) {
  return a.dt == MOE_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<__half>(a, s);
}

}  // namespace moe
