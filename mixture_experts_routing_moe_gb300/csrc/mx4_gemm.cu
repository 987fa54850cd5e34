// Grouped products of microscaled 4-bit rows on 5th-generation tensor cores (tcgen05.mma
// kind::mxf4, scales from tensor memory):
//   product   out[r, n] = sum_k A[r, k] B[e, n, k]
//   gate/up   the blocks of silu(A gate_e^T) * (A up_e^T), quantised in the epilogue
// over the ragged row groups offsets[e] .. offsets[e+1]-1.
//
// A persistent kernel walks tiles (expert, m-tile, n-tile) of 256 columns and 128 rows (a CTA) or
// 256 rows (a cluster of two CTAs, cta_group::2: each CTA holds 128 of the rows and half of the B
// rows, so a tile pulls a third fewer bytes through L2).  Roles in each CTA:
//   warp 0      loads, for each 256-deep K slice, the codes of its A and B rows (128 bytes a row) by
//               TMA into a ring.  For gate/up the B tile holds gate rows 0-63, up rows 0-63, gate
//               rows 64-127, up rows 64-127 of 128 columns of a.  (Warps 0 and 1 run their loops with
//               all lanes; an elected one issues.)
//   warp 1      (of CTA 0) copies each slice's scales to tensor memory and issues its four K = 64
//               MMAs (N = 256); tcgen05.commit frees the slot.
//   warps 4-6   scales of A and of the two halves of B: each lane holds 32 bytes (four slices) of
//               four rows in registers, loads the next 32 ahead, and writes each slice's words to
//               the chunk layout, 16 bytes at a time.  Groups start at any row, so no bulk copy of
//               a fixed box would do.
//   warps 8-15  epilogue: each warp takes 32 rows x 128 columns of the accumulator into registers
//               at once and frees it, so the next tile's MMAs run while it converts and stores.
//               (256 accumulator columns and the scales leave no room for a second accumulator.)
// Waits are bounded; on expiry the status word records the timeout and every role leaves.
//
// What bounds it: at 8192^3 it runs in 159-161 us, 6.9 PFLOP/s, the tensor pipe 80 % active (in K =
// 64 steps); without the scales (skipped, to time the rest) it takes 154, so the tensor pipe and
// its operands' way through shared memory are what is left.  Deep K keeps that (K = 14336: 6.6); at
// K = 2048 a tile is 8 slices, and the 1400 cycles in which the accumulator is emptied while no MMA
// can run are a fifth of it (3.4 with groups that fill 78 % of their tiles).  On the way there, at
// 8192^3: scales four bytes at a time per slice, 671 us (the L1 tag stage); pairs with a full
// release at cluster scope for each slice, 467 (it waits for the warp's loads in flight), releasing
// shared memory only, 250; 16-byte chunk stores, 238; whole-warp issue loops with an elected lane,
// 195; two slices behind one proxy fence, 184; scale rows located once a tile and loaded 32 bytes
// at a time, 163.
#include "launch.h"
#include "mx4.cuh"
#include "mx4_mma.cuh"
#include "tiles.cuh"

namespace moe {
namespace {
using namespace tc;
using namespace mx4;

constexpr int BM = 128, BN = 256;  // rows of a CTA, columns of a tile
constexpr int SF_BYTES = 6 * kScaleChunk;  // a slice: 2 chunks of A, 2 x 2 (K chunk, row half) of B
constexpr int kThreads = 512;
// Registers of a thread of each warpgroup (the launch gives 128 to each; 72 + 104 + 2 * 168 = 512
// = 4 * 128 are taken): the epilogue holds 128 accumulator values at once.
constexpr int kRegsIssue = 72, kRegsScales = 104, kRegsEpilogue = 168;
constexpr int kMaxExperts = 1024;
constexpr int kBarBytes = 256;
constexpr int kTurnBytes = 1024;  // an epilogue warp's: 32 rows x 32 bytes
constexpr uint32_t kTmemCols = 512, kScaleCol = 256;

// CG: CTAs of a tile
template <int CG>
struct Shape {
  static constexpr int STAGES = CG == 2 ? 6 : 4;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN / CG * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * (STAGE_BYTES + SF_BYTES) + kBarBytes +
                                 (kMaxExperts + 4) * sizeof(int) + 8 * kTurnBytes;
};
static_assert(Shape<1>::SMEM <= 232448 && Shape<2>::SMEM <= 232448, "shared memory of a CTA");

struct Params {
  const int32_t* offsets;  // null: one group of `rows` rows
  int64_t rows;
  const uint8_t* a_scales;
  const uint8_t* b_scales;   // gate for the gate/up product
  const uint8_t* b2_scales;  // up
  int64_t scale_pitch;       // of a row of K values
  int scales_align;          // see load_scales()
  int E, N, KB, NT;          // N: rows of one expert's B (gate/up: I); KB: 256-deep slices
  void* out;
  int store;                 // bytes of a store: 32 or 16 where they divide the pitch and the base
  uint8_t* codes;            // gate/up: rows of N values in blocks
  uint8_t* scales;
  unsigned* status;
  int zero_status;
};

// 32 consecutive bytes of a row's scales from byte `at` (a multiple of 32) on; bytes past the row
// are zero.  align: the largest of 32, 16 and 4 that divides the pitch and the bases.  One 32-byte
// load a row asks L2 once a sector; two of 16 bytes ask twice, as the little L1 that the ring
// leaves does not hold the tile's 384 lines between them.
__device__ __forceinline__ void load_scales(const uint8_t* row, int at, int pitch, int align,
                                            uint32_t* w) {
  if (align == 32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0u;
    if (at < pitch)
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                     "=r"(w[6]), "=r"(w[7])
                   : "l"(row + at));
  } else if (align == 16) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (at + 16 * j < pitch) v = ld_nc_v4(row + at + 16 * j);
      w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = at + 4 * j < pitch ? __ldg(reinterpret_cast<const uint32_t*>(row + at + 4 * j)) : 0u;
  }
}

__device__ __forceinline__ void st_v8(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
// 32 accumulator columns of a row, 32 bytes (a whole sector; 16 cost twice the requests) or 16 at a
// time; the last columns of a row of a ragged N one by one.
template <typename T>
__device__ __forceinline__ void store_row(T* row, const float* v, int col0, int N, int store) {
  constexpr int W = 16 / sizeof(T);
  if (col0 + 32 <= N) {
#pragma unroll
    for (int i = 0; i < 32 / W; i += 2) {
      Vec16<T> q, r;
      q.from_float(v + i * W);
      r.from_float(v + (i + 1) * W);
      if (store == 32) {
        st_v8(row + col0 + i * W, q.u, r.u);
      } else {
        st_v4(row + col0 + i * W, q.u);
        st_v4(row + col0 + (i + 1) * W, r.u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (col0 + i < N) row[col0 + i] = Dt<T>::from_f(v[i]);
  }
}
// A warp's 32 rows x 128 columns of an output whose rows are not 16-byte aligned (out: row 0, the
// warp's first column; rows, cols: how many of them exist): 32 bytes of each row at a time go through
// shared memory, so that a store's lanes write neighbouring elements of two (f32: four) rows.  With
// each lane writing its own row, element by element, 5467 x 6895 f16 with K = 512 took 342 us; this
// way, 74.  (The pair kernel spills nine registers for it.)
template <typename T>
__device__ __forceinline__ void store_turned(T* out, int64_t pitch, const uint32_t (&acc)[4][32],
                                             int rows, int cols, uint8_t* turn, int lane) {
  constexpr int CW = 32 / sizeof(T), RW = 32 / CW;  // columns of a piece, rows of a store
  const int rsub = lane / CW, col = lane % CW;
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += CW) {
    if (c0 < cols) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Vec16<T> q;
#pragma unroll
        for (int i = 0; i < Vec16<T>::N; ++i) {
          const int e = c0 + h * Vec16<T>::N + i;
          q.e[i] = Dt<T>::from_f(__uint_as_float(acc[e / 32][e % 32]));
        }
        *reinterpret_cast<uint4*>(turn + raw_offset(lane, h)) = q.u;
      }
      __syncwarp();
#pragma unroll 4
      for (int r = 0; r < 32; r += RW) {
        const int rr = r + rsub, at = col * (int)sizeof(T);
        const T v = *reinterpret_cast<const T*>(turn + raw_offset(rr, at >> 4) + (at & 15));
        if (rr < rows && c0 + col < cols) out[rr * pitch + c0 + col] = v;
      }
      __syncwarp();
    }
  }
}

// silu(g) u to a few units of FP32 (quantising it moves a value near a border between codes by a whole
// step), for any g that FP32 holds.  With e = exp(-|g| / 2), 1 / (1 + exp(-g)) is 1 / (1 + e^2) for
// g >= 0 and e^2 / (1 + e^2) below: the divisor stays in [1, 2], and g e e leaves the normal numbers
// only where silu(g) does.  e is a power of two of h = -|g| log2(e) / 2, whose rounding (and that of the
// constant) l makes up for.  (expf and a division take twice the instructions, more than the MMAs of a
// tile can hide: prefill experts 976 -> 1248 us, decode 54 -> 68.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float x = fabsf(g);
  const float c = -0.72134752f, c_lo = -9.6298e-9f;  // -log2(e) / 2
  const float h = x * c, l = fmaf(x, c_lo, fmaf(x, c, -h));
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(h));
  e = fmaf(e * l, 0.69314718f, e);  // 2^(h + l), l at most 2^-18
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, e, 1.f)));
  const float m = g < 0.f ? e : 1.f;
  return g * m * m * r * u;
}

// What the epilogue writes: the blocks of a; rows that are 16-byte aligned; other rows.
enum Kind { kGateUp, kRows, kTurned };

template <int CG, int KIND, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    moe_mx4_gemm(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                 const __grid_constant__ CUtensorMap mapB2, const Params p) {
  constexpr bool GATEUP = KIND == kGateUp;
  using S = Shape<CG>;
  constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES;
  extern __shared__ uint8_t mx4_smem_raw[];
  const uint32_t raw = smem_u32(mx4_smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = mx4_smem_raw + (base - raw);
  const uint32_t sf_base = base + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + STAGES * (STAGE_BYTES + SF_BYTES));
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };               // CTA 0's is used
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };   // each CTA's own
  const uint32_t tfull = bar0 + 8u * (2 * STAGES), tempty = tfull + 8, drain_bar = tfull + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 3);
  volatile int* abort_f = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* pref = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);
  uint8_t* turn = reinterpret_cast<uint8_t*>(pref + (kMaxExperts + 4));  // 16-byte aligned

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)cluster_rank() : 0;
  const bool leader = rank == 0;
  const int first = CG == 2 ? (int)cluster_id_x() : (int)blockIdx.x;
  const int step = CG == 2 ? (int)ncluster_x() : (int)gridDim.x;
  if (p.zero_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1 + 3 * CG);  // the producer's expect_tx and the scale warps
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 8 * CG);
    mbar_init(drain_bar, 1);
    *abort_f = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (CG == 2) tmem_alloc2(smem_u32(tmem_slot), kTmemCols);
    else tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  }
  // first row of group e, kept inside [0, rows] whatever the caller's array holds
  auto offset_of = [&](int e) {
    const int64_t v = p.offsets ? (int64_t)__ldg(p.offsets + e) : (e ? p.rows : 0);
    return (int)min(max(v, (int64_t)0), p.rows);
  };
  int* offs = reinterpret_cast<int*>(turn);  // until the prefix is built
  static_assert((kMaxExperts + 1) * sizeof(int) <= 8 * kTurnBytes, "offsets fit");
  for (int i = threadIdx.x; i <= p.E; i += kThreads) offs[i] = offset_of(i);
  __syncthreads();
  if (warp == 2)
    build_expert_prefix(
        offs, p.E, [](int n) { return n > 0 ? (n + BM * CG - 1) / (BM * CG) : 0; }, pref, lane);
  if (threadIdx.x == 0) {
    tma_prefetch(&mapA);
    tma_prefetch(&mapB);
    if (GATEUP) tma_prefetch(&mapB2);
  }
  tc_fence_before();
  if (CG == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = pref[p.E] * p.NT;
  // an arrival on the same barrier of CTA 0
  auto arrive_leader = [&](uint32_t bar) {
    if (leader) mbar_arrive(bar);
    else mbar_arrive_cluster_shared(map_to_rank(bar, 0));
  };
  // tile t -> this CTA's first row, end of the group's rows, expert, n-tile
  struct Tile {
    int r0, r1, e, n;
  };
  auto tile_of = [&](int t) {
    Tile x;
    x.e = find_expert(pref, p.E, t / p.NT);
    const int local = t - pref[x.e] * p.NT, mt = pref[x.e + 1] - pref[x.e];
    // eight m-tiles beside one n-tile, then the next n-tile
    const int g0 = local / (8 * p.NT) * 8, gm = min(8, mt - g0), q = local - g0 * p.NT;
    x.n = q / gm;
    x.r0 = offset_of(x.e) + (g0 + q % gm) * (BM * CG) + rank * BM;
    x.r1 = offset_of(x.e + 1);
    return x;
  };

  if (warp < 4) {
    set_max_regs_dec<kRegsIssue>();
    if (warp == 0) {
      int stage = 0, armed = 0;
      uint32_t phase = 0;
      bool stop = false;
      const uint64_t pol = policy_evict_normal();
      for (int t = first; t < total && !stop; t += step) {
        const Tile x = tile_of(t);
        const int b_row = x.e * p.N + x.n * (GATEUP ? BN / 2 : BN) +
                          rank * (GATEUP ? BN / 4 : BN / 2);
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!__all_sync(0xFFFFFFFFu,
                          wait_bounded(empty_bar(stage), phase ^ 1u, abort_f, p.status))) {
            stop = true;
            break;
          }
          const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + S::A_BYTES;
          const uint32_t fb = CG == 2 ? map_to_rank(full_bar(stage), 0) : full_bar(stage);
          auto load = [&](uint32_t dst, const CUtensorMap* m, int row) {
            if (CG == 2) tma_load_2d_pair(dst, m, fb, kb * 128, row, pol);
            else tma_load_2d(dst, m, fb, kb * 128, row, pol);
          };
          if (elect_one()) {
            if (leader) mbar_expect_tx(full_bar(stage), CG * STAGE_BYTES);
            load(sa, &mapA, x.r0);
            if (GATEUP) {
#pragma unroll
              for (int h = 0; h < 2 / CG; ++h) {
                load(sb + h * 128 * 128, &mapB, b_row + h * 64);
                load(sb + h * 128 * 128 + 64 * 128, &mapB2, b_row + h * 64);
              }
            } else {
              load(sb, &mapB, b_row);
            }
          }
          ++armed;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (stop && leader) {  // let copies still in flight land
        const long long until = clock64() + kWaitLimit;
        for (int i = 0; i < min(armed, STAGES); ++i) {
          if (stage == 0) {
            stage = STAGES - 1;
            phase ^= 1u;
          } else {
            --stage;
          }
          wait_until(full_bar(stage), phase, until);
        }
      }
    }
    if (warp == 1 && leader) {
      constexpr uint32_t idesc0 = make_idesc_mxf4(BM * CG, BN, 0);
      constexpr uint32_t idesc2 = make_idesc_mxf4(BM * CG, BN, 2);
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, CG == 2
                                           ? wait_bounded_cluster(bar, parity, abort_f, p.status)
                                           : wait_bounded(bar, parity, abort_f, p.status));
      };
      auto copy = [&](uint32_t taddr, uint32_t chunk) {
        if (CG == 2) tmem_cp_scale2(taddr, make_sdesc_scale(chunk));
        else tmem_cp_scale(taddr, make_sdesc_scale(chunk));
      };
      int stage = 0;
      uint32_t phase = 0, tphase = 0;
      bool stop = false;
      for (int t = first; t < total && !stop; t += step) {
        if (!wait(tempty, tphase ^ 1u)) break;
        tphase ^= 1u;
        tc_fence_after();
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!wait(full_bar(stage), phase)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + S::A_BYTES;
          const uint32_t sf = sf_base + stage * SF_BYTES;
          const uint64_t da = make_sdesc(sa), db = make_sdesc(sb);
          // a slot of columns for each stage, so that the copies need not wait for the MMAs of the
          // slice before: 128 values (c) take 4 columns for A and 8 for the two halves of B
          const uint32_t cols = tmem + kScaleCol + stage * 24;
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              copy(cols + c * 12, sf + c * kScaleChunk);
              copy(cols + c * 12 + 4, sf + (2 + 2 * c) * kScaleChunk);
              copy(cols + c * 12 + 8, sf + (3 + 2 * c) * kScaleChunk);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t ca = cols + (k >> 1) * 12, cb = ca + 4;
              const uint32_t idesc = (k & 1) ? idesc2 : idesc0, more = (kb | k) != 0;
              if (CG == 2) umma2_mxf4(tmem, da + 2u * k, db + 2u * k, idesc, ca, cb, more);
              else umma_mxf4(tmem, da + 2u * k, db + 2u * k, idesc, ca, cb, more);
            }
            if (CG == 2) umma_commit2(empty_bar(stage), 0x3);
            else umma_commit(empty_bar(stage));
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (stop) break;
        if (elect_one()) {
          if (CG == 2) umma_commit2(tfull, 0x3);
          else umma_commit(tfull);
        }
      }
      // arrives once every MMA issued above has completed
      if (elect_one()) {
        if (CG == 2) umma_commit2(drain_bar, 0x1);
        else umma_commit(drain_bar);
      }
      wait_drain(drain_bar, 0);
    }
  } else if (warp < 8) {
    set_max_regs_dec<kRegsScales>();
    // scales: warp 4 takes the A rows, warps 5 and 6 the two halves of the B rows; lane l holds
    // rows l, l + 32, l + 64, l + 96, whose words are 16 consecutive bytes of a chunk
    const int part = warp - 4;
    const int pitch = (int)p.scale_pitch;
    const int align = p.scales_align;
    int stage = 0;
    uint32_t phase = 0;
    bool stop = part == 3;
    // quads of slices over all of this CTA's tiles; the next quad's words are loaded ahead
    const int quads = (p.KB + 3) / 4;
    uint32_t next[4][8];
    const uint8_t* src[4];
    auto point = [&](int t) {  // src: this lane's four rows of tile t
      const Tile x = tile_of(t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 32 * j + lane;
        if (part == 0) {
          src[j] = p.a_scales + min((int64_t)x.r0 + i, p.rows - 1) * pitch;
        } else {
          const int h = part - 1;
          int n = GATEUP ? x.n * (BN / 2) + h * 64 + (i & 63) : x.n * BN + h * 128 + i;
          n = min(n, p.N - 1);
          const uint8_t* b = GATEUP && j >= 2 ? p.b2_scales : p.b_scales;
          src[j] = b + ((int64_t)x.e * p.N + n) * pitch;
        }
      }
    };
    auto load_quad = [&](int quad) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        load_scales(src[j], quad * 32, pitch, align, next[j]);
      }
    };
    if (first < total && !stop) {
      point(first);
      load_quad(0);
    }
    // chunk (c, half) of B is chunk 2 + 2 c + half of a slice, chunk c of A is chunk c
    const uint32_t dst = sf_base + (part == 0 ? 0 : 1 + part) * kScaleChunk + lane * 16;
    const uint32_t chunk_step = (part == 0 ? 1 : 2) * kScaleChunk;
    for (int t = first; t < total && !stop; t += step) {
      for (int quad = 0; quad < quads && !stop; ++quad) {
        uint32_t now[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int w = 0; w < 8; ++w) now[j][w] = next[j][w];
        if (quad + 1 < quads) {
          load_quad(quad + 1);
        } else if (t + step < total) {
          point(t + step);
          load_quad(0);
        }
        // two slices at a time: a fence between the proxies and the arrivals behind it are a chain
        // of several hundred cycles, as long as a slice's MMAs
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const int n = min(2, p.KB - quad * 4 - k);
          if (n <= 0 || stop) continue;
          uint32_t bar[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if (z >= n || stop) continue;
            // (every lane waits: the warp's threads write together)
            if (!__all_sync(0xFFFFFFFFu,
                            wait_bounded(empty_bar(stage), phase ^ 1u, abort_f, p.status))) {
              stop = true;
              continue;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int w = 2 * (k + z) + c;
              st_shared_v4(dst + stage * SF_BYTES + c * chunk_step, now[0][w], now[1][w],
                           now[2][w], now[3][w]);
            }
            bar[z] = full_bar(stage);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (stop) continue;
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) {
            arrive_leader(bar[0]);
            if (n == 2) arrive_leader(bar[1]);
          }
        }
      }
    }
  } else {
    set_max_regs_inc<kRegsEpilogue>();
    const int q = warp & 3, h = warp >= 12;  // lane quarter, column half
    uint32_t tphase = 0;
    for (int t = first; t < total; t += step) {
      const Tile x = tile_of(t);
      const bool ok = wait_bounded(tfull, tphase, abort_f, p.status);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tphase ^= 1u;
      tc_fence_after();
      uint32_t acc[4][32];
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + h * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(taddr + c * 32, acc[c]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(tempty);
      const int row = x.r0 + q * 32 + lane;
      if (KIND == kTurned) {
        const int col0 = x.n * BN + h * 128;
        store_turned((T*)p.out + (int64_t)(x.r0 + q * 32) * p.N + col0, p.N, acc,
                     x.r1 - x.r0 - q * 32, p.N - col0, turn + (warp - 8) * kTurnBytes, lane);
      } else if (row < x.r1) {
        if (GATEUP) {
          // columns 0-63 gate, 64-127 up of a's columns n * 128 + h * 64 ..: two blocks
          const int64_t cp = code_pitch(p.N), sp = scale_pitch(p.N);
          const int blocks = (int)blocks_of(p.N);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int blk = x.n * 4 + h * 2 + c;
            if (blk >= blocks) continue;
            float a[32];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float g = __uint_as_float(acc[c][i]), u = __uint_as_float(acc[c + 2][i]);
              a[i] = blk * 32 + i < p.N ? silu_mul(g, u) : 0.f;
              top = max(top, __float_as_uint(a[i]) & 0x7FFFFFFFu);
            }
            const uint32_t b = scale_byte(top);
            const float inv = inv_scale(b);
            uint4 w = make_uint4(0, 0, 0, 0);
            if (b != 255u)
              w = make_uint4(codes8(a, inv), codes8(a + 8, inv), codes8(a + 16, inv),
                             codes8(a + 24, inv));
            st_v4(p.codes + row * cp + blk * 16, w);
            p.scales[row * sp + blk] = (uint8_t)b;
            if (blk == blocks - 1)
              for (int z = blocks; z & 3; ++z) p.scales[row * sp + z] = 0;
          }
        } else {
          T* orow = (T*)p.out + (int64_t)row * p.N;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            store_row(orow, reinterpret_cast<const float*>(acc[c]), x.n * BN + h * 128 + c * 32,
                      p.N, p.store);
        }
      }
    }
  }

  settle_after_abort(abort_f);
  tc_fence_before();
  __syncwarp();
  if (CG == 2) cluster_sync_all();  // no CTA leaves while its pair may still signal it
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2) tmem_dealloc2(tmem, kTmemCols);
    else tmem_dealloc(tmem, kTmemCols);
  }
}

int sm_count(cudaError_t* err) {
  int dev = 0, sms = 0;
  *err = cudaGetDevice(&dev);
  if (*err == cudaSuccess) *err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <int CG, int KIND, typename T>
cudaError_t launch_cg(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& b2,
                      const Params& p, int sms, cudaStream_t s) {
  auto kern = moe_mx4_gemm<CG, KIND, T>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Shape<CG>::SMEM);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<CG>::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 1 : 0;
  const int64_t rows_per = BM * CG;
  const int64_t upper = ((p.rows + rows_per - 1) / rows_per + p.E) * (int64_t)p.NT;  // >= tiles
  const int64_t fit = sms / CG;
  cfg.gridDim = dim3((unsigned)(CG * (upper < fit ? upper : fit)));
  return cudaLaunchKernelEx(&cfg, kern, a, b, b2, p);
}

// Pairs when groups average at least 160 rows; below that a pair's taller tiles multiply mostly
// padding, above it they read fewer bytes through L2.  Experts of 32 groups, H = 4096, I = 2048,
// one CTA against a pair: 64 rows a group 91 / 96 us, 96 95 / 102, 128 105 / 107, 192 119 / 112,
// 512 229 / 219.
bool use_pairs(int64_t rows, int E) { return rows >= (int64_t)160 * E; }

template <int KIND, typename T>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& b2,
                   const Params& p, cudaStream_t s) {
  cudaError_t err;
  const int sms = sm_count(&err);
  if (err != cudaSuccess) return err;
  return use_pairs(p.rows, p.E) ? launch_cg<2, KIND, T>(a, b, b2, p, sms, s)
                                : launch_cg<1, KIND, T>(a, b, b2, p, sms, s);
}

// Of 32, 16 and 4, the largest that divides the pitch and the three bases.
int scales_align(int64_t pitch, const void* a, const void* b, const void* c) {
  const uintptr_t all = (uintptr_t)pitch | (uintptr_t)a | (uintptr_t)b | (uintptr_t)c;
  return all % 32 == 0 ? 32 : all % 16 == 0 ? 16 : 4;
}

Params make_params(Mx4Rows a, int64_t rows, const int32_t* offsets, int E, int N, int K, int cols,
                   unsigned* status) {
  Params p{};
  p.offsets = offsets;
  p.rows = rows;
  p.a_scales = a.scales;
  p.scale_pitch = scale_pitch(K);
  p.E = E;
  p.N = N;
  p.KB = (K + 255) / 256;
  p.NT = (N + cols - 1) / cols;
  p.status = status;
  return p;
}

}  // namespace

cudaError_t launch_mx4_product(Mx4Rows a, int64_t rows, Mx4Rows b, const int32_t* offsets, int E,
                               int N, int K, void* out, int odt, unsigned* status,
                               bool zero_status, cudaStream_t s) {
  CUtensorMap ma, mb;
  const int64_t pitch = code_pitch(K);
  if (!make_map_bytes(&ma, a.codes, pitch, rows, BM) ||
      !make_map_bytes(&mb, b.codes, pitch, (int64_t)E * N, use_pairs(rows, E) ? BN / 2 : BN))
    return cudaErrorInvalidValue;
  Params p = make_params(a, rows, offsets, E, N, K, BN, status);
  p.b_scales = b.scales;
  p.scales_align = scales_align(p.scale_pitch, a.scales, b.scales, b.scales);
  p.out = out;
  const uintptr_t both = (uintptr_t)out | (uintptr_t)N * (odt == MOE_F32 ? 4 : 2);
  p.store = both % 32 == 0 ? 32 : both % 16 == 0 ? 16 : 1;
  p.zero_status = zero_status;
  const bool turned = p.store < 16;
  switch (odt) {
    case MOE_F32:
      return turned ? launch<kTurned, float>(ma, mb, mb, p, s) : launch<kRows, float>(ma, mb, mb, p, s);
    case MOE_F16:
      return turned ? launch<kTurned, __half>(ma, mb, mb, p, s)
                    : launch<kRows, __half>(ma, mb, mb, p, s);
    case MOE_BF16:
      return turned ? launch<kTurned, __nv_bfloat16>(ma, mb, mb, p, s)
                    : launch<kRows, __nv_bfloat16>(ma, mb, mb, p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx4_gate_up(Mx4Rows a, int64_t rows, Mx4Rows gate, Mx4Rows up,
                               const int32_t* offsets, int E, int I, int H, uint8_t* codes,
                               uint8_t* scales, unsigned* status, cudaStream_t s) {
  CUtensorMap ma, mg, mu;
  const int64_t pitch = code_pitch(H);
  if (!make_map_bytes(&ma, a.codes, pitch, rows, BM) ||
      !make_map_bytes(&mg, gate.codes, pitch, (int64_t)E * I, 64) ||
      !make_map_bytes(&mu, up.codes, pitch, (int64_t)E * I, 64))
    return cudaErrorInvalidValue;
  Params p = make_params(a, rows, offsets, E, I, H, BN / 2, status);
  p.b_scales = gate.scales;
  p.b2_scales = up.scales;
  p.scales_align = scales_align(p.scale_pitch, a.scales, gate.scales, up.scales);
  p.codes = codes;
  p.scales = scales;
  return launch<kGateUp, float>(ma, mg, mu, p, s);
}

}  // namespace moe
