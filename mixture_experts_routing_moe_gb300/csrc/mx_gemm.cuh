// Grouped products of microscaled rows, in 4 or in 8 bits (F: Fmt4 or Fmt8), on 5th-generation
// tensor cores (tcgen05.mma kind::mxf4 or kind::mxf8f6f4, scales from tensor memory):
//   product   out[r, n] = sum_k A[r, k] B[e, n, k]
//   gate/up   the blocks of silu(A gate_e^T) * (A up_e^T), quantised in the epilogue
// over the ragged row groups offsets[e] .. offsets[e+1]-1.
//
// A persistent kernel walks tiles (expert, m-tile, n-tile) of 256 columns and 128 rows (a CTA) or
// 256 rows (a cluster of two CTAs, cta_group::2: each CTA holds 128 of the rows and half of the B
// rows, so a tile pulls a third fewer bytes through L2), or in 8 bits of 64 or 128 columns and 128
// rows where few rows leave few tiles.  Roles in each CTA:
//   warp 0      loads, for each K slice (128 bytes a row: 256 values in 4 bits, 128 in 8), the codes
//               of its A and B rows by TMA into a ring.  For gate/up the B tile of 256 columns holds
//               gate rows 0-63, up rows 0-63, gate rows 64-127, up rows 64-127 of 128 columns of a.
//               (Warps 0 and 1 run their loops with all lanes; an elected one issues.)
//   warp 1      (of CTA 0) copies each slice's scales to tensor memory and issues its four MMAs of
//               32 bytes a row (K = 64 or 32); tcgen05.commit frees the slot.
//   warps 4-6   scales of A and of the two halves of B: each lane holds 32 bytes (four or eight
//               slices) of four rows in registers, loads the next 32 ahead, and writes each slice's
//               words to the chunk layout, 16 bytes at a time.  Groups start at any row, so no bulk
//               copy of a fixed box would do.
//   warps 8-15  epilogue: each warp takes 32 rows and half of the columns of the accumulator into
//               registers at once and frees it, so the next tile's MMAs run while it converts and
//               stores.  (256 accumulator columns and the scales leave no room for a second
//               accumulator.)
// Waits are bounded; on expiry the status word records the timeout and every role leaves.
//
// What bounds it, in 4 bits: at 8192^3 it runs in 152-157 us, 7.0-7.2 PFLOP/s, the tensor pipe 83 %
// active (in K = 64 steps).  Before the stores of 16-bit rows went by whole lines (store_lines) it took
// 159-161, and without the scales (skipped, to time the rest) 154, so the tensor pipe and its operands'
// way through shared memory are what is left.  Deep K kept that
// (K = 14336: 6.6); at K = 2048 a tile is 8 slices, and the 1400 cycles in which the accumulator is
// emptied while no MMA can run are a fifth of it (3.4 with groups that fill 78 % of their tiles).  On
// the way there, at 8192^3: scales four bytes at a time per slice, 671 us (the L1 tag stage); pairs
// with a full release at cluster scope for each slice, 467 (it waits for the warp's loads in flight),
// releasing shared memory only, 250; 16-byte chunk stores, 238; whole-warp issue loops with an
// elected lane, 195; two slices behind one proxy fence, 184; scale rows located once a tile and
// loaded 32 bytes at a time, 163.
// In 8 bits a slice's MMAs take twice as long (512 cycles), so the rest hides better: 8192^3 in
// 310-321 us by itself, 3.5 PFLOP/s, the tensor pipe 87 % active; under load, at the 1.4 GHz that its
// power leaves, 364-373.  A tile of 64 slices took 36300 cycles, of which 32800 are MMAs; the emptying
// is some 1000, and the next tile's first slices came late behind the stores (store_lines).  Raw
// scales that came by TMA instead of through the scale warps' loads made no difference there (363 and
// 371 us on two boxes) and few rows slower.
#pragma once

#include "launch.h"
#include "mx4.cuh"
#include "mx4_mma.cuh"
#include "mx8.cuh"
#include "tiles.cuh"

namespace moe {
namespace {
using namespace tc;

constexpr int BM = 128;  // rows of a CTA
constexpr int kWide = 256, kHalf = 128, kNarrow = 64;  // columns of a tile (BN)
constexpr int kThreads = 512;
// Registers of a thread of each warpgroup (the launch gives 128 to each; 72 + 104 + 2 * 168 = 512
// = 4 * 128 are taken): the epilogue holds 128 accumulator values at once.
constexpr int kRegsIssue = 72, kRegsScales = 104, kRegsEpilogue = 168;
constexpr int kMaxExperts = 1024;
constexpr int kBarBytes = 256;
constexpr int kTurnBytes = 1024;  // an epilogue warp's: 32 rows x 32 bytes
constexpr uint32_t kTmemCols = 512, kScaleCol = 256;

// What the two formats differ in.  A 128-byte slice of a row has CHUNKS x 128 values (a chunk holds the
// scales of 128 rows and four blocks).
struct Fmt4 {
  static constexpr int CHUNKS = 2, CODE_BYTES = 16;  // CODE_BYTES: of a block
  static __host__ __device__ int64_t code_pitch(int64_t K) { return mx4::code_pitch(K); }
  // MMA k of a slice: its scales are in chunk k / 2, bytes 0-1 or 2-3
  static constexpr int chunk_of(int k) { return k >> 1; }
  static constexpr uint32_t idesc(int M, int N, int k) { return make_idesc_mxf4(M, N, 2 * (k & 1)); }
  template <int CG>
  static __device__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                             uint32_t sfb, uint32_t more) {
    if (CG == 2) umma2_mxf4(d, a, b, idesc, sfa, sfb, more);
    else umma_mxf4(d, a, b, idesc, sfa, sfb, more);
  }
  // Scale byte of a block whose largest magnitude has the bits `top`, and its codes.
  static __device__ uint32_t block(const float* a, uint32_t top, uint4* out) {
    const uint32_t b = mx4::scale_byte(top);
    const float inv = mx4::inv_scale(b);
    uint4 w = make_uint4(0, 0, 0, 0);
    if (b != 255u)
      w = make_uint4(mx4::codes8(a, inv), mx4::codes8(a + 8, inv), mx4::codes8(a + 16, inv),
                     mx4::codes8(a + 24, inv));
    out[0] = w;
    return b;
  }
};
struct Fmt8 {
  static constexpr int CHUNKS = 1, CODE_BYTES = 32;
  static __host__ __device__ int64_t code_pitch(int64_t K) { return mx8::code_pitch(K); }
  static constexpr int chunk_of(int) { return 0; }
  static constexpr uint32_t idesc(int M, int N, int k) { return make_idesc_mxf8(M, N, k); }
  template <int CG>
  static __device__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                             uint32_t sfb, uint32_t more) {
    if (CG == 2) umma2_mxf8(d, a, b, idesc, sfa, sfb, more);
    else umma_mxf8(d, a, b, idesc, sfa, sfb, more);
  }
  static __device__ uint32_t block(const float* a, uint32_t top, uint4* out) {
    const uint32_t b = mx8::scale_byte(top);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = b == 255u ? 0u : mx8::codes4(a + 4 * i, mx8::inv_scale(b));
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return b;
  }
};

// CG: CTAs of a tile; BN: its columns
template <typename F, int CG, int BN>
struct Shape {
  static constexpr int STAGES = BN == kNarrow ? 8 : CG == 2 || BN == kHalf ? 6 : 4;
  // Epilogue halves of a tile's columns; of those of a half, the first half is gate's, the other up's.
  static constexpr int HALVES = BN >= 128 ? 2 : 1, HC = BN / HALVES, GC = HC / 2;
  // Rows of a copy of A.  Single CTAs, which few rows take, copy the rows that their group has and no
  // others: with 128 a slice, every CTA asked L2 for the few rows there are at the same time (a token's
  // 8 experts, H = 2048, I = 768: 1.5 us a slice).
  static constexpr int A_BOX = CG == 1 && F::CHUNKS == 1 ? 16 : BM;
  static constexpr int B_CHUNKS = (BN + 127) / 128;  // scale chunks of 128 B rows
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN / CG * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // scales of a slice: the chunks of A, then (chunk, row half) of B
  static constexpr int SF_BYTES = (1 + B_CHUNKS) * F::CHUNKS * kScaleChunk;
  static constexpr int SF_COLS = (1 + B_CHUNKS) * 4;  // columns of tensor memory of 128 values
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * (STAGE_BYTES + SF_BYTES) + kBarBytes +
                                 (kMaxExperts + 4) * sizeof(int) + 8 * kTurnBytes;
};
static_assert(Shape<Fmt4, 1, kWide>::SMEM <= 232448 && Shape<Fmt4, 2, kWide>::SMEM <= 232448 &&
                  Shape<Fmt8, 1, kWide>::SMEM <= 232448 && Shape<Fmt8, 2, kWide>::SMEM <= 232448 &&
                  Shape<Fmt8, 1, kNarrow>::SMEM <= 232448 && Shape<Fmt8, 1, kHalf>::SMEM <= 232448,
              "shared memory of a CTA");
static_assert(kScaleCol + 8 * Shape<Fmt8, 1, kNarrow>::SF_COLS <= kTmemCols &&
                  kScaleCol + 6 * Fmt4::CHUNKS * Shape<Fmt4, 2, kWide>::SF_COLS <= kTmemCols,
              "tensor memory");
static_assert((2 * 8 + 3 + 1) * 8 <= kBarBytes, "barriers");

struct Params {
  const int32_t* offsets;  // null: one group of `rows` rows
  int64_t rows;
  const uint8_t* a_scales;
  const uint8_t* b_scales;   // gate for the gate/up product
  const uint8_t* b2_scales;  // up
  int64_t scale_pitch;       // of a row of K values
  int scales_align;          // see load_scales()
  int E, N, KB, NT;          // N: rows of one expert's B (gate/up: I); KB: slices
  void* out;
  int store;                 // kRows: bytes of a store, 32 or 16
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
// 32 accumulator columns of a row, 32 bytes (a whole sector; 16 cost twice the requests) or 16 at a time;
// the last columns of a row of a ragged N one by one.  (FP32 rows by whole lines, as store_lines writes
// them, made one wave of short tiles slower, 3001 x 1000 with K = 1376 in 8 bits: 11.7 -> 13.3 us; 8192 x
// 8192 would gain, K = 2048 122 -> 109, K = 8192 334 -> 329.)
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
// V pieces of 16 bytes of each of a warp's 32 rows (a lane holds its row's; out: row 0, the warp's first
// byte; rows, bytes: how many of them exist, whole pieces).  They go through the warp's 1 KB of shared
// memory, 64 / V rows at a time (swizzled, so neither way has conflicts), and V lanes store V neighbouring
// pieces: whole lines of 128 bytes where V = 8.  With each lane writing 32 bytes of its own row at a time,
// the first slices of the next tile came 2500 cycles late behind the requests: 8192 x 8192 bf16 with
// K = 2048 took 99 to 104 us on three boxes (4 bits: 68), this way 91 to 96 (60), and without any store
// 80 (47).  2 or 4 KB a warp, the L2's eviction hints and stores spread over the next tile's time
// changed little (K = 2048 96.5, 91.4 against 91.6, and 90.2).
template <int V>
__device__ __forceinline__ void store_lines(uint8_t* out, int64_t pitch, const uint4 (&v)[V], int rows,
                                            int bytes, uint32_t turn, int lane) {
  static_assert(V == 2 || V == 4 || V == 8, "pieces of a row");
  constexpr int ROWS = 64 / V;
  auto at = [&](int row, int j) { return turn + (row * V + (j ^ (row / (8 / V) % V))) * 16; };
#pragma unroll
  for (int g = 0; g < 32 / ROWS; ++g) {
    if (lane / ROWS == g) {
#pragma unroll
      for (int j = 0; j < V; ++j) st_shared_v4(at(lane % ROWS, j), v[j].x, v[j].y, v[j].z, v[j].w);
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = (h * 32 + lane) / V, j = lane % V;
      const uint4 q = ld_shared_v4(at(row, j));
      if (g * ROWS + row < rows && j * 16 < bytes) st_v4(out + (g * ROWS + row) * pitch + j * 16, q);
    }
    __syncwarp();
  }
}
// A warp's 32 rows x 32 CH columns of an output whose rows are not 16-byte aligned (out: row 0, the
// warp's first column; rows, cols: how many of them exist): 32 bytes of each row at a time go through
// shared memory, so that a store's lanes write neighbouring elements of two (f32: four) rows.  With
// each lane writing its own row, element by element, 5467 x 6895 f16 with K = 512 took 342 us; this
// way, 74.  (The pair kernel spills nine registers for it.)
template <typename T, int CH>
__device__ __forceinline__ void store_turned(T* out, int64_t pitch, const uint32_t (&acc)[CH][32],
                                             int rows, int cols, uint8_t* turn, int lane) {
  constexpr int CW = 32 / sizeof(T), RW = 32 / CW;  // columns of a piece, rows of a store
  const int rsub = lane / CW, col = lane % CW;
#pragma unroll
  for (int c0 = 0; c0 < 32 * CH; c0 += CW) {
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

// What the epilogue writes: the blocks of a; rows that are 16-byte aligned, by lanes or (16 bits) by whole
// lines; other rows.
enum Kind { kGateUp, kRows, kLines, kTurned };

template <typename F, int CG, int BN, int KIND, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    moe_mx_gemm(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                 const __grid_constant__ CUtensorMap mapB2, const Params p) {
  constexpr bool GATEUP = KIND == kGateUp;
  using S = Shape<F, CG, BN>;
  constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES, SF_BYTES = S::SF_BYTES;
  constexpr int CHUNKS = F::CHUNKS, B_CHUNKS = S::B_CHUNKS, HC = S::HC, GC = S::GC;
  constexpr int GROUP = 8 / CHUNKS;  // slices whose scales are 32 bytes of a row
  extern __shared__ uint8_t mx_smem_raw[];
  const uint32_t raw = smem_u32(mx_smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = mx_smem_raw + (base - raw);
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
      mbar_init(full_bar(s), 1 + (1 + B_CHUNKS) * CG);  // the producer's expect_tx and the scale warps
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 4 * S::HALVES * CG);
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
            const int a_rows = S::A_BOX == BM ? BM : min(BM, x.r1 - x.r0);
            const int boxes = (a_rows + S::A_BOX - 1) / S::A_BOX;
            if (leader)
              mbar_expect_tx(full_bar(stage),
                             CG * (S::B_BYTES + boxes * S::A_BOX * 128));
            for (int i = 0; i < boxes; ++i) load(sa + i * S::A_BOX * 128, &mapA, x.r0 + i * S::A_BOX);
            if (GATEUP) {
#pragma unroll
              for (int h = 0; h < S::HALVES / CG; ++h) {
                load(sb + h * HC * 128, &mapB, b_row + h * GC);
                load(sb + h * HC * 128 + GC * 128, &mapB2, b_row + h * GC);
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
          const uint32_t cols = tmem + kScaleCol + stage * S::SF_COLS * CHUNKS;
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
              copy(cols + c * S::SF_COLS, sf + c * kScaleChunk);
#pragma unroll
              for (int h = 0; h < B_CHUNKS; ++h)
                copy(cols + c * S::SF_COLS + 4 + 4 * h,
                     sf + (CHUNKS + B_CHUNKS * c + h) * kScaleChunk);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t ca = cols + F::chunk_of(k) * S::SF_COLS, cb = ca + 4;
              F::template mma<CG>(tmem, da + 2u * k, db + 2u * k, F::idesc(BM * CG, BN, k), ca, cb,
                                  (kb | k) != 0);
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
    bool stop = part > B_CHUNKS;
    // groups of slices over all of this CTA's tiles; the next group's words are loaded ahead
    const int groups = (p.KB + GROUP - 1) / GROUP;
    uint32_t next[4][8];
    const uint8_t* src[4];
    auto point = [&](int t) {  // src: this lane's four rows of tile t
      const Tile x = tile_of(t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 32 * j + lane;
        if (part == 0) {
          src[j] = p.a_scales + min((int64_t)x.r0 + i, (S::A_BOX == BM ? p.rows : x.r1) - 1) * pitch;
        } else {
          const int h = part - 1;
          // (of a narrow tile's chunk, rows 64 to 127 are not used)
          int n = GATEUP ? x.n * (BN / 2) + (h * 128 + i) / HC * GC + i % GC
                         : x.n * BN + h * 128 + i;
          n = min(n, p.N - 1);
          const uint8_t* b = GATEUP && i % HC >= GC ? p.b2_scales : p.b_scales;
          src[j] = b + ((int64_t)x.e * p.N + n) * pitch;
        }
      }
    };
    auto load_group = [&](int group) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        load_scales(src[j], group * 32, pitch, align, next[j]);
      }
    };
    if (first < total && !stop) {
      point(first);
      load_group(0);
    }
    // chunk (c, half) of B is chunk CHUNKS + B_CHUNKS c + half of a slice, chunk c of A is chunk c
    const uint32_t dst = sf_base + (part == 0 ? 0 : CHUNKS - 1 + part) * kScaleChunk + lane * 16;
    const uint32_t chunk_step = (part == 0 ? 1 : B_CHUNKS) * kScaleChunk;
    for (int t = first; t < total && !stop; t += step) {
      for (int group = 0; group < groups && !stop; ++group) {
        uint32_t now[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int w = 0; w < 8; ++w) now[j][w] = next[j][w];
        if (group + 1 < groups) {
          load_group(group + 1);
        } else if (t + step < total) {
          point(t + step);
          load_group(0);
        }
        // two slices at a time: a fence between the proxies and the arrivals behind it are a chain
        // of several hundred cycles, as long as a slice's MMAs
#pragma unroll
        for (int k = 0; k < GROUP; k += 2) {
          const int n = min(2, p.KB - group * GROUP - k);
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
            for (int c = 0; c < CHUNKS; ++c) {
              const int w = CHUNKS * (k + z) + c;
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
    for (int t = h < S::HALVES ? first : total; t < total; t += step) {
      const Tile x = tile_of(t);
      const bool ok = wait_bounded(tfull, tphase, abort_f, p.status);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tphase ^= 1u;
      tc_fence_after();
      uint32_t acc[HC / 32][32];
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + h * HC;
#pragma unroll
      for (int c = 0; c < HC / 32; ++c) tmem_ld32(taddr + c * 32, acc[c]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(tempty);
      const int64_t row0 = x.r0 + q * 32;
      const int rows = x.r1 - (int)row0;  // of the warp's that the group has, or more
      if (rows <= 0) continue;
      uint8_t* my_turn = turn + (warp - 8) * kTurnBytes;
      if (GATEUP) {
        // GC columns gate, then GC up, of a's columns n * BN / 2 + h * GC ..: GC / 32 blocks
        constexpr int BLOCKS = GC / 32, PIECES = F::CODE_BYTES / 16;
        const int64_t cp = F::code_pitch(p.N), sp = mx4::scale_pitch(p.N);
        const int blocks = (int)mx4::blocks_of(p.N), blk0 = x.n * (BN / 64) + h * BLOCKS;
        uint4 codes[BLOCKS * PIECES];
        uint32_t scale = 0;  // bytes, the first block's lowest
#pragma unroll
        for (int c = 0; c < BLOCKS; ++c) {
          float a[32];
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float g = __uint_as_float(acc[c][i]), u = __uint_as_float(acc[c + BLOCKS][i]);
            a[i] = (blk0 + c) * 32 + i < p.N ? mx4::silu_mul(g, u) : 0.f;
            top = max(top, __float_as_uint(a[i]) & 0x7FFFFFFFu);
          }
          scale |= F::block(a, top, codes + c * PIECES) << (8 * c);
        }
        // (Single CTAs' lanes store their own rows: through shared memory the experts of 256 tokens, k = 8,
        // 128 experts took 57.8 us in place of 56.5 in 4 bits, those of 2000 118 and 115.)
        if (CG == 2)
          store_lines(p.codes + row0 * cp + (int64_t)blk0 * F::CODE_BYTES, cp, codes, rows,
                      (blocks - blk0) * F::CODE_BYTES, smem_u32(my_turn), lane);
        if (lane < rows && blk0 < blocks) {
          if (CG == 1) {
            uint8_t* at = p.codes + (row0 + lane) * cp + (int64_t)blk0 * F::CODE_BYTES;
#pragma unroll
            for (int c = 0; c < BLOCKS; ++c) {
              if (blk0 + c >= blocks) continue;
              if (PIECES == 2) st_v8(at + c * 32, codes[c * PIECES], codes[c * PIECES + PIECES - 1]);
              else st_v4(at + c * 16, codes[c]);
            }
          }
          // pitches are multiples of four, and a row's bytes past its last block are zero
          uint8_t* sc = p.scales + (row0 + lane) * sp + blk0;
          if (BLOCKS == 2 && blk0 + 1 < blocks) *reinterpret_cast<uint16_t*>(sc) = (uint16_t)scale;
          else *sc = (uint8_t)scale;
          const int last = min(blk0 + BLOCKS, blocks);
          if (last == blocks)
            for (int z = last; z & 3; ++z) sc[z - blk0] = 0;
        }
      } else if (KIND == kTurned) {
        const int col0 = x.n * BN + h * HC;
        store_turned((T*)p.out + row0 * p.N + col0, p.N, acc, rows, p.N - col0, my_turn, lane);
      } else if constexpr (KIND == kRows) {
        if (lane < rows) {
#pragma unroll
          for (int c = 0; c < HC / 32; ++c)
            store_row((T*)p.out + (row0 + lane) * p.N, reinterpret_cast<const float*>(acc[c]),
                      x.n * BN + h * HC + c * 32, p.N, p.store);
        }
      } else {
        constexpr int W = 16 / sizeof(T), C = 8 * W;  // columns of a piece and of a line
#pragma unroll
        for (int c = 0; c < HC / C; ++c) {
          const int col0 = x.n * BN + h * HC + c * C;
          uint4 line[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            Vec16<T> piece;
            const int e = c * C + j * W;
            piece.from_float(reinterpret_cast<const float*>(acc[e / 32]) + e % 32);
            line[j] = piece.u;
          }
          if (col0 < p.N)
            store_lines((uint8_t*)((T*)p.out + row0 * p.N + col0), (int64_t)p.N * sizeof(T), line, rows,
                        (p.N - col0) * (int)sizeof(T), smem_u32(my_turn), lane);
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

template <typename F, int CG, int BN, int KIND, typename T>
cudaError_t launch_cg(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& b2,
                      const Params& p, int sms, cudaStream_t s) {
  using S = Shape<F, CG, BN>;
  auto kern = moe_mx_gemm<F, CG, BN, KIND, T>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)S::SMEM);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::SMEM;
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
// 512 229 / 219.  In 8 bits: 64 147 / 157, 128 155 / 165, 160 184 / 171, 192 188 / 173, 512 353 / 310.
bool use_pairs(int64_t rows, int E) { return rows >= (int64_t)160 * E; }

template <typename F>
int a_box(int64_t rows, int E) {
  return use_pairs(rows, E) ? Shape<F, 2, kWide>::A_BOX : Shape<F, 1, kWide>::A_BOX;
}

// Columns of a tile (in 8 bits) of at most 128 rows.  A slice costs some 470 cycles of issue however narrow
// its tile is, so the narrowest pay only as long as every SM has one at most, and half ones where there
// are a few a SM, to deal them out evenly.  Experts, cold, with a row for each reached, at 64 / 128 / 256
// columns: 4 of 16, H = 1024, I = 512: 18.9 / 21.0 / 25.1 us; 8 of 128, H = 2048, I = 768: 31.2 / 27.1 /
// 33.2; 28 of them 55.8 / 49.6 / 53.7, 51 84.4 / 70.1 / 72.2; 2 of 8, H = 4096, I = 14336: 123 / 95 / 109;
// 5 of them 250 / 195 / 177; 61 of 256, H = 7168, I = 2048: 600 / 443 / 443.
template <typename F>
int tile_columns(int64_t rows, int E, int64_t columns, int sms) {
  if (F::CHUNKS != 1 || use_pairs(rows, E) || rows > BM) return kWide;
  const int64_t experts = rows < E ? rows : E;  // that rows can reach
  if (experts * ((columns + kNarrow - 1) / kNarrow) <= sms) return kNarrow;
  return experts * ((columns + kWide - 1) / kWide) <= 3 * (int64_t)sms ? kHalf : kWide;
}

// Whether wide tiles' rows of 16 bits go by whole lines: pairs' do, and single CTAs' when the output is at
// least three full tiles an SM, as the way through shared memory costs a tile some 1500 cycles that only the
// next tile's slices, which come earlier, make up for.  By lanes / by lines, in 4 bits: 64 rows in 16 groups,
// N = 768, K = 2048 7.0 / 7.9 us; 5000 in 32, N = 2048, K = 512 14.9 / 16.0; 256 tokens' experts 56.5 / 58.8,
// 2000 tokens' 114.8 / 112.9; 20000 in 128, N = 2048, K = 768 39.7 / 37.4.  In 8 bits, the same rows: 8.8 /
// 9.0; 15.3 / 16.2; layers 90.3 / 90.9, 183.1 / 181.8; 62.5 / 61.4.  Pairs: 3001 rows in 7, N = 1000,
// K = 1376 11.6 / 10.3 and 12.2 / 10.9; 10000 in 32, N = 2048, K = 512 29.1 / 25.6 in 8 bits; 4096 in one,
// N = 2048, K = 512 10.5 / 10.7 and 11.5 / 11.8.
bool by_lines(int64_t rows, int E, int64_t N, int sms) {
  return use_pairs(rows, E) || rows * N >= (int64_t)3 * BM * kWide * sms;
}

// KIND of a wide tile; narrow ones and pairs have only one of kRows and kLines.
template <typename F, int KIND, typename T>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& b2,
                   const Params& p, int bn, int sms, cudaStream_t s) {
  constexpr int SMALL = KIND == kLines ? kRows : KIND;
  constexpr int PAIR = KIND == kRows && sizeof(T) == 2 ? kLines : KIND;
  if constexpr (F::CHUNKS == 1) {
    if (bn == kNarrow) return launch_cg<F, 1, kNarrow, SMALL, T>(a, b, b2, p, sms, s);
    if (bn == kHalf) return launch_cg<F, 1, kHalf, SMALL, T>(a, b, b2, p, sms, s);
  }
  return use_pairs(p.rows, p.E) ? launch_cg<F, 2, kWide, PAIR, T>(a, b, b2, p, sms, s)
                                : launch_cg<F, 1, kWide, KIND, T>(a, b, b2, p, sms, s);
}

// Of 32, 16 and 4, the largest that divides the pitch and the three bases.
int scales_align(int64_t pitch, const void* a, const void* b, const void* c) {
  const uintptr_t all = (uintptr_t)pitch | (uintptr_t)a | (uintptr_t)b | (uintptr_t)c;
  return all % 32 == 0 ? 32 : all % 16 == 0 ? 16 : 4;
}

template <typename F>
Params make_params(MxRows a, int64_t rows, const int32_t* offsets, int E, int N, int K, int cols,
                   unsigned* status) {
  Params p{};
  p.offsets = offsets;
  p.rows = rows;
  p.a_scales = a.scales;
  p.scale_pitch = mx4::scale_pitch(K);
  p.E = E;
  p.N = N;
  p.KB = (K + 128 * F::CHUNKS - 1) / (128 * F::CHUNKS);
  p.NT = (N + cols - 1) / cols;
  p.status = status;
  return p;
}

template <typename F, typename T>
cudaError_t launch_product(MxRows a, int64_t rows, MxRows b, const int32_t* offsets, int E, int N,
                           int K, void* out, unsigned* status, bool zero_status, cudaStream_t s) {
  CUtensorMap ma, mb;
  cudaError_t err;
  const int sms = sm_count(&err);
  if (err != cudaSuccess) return err;
  const int bn = tile_columns<F>(rows, E, N, sms);
  const int64_t pitch = F::code_pitch(K);
  if (!make_map_bytes(&ma, a.codes, pitch, rows, a_box<F>(rows, E)) ||
      !make_map_bytes(&mb, b.codes, pitch, (int64_t)E * N, use_pairs(rows, E) ? bn / 2 : bn))
    return cudaErrorInvalidValue;
  Params p = make_params<F>(a, rows, offsets, E, N, K, bn, status);
  p.b_scales = b.scales;
  p.scales_align = scales_align(p.scale_pitch, a.scales, b.scales, b.scales);
  p.out = out;
  const uintptr_t both = (uintptr_t)out | (uintptr_t)N * sizeof(T);
  p.store = both % 32 ? 16 : 32;
  p.zero_status = zero_status;
  if (both % 16) return launch<F, kTurned, T>(ma, mb, mb, p, bn, sms, s);
  if constexpr (sizeof(T) == 2)
    if (by_lines(rows, E, N, sms)) return launch<F, kLines, T>(ma, mb, mb, p, bn, sms, s);
  return launch<F, kRows, T>(ma, mb, mb, p, bn, sms, s);
}

template <typename F>
cudaError_t launch_gate_up(MxRows a, int64_t rows, MxRows gate, MxRows up, const int32_t* offsets,
                           int E, int I, int H, uint8_t* codes, uint8_t* scales, unsigned* status,
                           bool zero_status, cudaStream_t s) {
  CUtensorMap ma, mg, mu;
  cudaError_t err;
  const int sms = sm_count(&err);
  if (err != cudaSuccess) return err;
  const int bn = tile_columns<F>(rows, E, 2 * (int64_t)I, sms);
  const int64_t pitch = F::code_pitch(H);
  const int box = bn == kWide ? Shape<F, 1, kWide>::GC : Shape<F, 1, kHalf>::GC;
  static_assert(Shape<F, 1, kHalf>::GC == Shape<F, 1, kNarrow>::GC, "rows of a copy of gate or up");
  if (!make_map_bytes(&ma, a.codes, pitch, rows, a_box<F>(rows, E)) ||
      !make_map_bytes(&mg, gate.codes, pitch, (int64_t)E * I, box) ||
      !make_map_bytes(&mu, up.codes, pitch, (int64_t)E * I, box))
    return cudaErrorInvalidValue;
  Params p = make_params<F>(a, rows, offsets, E, I, H, bn / 2, status);
  p.b_scales = gate.scales;
  p.b2_scales = up.scales;
  p.scales_align = scales_align(p.scale_pitch, a.scales, gate.scales, up.scales);
  p.codes = codes;
  p.scales = scales;
  p.zero_status = zero_status;
  return launch<F, kGateUp, float>(ma, mg, mu, p, bn, sms, s);
}

}  // namespace
}  // namespace moe
