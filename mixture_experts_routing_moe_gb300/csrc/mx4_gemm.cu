// Grouped products of microscaled 4-bit rows on 5th-generation tensor cores (tcgen05.mma
// kind::mxf4, scales from tensor memory):
//   product   out[r, n] = sum_k A[r, k] B[e, n, k]
//   gate/up   the blocks of silu(A gate_e^T) * (A up_e^T), quantised in the epilogue
// over the ragged row groups offsets[e] .. offsets[e+1]-1.
//
// A persistent kernel, one CTA per SM, walks 128 x 256 tiles (expert, m-tile, n-tile).  Roles:
//   warp 0      one thread loads, for each 256-deep K slice, the codes of 128 A rows and 256 B rows
//               (128 bytes a row) by TMA into a 4-stage ring.  For gate/up the B tile holds gate
//               rows 0-63, up rows 0-63, gate rows 64-127, up rows 64-127 of 128 columns of a.
//   warp 1      one thread copies each slice's scales to tensor memory and issues its four
//               K = 64 MMAs (M = 128, N = 256); tcgen05.commit frees the slot.
//   warps 2-3   gather the scales of the slice's 384 rows with 4-byte cp.async into the chunk
//               layout; groups start at any row, so no bulk copy of a fixed box would do.
//   warps 4-11  epilogue: each warp takes 32 rows x 128 columns of the accumulator into registers
//               at once and frees it, so the next tile's MMAs run while it converts and stores.
//               (256 accumulator columns and the scales leave no room for a second accumulator.)
// Waits are bounded; on expiry the status word records the timeout and every role leaves.
#include <atomic>

#include "launch.h"
#include "mx4.cuh"
#include "mx4_mma.cuh"
#include "tiles.cuh"

namespace moe {
namespace {
using namespace tc;
using namespace mx4;

constexpr int BM = 128, BN = 256, STAGES = 4;
constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
constexpr int SF_BYTES = 6 * kScaleChunk;  // A: 2 chunks; B: 2 x 2 (K chunk, row half)
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int kThreads = 384;
constexpr int kLoaders = 64, kLag = STAGES - 1;
constexpr int kMaxExperts = 1024;
constexpr int kBarBytes = 128;
constexpr size_t kSmemBytes = 1024 + (size_t)STAGES * (STAGE_BYTES + SF_BYTES) + kBarBytes +
                              2 * (kMaxExperts + 4) * sizeof(int);
constexpr uint32_t kTmemCols = 512, kScaleCol = 256;

struct Params {
  const int32_t* offsets;  // null: one group of `rows` rows
  int64_t rows;
  const uint8_t* a_scales;
  const uint8_t* b_scales;   // gate for the gate/up product
  const uint8_t* b2_scales;  // up
  int64_t scale_pitch;       // of a row of K values
  int E, N, KB, NT;          // N: rows of one expert's B (gate/up: I); KB: 256-deep slices
  void* out;
  uint8_t* codes;            // gate/up: rows of N values in blocks
  uint8_t* scales;
  unsigned* status;
  int zero_status;
};

template <typename T>
__device__ __forceinline__ void store_row(T* row, const float* v, int col0, int N, bool vec) {
  constexpr int W = 16 / sizeof(T);
  if (vec && col0 + 32 <= N) {
#pragma unroll
    for (int i = 0; i < 32 / W; ++i) {
      Vec16<T> q;
      q.from_float(v + i * W);
      st_v4(row + col0 + i * W, q.u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (col0 + i < N) row[col0 + i] = Dt<T>::from_f(v[i]);
  }
}

template <bool GATEUP, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    moe_mx4_gemm(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                 const __grid_constant__ CUtensorMap mapB2, const Params p) {
  extern __shared__ uint8_t mx4_smem_raw[];
  const uint32_t raw = smem_u32(mx4_smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = mx4_smem_raw + (base - raw);
  const uint32_t sf_base = base + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + STAGES * (STAGE_BYTES + SF_BYTES));
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t tfull = bar0 + 8u * (2 * STAGES), tempty = tfull + 8, drain_bar = tfull + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 3);
  volatile int* abort_f = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* pref = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);
  int* offs = pref + (kMaxExperts + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.zero_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1 + kLoaders);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 8);
    mbar_init(drain_bar, 1);
    *abort_f = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // a copy of the offsets, kept inside [0, rows] whatever the caller's array holds
  for (int i = threadIdx.x; i <= p.E; i += kThreads) {
    const int64_t v = p.offsets ? (int64_t)__ldg(p.offsets + i) : (i ? p.rows : 0);
    offs[i] = (int)min(max(v, (int64_t)0), p.rows);
  }
  __syncthreads();
  if (warp == 2)
    build_expert_prefix(offs, p.E, [](int n) { return n > 0 ? (n + BM - 1) / BM : 0; }, pref, lane);
  if (threadIdx.x == 0) {
    tma_prefetch(&mapA);
    tma_prefetch(&mapB);
    if (GATEUP) tma_prefetch(&mapB2);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = pref[p.E] * p.NT;
  // tile t -> first row, end of the group's rows, first row of the expert's B, n-tile
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
    x.r0 = offs[x.e] + (g0 + q % gm) * BM;
    x.r1 = offs[x.e + 1];
    return x;
  };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, armed = 0;
      uint32_t phase = 0;
      bool stop = false;
      const uint64_t pol = policy_evict_normal();
      for (int t = blockIdx.x; t < total && !stop; t += gridDim.x) {
        const Tile x = tile_of(t);
        const int b_row = x.e * p.N + x.n * (GATEUP ? BN / 2 : BN);
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_f, p.status)) {
            stop = true;
            break;
          }
          const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + A_BYTES, fb = full_bar(stage);
          mbar_expect_tx(fb, STAGE_BYTES);
          tma_load_2d(sa, &mapA, fb, kb * 128, x.r0, pol);
          if (GATEUP) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tma_load_2d(sb + h * 128 * 128, &mapB, fb, kb * 128, b_row + h * 64, pol);
              tma_load_2d(sb + h * 128 * 128 + 64 * 128, &mapB2, fb, kb * 128, b_row + h * 64, pol);
            }
          } else {
            tma_load_2d(sb, &mapB, fb, kb * 128, b_row, pol);
          }
          ++armed;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (*abort_f) {  // let copies still in flight land
        for (int i = 0; i < min(armed, STAGES); ++i) {
          if (stage == 0) {
            stage = STAGES - 1;
            phase ^= 1u;
          } else {
            --stage;
          }
          wait_drain(full_bar(stage), phase);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc0 = make_idesc_mxf4(BM, BN, 0), idesc2 = make_idesc_mxf4(BM, BN, 2);
      int stage = 0;
      uint32_t phase = 0, tphase = 0;
      bool stop = false;
      for (int t = blockIdx.x; t < total && !stop; t += gridDim.x) {
        if (!wait_bounded(tempty, tphase ^ 1u, abort_f, p.status)) break;
        tphase ^= 1u;
        tc_fence_after();
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!wait_bounded(full_bar(stage), phase, abort_f, p.status)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + A_BYTES;
          const uint32_t sf = sf_base + stage * SF_BYTES;
          const uint64_t da = make_sdesc(sa), db = make_sdesc(sb);
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // 128 values: A chunk c, B chunks (c, half)
            const uint32_t ca = tmem + kScaleCol + c * 12, cb = ca + 4;
            tmem_cp_scale(ca, make_sdesc_scale(sf + c * kScaleChunk));
            tmem_cp_scale(cb, make_sdesc_scale(sf + (2 + 2 * c) * kScaleChunk));
            tmem_cp_scale(cb + 4, make_sdesc_scale(sf + (3 + 2 * c) * kScaleChunk));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
              umma_mxf4(tmem, da + 2u * (2 * c + kk), db + 2u * (2 * c + kk), kk ? idesc2 : idesc0,
                        ca, cb, (kb | c | kk) != 0);
          }
          umma_commit(empty_bar(stage));
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!stop) umma_commit(tfull);
      }
      umma_commit(drain_bar);  // arrives once every MMA issued above has completed
      wait_drain(drain_bar, 0);
    }
  } else if (warp < 4) {
    // scales: thread i takes A rows i, i + 64 and B rows i, i + 64, i + 128, i + 192 of the tile
    const int i0 = threadIdx.x - 64;
    int stage = 0, pending = 0, done = 0;
    uint32_t phase = 0;
    bool stop = false;
    auto arrive_oldest = [&]() {
      fence_proxy_async_smem();
      mbar_arrive(full_bar(done));
      if (++done == STAGES) done = 0;
      --pending;
    };
    const int words = (int)(p.scale_pitch / 4);
    for (int t = blockIdx.x; t < total && !stop; t += gridDim.x) {
      const Tile x = tile_of(t);
      const uint8_t* src[6];
      uint32_t dst[6];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = i0 + 64 * j;
        const int64_t row = min((int64_t)x.r0 + r, p.rows - 1);
        src[j] = p.a_scales + row * p.scale_pitch;
        dst[j] = scale_chunk_offset(r);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = i0 + 64 * j;  // j selects gate 0, up 0, gate 1, up 1 of the gate/up tile
        int n = GATEUP ? x.n * (BN / 2) + (j >> 1) * 64 + i0 : x.n * BN + r;
        n = min(n, p.N - 1);
        const uint8_t* b = GATEUP && (j & 1) ? p.b2_scales : p.b_scales;
        src[2 + j] = b + ((int64_t)x.e * p.N + n) * p.scale_pitch;
        dst[2 + j] = (2 + (r >> 7)) * kScaleChunk + scale_chunk_offset(r & 127);
      }
      for (int kb = 0; kb < p.KB; ++kb) {
        if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_f, p.status)) {
          stop = true;
          break;
        }
        const uint32_t sf = sf_base + stage * SF_BYTES;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // a row's last slice may have no second chunk: its codes are the zeros TMA fills in, and
          // any finite scale will do
          const int w = min(kb * 2 + c, words - 1);
#pragma unroll
          for (int j = 0; j < 6; ++j)
            cp_async4(sf + dst[j] + (j < 2 ? c : 2 * c) * kScaleChunk, src[j] + w * 4);
        }
        cp_async_commit();
        if (++pending > kLag) {
          cp_async_wait<kLag>();
          arrive_oldest();
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    cp_async_wait<0>();
    while (pending > 0) arrive_oldest();
  } else {
    const int q = warp & 3, h = (warp >> 2) - 1;  // lane quarter, column half
    uint32_t tphase = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
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
      if (lane == 0) mbar_arrive(tempty);
      const int row = x.r0 + q * 32 + lane;
      if (row < x.r1) {
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
              a[i] = blk * 32 + i < p.N ? g / (1.f + expf(-g)) * u : 0.f;
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
          const bool vec = ((uintptr_t)p.out & 15u) == 0 && (p.N * sizeof(T)) % 16 == 0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            store_row(orow, reinterpret_cast<const float*>(acc[c]), x.n * BN + h * 128 + c * 32,
                      p.N, vec);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

int sm_count(cudaError_t* err) {
  int dev = 0, sms = 0;
  *err = cudaGetDevice(&dev);
  if (*err == cudaSuccess) *err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <bool GATEUP, typename T>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& b2,
                   const Params& p, cudaStream_t s) {
  cudaError_t err;
  const int sms = sm_count(&err);
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(moe_mx4_gemm<GATEUP, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSmemBytes);
  if (err != cudaSuccess) return err;
  const int64_t upper = ((p.rows + BM - 1) / BM + p.E) * (int64_t)p.NT;  // >= number of tiles
  moe_mx4_gemm<GATEUP, T>
      <<<(unsigned)(upper < sms ? upper : sms), kThreads, kSmemBytes, s>>>(a, b, b2, p);
  return cudaGetLastError();
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
      !make_map_bytes(&mb, b.codes, pitch, (int64_t)E * N, BN))
    return cudaErrorInvalidValue;
  Params p = make_params(a, rows, offsets, E, N, K, BN, status);
  p.b_scales = b.scales;
  p.out = out;
  p.zero_status = zero_status;
  switch (odt) {
    case MOE_F32: return launch<false, float>(ma, mb, mb, p, s);
    case MOE_F16: return launch<false, __half>(ma, mb, mb, p, s);
    case MOE_BF16: return launch<false, __nv_bfloat16>(ma, mb, mb, p, s);
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
  p.codes = codes;
  p.scales = scales;
  return launch<true, float>(ma, mg, mu, p, s);
}

}  // namespace moe
