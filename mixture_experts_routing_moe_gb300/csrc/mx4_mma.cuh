// Inline-PTX wrappers of the block-scaled tensor instructions the microscaled kernels use, beside
// those of tcgen05.cuh.
//
// tcgen05.mma kind::mxf4 multiplies packed e2m1 operands (128-byte swizzled K-major tiles, 256
// values a 128-byte row; one instruction takes K = 64, 32 bytes of a row) with one power-of-two
// scale for each 32 values of each row, read from tensor memory.  Scales of 128 rows and four
// blocks (128 values) are one 512-byte chunk in shared memory, the four bytes of row r at
// (r % 32) * 16 + (r / 32) * 4; tcgen05.cp 32x128b.warpx4 spreads it over four 32-bit columns
// (column j: rows 32 j .. 32 j + 31, repeated in each 32-lane quarter).  Each K = 64 step uses two
// of the four bytes, named by the scale ids of the instruction descriptor (0 or 2).
// kind::mxf8f6f4 does the same for e4m3 operands: 128 values a 128-byte row, K = 32 an instruction, one
// of the four bytes (0 to 3).
#pragma once

#include "tcgen05.cuh"

namespace moe {
namespace tc {

// One lane of a converged warp.  Roles that issue tensor or TMA instructions run their loops with
// the whole warp and predicate the instructions on this: descriptors and addresses then stay in
// uniform registers, where a loop of one lane has to move each of them there.
static __device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

constexpr int kScaleChunk = 512;  // bytes: 128 rows x 4 blocks

// Byte offset in a chunk of row r's four scales.
static __device__ __forceinline__ uint32_t scale_chunk_offset(int r) {
  return (uint32_t)((r & 31) * 16 + (r >> 5) * 4);
}
// Shared-memory descriptor of a scale chunk: no swizzle, 8-row groups of 16-byte rows 128 bytes
// apart.
static __device__ __forceinline__ uint64_t make_sdesc_scale(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
static __device__ __forceinline__ void tmem_cp_scale(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
// Instruction descriptor of kind::mxf4: e2m1 (1) x e2m1 (1), both K-major, scales ue8m0; N >> 3 at
// bit 17, M >> 7 at bit 27, scale ids of B at bit 4 and of A at bit 29.
static __host__ __device__ constexpr uint32_t make_idesc_mxf4(int M, int N, int sf_id) {
  return ((uint32_t)sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         (1u << 23) | ((uint32_t)(M >> 7) << 27) | ((uint32_t)sf_id << 29);
}
static __device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                 uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// kind::mxf8f6f4 with e4m3 (0) operands of a byte a value: one instruction takes K = 32, again 32
// bytes of a row, and one of the four scale bytes, named by the scale id (0 to 3).
static __host__ __device__ constexpr uint32_t make_idesc_mxf8(int M, int N, int sf_id) {
  return ((uint32_t)sf_id << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 7) << 27) | ((uint32_t)sf_id << 29);
}
static __device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                 uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// The same instructions for a CTA pair, issued by CTA 0: the copy moves each CTA's chunk into
// that CTA's tensor memory, and the MMA reads both CTAs' operands at the same offsets.
static __device__ __forceinline__ void tmem_cp_scale2(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
static __device__ __forceinline__ void umma2_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                  uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
static __device__ __forceinline__ void umma2_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                  uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Waits for a phase, or until clock64() reaches `until` (after an abort, while copies land).
static __device__ __forceinline__ void wait_until(uint32_t bar, uint32_t parity, long long until) {
  while (!mbar_try_wait(bar, parity) && clock64() < until) {
  }
}

// After an abort, before the CTA's shared memory may go to another: copies that no wait saw land had
// 2^24 cycles (8 ms) to do so.
static __device__ __forceinline__ void settle_after_abort(volatile int* abort_f) {
  if (!*abort_f) return;
  const long long until = clock64() + (1 << 24);
  while (clock64() < until) __nanosleep(1000);
}

// Register budget of the calling warpgroup (every warp of it executes this).
template <int N>
static __device__ __forceinline__ void set_max_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
static __device__ __forceinline__ void set_max_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

static __device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Scale bytes on their way from global memory to the chunk layout wait as raw rows of 32 bytes, 16-
// byte half h of row i at i * 32 + 16 (h ^ (i / 4 % 2)), so that eight lanes read eight rows' halves
// without bank conflicts.  One warp copies them in, asynchronously, and another one writes the
// chunks: the fence between the proxies that follows each chunk waits for the issuing warp's own
// global accesses, so a warp that did both would wait for its next rows at every slice.
static __device__ __forceinline__ uint32_t raw_offset(int row, int half) {
  return (uint32_t)(row * 32 + ((half ^ (row >> 2 & 1)) * 16));
}
// Sixteen bytes past L1; zeros where `in` is false (nothing is read then).  (Four bytes can only be
// copied through L1, which may hold a line from before it was written elsewhere.)
static __device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
// One arrival on `bar` once this thread's copies so far have landed.
static __device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
static __device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
// Arrival on a barrier of another CTA of the cluster that releases this thread's (and, by
// cumulativity, its warp's) shared-memory writes only: a full release at cluster scope also waits
// for the warp's global accesses in flight.
static __device__ __forceinline__ void mbar_arrive_cluster_shared(uint32_t cluster_addr) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
      : "memory");
}
// Wait of wait_bounded() for a phase that threads of the other CTA complete too (acquire at
// cluster scope).
static __device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
static __device__ __forceinline__ bool wait_bounded_cluster(uint32_t bar, uint32_t parity,
                                                            volatile int* abort_f,
                                                            unsigned* status) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (*abort_f) return false;
    if (clock64() - t0 > kWaitLimit) {
      *abort_f = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

// 2-D map over a row-major byte matrix [rows, pitch], box 128 bytes x box_rows, 128-byte swizzle;
// bytes past the end read as zero.  pitch is a multiple of 16.
static inline bool make_map_bytes(CUtensorMap* m, const void* ptr, int64_t pitch, int64_t rows,
                                  int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)pitch};
  cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  auto encode = [&]() {
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {  // the thread's first call of CUDA: none is current yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
    r = encode();
  }
  return r == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace moe
