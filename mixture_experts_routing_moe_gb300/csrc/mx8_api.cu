// C-ABI entry points of the microscaled 8-bit operators (declared in include/moe_mx8.h): host-side
// validation, workspace layout and the launch sequence.
#include <stdint.h>

#include "launch.h"
#include "mx8.cuh"
#include "mx_checks.h"

using namespace moe;
using namespace moe::mx8;
using namespace moe::mx;

namespace {

struct Cursor {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  }
};

struct ExpertsLayout {
  size_t ac, as, total;
};
ExpertsLayout experts_layout(int64_t rows, int64_t I) {
  ExpertsLayout l;
  Cursor c;
  c.take(kWsHeader);
  l.ac = c.take((size_t)rows * code_pitch(I));
  l.as = c.take((size_t)rows * scale_pitch(I));
  l.total = c.off;
  return l;
}

struct ForwardLayout {
  size_t ros, tor, offsets, hist, xc, xs, y, ac, as, total;
};
ForwardLayout forward_layout(int64_t T, int64_t E, int64_t H, int64_t I, int k, int odt) {
  const int64_t R = T * k;
  ForwardLayout l;
  Cursor c;
  c.take(kWsHeader);
  l.ros = c.take((size_t)R * 4);
  l.tor = c.take((size_t)R * 4);
  l.offsets = c.take((size_t)(E + 1) * 4);
  l.hist = c.take(dispatch_scratch_bytes(R, (int)E));
  // y takes the place of the dispatched rows, which the first product has read
  l.xc = l.y = c.off;
  c.take((size_t)R * code_pitch(H));
  l.xs = c.take((size_t)R * scale_pitch(H));
  const size_t y_end = l.y + align_up((size_t)R * H * dtype_size(odt), 256);
  if (c.off < y_end) c.off = y_end;
  l.ac = c.take((size_t)R * code_pitch(I));
  l.as = c.take((size_t)R * scale_pitch(I));
  l.total = c.off;
  return l;
}

int check_route_shape(int64_t T, int64_t E, int top_k) {
  if (T < 0 || E < 1 || E > kMaxE || top_k < 1 || top_k > E || T >= kMaxRows ||
      T * top_k >= kMaxRows)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_mx8_code_bytes(int64_t K) { return dim_ok(K) ? (size_t)code_pitch(K) : 0; }
size_t moe_mx8_scale_bytes(int64_t K) { return dim_ok(K) ? (size_t)scale_pitch(K) : 0; }

int moe_mx8_quantize(const void* x, int xdt, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                     uint8_t* scales, moe_stream_t stream) {
  if (!dtype_size(xdt)) return MOE_ERR_DTYPE;
  if (rows < 0 || rows >= kMaxRows || !dim_ok(K) || ldx < K || ldx >= ((int64_t)1 << 31))
    return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x) return MOE_ERR_NULL;
  if (int st = check_operand(codes, scales)) return st;
  if (!aligned(x, dtype_size(xdt))) return MOE_ERR_ALIGN;
  return cuda_status(
      launch_mx8_quantize(x, xdt, rows, K, ldx, codes, scales, (cudaStream_t)stream));
}

int moe_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                       void* out, int odt, int64_t ldo, moe_stream_t stream) {
  if (!dtype_size(odt)) return MOE_ERR_DTYPE;
  if (rows < 0 || rows >= kMaxRows || !dim_ok(K) || ldo < K || ldo >= ((int64_t)1 << 31))
    return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!out) return MOE_ERR_NULL;
  if (int st = check_operand(codes, scales)) return st;
  if (!aligned(out, dtype_size(odt))) return MOE_ERR_ALIGN;
  return cuda_status(
      launch_mx8_dequantize(codes, scales, rows, K, out, odt, ldo, (cudaStream_t)stream));
}

int moe_mx8_dispatch(const uint8_t* codes, const uint8_t* scales, int64_t T, int64_t H,
                     const uint32_t* idx, int64_t E, int top_k, uint8_t* x_codes,
                     uint8_t* x_scales, int32_t* offsets, uint32_t* token_of_row,
                     uint32_t* row_of_slot, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (int st = check_route_shape(T, E, top_k)) return st;
  if (!dim_ok(H)) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!idx || !offsets || !token_of_row || !row_of_slot) return MOE_ERR_NULL;
  if (int st = check_operand(codes, scales)) return st;
  if (int st = check_operand(x_codes, x_scales)) return st;
  if (!aligned(idx, 4) || !aligned(offsets, 4) || !aligned(token_of_row, 4) ||
      !aligned(row_of_slot, 4))
    return MOE_ERR_ALIGN;
  if (!ws || !aligned(ws, 16) || ws_bytes < moe_dispatch_workspace_bytes(T, E, top_k))
    return MOE_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t err = cudaMemsetAsync(ws, 0, sizeof(unsigned), s);
  if (err == cudaSuccess)
    err = launch_dispatch_map(T, idx, (int)E, top_k, offsets, token_of_row, row_of_slot,
                              (int32_t*)((uint8_t*)ws + kWsHeader), (unsigned*)ws, s);
  if (err == cudaSuccess)
    err = launch_dispatch_block_rows(codes, scales, T, code_pitch(H), scale_pitch(H), top_k,
                                     row_of_slot, x_codes, x_scales, s);
  return cuda_status(err);
}

size_t moe_mx8_product_workspace_bytes(void) { return kWsHeader; }

int moe_mx8_product(const uint8_t* a_codes, const uint8_t* a_scales, int64_t rows,
                    const uint8_t* b_codes, const uint8_t* b_scales, const int32_t* offsets,
                    int64_t E, int64_t N, int64_t K, void* out, int odt, void* ws,
                    size_t ws_bytes, moe_stream_t stream) {
  if (!dtype_size(odt)) return MOE_ERR_DTYPE;
  if (int st = check_product_shape(rows, E, N, K)) return st;
  if (!offsets && E != 1) return MOE_ERR_NULL;
  if (int st = check_operand(b_codes, b_scales)) return st;
  if (rows == 0) return MOE_OK;
  if (int st = check_operand(a_codes, a_scales)) return st;
  if (!out) return MOE_ERR_NULL;
  if (!aligned(out, dtype_size(odt)) || !aligned(offsets, 4)) return MOE_ERR_ALIGN;
  if (int st = check_ws(ws, ws_bytes, kWsHeader)) return st;
  return cuda_status(launch_mx8_product({a_codes, a_scales}, rows, {b_codes, b_scales}, offsets,
                                        (int)E, (int)N, (int)K, out, odt, (unsigned*)ws, true,
                                        (cudaStream_t)stream));
}

size_t moe_mx8_experts_workspace_bytes(int64_t rows, int64_t I) {
  if (rows < 0 || rows >= kMaxRows || !dim_ok(I)) return 0;
  return experts_layout(rows, I).total;
}

int moe_mx8_experts_forward_dispatched(const uint8_t* x_codes, const uint8_t* x_scales,
                                       const int32_t* offsets, int64_t rows,
                                       const uint8_t* gate_codes, const uint8_t* gate_scales,
                                       const uint8_t* up_codes, const uint8_t* up_scales,
                                       const uint8_t* down_codes, const uint8_t* down_scales,
                                       int64_t E, int64_t H, int64_t I, void* y, int odt, void* ws,
                                       size_t ws_bytes, moe_stream_t stream) {
  if (!dtype_size(odt)) return MOE_ERR_DTYPE;
  if (int st = check_product_shape(rows, E, I, H)) return st;
  if (int st = check_product_shape(rows, E, H, I)) return st;
  if (int st = check_operand(gate_codes, gate_scales)) return st;
  if (int st = check_operand(up_codes, up_scales)) return st;
  if (int st = check_operand(down_codes, down_scales)) return st;
  if (!offsets) return MOE_ERR_NULL;
  if (rows == 0) return MOE_OK;
  if (int st = check_operand(x_codes, x_scales)) return st;
  if (!y) return MOE_ERR_NULL;
  if (!aligned(y, dtype_size(odt)) || !aligned(offsets, 4)) return MOE_ERR_ALIGN;
  const ExpertsLayout l = experts_layout(rows, I);
  if (int st = check_ws(ws, ws_bytes, l.total)) return st;
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t* b = (uint8_t*)ws;
  cudaError_t err = launch_mx8_gate_up({x_codes, x_scales}, rows, {gate_codes, gate_scales},
                                       {up_codes, up_scales}, offsets, (int)E, (int)I, (int)H,
                                       b + l.ac, b + l.as, (unsigned*)ws, true, s);
  if (err == cudaSuccess)
    err = launch_mx8_product({b + l.ac, b + l.as}, rows, {down_codes, down_scales}, offsets, (int)E,
                             (int)H, (int)I, y, odt, (unsigned*)ws, false, s);
  return cuda_status(err);
}

size_t moe_mx8_forward_workspace_bytes(int64_t T, int64_t E, int64_t H, int64_t I, int top_k,
                                       int odt) {
  if (!dtype_size(odt) || check_route_shape(T, E, top_k) != MOE_OK ||
      check_product_shape(T * top_k, E, I, H) != MOE_OK ||
      check_product_shape(T * top_k, E, H, I) != MOE_OK)
    return 0;
  return forward_layout(T, E, H, I, top_k, odt).total;
}

int moe_mx8_forward(const uint8_t* x_codes, const uint8_t* x_scales, const uint32_t* idx,
                    const void* w, int wdt, const uint8_t* gate_codes, const uint8_t* gate_scales,
                    const uint8_t* up_codes, const uint8_t* up_scales, const uint8_t* down_codes,
                    const uint8_t* down_scales, int64_t T, int64_t E, int64_t H, int64_t I,
                    int top_k, void* out, int odt, void* ws, size_t ws_bytes,
                    moe_stream_t stream) {
  if (!dtype_size(odt) || !dtype_size(wdt)) return MOE_ERR_DTYPE;
  if (int st = check_route_shape(T, E, top_k)) return st;
  const int64_t R = T * top_k;
  if (int st = check_product_shape(R, E, I, H)) return st;
  if (int st = check_product_shape(R, E, H, I)) return st;
  if (int st = check_operand(gate_codes, gate_scales)) return st;
  if (int st = check_operand(up_codes, up_scales)) return st;
  if (int st = check_operand(down_codes, down_scales)) return st;
  if (T == 0) return MOE_OK;
  if (int st = check_operand(x_codes, x_scales)) return st;
  if (!idx || !w || !out) return MOE_ERR_NULL;
  if (!aligned(idx, 4) || !aligned(w, dtype_size(wdt)) || !aligned(out, dtype_size(odt)))
    return MOE_ERR_ALIGN;
  const ForwardLayout l = forward_layout(T, E, H, I, top_k, odt);
  if (int st = check_ws(ws, ws_bytes, l.total)) return st;
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t* b = (uint8_t*)ws;
  unsigned* status = (unsigned*)ws;
  int32_t* offsets = (int32_t*)(b + l.offsets);
  uint32_t* ros = (uint32_t*)(b + l.ros);
  cudaError_t err;
  if (R <= kFewSlots) {
    err = launch_dispatch_few_blocks(x_codes, x_scales, T, code_pitch(H), scale_pitch(H), idx, (int)E,
                                     top_k, offsets, ros, b + l.xc, b + l.xs, status, s);
  } else {
    err = cudaMemsetAsync(status, 0, sizeof(unsigned), s);
    if (err == cudaSuccess)
      err = launch_dispatch_map(T, idx, (int)E, top_k, offsets, (uint32_t*)(b + l.tor), ros,
                                (int32_t*)(b + l.hist), status, s);
    if (err == cudaSuccess)
      err = launch_dispatch_block_rows(x_codes, x_scales, T, code_pitch(H), scale_pitch(H), top_k, ros,
                                       b + l.xc, b + l.xs, s);
  }
  if (err == cudaSuccess)
    err = launch_mx8_gate_up({b + l.xc, b + l.xs}, R, {gate_codes, gate_scales},
                             {up_codes, up_scales}, offsets, (int)E, (int)I, (int)H, b + l.ac,
                             b + l.as, status, false, s);
  if (err == cudaSuccess)
    err = launch_mx8_product({b + l.ac, b + l.as}, R, {down_codes, down_scales}, offsets, (int)E,
                             (int)H, (int)I, b + l.y, odt, status, false, s);
  if (err == cudaSuccess)
    err = launch_combine(b + l.y, odt, ros, w, wdt, T, H, top_k, out, s);
  return cuda_status(err);
}

}  // extern "C"
