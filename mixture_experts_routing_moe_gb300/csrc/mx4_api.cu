// C-ABI entry points of the microscaled 4-bit operators (declared in include/moe_mx4.h): host-side
// validation, workspace layout and the launch sequence.
#include <stdint.h>

#include "launch.h"
#include "mx4.cuh"

using namespace moe;
using namespace moe::mx4;

namespace {

constexpr int kMaxE = 1024;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1024;  // a tile past the last row stays an int
constexpr int64_t kMaxDim = (int64_t)1 << 24;

int dtype_size(int dt) { return dt == MOE_F32 ? 4 : (dt == MOE_F16 || dt == MOE_BF16) ? 2 : 0; }
bool aligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool dim_ok(int64_t v) { return v >= 1 && v < kMaxDim; }

// rows x [N or I] products: row and tile numbers are 32-bit ints in the kernels
int check_product_shape(int64_t rows, int64_t E, int64_t N, int64_t K) {
  if (rows < 0 || rows >= kMaxRows || E < 1 || E > kMaxE || !dim_ok(N) || !dim_ok(K))
    return MOE_ERR_SHAPE;
  if (E * N >= kMaxRows) return MOE_ERR_SHAPE;
  if (((rows + 127) / 128 + E) * ((N + 127) / 128) >= kMaxRows) return MOE_ERR_SHAPE;
  return MOE_OK;
}
// The alignment of one operand in blocks; null pointers are MOE_ERR_NULL.
int check_operand(const uint8_t* codes, const uint8_t* scales) {
  if (!codes || !scales) return MOE_ERR_NULL;
  return aligned(codes, 16) && aligned(scales, 4) ? MOE_OK : MOE_ERR_ALIGN;
}
int check_ws(const void* ws, size_t have, size_t need) {
  return ws && aligned(ws, 256) && have >= need ? MOE_OK : MOE_ERR_WORKSPACE;
}

struct ExpertsLayout {
  size_t xc, xs, ac, as, total;
};
ExpertsLayout experts_layout(int64_t rows, int64_t H, int64_t I) {
  ExpertsLayout l;
  size_t off = kWsHeader;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  l.xc = take((size_t)rows * code_pitch(H));
  l.xs = take((size_t)rows * scale_pitch(H));
  l.ac = take((size_t)rows * code_pitch(I));
  l.as = take((size_t)rows * scale_pitch(I));
  l.total = off;
  return l;
}

int check_tokens_shape(int64_t T, int64_t E, int64_t H, int64_t I, int k, int dt) {
  if (dt != MOE_F16 && dt != MOE_BF16) return MOE_ERR_DTYPE;
  if (T < 0 || T > kMx4TokensMaxT || E < 1 || E > kMaxE || k < 1 || k > E || k > kMx4TokensMaxK ||
      T * k > kMx4TokensMaxSlots || !dim_ok(H) || !dim_ok(I) || E * H >= kMaxRows ||
      E * I >= kMaxRows)
    return MOE_ERR_SHAPE;
  return H % 128 || I % 128 ? MOE_ERR_ALIGN : MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_mx4_code_bytes(int64_t K) { return dim_ok(K) ? (size_t)code_pitch(K) : 0; }
size_t moe_mx4_scale_bytes(int64_t K) { return dim_ok(K) ? (size_t)scale_pitch(K) : 0; }

int moe_mx4_quantize(const void* x, int xdt, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                     uint8_t* scales, moe_stream_t stream) {
  if (!dtype_size(xdt)) return MOE_ERR_DTYPE;
  if (rows < 0 || rows >= kMaxRows || !dim_ok(K) || ldx < K || ldx >= ((int64_t)1 << 31))
    return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x) return MOE_ERR_NULL;
  if (int st = check_operand(codes, scales)) return st;
  if (!aligned(x, dtype_size(xdt))) return MOE_ERR_ALIGN;
  return cuda_status(launch_mx4_quantize(x, xdt, rows, K, ldx, codes, scales, nullptr,
                                         (cudaStream_t)stream));
}

int moe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                       void* out, int odt, int64_t ldo, moe_stream_t stream) {
  if (!dtype_size(odt)) return MOE_ERR_DTYPE;
  if (rows < 0 || rows >= kMaxRows || !dim_ok(K) || ldo < K || ldo >= ((int64_t)1 << 31))
    return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!out) return MOE_ERR_NULL;
  if (int st = check_operand(codes, scales)) return st;
  if (!aligned(out, dtype_size(odt))) return MOE_ERR_ALIGN;
  return cuda_status(
      launch_mx4_dequantize(codes, scales, rows, K, out, odt, ldo, (cudaStream_t)stream));
}

size_t moe_mx4_product_workspace_bytes(void) { return kWsHeader; }

int moe_mx4_product(const uint8_t* a_codes, const uint8_t* a_scales, int64_t rows,
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
  return cuda_status(launch_mx4_product({a_codes, a_scales}, rows, {b_codes, b_scales}, offsets,
                                        (int)E, (int)N, (int)K, out, odt, (unsigned*)ws, true,
                                        (cudaStream_t)stream));
}

size_t moe_mx4_experts_workspace_bytes(int64_t rows, int64_t H, int64_t I) {
  if (rows < 0 || rows >= kMaxRows || !dim_ok(H) || !dim_ok(I)) return 0;
  return experts_layout(rows, H, I).total;
}

int moe_mx4_experts_forward_dispatched(const void* x_d, int xdt, const int32_t* offsets,
                                       int64_t rows, const uint8_t* gate_codes,
                                       const uint8_t* gate_scales, const uint8_t* up_codes,
                                       const uint8_t* up_scales, const uint8_t* down_codes,
                                       const uint8_t* down_scales, int64_t E, int64_t H, int64_t I,
                                       void* y, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!dtype_size(xdt)) return MOE_ERR_DTYPE;
  if (int st = check_product_shape(rows, E, I, H)) return st;
  if (int st = check_product_shape(rows, E, H, I)) return st;
  if (int st = check_operand(gate_codes, gate_scales)) return st;
  if (int st = check_operand(up_codes, up_scales)) return st;
  if (int st = check_operand(down_codes, down_scales)) return st;
  if (!offsets) return MOE_ERR_NULL;
  if (rows == 0) return MOE_OK;
  if (!x_d || !y) return MOE_ERR_NULL;
  if (!aligned(x_d, dtype_size(xdt)) || !aligned(y, dtype_size(xdt)) || !aligned(offsets, 4))
    return MOE_ERR_ALIGN;
  const ExpertsLayout l = experts_layout(rows, H, I);
  if (int st = check_ws(ws, ws_bytes, l.total)) return st;
  cudaStream_t s = (cudaStream_t)stream;
  unsigned* status = (unsigned*)ws;
  uint8_t* b = (uint8_t*)ws;
  cudaError_t err =
      launch_mx4_quantize(x_d, xdt, rows, H, H, b + l.xc, b + l.xs, status, s);
  if (err == cudaSuccess)
    err = launch_mx4_gate_up({b + l.xc, b + l.xs}, rows, {gate_codes, gate_scales},
                             {up_codes, up_scales}, offsets, (int)E, (int)I, (int)H, b + l.ac,
                             b + l.as, status, s);
  if (err == cudaSuccess)
    err = launch_mx4_product({b + l.ac, b + l.as}, rows, {down_codes, down_scales}, offsets, (int)E,
                             (int)H, (int)I, y, xdt, status, false, s);
  return cuda_status(err);
}

size_t moe_mx4_tokens_workspace_bytes(int64_t T, int64_t E, int64_t H, int64_t I, int top_k,
                                      int dt) {
  if (check_tokens_shape(T, E, H, I, top_k, dt) != MOE_OK) return 0;
  return mx4_tokens_layout(T, E, H, I, top_k).total;
}

int moe_mx4_forward_tokens(const void* x, const void* router, int dt, const uint8_t* gate_codes,
                           const uint8_t* gate_scales, const uint8_t* up_codes,
                           const uint8_t* up_scales, const uint8_t* down_codes,
                           const uint8_t* down_scales, int64_t T, int64_t E, int64_t H, int64_t I,
                           int top_k, int renormalize, void* out, uint32_t* idx, float* w,
                           void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (int st = check_tokens_shape(T, E, H, I, top_k, dt)) return st;
  if (int st = check_operand(gate_codes, gate_scales)) return st;
  if (int st = check_operand(up_codes, up_scales)) return st;
  if (int st = check_operand(down_codes, down_scales)) return st;
  if (!router) return MOE_ERR_NULL;
  if (T == 0) return MOE_OK;
  if (!x || !out) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(router, 16) || !aligned(out, 2) || !aligned(idx, 4) ||
      !aligned(w, 4))
    return MOE_ERR_ALIGN;
  if (int st = check_ws(ws, ws_bytes, mx4_tokens_layout(T, E, H, I, top_k).total)) return st;
  Mx4TokensArgs a{};
  a.x = x;
  a.router = router;
  a.dt = dt;
  a.T = (int)T;
  a.E = (int)E;
  a.H = (int)H;
  a.I = (int)I;
  a.k = top_k;
  a.renorm = renormalize != 0;
  a.gate = {gate_codes, gate_scales};
  a.up = {up_codes, up_scales};
  a.down = {down_codes, down_scales};
  a.out = out;
  a.idx = idx;
  a.w = w;
  a.ws = (uint8_t*)ws;
  return cuda_status(launch_mx4_tokens(a, (cudaStream_t)stream));
}

}  // extern "C"
