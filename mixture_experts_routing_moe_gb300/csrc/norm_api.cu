// C-ABI entry points of the residual norm (declared in include/moe_front.h): host-side validation.
#include <math.h>
#include <stdint.h>

#include "../../include/moe_front.h"
#include "mx_checks.h"
#include "norm.cuh"

using namespace moe;
using namespace moe::mx;

namespace {

bool ld_ok(int64_t ld, int64_t H) { return ld >= H && ld < ((int64_t)1 << 31); }
int check_rows(int dt, int wdt, int64_t T, int64_t H) {
  if (!dtype_size(dt) || (wdt != dt && wdt != MOE_F32)) return MOE_ERR_DTYPE;
  return T < 0 || T >= kMaxRows || !dim_ok(H) ? MOE_ERR_SHAPE : MOE_OK;
}

}  // namespace

extern "C" {

int moe_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                 int wdt, int dt, int64_t T, int64_t H, float eps, void* sum, int64_t lds, void* y,
                 int64_t ldy, uint8_t* codes, uint8_t* scales, float* rstd, moe_stream_t stream) {
  if (int st = check_rows(dt, wdt, T, H)) return st;
  if (!ld_ok(ldx, H) || (residual && !ld_ok(ldr, H)) || (sum && !ld_ok(lds, H)) ||
      (y && !ld_ok(ldy, H)))
    return MOE_ERR_SHAPE;
  if (!(eps >= 0.f) || !isfinite(eps)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !weight || (codes == nullptr) != (scales == nullptr)) return MOE_ERR_NULL;
  const unsigned es = dtype_size(dt);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(weight, dtype_size(wdt)) ||
      !aligned(sum, es) || !aligned(y, es) || !aligned(rstd, 4) || !aligned(codes, 16) ||
      !aligned(scales, 4))
    return MOE_ERR_ALIGN;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.w32 = wdt == MOE_F32;
  a.T = T;
  a.H = H;
  a.ldx = ldx;
  a.ldr = ldr;
  a.lds = lds;
  a.ldy = ldy;
  a.eps = eps;
  a.sum = sum;
  a.y = y;
  a.codes = codes;
  a.scales = scales;
  a.rstd = rstd;
  return cuda_status(launch_rms_norm(a, dt, (cudaStream_t)stream));
}

size_t moe_rms_norm_backward_workspace_bytes(int64_t T, int64_t H, int dt) {
  if (check_rows(dt, dt, T, H) != MOE_OK) return 0;
  return kWsHeader + align_up(rms_norm_backward_scratch_bytes(T, H), 256);
}

int moe_rms_norm_backward(const void* dy, int64_t lddy, const void* s, int64_t lds,
                          const void* weight, int wdt, const float* rstd, const void* dsum,
                          int64_t ldds, int dt, int64_t T, int64_t H, void* dx, int64_t lddx,
                          float* dweight, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (int st = check_rows(dt, wdt, T, H)) return st;
  if (!ld_ok(lddy, H) || !ld_ok(lds, H) || (dsum && !ld_ok(ldds, H)) || (dx && !ld_ok(lddx, H)))
    return MOE_ERR_SHAPE;
  cudaStream_t st = (cudaStream_t)stream;
  if (!aligned(dweight, 4)) return MOE_ERR_ALIGN;
  if (T == 0)  // no rows: the weight's gradient is zero
    return dweight ? cuda_status(cudaMemsetAsync(dweight, 0, (size_t)H * sizeof(float), st)) : MOE_OK;
  if (!dy || !s || !weight || !rstd) return MOE_ERR_NULL;
  const unsigned es = dtype_size(dt);
  if (!aligned(dy, es) || !aligned(s, es) || !aligned(weight, dtype_size(wdt)) ||
      !aligned(rstd, 4) || !aligned(dsum, es) || !aligned(dx, es))
    return MOE_ERR_ALIGN;
  if (dweight)
    if (int bad = check_ws(ws, ws_bytes, moe_rms_norm_backward_workspace_bytes(T, H, dt))) return bad;
  if (!dx && !dweight) return MOE_OK;
  NormGradArgs a{};
  a.dy = dy;
  a.s = s;
  a.weight = weight;
  a.w32 = wdt == MOE_F32;
  a.rstd = rstd;
  a.dsum = dsum;
  a.T = T;
  a.H = H;
  a.lddy = lddy;
  a.lds = lds;
  a.ldds = ldds;
  a.lddx = lddx;
  a.dx = dx;
  a.dweight = dweight;
  a.part_dw = dweight ? (float*)((uint8_t*)ws + kWsHeader) : nullptr;
  return cuda_status(launch_rms_norm_backward(a, dt, st));
}

}  // extern "C"
