/*
 * moe_front.h — C ABI of what stands in front of libmoe's experts: the residual stream's norm, with
 * its result in 16 or 32 bits (for the router and the experts of moe.h) and in 8-bit blocks (for
 * those of moe_mx8.h), its gradient, and group-limited softmax routing.
 *
 * The conventions of moe.h hold here too: device pointers owned by the caller, work enqueued on
 * `stream`, every argument checked on the host before anything is enqueued, the status codes of
 * moe.h, no allocation and no synchronisation.
 */
#ifndef MOE_FRONT_H_
#define MOE_FRONT_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_rms_norm — s = x + residual (rounded to dt), y = s (mean(s^2) + eps)^(-1/2) weight.
 * x, residual (NULL: none, s = x) [T, H] of dtype dt, row t at t * ldx / ldr elements; weight [H] of
 * dtype wdt: dt or MOE_F32.  Outputs, each of which may be NULL:
 *   sum [T, H] of dt, row t at t * lds: s;
 *   y [T, H] of dt, row t at t * ldy: rounded once from FP32;
 *   codes, scales: y in the blocks of moe_mx8_quantize, taken from the FP32 values (both or none);
 *   rstd [T] float: (mean(s^2) + eps)^(-1/2), for moe_rms_norm_backward.
 * The mean is FP32: squares past its range give rstd 0.  Rows whose squares are below it are normalised
 * like others (with an rstd of infinity where it is past FP32's range: root mean squares below 2^-128).
 * A NaN or an infinity stays in its row.  Weights are numbers: an infinite one makes its column of y
 * infinite or NaN, and its blocks 255.
 * sum may be x or residual itself, y may be x, with the same row stride; other overlaps are not
 * allowed.
 * Limits: 0 <= T < 2^31 - 1024, 1 <= H < 2^24, H <= ld < 2^31 (else MOE_ERR_SHAPE); eps finite and
 * >= 0 (else MOE_ERR_ARG).  Alignment: 16 bytes for codes and 4 for scales (else MOE_ERR_ALIGN); none
 * for the rest (16-byte aligned rows take a vectorised path).
 */
int moe_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                 int wdt, int dt, int64_t T, int64_t H, float eps, void* sum, int64_t lds, void* y,
                 int64_t ldy, uint8_t* codes, uint8_t* scales, float* rstd, moe_stream_t stream);

/*
 * moe_rms_norm_backward — the gradient of y, and of s along the residual stream, back to s (which is
 * that of x and of the residual alike) and to the weight.  With n = s rstd:
 *   dx = dsum + rstd (dy weight - n mean(dy weight n)),  dweight = sum over rows of dy n
 * dy, s (the sum of the forward, or its x without a residual), dsum (NULL: none) [T, H] of dt with
 * row strides; rstd [T] of the forward.  dx [T, H] of dt, rounded once, and dweight [H] FP32; either
 * may be NULL.  dx may be dy or dsum itself, with the same row stride.  dweight is summed in a fixed
 * order: it repeats bit for bit.
 * ws: at least moe_rms_norm_backward_workspace_bytes(T, H, dt) bytes, 256-byte aligned (with
 * dweight only).
 */
size_t moe_rms_norm_backward_workspace_bytes(int64_t T, int64_t H, int dt);
int moe_rms_norm_backward(const void* dy, int64_t lddy, const void* s, int64_t lds,
                          const void* weight, int wdt, const float* rstd, const void* dsum,
                          int64_t ldds, int dt, int64_t T, int64_t H, void* dx, int64_t lddx,
                          float* dweight, void* ws, size_t ws_bytes, moe_stream_t stream);

/*
 * moe_route_softmax_grouped — as moe_route_sigmoid_grouped, with softmax scores: p = softmax(logits)
 * over all E experts, c = p + bias[e] (bias: FP32 [E], or NULL for none; it changes the selection
 * only).  A group scores its largest c, or with group_top_two != 0 the sum of its two largest;
 * the `selected_groups` best groups are kept (ties: lower group id), then the top_k experts inside
 * them by c (ties: lower id), listed in that order.  w = p of the chosen experts, divided by their
 * sum if renormalize != 0, times `scale`, rounded to `ldt`.
 * The selection is decided in float64; without a bias experts (and groups by their largest) are ranked
 * by their logits, which is the ranking of the exact softmax.  A bias of -inf leaves an expert out
 * as long as others are left.  Rows holding a NaN, a +inf or only -inf logits, and all rows with a NaN
 * bias, get NaN weights and ids 0..k-1.
 * Limits, types and alignment: those of moe_route_sigmoid_grouped.  The gradient of the weights is
 * moe_selected_router_backward's, with MOE_SCORE_SOFTMAX.
 */
int moe_route_softmax_grouped(const void* logits, int ldt, const float* bias, int64_t T, int64_t E,
                              int top_k, int groups, int selected_groups, int group_top_two,
                              int renormalize, float scale, uint32_t* idx, void* w,
                              moe_stream_t stream);

/*
 * moe_forward_softmax_grouped — moe_forward_sigmoid_grouped with the router above, as staged launches
 * for batches of every size.  Workspace: moe_forward_workspace_bytes(T, E, H, I, top_k, ldt, wdt).
 */
int moe_forward_softmax_grouped(const void* x, const void* logits, int ldt, const float* bias,
                                const void* gate, const void* up, const void* down, int wdt,
                                int64_t T, int64_t E, int64_t H, int64_t I, int top_k, int groups,
                                int selected_groups, int group_top_two, int renormalize,
                                float scale, void* out, void* ws, size_t ws_bytes,
                                moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_FRONT_H_ */
