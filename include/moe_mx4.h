/*
 * moe_mx4.h — C ABI of libmoe's microscaled 4-bit (MXFP4) operators: quantisation, grouped
 * product, SwiGLU experts, and a whole MoE layer for a few tokens.
 *
 * The ruDNN pages require unquantised router logits and weights (docs/de/README.md §4); these
 * entry points stand beside the layer of moe.h for callers whose expert weights are held in 4
 * bits.  The conventions of moe.h hold here too: device pointers owned by the caller, work
 * enqueued on `stream`, every argument checked on the host before anything is enqueued, the
 * status codes of moe.h, no allocation and no synchronisation, one workspace for one call in
 * flight, the device status word in its first 256 bytes (moe_device_status()).
 *
 * The format (OCP Microscaling Formats, MXFP4).  A row of K values is cut into ceil(K / 32)
 * blocks of 32.  A block is
 *   codes   16 bytes of e2m1 codes, two a byte, the even position in the low nibble; code
 *           s x1 x0 m stands for (-1)^s { 0, 0.5, 1, 1.5, 2, 3, 4, 6 };
 *   scale   one byte b standing for 2^(b - 127); 255 makes every value of the block a NaN.
 * codes  [rows, 16 ceil(K / 32)] uint8, 16-byte aligned; a last short block is filled with
 *        zero codes.
 * scales [rows, 4 ceil(K / 128)] uint8, 4-byte aligned; the bytes past the last block are 0.
 * Limits (MOE_ERR_SHAPE past them): K, N, H, I >= 1 and below 2^24; 1 <= E <= 1024; row strides
 * below 2^31 elements; rows, and the weight rows E N, E H, E I, below 2^31 - 1024; for the products,
 * (ceil(rows / 128) + E) ceil(N / 128) below 2^31 - 1024 (N: H and I for the experts).
 */
#ifndef MOE_MX4_H_
#define MOE_MX4_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one row of codes / scales of K values (0 for K < 1). */
size_t moe_mx4_code_bytes(int64_t K);
size_t moe_mx4_scale_bytes(int64_t K);

/*
 * moe_mx4_quantize — rows of x to blocks.
 * Scale: floor(log2(max |x|)) - 2 clamped to [-127, 127], so the largest magnitude lands in
 * [4, 8); a block of zeros gets byte 0.  Each x 2^-scale goes to the nearest code, ties to the
 * even one, magnitudes above 6 to 6; signs (of zeros too) are kept.  A block holding an infinity
 * or a NaN gets scale byte 255 and zero codes.
 * x [rows, K] of dtype xdt (f32 / f16 / bf16), row r at x + r * ldx elements, ldx >= K.
 * Alignment: none for x (16-byte aligned rows take a vectorised path).
 */
int moe_mx4_quantize(const void* x, int xdt, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                     uint8_t* scales, moe_stream_t stream);

/*
 * moe_mx4_dequantize — the values the blocks stand for, rounded once to odt.
 * out [rows, K], row r at out + r * ldo elements, ldo >= K; elements between rows are not written.
 */
int moe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                       void* out, int odt, int64_t ldo, moe_stream_t stream);

/*
 * moe_mx4_product — out[r, n] = sum_k A[r, k] B[e, n, k] for the rows r of group e.
 * A: a_codes / a_scales, [rows] rows of K values.  B: b_codes / b_scales, [E, N] rows of K.
 * offsets [E + 1] int32 on the device (non-decreasing, offsets[0] = 0, offsets[E] <= rows): rows
 * offsets[e] .. offsets[e+1]-1 are group e; rows past offsets[E] are not written.  NULL with
 * E = 1: every row.  FP32 accumulation, rounded once to odt; out [rows, N].
 * A NaN block makes the results that read it NaN.
 * ws: at least moe_mx4_product_workspace_bytes() bytes, 256-byte aligned.
 */
size_t moe_mx4_product_workspace_bytes(void);
int moe_mx4_product(const uint8_t* a_codes, const uint8_t* a_scales, int64_t rows,
                    const uint8_t* b_codes, const uint8_t* b_scales, const int32_t* offsets,
                    int64_t E, int64_t N, int64_t K, void* out, int odt, void* ws,
                    size_t ws_bytes, moe_stream_t stream);

/*
 * moe_mx4_experts_forward_dispatched — moe_experts_forward_dispatched with weights and
 * activations in blocks.  With Q the trip of moe_mx4_quantize over rows of H or I values:
 *   g = Q(x_d[r]) gate[e]^T,  u = Q(x_d[r]) up[e]^T,  a = Q(silu(g) u),  y[r] = a down[e]^T
 * g, u and silu(g) u are FP32 (not rounded before they are quantised), y is rounded once to xdt.
 * x_d, y [rows, H] of dtype xdt, contiguous; gate, up [E, I] rows of H values, down [E, H] rows
 * of I values; offsets as above, not NULL.
 * ws: at least moe_mx4_experts_workspace_bytes(rows, H, I) bytes, 256-byte aligned.
 */
size_t moe_mx4_experts_workspace_bytes(int64_t rows, int64_t H, int64_t I);
int moe_mx4_experts_forward_dispatched(const void* x_d, int xdt, const int32_t* offsets,
                                       int64_t rows, const uint8_t* gate_codes,
                                       const uint8_t* gate_scales, const uint8_t* up_codes,
                                       const uint8_t* up_scales, const uint8_t* down_codes,
                                       const uint8_t* down_scales, int64_t E, int64_t H, int64_t I,
                                       void* y, void* ws, size_t ws_bytes, moe_stream_t stream);

/*
 * moe_mx4_forward_tokens — a whole layer for a few tokens: router, top-k, experts, combine.
 *   logits = x router^T (FP32), idx and weights as moe_route selects them (softmax over all E,
 *   ties to the lower id, renormalize as there) with FP32 weights,
 *   a = silu(x gate[e]^T) (x up[e]^T) in FP32, rounded once to dt,
 *   out[t] = sum_j w[t, j] (a_j down[e_j]^T), FP32 in the order j = 0 .. top_k-1, rounded once.
 * x [T, H], router [E, H] and out [T, H] of dtype dt (f16 / bf16), weights as for the experts
 * above.  The activations are not quantised: they enter the products to within 2^-23 of the
 * largest value of their block of 32 (2^-128 where that is smaller), which is what one rounding of an
 * FP32 sum that holds it costs; bf16 values down to 2^-15 of the largest are exact, f16 values down
 * to 2^-12.  A token holding an infinity or a NaN gets NaN.
 * idx [T, top_k] uint32 and w [T, top_k] float receive the selection; either may be NULL.
 * Two launches, the second a cooperative one; if its CTAs cannot all be resident (another context
 * holds SMs) the call returns MOE_ERR_CUDA.
 * Limits: T <= 64, top_k <= min(E, 32), T * top_k <= 1024 (else MOE_ERR_SHAPE); H and I multiples
 * of 128, x and router 16-byte aligned (else MOE_ERR_ALIGN).
 * ws: at least moe_mx4_tokens_workspace_bytes(...) bytes (0 for sizes out of range), 256-byte
 * aligned.
 */
size_t moe_mx4_tokens_workspace_bytes(int64_t T, int64_t E, int64_t H, int64_t I, int top_k,
                                      int dt);
int moe_mx4_forward_tokens(const void* x, const void* router, int dt, const uint8_t* gate_codes,
                           const uint8_t* gate_scales, const uint8_t* up_codes,
                           const uint8_t* up_scales, const uint8_t* down_codes,
                           const uint8_t* down_scales, int64_t T, int64_t E, int64_t H, int64_t I,
                           int top_k, int renormalize, void* out, uint32_t* idx, float* w,
                           void* ws, size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_MX4_H_ */
