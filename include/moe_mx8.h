/*
 * moe_mx8.h — C ABI of libmoe's microscaled 8-bit (MXFP8) operators: quantisation, dispatch of rows
 * in blocks, grouped product, SwiGLU experts, and the layer from routed tokens on.
 *
 * They stand beside the 4-bit operators of moe_mx4.h, for weights and activations that 4 bits would
 * cost too much, with the same conventions (those of moe.h): device pointers owned by the caller,
 * work enqueued on `stream`, every argument checked on the host before anything is enqueued, the
 * status codes of moe.h, no allocation and no synchronisation, one workspace for one call in
 * flight, the device status word in its first 256 bytes (moe_device_status()).
 *
 * The format (OCP Microscaling Formats, MXFP8 with e4m3 elements).  A row of K values is cut into
 * ceil(K / 32) blocks of 32.  A block is
 *   codes   32 bytes of e4m3 codes (sign, 4 bits of exponent with bias 7, 3 bits behind the first;
 *           0x7F and 0xFF are NaN, the largest magnitude is 448);
 *   scale   one byte b standing for 2^(b - 127); 255 makes every value of the block a NaN.
 * codes  [rows, 32 ceil(K / 32)] uint8, 16-byte aligned; a last short block is filled with
 *        zero codes.
 * scales [rows, 4 ceil(K / 128)] uint8, 4-byte aligned; the bytes past the last block are 0.
 * Limits (MOE_ERR_SHAPE past them): those of moe_mx4.h.
 */
#ifndef MOE_MX8_H_
#define MOE_MX8_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one row of codes / scales of K values (0 for K < 1). */
size_t moe_mx8_code_bytes(int64_t K);
size_t moe_mx8_scale_bytes(int64_t K);

/*
 * moe_mx8_quantize — rows of x to blocks.
 * Scale: the least power of two that leaves max |x| at most 448, clamped to [2^-127, 2^127], so no
 * value saturates.  Each x 2^-scale goes to the nearest code, ties to the even one; signs (of zeros
 * too) are kept.  A block of zeros gets byte 0; one holding an infinity or a NaN gets byte 255 and
 * zero codes.
 * x [rows, K] of dtype xdt (f32 / f16 / bf16), row r at x + r * ldx elements, ldx >= K.
 * Alignment: none for x (16-byte aligned rows take a vectorised path).
 */
int moe_mx8_quantize(const void* x, int xdt, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                     uint8_t* scales, moe_stream_t stream);

/*
 * moe_mx8_dequantize — the values the blocks stand for, rounded once to odt.
 * out [rows, K], row r at out + r * ldo elements, ldo >= K; elements between rows are not written.
 */
int moe_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                       void* out, int odt, int64_t ldo, moe_stream_t stream);

/*
 * moe_mx8_dispatch — moe_dispatch for tokens in blocks: codes / scales [T] rows of H values.
 * x_codes, x_scales [T * top_k] rows; the other arguments, ids >= E and the workspace as there.
 * Alignment: codes and x_codes 16 bytes, scales and x_scales 4, ws 16.
 */
int moe_mx8_dispatch(const uint8_t* codes, const uint8_t* scales, int64_t T, int64_t H,
                     const uint32_t* idx, int64_t E, int top_k, uint8_t* x_codes,
                     uint8_t* x_scales, int32_t* offsets, uint32_t* token_of_row,
                     uint32_t* row_of_slot, void* ws, size_t ws_bytes, moe_stream_t stream);

/*
 * moe_mx8_product — out[r, n] = sum_k A[r, k] B[e, n, k] for the rows r of group e.
 * As moe_mx4_product, with both operands in 8-bit blocks.
 */
size_t moe_mx8_product_workspace_bytes(void);
int moe_mx8_product(const uint8_t* a_codes, const uint8_t* a_scales, int64_t rows,
                    const uint8_t* b_codes, const uint8_t* b_scales, const int32_t* offsets,
                    int64_t E, int64_t N, int64_t K, void* out, int odt, void* ws,
                    size_t ws_bytes, moe_stream_t stream);

/*
 * moe_mx8_experts_forward_dispatched — SwiGLU experts over dispatched rows in blocks (from
 * moe_mx8_dispatch, or dispatched rows that moe_mx8_quantize took).  With Q the trip of
 * moe_mx8_quantize over rows of I values:
 *   g = x gate[e]^T,  u = x up[e]^T,  a = Q(silu(g) u),  y[r] = a down[e]^T
 * g, u and silu(g) u are FP32 (not rounded before they are quantised), y is rounded once to odt.
 * x [rows] rows of H values; gate, up [E, I] rows of H, down [E, H] rows of I; y [rows, H],
 * contiguous; offsets [E + 1] as for the product, not NULL.
 * ws: at least moe_mx8_experts_workspace_bytes(rows, I) bytes, 256-byte aligned.
 */
size_t moe_mx8_experts_workspace_bytes(int64_t rows, int64_t I);
int moe_mx8_experts_forward_dispatched(const uint8_t* x_codes, const uint8_t* x_scales,
                                       const int32_t* offsets, int64_t rows,
                                       const uint8_t* gate_codes, const uint8_t* gate_scales,
                                       const uint8_t* up_codes, const uint8_t* up_scales,
                                       const uint8_t* down_codes, const uint8_t* down_scales,
                                       int64_t E, int64_t H, int64_t I, void* y, int odt, void* ws,
                                       size_t ws_bytes, moe_stream_t stream);

/*
 * moe_mx8_forward — the layer from routed tokens in blocks on: dispatch, experts, combine.
 *   out[t] = sum_j w[t, j] y_j, y_j expert idx[t, j]'s output for token t, rounded to odt, summed in
 *   FP32 in the order j = 0 .. top_k-1 and rounded once.
 * x [T] rows of H values in blocks; idx [T, top_k] and w [T, top_k] (dtype wdt) from any of the
 * routers; weights as above; out [T, H] of dtype odt.  A token with an id >= E gets NaN, and the
 * device status MOE_ERR_INDEX.
 * ws: at least moe_mx8_forward_workspace_bytes(...) bytes (0 for sizes out of range), 256-byte
 * aligned.
 */
size_t moe_mx8_forward_workspace_bytes(int64_t T, int64_t E, int64_t H, int64_t I, int top_k,
                                       int odt);
int moe_mx8_forward(const uint8_t* x_codes, const uint8_t* x_scales, const uint32_t* idx,
                    const void* w, int wdt, const uint8_t* gate_codes, const uint8_t* gate_scales,
                    const uint8_t* up_codes, const uint8_t* up_scales, const uint8_t* down_codes,
                    const uint8_t* down_scales, int64_t T, int64_t E, int64_t H, int64_t I,
                    int top_k, void* out, int odt, void* ws, size_t ws_bytes,
                    moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_MX8_H_ */
