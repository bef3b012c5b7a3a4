/*
 * nvfp4_ffn.h - C ABI of the feed-forward block in 16 bits beside the NVFP4 layer
 * (nvfp4_moe.h), for AMD Instinct MI355X (gfx950): the norm before it, products
 * with an epilogue, the gated projections, their gradients, and rows kept in 8
 * bits. Dense (a shared expert), or by the rows of an nvfp4_moe_plan.
 *
 * A block's forward and backward pass:
 *   nvfp4_ffn_rmsnorm          s = x + residual, its norm, in 16 or 8 bits
 *   nvfp4_ffn_gated            h = act(x Wg^T) * (x Wu^T)
 *   nvfp4_ffn_linear           y = act(h W^T + bias) + residual
 *   nvfp4_ffn_linear_dz, _dx, _dw;  nvfp4_ffn_gated_dz or _again, _dx, _dw (those of linear)
 *   nvfp4_ffn_rmsnorm_backward
 *
 * Types. Rows and weights are fp16 or bf16 (`dtype`: NVFP4_MOE_F16, NVFP4_MOE_BF16;
 * norms and rows in 8 bits take fp32 too). Products are accumulated in fp32, epilogues,
 * norms and column sums computed in fp32, and each output is rounded once.
 *
 * Rows in 8 bits: codes uint8 [rows][n] (E4M3) and scales uint8 [rows][n / 32]: 32
 * elements v have the scale 2^(byte - 127), the least from 2^-126 (byte 1) on under
 * which the largest |v| / scale is at most 448, and code = E4M3(v / scale), to
 * nearest, ties to even. Byte 255: the 32 held an infinity or NaN, and their values
 * are NaN. n % 32 == 0.
 *
 * Plans. With a plan rows are sorted by expert: expert e has rows offsets[e] ..
 * offsets[e + 1] - 1 and the e-th of `experts` stacked weights and biases. Rows from
 * offsets[experts] on have no expert. Nothing is read or stored outside the operands,
 * whatever the tables hold.
 *
 * Ownership, errors and threading as in nvfp4_moe.h: the caller owns every buffer,
 * nothing is allocated or synchronised, calls are stream-ordered and may be captured in
 * a HIP graph, arguments are checked before any HIP call (NVFP4_ERR_INVALID for sizes,
 * types and null pointers, NVFP4_ERR_MISALIGNED for addresses and strides,
 * NVFP4_ERR_WORKSPACE). Results do not depend on timing: no sum's order does. Strides
 * count elements; outputs have rows without gaps unless a stride is given. Outputs may not
 * overlap inputs. Calls with no work (0 rows) are NVFP4_OK and launch nothing, except
 * gradients of weights, which are then 0. rows < 2^31.
 *
 * Products need n % 8 == 0 and k % 8 == 0, both 1 .. 2^20, and addresses and rows of
 * operands at multiples of 16 bytes; an expert's weights stay below 2^31 bytes, and rows of x and dz lie less than 2^22
 * elements apart. A product has fewer than 2^23 tiles of 256 x 256 (2^31 - 2^15 rows of up to 256 columns, 2^24 rows of
 * 30000).
 */
#ifndef NVFP4_FFN_H
#define NVFP4_FFN_H

#include "nvfp4_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations: z, max(z, 0), z / (1 + e^-z), z Phi(z) with the normal distribution Phi.
 * Results below about 2^-119 may be 0; at infinities all take their limits. */
#define NVFP4_FFN_NONE 0
#define NVFP4_FFN_RELU 1
#define NVFP4_FFN_SILU 2
#define NVFP4_FFN_GELU 3

/* Rows sorted by expert, as nvfp4_moe_plan gives them. */
typedef struct nvfp4_ffn_plan {
  int32_t experts;           /* 1 .. NVFP4_MOE_MAX_EXPERTS */
  int32_t topk;              /* 1 .. NVFP4_MOE_MAX_TOPK: slots of a token */
  const int32_t* offsets;    /* device int32 [experts + 1] */
  const int32_t* row_slots;  /* device int32 [rows]: slot of a row; read where rows are gathered from tokens */
} nvfp4_ffn_plan;

/*
 * nvfp4_ffn_rmsnorm - s = x + residual, rounded to `dtype`; y = s * rstd * weight with
 * rstd = 1 / sqrt(mean of s^2 over the row + eps).
 *   x         device [rows][n] of dtype (fp32, fp16, bf16), rows x_stride apart; 1 <= n <= 65536
 *   residual  as x, rows residual_stride apart, or NULL: then s is x and `sum` is not written
 *   weight    device [n], fp32 (weight_f32 = 1) or of dtype; NULL: 1
 *   sum       device [rows][n] of dtype; it may be the address of x or residual with their stride n
 *   y         device [rows][n] of dtype, or NULL
 *   codes, scales  y in 8 bits (of the fp32 y, not of the rounded one), or both NULL
 *   rstd      device fp32 [rows], or NULL
 */
int nvfp4_ffn_rmsnorm(const void* x, int dtype, int64_t rows, int n, int64_t x_stride, const void* residual,
                      int64_t residual_stride, const void* weight, int weight_f32, float eps, void* sum, void* y,
                      void* codes, void* scales, float* rstd, void* stream);

/*
 * nvfp4_ffn_rmsnorm_backward - with h = s * rstd:
 *   dx = rstd * (weight dy - h * mean of (weight dy h) over the row) + dsum
 *   dweight = sum over rows of dy h
 * dx is the gradient of x and of the residual. dsum [rows][n]: a gradient that reaches
 * s otherwise, or NULL. dweight has the weight's type (weight NULL: dweight NULL).
 * workspace: device, 256-byte aligned, nvfp4_ffn_rmsnorm_workspace_bytes bytes (with dweight).
 */
int nvfp4_ffn_rmsnorm_backward(const void* dy, int64_t dy_stride, const void* s, int64_t s_stride, int dtype,
                               int64_t rows, int n, const void* weight, int weight_f32, const float* rstd,
                               const void* dsum, int64_t dsum_stride, void* dx, void* dweight, void* workspace,
                               size_t workspace_bytes, void* stream);
size_t nvfp4_ffn_rmsnorm_workspace_bytes(int64_t rows, int n);

/* nvfp4_ffn_quantize8 - rows to 8 bits; nvfp4_ffn_dequantize8 - their values, rounded to dtype. */
int nvfp4_ffn_quantize8(const void* x, int dtype, int64_t rows, int n, int64_t x_stride, void* codes, void* scales,
                        void* stream);
int nvfp4_ffn_dequantize8(const void* codes, const void* scales, int64_t rows, int n, void* out, int dtype,
                          int64_t out_stride, void* stream);

/*
 * nvfp4_ffn_gather - tokens' rows at the rows of their slots: out[r] = x[row_slots[r] / topk].
 * x: [tokens][n] of dtype, rows x_stride apart, n % 8 == 0, or (x NULL) codes and scales of
 * rows in 8 bits, n % 32 == 0. out: [tokens * topk][n] of dtype; rows of no expert are not written.
 */
int nvfp4_ffn_gather(const void* x, int64_t x_stride, const void* codes, const void* scales, int dtype, int64_t tokens,
                     int n, const nvfp4_ffn_plan* plan, void* out, void* stream);

/*
 * nvfp4_ffn_linear - z = x W^T + bias, y = act(z) + residual.
 *   x         device [rows][k] of dtype, rows x_stride apart
 *   w         device [n][k] of dtype, with a plan [experts][n][k]
 *   bias      device [n] or [experts][n], fp32 (bias_f32 = 1) or of dtype, or NULL
 *   residual  device [rows][n] of dtype, rows residual_stride apart, or NULL
 *   z         device [rows][n] of dtype: z as the gradient needs it, or NULL
 *   y         device [rows][n] of dtype
 *   clear     rows of no expert: 0 leaves them as they were in y and z, 1 writes 0
 *   workspace device, 256-byte aligned, nvfp4_ffn_product_workspace_bytes(rows, n, k, experts) bytes (may be 0)
 */
int nvfp4_ffn_linear(const void* x, int64_t x_stride, const void* w, const void* bias, int bias_f32, int act,
                     const void* residual, int64_t residual_stride, void* z, void* y, int dtype, int64_t rows, int n,
                     int k, const nvfp4_ffn_plan* plan, int clear, void* workspace, size_t workspace_bytes, void* stream);

/*
 * nvfp4_ffn_gated - g = x Wg^T, u = x Wu^T, h = act(g) * u; act not NVFP4_FFN_NONE.
 *   x         device [rows][k]; with a plan [tokens][k] below 2^31 bytes, rows = tokens * topk, each row its token's
 *   w         device [2 * inner][k], Wg's rows first; with a plan [experts][2 * inner][k]
 *   h         device [rows][inner]
 *   kept      device [rows][2 * inner] of dtype: g, then u, rounded; or NULL
 *   codes, scales  the same in 8 bits (of the fp32 values; inner % 32 == 0); or both NULL
 *   clear     as in nvfp4_ffn_linear, for h and what is kept
 *   workspace nvfp4_ffn_product_workspace_bytes(rows, 2 * inner, k, experts) bytes
 */
int nvfp4_ffn_gated(const void* x, int64_t x_stride, const void* w, int act, void* h, void* kept, void* codes,
                    void* scales, int dtype, int64_t rows, int inner, int k, const nvfp4_ffn_plan* plan, int clear,
                    void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace of a product [rows][k] x [n][k] (also of nvfp4_ffn_linear_dx with n and k in turn: [rows][n] x
 * [k][n]); experts 0: dense, else the plan's. */
size_t nvfp4_ffn_product_workspace_bytes(int64_t rows, int n, int k, int experts);

/*
 * nvfp4_ffn_product_parts - how a product is computed: the number of its launches over rows (1 or 2; 0 for arguments
 * that are none), and for each four values in `parts` (host, int32 [8]): its rows, the tile's rows and columns
 * (0, 0: the kernel of few rows), the parts of k. Those are the choice for a device of the current one's compute units
 * and rows without gaps: where rows lie so far apart that 320 of them are beyond 32-bit offsets, tiles of 256 rows take
 * the place of tiles of 320.
 *   kind   NVFP4_FFN_FORWARD, _FORWARD_CODES (gated with codes), _DX or _DW; rows, n, k, experts as for the call
 */
#define NVFP4_FFN_FORWARD 0
#define NVFP4_FFN_FORWARD_CODES 1
#define NVFP4_FFN_DX 2
#define NVFP4_FFN_DW 3
int nvfp4_ffn_product_parts(int kind, int64_t rows, int n, int k, int experts, int32_t* parts);

/*
 * nvfp4_ffn_linear_dz - dz = dy act'(z), rounded to dtype, and dbias = sum over an expert's
 * rows of the unrounded dz.
 *   dy, z     device [rows][n] of dtype, rows dy_stride apart and without gaps; z NULL with NVFP4_FFN_NONE
 *   dz        device [rows][n], or NULL (NVFP4_FFN_NONE: dz is dy); rows of no expert are not written
 *   dbias     device [n] or [experts][n], fp32 (bias_f32 = 1) or of dtype, or NULL
 *   workspace nvfp4_ffn_dz_workspace_bytes bytes (with dbias)
 */
int nvfp4_ffn_linear_dz(const void* dy, int64_t dy_stride, const void* z, int act, void* dz, void* dbias, int bias_f32,
                        int dtype, int64_t rows, int n, const nvfp4_ffn_plan* plan, void* workspace,
                        size_t workspace_bytes, void* stream);
size_t nvfp4_ffn_dz_workspace_bytes(int64_t rows, int n, int experts);

/*
 * nvfp4_ffn_gated_dz - dz [rows][2 * inner] = (dh u act'(g), dh act(g)) from g and u as they
 * were kept (kept, or codes and scales), rounded to dtype. Rows of no expert are not written.
 */
int nvfp4_ffn_gated_dz(const void* dh, int64_t dh_stride, const void* kept, const void* codes, const void* scales, int act,
                       void* dz, int dtype, int64_t rows, int inner, const nvfp4_ffn_plan* plan, void* stream);

/*
 * nvfp4_ffn_gated_again - the same dz with g and u computed again from x (as in nvfp4_ffn_gated) and not rounded on the
 * way: nothing of the forward pass need be kept but x. Rows of no expert are not written.
 */
int nvfp4_ffn_gated_again(const void* dh, int64_t dh_stride, const void* x, int64_t x_stride, const void* w, int act,
                          void* dz, int dtype, int64_t rows, int inner, int k, const nvfp4_ffn_plan* plan,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * nvfp4_ffn_linear_dx - dx [rows][k] = dz W; dz device [rows][n], rows dz_stride apart; w as in nvfp4_ffn_linear.
 * nvfp4_ffn_linear_dx_ex - the same, dx fp32 (dx_f32 = 1: rows of slots that are yet to be added) or of dtype.
 * nvfp4_ffn_linear_dw - dW [n][k], with a plan [experts][n][k], = dz^T x over an expert's rows (an expert
 * without rows: 0), fp32 (dw_f32 = 1) or of dtype; x device [rows][k], sorted by expert with a plan;
 * workspace: nvfp4_ffn_dw_workspace_bytes bytes (may be 0).
 */
int nvfp4_ffn_linear_dx(const void* dz, int64_t dz_stride, const void* w, void* dx, int dtype, int64_t rows, int n, int k,
                        const nvfp4_ffn_plan* plan, int clear, void* workspace, size_t workspace_bytes, void* stream);
int nvfp4_ffn_linear_dx_ex(const void* dz, int64_t dz_stride, const void* w, void* dx, int dx_f32, int dtype, int64_t rows,
                           int n, int k, const nvfp4_ffn_plan* plan, int clear, void* workspace, size_t workspace_bytes,
                           void* stream);
int nvfp4_ffn_linear_dw(const void* dz, int64_t dz_stride, const void* x, int64_t x_stride, void* dw, int dw_f32, int dtype,
                        int64_t rows, int n, int k, const nvfp4_ffn_plan* plan, void* workspace, size_t workspace_bytes,
                        void* stream);
size_t nvfp4_ffn_dw_workspace_bytes(int64_t rows, int n, int k, int experts);

/* The hipError_t of the last failed HIP call of these entry points on the calling
 * thread (0 if none). */
int nvfp4_ffn_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_FFN_H */
