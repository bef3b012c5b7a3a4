/*
 * nvfp4_moe.h - C ABI of the operators around the NVFP4 grouped GEMM
 * (nvfp4_grouped_gemm.h) in a layer of experts, for AMD Instinct MI355X
 * (gfx950): routing, the plan that sorts rows by expert, quantisation to NVFP4
 * operands, the combine, and the experts' products of a few tokens.
 *
 * A layer runs, per batch of tokens:
 *   nvfp4_moe_route       logits -> expert ids and weights of every slot
 *   nvfp4_moe_plan        ids -> rows sorted by expert, group tables
 *   nvfp4_moe_dispatch    x -> A, SFA of every expert's rows
 *   nvfp4_grouped_gemm_device, nvfp4_moe_swiglu, nvfp4_grouped_gemm_device
 *   nvfp4_moe_combine     experts' rows -> tokens
 * or, for a few tokens, nvfp4_moe_few_tokens twice in place of the middle four.
 *
 * Terms. A slot is a (token, choice) pair, numbered token * topk + choice. A
 * row is a place among the rows sorted by expert. A slot whose id is outside
 * 0 .. experts-1 has no expert: it has row -1, weight-sum share 0 and gradient
 * 0, and whatever its weight holds is not used.
 *
 * NVFP4 operands are those of nvfp4_grouped_gemm.h: codes uint8 [rows][k/2],
 * low nibble first; scales in atoms of 128 rows x 64 K-elements, 512 bytes.
 * Operands sorted by expert keep their codes row after row, without gaps;
 * every expert's scales begin at an atom row of their own: expert e's rows are
 * offsets[e] .. offsets[e+1]-1, its scale tensor is at
 * sfa + atoms[e] * ceil(k/64) * 512.
 *
 * Ownership, errors and threading as in nvfp4_grouped_gemm.h: the caller owns
 * every buffer, nothing is allocated or synchronised, calls are stream-ordered
 * and may be captured in a HIP graph, arguments are checked before any HIP
 * call with the same return codes (NVFP4_ERR_INVALID for sizes, types and null
 * pointers, NVFP4_ERR_MISALIGNED for addresses, NVFP4_ERR_WORKSPACE). Results
 * do not depend on timing: no sum's order does. Strides count elements.
 * Outputs may not overlap inputs. A call that would need more than about 2^31
 * threads is NVFP4_ERR_INVALID (2^23 workgroups of 256: 2^34 elements of rows to
 * quantise). Calls with no work (0 tokens or rows) are
 * NVFP4_OK and launch nothing, except that nvfp4_moe_plan of 0 tokens writes
 * its offsets.
 */
#ifndef NVFP4_MOE_H
#define NVFP4_MOE_H

#include "nvfp4_grouped_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define NVFP4_MOE_F32 0
#define NVFP4_MOE_F16 1
#define NVFP4_MOE_BF16 2

#define NVFP4_MOE_MAX_EXPERTS 512
#define NVFP4_MOE_MAX_TOPK 16
#define NVFP4_MOE_MAX_GROUPS 64
#define NVFP4_MOE_MAX_FEW_SLOTS 4096
#define NVFP4_MOE_MAX_PRODUCTS 4

#define NVFP4_MOE_SOFTMAX 0
#define NVFP4_MOE_SIGMOID 1

/* How nvfp4_moe_route scores and chooses. */
typedef struct nvfp4_moe_choice {
  int32_t score;        /* NVFP4_MOE_SOFTMAX (over all experts) or NVFP4_MOE_SIGMOID */
  int32_t topk;         /* experts of a token: 1 .. min(16, topk_groups * experts / groups) */
  int32_t groups;       /* 1 .. 64, divides experts; 1: no groups */
  int32_t topk_groups;  /* groups that stay eligible: 1 .. groups */
  int32_t group_best;   /* a group's value: the sum of its best 1 or 2 choice values */
  int32_t renormalize;  /* divide the weights of a token by their sum */
  float scale;          /* factor on the weights */
} nvfp4_moe_choice;

/*
 * nvfp4_moe_route - scores, choice and weights of every token.
 *
 *   s = score(x). Choice value v = x where there is neither bias nor groups,
 *   else s + bias (bias NULL: s), compared in fp64. With groups, the
 *   topk_groups groups of the largest value stay eligible. The topk largest v
 *   among the eligible experts are chosen, in falling order; equal values go to
 *   the lowest index (fp64 values within 2^-42 of each other, or that part of values
 *   beyond 1, may count as equal).
 *   w = scale * s / (renormalize ? sum of the chosen s : 1); the bias has no
 *   part in it.
 * A logit of -inf masks its expert: score 0 and never chosen. A token with
 * fewer eligible experts than topk gets id -1 and weight 0 in the other slots.
 * For the choice, a NaN logit counts as -inf and +inf as the largest fp32. A NaN
 * logit, and with softmax one of +inf, makes the weights of its token's chosen
 * experts NaN. A choice value of NaN or -inf
 * (through the bias) is never chosen either. A sum of scores that is 0 counts
 * as 1. Sums are those of the scores themselves, also where these lie below fp32's
 * range; a sigmoid of a logit below -708 (2^-1021) counts as 0.
 *
 *   logits   device [tokens][experts] of `dtype`, rows `row_stride` elements apart; tokens < 2^26
 *   bias     device fp32 [experts], or NULL
 *   ids      device int32 [tokens][topk]
 *   weights  device fp32 [tokens][topk]
 */
int nvfp4_moe_route(const void* logits, int dtype, int64_t tokens, int experts, int64_t row_stride,
                    const float* bias, const nvfp4_moe_choice* choice, int32_t* ids, float* weights,
                    void* stream);

/*
 * nvfp4_moe_route_backward - d logits from d weights: the gradient of
 * nvfp4_moe_route with the choice held fixed (groups and bias have no part).
 * Every element of dlogits [tokens][experts], of `dtype`, is written. `ids` as
 * nvfp4_moe_route gave them (a token's ids differ; -1: no gradient); the bias
 * gets no gradient. A logit of an expert that was not chosen is read only where the
 * weights are a softmax that is not renormalised: a NaN there makes no other
 * gradient NaN, though it made the weights so.
 */
int nvfp4_moe_route_backward(const void* logits, int dtype, int64_t tokens, int experts, int64_t row_stride,
                             const nvfp4_moe_choice* choice, const int32_t* ids, const float* dweights,
                             void* dlogits, int64_t dlogits_stride, void* stream);

/* A grouped product whose group tables nvfp4_moe_plan writes: expert e is a
 * group of m = its rows, with A, C and SFA of the rows sorted by expert and
 * the e-th of `experts` stacked weights. Addresses are device addresses. */
typedef struct nvfp4_moe_product {
  int32_t n, k;             /* n % 8 == 0, k % 32 == 0 */
  uint64_t a, b, c;         /* codes [rows][k/2], codes [experts][n][k/2], fp16 [rows][n] */
  uint64_t sfa, sfb;        /* scales of the rows; [experts][nvfp4_sf_bytes(n, k, 1)] */
  uint64_t sizes, abc, sf;  /* tables to write: int32 [experts][4], uint64 [experts][3], uint64 [experts][2] */
} nvfp4_moe_product;

/*
 * nvfp4_moe_plan - sort slots by expert, stably (slot order within an expert).
 *
 *   ids        device int32 [tokens][topk]
 *   offsets    device int32 [experts+1]: first row of each expert, then the number of rows
 *   atoms      device int32 [experts+1]: first scale-atom row of each expert, then their number
 *   slot_rows  device int32 [tokens*topk]: row of a slot, or -1
 *   row_slots  device int32 [tokens*topk]: slot of a row; -1 from offsets[experts] on
 *   products   host array of num_products (0 .. 4) products whose tables to fill, or NULL
 *   workspace  device, 256-byte aligned, nvfp4_moe_plan_workspace_bytes (may be 0) bytes
 * tokens * topk <= 2^30.
 */
int nvfp4_moe_plan(const int32_t* ids, int64_t tokens, int topk, int experts, int32_t* offsets, int32_t* atoms,
                   int32_t* slot_rows, int32_t* row_slots, const nvfp4_moe_product* products, int num_products,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * nvfp4_moe_plan_ex - as nvfp4_moe_plan, with a copy of the ids that belongs to
 * the plan, for callers whose ids are rewritten while the plan is in use:
 *   slot_ids   device int32 [tokens*topk]: expert of a slot, or -1 where it has none; or NULL
 */
int nvfp4_moe_plan_ex(const int32_t* ids, int64_t tokens, int topk, int experts, int32_t* offsets, int32_t* atoms,
                      int32_t* slot_rows, int32_t* row_slots, int32_t* slot_ids, const nvfp4_moe_product* products,
                      int num_products, void* workspace, size_t workspace_bytes, void* stream);
size_t nvfp4_moe_plan_workspace_bytes(int64_t tokens, int topk, int experts);

/* Bytes of the scales of up to `rows` rows sorted by expert: room for any
 * spread of the rows over the experts. 0 if an argument is not valid. */
size_t nvfp4_moe_sf_bytes(int64_t rows, int experts, int k);

/*
 * nvfp4_moe_quantize - rows to NVFP4: for every 16 elements v = x * scale
 * (rounded to fp32) of a row
 *     s = E4M3(max|v| / 6), at most 448;  code = E2M1(v / s), at most 6
 * each rounded once from the exact quotient, to nearest, ties to even. A block
 * whose s rounds to 0 has codes 0. A block that holds an infinity or NaN gets
 * scale NaN, so that products with it are NaN.
 *
 *   x    device [l][m][k] of `dtype`, rows row_stride and batches batch_stride elements apart
 *   a    device uint8 [l][m][k/2], sfa: device uint8 [nvfp4_sf_bytes(m, k, l)], both 16-byte aligned
 * k % 32 == 0. Scales of rows past m in a batch's last atom row are written as 0
 * or not at all.
 */
int nvfp4_moe_quantize(const void* x, int dtype, int l, int64_t m, int k, int64_t batch_stride, int64_t row_stride,
                       float scale, void* a, void* sfa, void* stream);

/*
 * nvfp4_moe_dispatch - as nvfp4_moe_quantize for x [tokens][k], each token's
 * row written to the rows of its slots in the plan (ids, and slot_rows, row_slots,
 * offsets and atoms of nvfp4_moe_plan for them). A row's expert is the one whose
 * rows hold it; ids say where that is looked for first, and may have been rewritten
 * since. Nothing is stored outside a and sfa, whatever the tables hold.
 *   a          device uint8 [tokens*topk][k/2]
 *   sfa        device uint8 [nvfp4_moe_sf_bytes(tokens*topk, experts, k)]
 *   workspace  device, 256-byte aligned, nvfp4_moe_dispatch_workspace_bytes (may be 0) bytes
 */
int nvfp4_moe_dispatch(const void* x, int dtype, int64_t tokens, int topk, int k, int64_t row_stride, float scale,
                       const int32_t* ids, const int32_t* slot_rows, const int32_t* row_slots,
                       const int32_t* offsets, const int32_t* atoms, int experts, void* a, void* sfa,
                       void* workspace, size_t workspace_bytes, void* stream);
size_t nvfp4_moe_dispatch_workspace_bytes(int64_t tokens, int topk, int k);

/*
 * nvfp4_moe_swiglu - as nvfp4_moe_quantize for v = silu(g * alpha) * (u * alpha)
 * * scale of rows sorted by expert, c [rows][2k] with g in columns 0 .. k-1 and
 * u in k .. 2k-1; codes and scales are those of the exact v (evaluated in fp64
 * where fp32 cannot tell; a v beyond fp32 counts as infinite).
 *   alpha    device fp32 [experts], or NULL for 1
 *   offsets, atoms  of the plan, or both NULL with experts == 1: `rows` rows of one group
 * rows is the size of c; rows from offsets[experts] on are not touched.
 */
int nvfp4_moe_swiglu(const void* c, int dtype, int64_t rows, int k, int64_t row_stride, const float* alpha,
                     float scale, const int32_t* offsets, const int32_t* atoms, int experts, void* a, void* sfa,
                     void* stream);

/*
 * nvfp4_moe_dequantize - the values code * scale of NVFP4 rows, as `dtype`
 * (exact in fp16 and fp32, and in bf16), out [l][m][k], rows row_stride elements
 * apart and batches m rows. With offsets and atoms (l == 1): of rows sorted by
 * expert, m the most rows there can be; rows from offsets[experts] on are not touched.
 */
int nvfp4_moe_dequantize(const void* a, const void* sfa, int l, int64_t m, int k, const int32_t* offsets,
                         const int32_t* atoms, int experts, void* out, int dtype, int64_t row_stride, void* stream);

/*
 * nvfp4_moe_combine - y[t] = residual[t] + sum over the slots j of t, in slot
 * order, of weights[t][j] * alpha[ids[t][j]] * c[slot_rows[t][j]], summed in
 * fp32 and rounded once to out_dtype. Slots whose row is not in 0 .. c_rows - 1
 * add nothing and read nothing.
 *   c          device [c_rows][n] of c_dtype (fp16 or bf16 or fp32), rows c_stride apart; NULL if c_rows is 0
 *   slot_rows  NULL: the row of a slot is the slot (then c_rows >= tokens*topk)
 *   weights    fp32 [tokens][topk], NULL: 1
 *   alpha      fp32 [experts], NULL: 1; needs ids
 *   ids        int32 [tokens][topk]; where given, a slot whose id is not in 0 .. experts - 1 adds nothing
 *   experts    their number; without alpha it may be 0 or less: then no id is too large
 *   residual   [tokens][n] of out_dtype, rows out_stride apart, or NULL
 *   out        [tokens][n] of out_dtype, rows out_stride apart
 */
int nvfp4_moe_combine(const void* c, int c_dtype, int64_t c_stride, int64_t c_rows, int64_t tokens, int topk, int n,
                      const int32_t* slot_rows, const float* weights, const float* alpha, const int32_t* ids,
                      int experts, const void* residual, void* out, int out_dtype, int64_t out_stride, void* stream);

/*
 * nvfp4_moe_combine_backward - gradients of nvfp4_moe_combine:
 *   dc[slot_rows[t][j]] = weights[t][j] * alpha * dy[t]   (of c_dtype, rows c_stride apart)
 *   dweights[t][j] = alpha * sum over n of dy[t] * c[slot_rows[t][j]]   (fp32)
 * Rows of dc that no slot names are not written; rows of slots without an expert
 * are 0, and so are dweights of slots without a row or an expert. No two slots
 * may name one row. The residual's gradient is dy.
 */
int nvfp4_moe_combine_backward(const void* dy, int dy_dtype, int64_t dy_stride, const void* c, int c_dtype,
                               int64_t c_stride, int64_t c_rows, int64_t tokens, int topk, int n,
                               const int32_t* slot_rows, const float* weights, const float* alpha, const int32_t* ids,
                               int experts, void* dc, float* dweights, void* stream);

/*
 * nvfp4_moe_few_tokens - the experts' product of a few tokens with activations
 * as they are (fp16 or bf16), one output row per slot:
 *   y[t][j] = alpha[e] * W_e x,  e = ids[t][j]
 *   swiglu: silu(y[0 .. n/2-1]) * y[n/2 .. n-1]
 * The weights of an expert are read once for a pass of its slots: as many as there
 * are tokens, rounded up to a power of two, 16 at most (an expert that a token names
 * several times may take more passes than one).
 * Products are accumulated in fp32. Slots without an expert give zeros.
 *   x      device [tokens][k], or with per_slot [tokens*topk][k], rows x_stride apart
 *   b, sfb device uint8 [experts][n][k/2] and [experts][nvfp4_sf_bytes(n, k, 1)], 16-byte aligned
 *   out    device [tokens*topk][n, or n/2 with swiglu] of out_dtype, rows without gaps
 * tokens * topk <= NVFP4_MOE_MAX_FEW_SLOTS; k % 32 == 0; n % 8 == 0
 * (swiglu: n % 16 == 0); the codes of an expert below 2^31 bytes.
 */
int nvfp4_moe_few_tokens(const void* x, int dtype, int64_t x_stride, int per_slot, const int32_t* ids,
                         int64_t tokens, int topk, int experts, int n, int k, const void* b, const void* sfb,
                         const float* alpha, int swiglu, void* out, int out_dtype, void* stream);

/* The hipError_t of the last failed HIP call of these entry points on the
 * calling thread (0 if none). */
int nvfp4_moe_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_MOE_H */
