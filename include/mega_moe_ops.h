/*
 * mega_moe_ops.h -- operators around the fused MoE layer of mega_moe.h, for one GPU (MI355X, gfx950):
 *   - products grouped by expert with ragged row counts, and their gradients (training the experts);
 *   - the router: choosing and weighing the experts of every token (topk_idx / topk_weights as
 *     mega_moe_forward takes them), its gradient, and the ordering of the chosen pairs by expert that
 *     the grouped products read;
 *   - a projection shared by many requests that each bring a low-rank adapter;
 *   - the root-mean-square norm in front of the layer, in 16 and in 8 bits, and its gradient;
 *   - SwiGLU between the experts' products and its gradient, and activations kept in 8 bits for the backward pass.
 *
 * Conventions are those of mega_moe.h: 0 or a negative MEGA_MOE_ERR_* code, nothing throws; device
 * pointers (16-byte aligned unless the comment says otherwise), dense row-major tensors; work is enqueued
 * on `stream` (a stream of the current HIP device, on which all pointers live) and is asynchronous.  No
 * call allocates, synchronises or keeps anything from one call to the next; every call may be captured
 * into a HIP graph (kernels only) and two calls may run at once on different streams as long as their
 * outputs and workspaces are apart.  Inputs and outputs must not overlap.  Results do not depend on the
 * order in which work-groups run: a call repeated on the same inputs gives the same bits.
 *
 * device_status: uint32 (device, 4-byte aligned) or NULL.  Conditions only the device can see are OR-ed
 * into it as MEGA_MOE_STATUS_* bits; nothing is written when there is none.  The caller zeroes it.
 */
#ifndef MEGA_MOE_OPS_H
#define MEGA_MOE_OPS_H

#include "mega_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define MEGA_MOE_BF16 0
#define MEGA_MOE_FP16 1
#define MEGA_MOE_FP32 2

#define MEGA_MOE_MAX_GROUP_ROWS (1 << 26)   /* rows of a grouped product or an adapter projection */
#define MEGA_MOE_MAX_GROUP_COLS 65536       /* its n and k */
#define MEGA_MOE_MAX_PAIRS 2147418112       /* 2^31 - 2^16: chosen (token, expert) pairs */
#define MEGA_MOE_MAX_REQUESTS 4096          /* requests of an adapter projection */
#define MEGA_MOE_MAX_NORM_COLS 16384        /* columns of a normalised row */

/* ------------------------------------------------------------------ products grouped by expert
 * Rows are sorted by group: group e owns rows offsets[e] .. offsets[e+1]-1 of the row tensors (any count,
 * zero included) and the weight w[e] of the same layout as the layer's unpacked W1 / W2.
 *   forward          y[m]  = x[m] w[e]^T              x [rows][k], w [groups][n][k] -> y [rows][n]
 *   backward_rows    dx[m] = dy[m] w[e]               dy [rows][n], w              -> dx [rows][k]
 *   backward_weight  dw[e] = sum over m of dy[m]^T x[m]   dy, x                    -> dw [groups][n][k]
 * Sums are held in fp32 and rounded once to the output's type.
 *   offsets    int32 [groups + 1] (device), not decreasing, 0 <= offsets[0], offsets[groups] <= rows.
 *              Rows before offsets[0] and from offsets[groups] on are neither read nor written.  Entries
 *              that break this are clamped into 0 .. rows (a decreasing pair is an empty group), and
 *              MEGA_MOE_STATUS_BAD_LAYOUT is latched; which rows are then written is not defined.
 *   rows       rows of the row tensors, 0 .. MEGA_MOE_MAX_GROUP_ROWS
 *   n, k       multiples of 8, 8 .. MEGA_MOE_MAX_GROUP_COLS
 *   groups     1 .. MEGA_MOE_MAX_LOCAL_EXPERTS
 *   dtype      MEGA_MOE_BF16 or MEGA_MOE_FP16, of every operand
 *   out_dtype  (backward_weight) dtype or MEGA_MOE_FP32
 *   accumulate (backward_weight) nonzero: dw += instead of dw =, with out_dtype MEGA_MOE_FP32 only
 *   workspace  (backward_weight) mega_moe_grouped_weight_workspace_bytes() bytes, 0 for most sizes (NULL then): few
 *              and small weights with many rows split the sum; its contents do not matter
 * backward_weight writes zeros for a group without rows (leaves it as it was when accumulating).
 * With rows == 0, forward and backward_rows do nothing and the row pointers may be NULL.
 * Errors: INVALID_ARG (null or misaligned pointer, negative size), UNSUPPORTED (size or type outside the
 * limits, or an output of more than 2^22 tiles of 128 x 128, a last one per group among them; of the weight gradient,
 * of more than 2^21 tiles of 256 x 256), WORKSPACE_TOO_SMALL, HIP. */
int32_t mega_moe_grouped_forward(const void* x, const void* w, const int32_t* offsets, void* y, int64_t rows,
                                 int32_t n, int32_t k, int32_t groups, int32_t dtype, uint32_t* device_status,
                                 void* stream);
int32_t mega_moe_grouped_backward_rows(const void* dy, const void* w, const int32_t* offsets, void* dx,
                                       int64_t rows, int32_t n, int32_t k, int32_t groups, int32_t dtype,
                                       uint32_t* device_status, void* stream);
int32_t mega_moe_grouped_backward_weight(const void* dy, const void* x, const int32_t* offsets, void* dw,
                                         int64_t rows, int32_t n, int32_t k, int32_t groups, int32_t dtype,
                                         int32_t out_dtype, int32_t accumulate, void* workspace,
                                         uint64_t workspace_bytes, uint32_t* device_status, void* stream);
int32_t mega_moe_grouped_weight_workspace_bytes(int64_t rows, int32_t n, int32_t k, int32_t groups,
                                                uint64_t* bytes_out /* host */);

/* ------------------------------------------------------------------ router */
#define MEGA_MOE_SCORE_SOFTMAX 0   /* s = softmax of the token's logits over all its unmasked experts */
#define MEGA_MOE_SCORE_SIGMOID 1   /* s = 1 / (1 + exp(-logit))                                       */

typedef struct mega_moe_router_config {
    int64_t tokens;        /* T >= 0; T * topk at most MEGA_MOE_MAX_PAIRS                              */
    int32_t num_experts;   /* E: 1 .. MEGA_MOE_MAX_EXPERTS                                             */
    int32_t topk;          /* K: 1 .. min(E, MEGA_MOE_MAX_TOPK)                                        */
    int32_t score;         /* MEGA_MOE_SCORE_*                                                         */
    int32_t num_groups;    /* experts in equal consecutive groups; divides E; 1 .. 64                  */
    int32_t topk_groups;   /* groups a token may choose from, 1 .. num_groups                          */
    int32_t group_top;     /* a group is worth the sum of its group_top best experts: 1 or 2           */
    int32_t renormalize;   /* nonzero: the chosen scores are divided by their sum                      */
    float scale;           /* factor of every weight, finite                                           */
    int32_t dtype;         /* of logits (and dlogits): MEGA_MOE_BF16, _FP16 or _FP32                   */
} mega_moe_router_config;

/* For every token: the K experts that rank highest, and their weights.
 *   logits        dtype [T][E].  -inf or NaN masks an expert of that token: it scores 0 and is never
 *                 chosen.  +inf counts as the largest fp32 number.
 *   bias          float [E] or NULL: added to the scores for the choice only, not in the weights.  An
 *                 expert whose biased score is -inf or NaN is not chosen.
 *   topk_idx      int64 [T][K]: expert ids, highest rank first; equal ranks: the lower id first.  A token
 *                 with fewer than K experts to choose from gets -1 (no expert) in the places left.
 *   topk_weights  float [T][K]: scale * s, or scale * s / (sum of the chosen s) when renormalizing; 0 where
 *                 topk_idx is -1, and all 0 where the sum is 0 (sigmoid scores of logits below -709, whose
 *                 exp(-logit) is beyond fp64; in the renormalized softmax the experts that were not
 *                 chosen cancel out, and it is not)
 * Rank: s + bias; without a bias the logit itself, whose order is that of s.  With num_groups > 1 only
 * experts of the topk_groups best groups are eligible; a group's worth is the sum of its group_top
 * highest ranks over unmasked experts (without a bias and with group_top 2: of their s), equal worths: the lower
 * group.  Scores and ranks are computed in fp64, so that a choice between close scores does not hang on
 * fp32 rounding.
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int32_t mega_moe_router_topk(const mega_moe_router_config* cfg, const void* logits, const float* bias,
                             int64_t* topk_idx, float* topk_weights, void* stream);

/* Gradient of the weights with respect to the logits, with the choice held fixed (a bias gets none).
 *   dweights  float [T][K], topk_idx int64 [T][K] as the forward pass returned it (entries outside
 *             0 .. E-1 are ignored; an expert named twice counts twice), logits as in the forward pass
 *   dlogits   dtype [T][E]: every entry written; 0 for masked experts
 * The scores are computed again from the logits.  num_groups, topk_groups and group_top are not used.
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int32_t mega_moe_router_backward(const mega_moe_router_config* cfg, const float* dweights, const void* logits,
                                 const int64_t* topk_idx, void* dlogits, void* stream);

/* Order chosen pairs by expert, for the grouped products: pair p = t*K + k goes to expert topk_idx[p].
 *   topk_idx   int64 [pairs]; entries outside first_expert .. first_expert + num_local_experts - 1
 *              belong to no group here
 *   offsets    int32 [num_local_experts + 1]: first place of every local expert's pairs, and their number
 *   order      int32 [pairs]: order[i] = pair at place i; pairs of one expert in increasing order; -1 from
 *              offsets[num_local_experts] on
 *   slot       int32 [pairs]: the place of pair p, -1 if it belongs to no group here
 *   workspace  mega_moe_group_workspace_bytes() bytes (may be NULL at 0); its contents do not matter
 * pairs 0 .. MEGA_MOE_MAX_PAIRS (pointers of pair arrays may be NULL at 0); num_local_experts 1 .. MEGA_MOE_MAX_EXPERTS.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE_TOO_SMALL, HIP. */
int32_t mega_moe_group_workspace_bytes(int64_t pairs, int32_t num_local_experts, uint64_t* bytes_out /* host */);
int32_t mega_moe_group_by_expert(const int64_t* topk_idx, int64_t pairs, int32_t first_expert,
                                 int32_t num_local_experts, int32_t* offsets, int32_t* order, int32_t* slot,
                                 void* workspace, uint64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ low-rank adapters
 * One projection for the rows of many requests, each with an adapter of its own (or none):
 *   y[m] = x[m] w^T + scales[a] * (x[m] a_a^T) b_a^T,   a = adapter[r] of the request r that owns row m
 *   x        dtype [rows][k], w dtype [n][k], y dtype [rows][n]
 *   a        dtype [adapters][rank][k], b dtype [adapters][n][rank], scales float [adapters]
 *   offsets  int32 [requests + 1] as for the grouped products: request r owns rows offsets[r] ..
 *            offsets[r+1]-1.  Rows that belong to no request get the shared projection alone.
 *   adapter  int32 [requests]: -1 for none; several requests may name the same adapter.  An entry outside
 *            -1 .. adapters-1 counts as none and latches MEGA_MOE_STATUS_BAD_EXPERT_ID
 *   rank     a multiple of 8, 8 .. 256 (adapters of lower rank are padded with zeros)
 *   requests 0 .. MEGA_MOE_MAX_REQUESTS; adapters 1 .. 65536; rows, n, k, dtype as above
 *   workspace mega_moe_adapter_workspace_bytes() bytes; its contents do not matter
 * The shared sum, x a^T and the adapter's sum are held in fp32; scales[a] * x a^T enters the second product as
 * the sum of two 16-bit numbers, the value rounded and the rounded remainder: an error of 2^-16 of it in bf16 and 2^-22
 * in fp16, where a power of two per row and 32 ranks gives it fp32's range (and values below 2^-39 of the largest of
 * their 32 count as 0).
 * Errors: INVALID_ARG, UNSUPPORTED (size or type outside the limits, or a y of more than 2^23 tiles of 64 x 128),
 * WORKSPACE_TOO_SMALL, HIP. */
int32_t mega_moe_adapter_workspace_bytes(int64_t rows, int32_t n, int32_t k, int32_t rank, int32_t requests,
                                         uint64_t* bytes_out /* host */);
int32_t mega_moe_adapter_forward(const void* x, const void* w, const void* a, const void* b, const float* scales,
                                 const int32_t* offsets, const int32_t* adapter, void* y, int64_t rows, int32_t n,
                                 int32_t k, int32_t rank, int32_t requests, int32_t adapters, int32_t dtype,
                                 void* workspace, uint64_t workspace_bytes, uint32_t* device_status, void* stream);

/* ------------------------------------------------------------------ 8-bit rows
 * Rows in 8 bits as the layer takes its tokens: codes uint8 [rows][cols] (e4m3fn) and scales float [rows][ceil(cols / 128)],
 * one per row and 128 columns (the last block may be shorter); the value is code * scale.  Every scale that is written
 * here is a power of two, 2^ceil(log2(largest / 448)) of the largest magnitude of its block (2^-126 at least): no value
 * saturates, each is rounded once to four significant bits (to nearest, ties to even; below 2^-6 scales to multiples of
 * 2^-9 scales; what would become 2^128 becomes 1.875 * 2^127), and code * scale is exact in bf16 and fp16.  A block that holds an infinity or a NaN becomes NaN
 * throughout, with scale 1.  Scales that are read may be any numbers.
 * The row operators below take rows of any length from 1 on, and pointers that are aligned to their element type
 * (codes: to nothing).
 *   quantize_rows    x dtype [rows][cols] -> codes, scales
 *   dequantize_rows  codes, scales -> y dtype [rows][cols], rounded to dtype where that has fewer bits (fp16: 65536, to which
 *                    four bits round fp16's largest numbers, comes back as 65504)
 *   rows   0 .. MEGA_MOE_MAX_GROUP_ROWS (pointers may be NULL at 0), cols 1 .. MEGA_MOE_MAX_GROUP_COLS
 *   dtype  MEGA_MOE_BF16, _FP16 or _FP32
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int32_t mega_moe_quantize_rows(const void* x, uint8_t* codes, float* scales, int64_t rows, int32_t cols, int32_t dtype, void* stream);
int32_t mega_moe_dequantize_rows(const uint8_t* codes, const float* scales, void* y, int64_t rows, int32_t cols, int32_t dtype,
                                 void* stream);

/* The weight gradient of the grouped products from rows kept in 8 bits:
 *   dw[e] = sum over the rows m of group e of dy[m]^T x[m],   x[m] = codes * scales
 *   dy dtype [rows][n], codes uint8 [rows][k], scales float [rows][ceil(k / 128)].  A value enters the product in dtype:
 *   exactly with scales that are powers of two, unless it leaves fp16's range (as in dequantize_rows), else rounded.
 * Everything else, the limits and errors included, as for mega_moe_grouped_backward_weight, but codes are 8-byte and scales
 * 4-byte aligned, codes and scales of rows of no group may be read (and count for nothing), and
 *   workspace  mega_moe_grouped_codes_workspace_bytes() bytes: for the parts of a split sum, and with many tiles of dw for
 *              the rows in 16 bits */
int32_t mega_moe_grouped_codes_workspace_bytes(int64_t rows, int32_t n, int32_t k, int32_t groups, uint64_t* bytes_out /* host */);
int32_t mega_moe_grouped_backward_weight_codes(const void* dy, const uint8_t* codes, const float* scales, const int32_t* offsets,
                                               void* dw, int64_t rows, int32_t n, int32_t k, int32_t groups, int32_t dtype,
                                               int32_t out_dtype, int32_t accumulate, void* workspace, uint64_t workspace_bytes,
                                               uint32_t* device_status, void* stream);

/* ------------------------------------------------------------------ norm
 * Root-mean-square norm of rows, with the residual's addition:
 *   v = x + residual,  h = v rounded,  y = v w / sqrt(mean over the row of v^2 + eps)
 *   x         dtype [rows][hidden], or NULL: v = residual (a residual stream of its own type, without an addition)
 *   residual  residual_dtype [rows][hidden], or NULL: v = x
 *   weight    weight_dtype [hidden]
 *   h         residual_dtype [rows][hidden] or NULL; y dtype [rows][hidden] or NULL; codes and scales (8-bit rows of y) or
 *             both NULL; at least one of the three
 *   dtype     MEGA_MOE_BF16, _FP16 or _FP32; residual_dtype, weight_dtype: dtype or MEGA_MOE_FP32
 *   rows 0 .. MEGA_MOE_MAX_GROUP_ROWS (pointers may be NULL at 0), hidden 1 .. MEGA_MOE_MAX_NORM_COLS; eps >= 0, finite
 * v is fp32; y and the codes are computed from v, not from h, and rounded once each.  Without codes the squares and products
 * are fp32's (values from 1.8e19 on give y = 0); codes are those of the exact v w / sqrt(...), and y beside them is within
 * half a step of fp32 of it before its rounding, so that it may differ in its last bit from a call without codes.
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int32_t mega_moe_rms_norm(const void* x, const void* residual, const void* weight, void* h, void* y, uint8_t* codes, float* scales,
                          int64_t rows, int32_t hidden, float eps, int32_t dtype, int32_t residual_dtype, int32_t weight_dtype,
                          void* stream);

/* Its gradient: with r = 1 / sqrt(mean h^2 + eps), n = h r and g = dy w,
 *   dx = r (g - n mean(g n)) + dresidual,   dweight = sum over the rows of dy n
 * dx is the gradient of v, and so of x and of residual alike; dresidual is what reached h from elsewhere.
 *   dy         dtype [rows][hidden]
 *   h          residual_dtype [rows][hidden] with h_scales NULL, or codes with their h_scales (8-bit rows)
 *   dresidual  residual_dtype [rows][hidden] or NULL; dx residual_dtype [rows][hidden]; dweight float [hidden]
 *   workspace  mega_moe_norm_workspace_bytes() bytes, 4-byte aligned (may be NULL with rows 0); its contents do not matter
 * With rows 0 dweight is zeros.  Sums are fp32, dweight's in an order that depends on the sizes alone.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE_TOO_SMALL, HIP. */
int32_t mega_moe_norm_workspace_bytes(int64_t rows, int32_t hidden, uint64_t* bytes_out /* host */);
int32_t mega_moe_rms_norm_backward(const void* dy, const void* h, const float* h_scales, const void* weight, const void* dresidual,
                                   void* dx, float* dweight, int64_t rows, int32_t hidden, float eps, int32_t dtype,
                                   int32_t residual_dtype, int32_t weight_dtype, void* workspace, uint64_t workspace_bytes,
                                   void* stream);

/* ------------------------------------------------------------------ SwiGLU
 * Between the experts' two products: a row of gate_up is gate | up, inter columns each,
 *   act = gate / (1 + exp(-gate)) * up
 *   gate_up  dtype [rows][2 inter], act dtype [rows][inter]; dtype MEGA_MOE_BF16 or MEGA_MOE_FP16
 *   codes    uint8 [rows][2 inter] and scales float [rows][2][ceil(inter / 128)], or both NULL: gate_up in 8 bits for the
 *            backward pass; gate and up are 8-bit rows of their own
 *   offsets  int32 [groups + 1] as for the grouped products, or NULL (all rows): only rows offsets[0] .. offsets[groups]-1 are
 *            read and written; entries outside 0 .. rows are clamped and latch MEGA_MOE_STATUS_BAD_LAYOUT
 *   rows 0 .. MEGA_MOE_MAX_GROUP_ROWS (pointers may be NULL at 0), inter 1 .. MEGA_MOE_MAX_GROUP_COLS
 * backward, with s = 1 / (1 + exp(-gate)):
 *   dgate = dact up s (1 + gate (1 - s)),  dup = dact gate s  -> dgate_up dtype [rows][2 inter]
 *   gate_up  dtype [rows][2 inter] with scales NULL, or codes with their scales
 *   act      dtype [rows][inter] or NULL: act again, for the gradient of the second product's weights
 * Arithmetic is fp32, every output rounded once.
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int32_t mega_moe_swiglu(const void* gate_up, void* act, uint8_t* codes, float* scales, const int32_t* offsets, int32_t groups,
                        int64_t rows, int32_t inter, int32_t dtype, uint32_t* device_status, void* stream);
int32_t mega_moe_swiglu_backward(const void* dact, const void* gate_up, const float* scales, void* dgate_up, void* act,
                                 const int32_t* offsets, int32_t groups, int64_t rows, int32_t inter, int32_t dtype,
                                 uint32_t* device_status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MEGA_MOE_OPS_H */
