/*
 * mega_moe_ops.h -- operators around the fused MoE layer of mega_moe.h, for one GPU (MI355X, gfx950):
 *   - products grouped by expert with ragged row counts, and their gradients (training the experts).
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

#define MEGA_MOE_MAX_GROUP_ROWS (1 << 26)   /* rows of a grouped product */
#define MEGA_MOE_MAX_GROUP_COLS 65536       /* its n and k */

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
 * backward_weight writes zeros for a group without rows (leaves it as it was when accumulating).
 * With rows == 0, forward and backward_rows do nothing and the row pointers may be NULL.
 * Errors: INVALID_ARG (null or misaligned pointer, negative size), UNSUPPORTED (size or type outside the
 * limits), HIP. */
int32_t mega_moe_grouped_forward(const void* x, const void* w, const int32_t* offsets, void* y, int64_t rows,
                                 int32_t n, int32_t k, int32_t groups, int32_t dtype, uint32_t* device_status,
                                 void* stream);
int32_t mega_moe_grouped_backward_rows(const void* dy, const void* w, const int32_t* offsets, void* dx,
                                       int64_t rows, int32_t n, int32_t k, int32_t groups, int32_t dtype,
                                       uint32_t* device_status, void* stream);
int32_t mega_moe_grouped_backward_weight(const void* dy, const void* x, const int32_t* offsets, void* dw,
                                         int64_t rows, int32_t n, int32_t k, int32_t groups, int32_t dtype,
                                         int32_t out_dtype, int32_t accumulate, uint32_t* device_status,
                                         void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MEGA_MOE_OPS_H */
