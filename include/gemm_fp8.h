/*
 * gemm_fp8.h -- C ABI of the 8-bit floating-point operators of the GEMM
 * library: quantisation with one FP32 scale for each 128 values along the
 * summed axis, the matrix product of two such matrices, and the RMS norm that
 * feeds it with its gradient.
 *
 * Conventions are those of gemm_pipelined.h: device pointers owned by the
 * caller, calls asynchronous on the caller's stream, argument errors found on
 * the host before anything is launched (the outputs are then untouched), the
 * return codes GP_OK and GP_ERR_*, and the per-thread record of the last call
 * read by gemm_stats().  The kernels are launched as programmatic dependents
 * of the work before them, and touch memory only once it has completed.
 * The norm's gradient keeps partial sums in a workspace that the caller
 * passes, and no other call needs one: none allocates, and calls may be captured
 * in a graph (once one call on the device has let the library load its code).
 * Results do not depend on timing: partial sums meet in a fixed order.
 *
 * 8-bit matrices
 * --------------
 * A matrix of `rows` x `cols` stores element (r, c) as the 8-bit code at
 * data[r * ld + c], ld a multiple of 16 and data 16-byte aligned, so that rows
 * begin on 16-byte boundaries (cols itself may be any number).  The value it
 * stands for is
 *     code(r, c) * scales[(r / group) * stride_row + (c / 128) * stride_col]
 * with group 1 (a scale for each row's 128 values: activations, gradients) or
 * 128 (a scale for each 128 x 128 block: weights).  The last group of a row
 * or column may be shorter.  Scales are FP32, in any element strides.
 *
 * Quantisation of a group with largest magnitude amax:
 *     scale = max(amax / FMAX, 2^-64)          FMAX: 448 (E4M3), 57344 (E5M2)
 *     code  = round_to_nearest_even(x * (1 / scale)), saturated at +-FMAX
 * in FP32.  A group of zeros has the scale 2^-64 and codes of zero.  A group
 * that holds a NaN has a NaN scale and NaN codes; one that holds an infinity
 * (and no NaN) has an infinite scale, NaN for the infinity (E4M3 has none) and
 * zeros elsewhere: what follows sees NaN in every result that the group takes
 * part in, in both cases.
 */
#ifndef GEMM_FP8_H
#define GEMM_FP8_H

#include <stdint.h>

#include "gemm_pipelined.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit formats. */
typedef enum {
    GP_E4M3 = 0, /* 4 exponent and 3 mantissa bits, no infinities, largest 448 */
    GP_E5M2 = 1  /* 5 exponent and 2 mantissa bits, largest 57344 (gradients) */
} gp_fp8_format;

/* Types of unquantised matrices and vectors. */
typedef enum {
    GP_REAL_F16 = 0,
    GP_REAL_BF16 = 1,
    GP_REAL_F32 = 2
} gp_real;

/* gp_plan.dtype of a gemm_fp8 call as gemm_stats() reports it (gemm_pipelined takes no such type). */
#define GP_PLAN_FP8 16

/* One 8-bit matrix with its scales (see above).  Inputs are not written. */
typedef struct gp_fp8_matrix {
    void* data;
    float* scales;
    int64_t ld;                  /* elements (= bytes) between rows, a multiple of 16 */
    int64_t stride_row;          /* elements between the scales of neighbouring row groups */
    int64_t stride_col;          /* elements between the scales of neighbouring groups of 128 columns */
    int32_t format;              /* gp_fp8_format */
    int32_t group;               /* rows that share a scale: 1 or 128 */
} gp_fp8_matrix;

/* Options of gemm_fp8.  Zero-initialise and set what you need. */
typedef struct gp_fp8_options {
    uint64_t timeout_ns;         /* limit of every bounded wait inside the kernel (0 = 1 s; waits of the K loop count
                                    with a 32-bit clock, and give up after 4 s where it is longer) */
    int32_t bn;                  /* force the tile width on the tensor cores' N side: 16, 32, 64, 128 or 256 (0 = the
                                    planner's choice; other values, and 256 on one SM: GP_ERR_UNSUPPORTED) */
    int32_t no_split;            /* 1: never share a tile's K loop among CTAs */
    int32_t inject_lost_load;    /* test hook: the TMA producer skips the last tile load of the problem (2: the first),
                                    so a consumer wait runs out and the call reports GP_ERR_TIMEOUT (no GPU fault); not
                                    with bn 256 (GP_ERR_UNSUPPORTED), whose tiles two CTAs share */
} gp_fp8_options;

/*
 * gemm_fp8 -- C = A x B^T (+ addend).
 *   A        M x K, B: N x K, 8-bit matrices as above (each with its own format and group).
 *   C        row-major M x N of type out_type (gp_real), ldc elements between rows.
 *   addend   NULL, or a row-major M x N matrix of type out_type with ld_add elements between rows, added in FP32
 *            before the one rounding to out_type; may be C itself (same pointer and ld), not overlap it otherwise.
 * Products of 128 along K are summed by the tensor cores in FP32, scaled by
 * the product of the two scales (formed in FP32: where that overflows, so does
 * the result) and added to FP32 sums.
 * M == 0 or N == 0: nothing is launched.  K == 0: C = addend, or zeros.
 * After GP_ERR_TIMEOUT, C is incomplete: a tile whose K loop did not come to its
 * end is not written, and which these are is not reported.
 * GP_ERR_ARG: NULL A, B or scales with K > 0, NULL C, bad enums, group not 1
 * or 128, an ld below the columns (K, or N for C and addend), a negative size.
 * GP_ERR_UNSUPPORTED: an 8-bit matrix not 16-byte aligned or with ld % 16 != 0;
 * C, addend or scales not aligned to their element.  GP_ERR_SIZE: a size above
 * 2^31 - 256, or more than 2^30 output tiles.
 */
int gemm_fp8(const gp_fp8_matrix* A, const gp_fp8_matrix* B, void* C, int64_t ldc, const void* addend,
             int64_t ld_add, int64_t M, int64_t N, int64_t K, int out_type, void* stream,
             const gp_fp8_options* opts);

/*
 * gemm_fp8_plan -- the tile, ring and split that gemm_fp8 would choose for
 * a_group x b_group scales on a device with `sms` SMs (0: the current device;
 * without one, as on 152 SMs with gp_plan.grid left 0).  gp_plan.bm counts the
 * rows of the operand that fills the tensor cores' M side, bn those of the
 * other; gp_plan.layout is 1 where that operand is B (the roles are swapped);
 * gp_plan.k_splits CTAs, one cluster, share each tile's K loop.
 */
int gemm_fp8_plan(int64_t M, int64_t N, int64_t K, int a_group, int b_group, int sms, const gp_fp8_options* opts,
                  gp_plan* out);

/*
 * fp8_quantize -- the 8-bit matrix q of x, and/or qt of its transpose.
 *   x      row-major rows x cols of type `type`, ldx elements between rows.
 *   q      NULL, or the rows x cols matrix to write (data, scales, format, group, ld, strides set by the caller).
 *   qt     NULL, or the cols x rows matrix to write: the transpose, quantised along x's columns (groups of 128
 *          rows of x).  q and qt have the same format and group; with group 128 both hold the same codes and
 *          scales, transposed.
 * One pass over x.  rows == 0 or cols == 0: nothing is launched.  Bytes between
 * the columns and ld are not written.
 */
int fp8_quantize(const void* x, int64_t ldx, int64_t rows, int64_t cols, int type, const gp_fp8_matrix* q,
                 const gp_fp8_matrix* qt, void* stream);

/*
 * fp8_rmsnorm -- residual addition, RMS norm and quantisation.
 *     h    = x + residual, rounded to `type` (x itself without a residual)
 *     rstd = 1 / sqrt(mean(h^2) + eps)        over the row, in FP32
 *     y    = h * rstd * weight                in FP32
 *     q    = y in 8 bits, group 1
 *   x, residual (or NULL), h, y: row-major rows x cols of type `type`.
 *   weight  cols values of type weight_type.
 *   h_out   the sum (NULL: not written; may be x or residual itself).
 *   rstd    rows FP32 values (NULL: not written).
 *   y_out   y rounded to `type` (NULL: not written).
 *   q       NULL, or the 8-bit matrix to write (group 1).
 * The norm is of the rounded h, so that the gradient computed from the stored
 * h is that of the function that ran.  rows == 0: nothing is launched.  cols == 0:
rstd is filled with NaN (the mean of no values).
 * GP_ERR_SIZE: rows of 2^31 or more, cols above 2^30 (here and in the gradient).
 */
int fp8_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ld_res, const void* weight, int weight_type,
                float eps, int64_t rows, int64_t cols, int type, void* h_out, int64_t ld_h, float* rstd, void* y_out,
                int64_t ld_y, const gp_fp8_matrix* q, void* stream);

/*
 * fp8_rmsnorm_backward -- gradient of y = h * rstd * weight.
 *     g  = dy * weight
 *     dx = rstd * (g - h * rstd * mean(g * h * rstd)) (+ dres)      rounded once to `type`
 *     dw = sum over rows of dy * h * rstd                           FP32
 *   dy, h, dres (or NULL: the gradient that reaches h past the norm) and dx: row-major rows x cols of type `type`.
 *   dx is the gradient of h, so of x and of residual; it may be dy, h or dres itself.
 *   rstd    rows FP32 values, as fp8_rmsnorm stored them.
 *   dw      cols FP32 values, written (not added to); NULL: not computed.  With rows == 0 it is filled with zeros.
 *   workspace  16-byte aligned, workspace_bytes at least what fp8_rmsnorm_backward_workspace says for this device
 *           (else GP_ERR_ARG): the call's own until it has run.  Where that is 0 (few rows), and without dw, NULL does.
 */
int fp8_rmsnorm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const void* dres, int64_t ld_dres,
                         const void* weight, int weight_type, const float* rstd, int64_t rows, int64_t cols, int type,
                         void* dx, int64_t ld_dx, float* dw, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace of a call with dw on a device with `sms` SMs (0: the current device; without one, as on 152 SMs). */
int fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int sms, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_FP8_H */
