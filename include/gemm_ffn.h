/*
 * gemm_ffn.h -- C ABI of the feed-forward operators in 16 bits: a product with
 * bias, activation and residual in its epilogue, the gated product of two
 * weights in one kernel, what their backward pass needs kept in the inputs'
 * type or in 8 bits, and the gradients.
 *
 * Conventions are those of gemm_pipelined.h and gemm_fp8.h: device pointers
 * owned by the caller, calls asynchronous on the caller's stream, argument
 * errors found on the host before anything is launched (the outputs are then
 * untouched), the return codes GP_OK and GP_ERR_*, and the per-thread record of
 * the last call read by gemm_stats().  The kernels are launched as programmatic
 * dependents of the work before them, and touch memory only once it has
 * completed.  None of these calls allocates; the one that needs a workspace
 * takes it from the caller, so calls may be captured in a graph (once one call
 * on the device has let the library load its code).  Results do not depend on
 * timing: partial sums meet in a fixed order.
 *
 * Matrices are row-major with `ld` elements between rows.  `type` is GP_REAL_F16
 * or GP_REAL_BF16; an output type is `type` or GP_REAL_F32.  Operands of a
 * product (x, weights, dz) begin their rows on 16-byte boundaries: pointers
 * 16-byte aligned, ld a multiple of 8 (ffn_pack_rows lays out others); columns
 * may be any number.  Other matrices need the alignment of their elements only,
 * and are faster with rows on 16-byte boundaries.
 *
 * Products are summed in FP32 by the tensor cores, which cut instead of
 * rounding.  That sum is restarted, and the parts are added in FP32, every 768 of
 * the summed axis where an output is FP32, or 8-bit codes with FP32 scales; else
 * every 4096 (FP16) or 32768 (BF16), so that what is cut stays below the
 * output's own rounding.
 * Everything up to an output's one rounding is FP32.
 * Outputs do not overlap operands, except where it says so.
 *
 * Activations (act'(0) of relu is 0):
 *     relu = max(z, 0)     gelu = z Phi(z)     silu = z sigmoid(z)     sigmoid = 1 / (1 + exp(-z))
 *     gelu_tanh = z sigmoid(2 sqrt(2 / pi) (z + 0.044715 z^3))   ( = z/2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) )
 *
 * They are formed from ex2.approx and rcp.approx: off by up to 1e-6 relative for
 * z > -3, and by 1e-5 in the tail towards -12 (gelu_tanh 8.5e-6, gelu 3.4e-6,
 * silu and sigmoid 8e-7 measured); below 2^-126 they are 0.
 *
 * Values kept for the backward pass are those before the activation, either
 * rounded to `type`, or in 8 bits as fp8_quantize would make them of the FP32
 * values: E4M3 codes with one FP32 scale for each row's 128 values (group 1).
 */
#ifndef GEMM_FFN_H
#define GEMM_FFN_H

#include <stdint.h>

#include "gemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GP_ACT_NONE = 0,
    GP_ACT_RELU = 1,
    GP_ACT_GELU = 2,
    GP_ACT_GELU_TANH = 3,
    GP_ACT_SILU = 4,
    GP_ACT_SIGMOID = 5
} gp_activation;

/* gp_plan.dtype of these calls as gemm_stats() reports it. */
#define GP_PLAN_FFN 17

/* Options of the products.  Zero-initialise and set what you need; NULL: all zero. */
typedef struct gp_ffn_options {
    uint64_t timeout_ns;         /* limit of every bounded wait inside the kernel (0 = 1 s) */
    int32_t tile;                /* force the tile: 256 (256 x 256 of two CTAs), 128 (128 x 128), or so many rows of the
                                    output x 128 columns by a cluster that may share the K loop: 16, 32, 64 (gemm_gated
                                    up to here, gemm_weight_grad from here on) or 129 (128 rows); these not where values
                                    are kept in 8 bits.  0 = the planner's choice.  Other values, and tiles that the
                                    call does not have: GP_ERR_UNSUPPORTED */
    int32_t k_splits;            /* tiles of a cluster: the CTAs that share a tile's K loop, 1, 2, 4 or 8 (at most 4
                                    with 16); 0 = the planner's choice.  Others: GP_ERR_UNSUPPORTED.  The tiles of 128
                                    x 128 and 256 x 256 do not look at it, whether forced or the planner's choice */
    int32_t inject_lost_load;    /* test hook: the TMA producer skips the last tile load of the problem, so a consumer
                                    wait runs out and the call reports GP_ERR_TIMEOUT (no GPU fault); not with tile 256
                                    (GP_ERR_UNSUPPORTED), and the planner does not choose that then */
    int32_t continues;           /* 1: gemm_stats() speaks of this call and the one before it by this thread (on the same
                                    device and stream) together: a wait that gave up in either is GP_ERR_TIMEOUT, the
                                    rest of the record is this call's.  Several calls may go on so */
} gp_ffn_options;

/*
 * gemm_linear -- z = x W^T + bias, y = act(z) + residual.
 */
typedef struct gp_linear {
    const void* x;               /* M x K */
    const void* weight;          /* N x K */
    const void* bias;            /* N values of bias_type; NULL: none */
    const void* residual;        /* M x N of out_type, added in FP32 before the rounding; NULL: none.  May be y itself
                                    (same pointer and ld), not overlap it otherwise */
    void* y;                     /* M x N of out_type */
    void* z;                     /* NULL, or M x N of `type`: z kept as it is */
    gp_fp8_matrix q;             /* data NULL, or M x N: z kept in 8 bits (E4M3, group 1).  z or q, not both */
    int64_t M, N, K;
    int64_t ldx, ldw, ld_res, ldy, ldz;
    int32_t type, out_type, bias_type, activation;
} gp_linear;

/*
 * M == 0 or N == 0: nothing is launched.  K == 0: z = bias, or zeros.
 * GP_ERR_ARG: NULL x or weight with K > 0, NULL y, bad enums, an ld below the
 * columns, both z and q, a q that is not E4M3 with group 1, a negative size.
 * GP_ERR_UNSUPPORTED: x or weight off 16-byte boundaries (see above), q not
 * 16-byte aligned or with ld % 16 != 0, others not aligned to their element.
 * GP_ERR_SIZE: a size above 2^31 - 256, or more than 2^30 output tiles.  After
 * GP_ERR_TIMEOUT the outputs are incomplete: tiles whose K loop did not come to
 * its end are not written.  (All of this holds for the other products too.)
 */
int gemm_linear(const gp_linear* args, void* stream, const gp_ffn_options* opts);

/*
 * gemm_gated -- g = x Wg^T, u = x Wu^T, h = act(g) * u, in one kernel.
 */
typedef struct gp_gated {
    const void* x;               /* M x K */
    const void* gate;            /* N x K */
    const void* up;              /* N x K */
    void* h;                     /* M x N of `type` */
    void *z_gate, *z_up;         /* NULL both, or M x N of `type`: g and u kept as they are */
    gp_fp8_matrix q_gate, q_up;  /* data NULL both, or M x N: g and u kept in 8 bits.  Not with z_gate, z_up */
    int64_t M, N, K;
    int64_t ldx, ld_gate, ld_up, ldh, ld_zg, ld_zu;
    int32_t type, activation;
} gp_gated;

int gemm_gated(const gp_gated* args, void* stream, const gp_ffn_options* opts);

/*
 * gemm_input_grad -- dx = dz_0 W_0 (+ dz_1 W_1): the gradient that a product x W^T, or a pair of them, sends to x.
 */
typedef struct gp_input_grad {
    const void* dz[2];           /* M x N */
    const void* weight[2];       /* N x K */
    void* dx;                    /* M x K of out_type */
    int64_t M, N, K;
    int64_t ld_dz[2], ldw[2], ld_dx;
    int32_t type, out_type;
    int32_t count;               /* 1 or 2 */
    int32_t reserved;
} gp_input_grad;

/* N == 0: dx is zeros. */
int gemm_input_grad(const gp_input_grad* args, void* stream, const gp_ffn_options* opts);

/*
 * gemm_weight_grad -- dw_i = dz_i^T x (+ addend_i), i < count: the gradients of the weights of products that share x.
 */
typedef struct gp_weight_grad {
    const void* dz[2];           /* M x N */
    const void* x;               /* M x K */
    const void* addend[2];       /* N x K of out_type, added in FP32 before the rounding, NULL: none (both or neither
                                    of two).  May be dw_i itself, not overlap it otherwise */
    void* dw[2];                 /* N x K of out_type; not the same one twice (GP_ERR_ARG) */
    int64_t M, N, K;
    int64_t ld_dz[2], ldx, ld_add[2], ld_dw[2];
    int32_t type, out_type;
    int32_t count;
    int32_t reserved;
} gp_weight_grad;

/* M == 0: dw_i = addend_i, or zeros. */
int gemm_weight_grad(const gp_weight_grad* args, void* stream, const gp_ffn_options* opts);

/*
 * gemm_ffn_plan -- the kernel and tile that a call would choose on a device with `sms` SMs (0: the current device;
 * without one, as on 152 SMs with gp_plan.grid left 0).  op: 0 gemm_linear, 1 gemm_gated, 2 gemm_input_grad,
 * 3 gemm_weight_grad; M, N, K and count as in that call; kept: the sum of 1 where values are kept in 8 bits (gradients:
 * FP32 is written), 2 where FP32 is written, 4 where the type is GP_REAL_F16 (gemm_gated: not 2; others: GP_ERR_ARG).
 * gp_plan.bm x bn is the tile (where layout is 1, bm counts columns of the output and bn rows); k_splits CTAs, one cluster,
 * share each tile's K loop; the last half_tiles tiles (after dp_tiles whole ones) run as two halves of their columns each.
 */
int gemm_ffn_plan(int op, int64_t M, int64_t N, int64_t K, int count, int kept, int sms, const gp_ffn_options* opts,
                  gp_plan* out);

/*
 * ffn_act_backward -- dz = dy * act'(z), rounded once to `type`, and dbias = sum over rows of dy * act'(z) in FP32.
 */
typedef struct gp_act_backward {
    const void* dy;              /* M x N */
    const void* z;               /* M x N of `type`, or NULL */
    gp_fp8_matrix q;             /* or z in 8 bits (group 1, either format); data NULL: not.  With GP_ACT_NONE neither */
    void* dz;                    /* M x N of `type` (may be dy itself); NULL: not written */
    float* dbias;                /* N values; NULL: not computed */
    void* workspace;             /* 16-byte aligned, ffn_act_backward_workspace() bytes at least; the call's own until it
                                    has run.  NULL where that is 0, and without dbias */
    int64_t workspace_bytes;
    int64_t M, N;
    int64_t ld_dy, ldz, ld_dz;
    int32_t type, activation;
} gp_act_backward;

/* M == 0: dbias is zeros.  GP_ERR_ARG: a workspace that is too small; neither or both of z and q (with GP_ACT_NONE: any). */
int ffn_act_backward(const gp_act_backward* args, void* stream);
int ffn_act_backward_workspace(int64_t M, int64_t N, int sms, int64_t* bytes);

/*
 * ffn_gated_backward -- of h = act(g) * u:  dg = dh * u * act'(g),  du = dh * act(g), and h once more.
 */
typedef struct gp_gated_backward {
    const void* dh;              /* M x N */
    const void *z_gate, *z_up;   /* g and u of `type`, or NULL both */
    gp_fp8_matrix q_gate, q_up;  /* or both in 8 bits (group 1) */
    void *dgate, *dup;           /* M x N of `type` (one of them may be dh itself; not the same one twice: GP_ERR_ARG) */
    void* h;                     /* M x N of `type`; NULL: not written */
    int64_t M, N;
    int64_t ld_dh, ld_zg, ld_zu, ld_dgate, ld_dup, ldh;
    int32_t type, activation;
} gp_gated_backward;

int ffn_gated_backward(const gp_gated_backward* args, void* stream);

/* ffn_pack_rows -- copies a rows x cols matrix of 16-bit elements (ld_src between rows) to one whose rows begin on
 * 16-byte boundaries (dst 16-byte aligned, ld_dst a multiple of 8, both as the products want them). */
int ffn_pack_rows(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int64_t rows, int64_t cols, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_FFN_H */
