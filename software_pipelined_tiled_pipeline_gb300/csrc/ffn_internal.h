// ffn_internal.h -- declarations shared by the feed-forward entry points and kernels.
#pragma once
#include "fp8_internal.h"
#include "gemm_ffn.h"

namespace gp {

enum FfnOp { kFfnLinear = 0, kFfnGated = 1, kFfnInputGrad = 2, kFfnWeightGrad = 3 };

constexpr int kFfnBK = 64;             // summed axis per ring slot: 128 bytes of 16-bit values
constexpr int kFfnRestart = 12;        // K blocks between restarts of the accumulator where more than 16 bits leave
// The same where 16 bits leave: 4096 products in FP16, 32768 in BF16.  The tensor cores cut a sum by 2^-23 of its products'
// magnitudes at most per product (16 at once: 1.0e-7 on average with operands of one sign, 6.4e-9 a product), so this loses
// half a spacing of the output at most, and 2.6e-5 and 1.7e-4 were measured, a twentieth of that.  Without restarts FP16
// lost 8.4e-4 after 131072 products, always towards zero: more than its rounding (4.9e-4).  Held sums cost the ring a
// little: FP16 4096 x 4096 x 8192 163 -> 169 us.
constexpr int kFfnRestartF16 = 64, kFfnRestartBF16 = 512;
constexpr int64_t kFfnMaxTiles = int64_t(1) << 30;   // tile numbers plus a grid stay below 2^31

// 8-bit codes with a scale for each row's 128 values, as the kernels see them.
struct FfnCodes {
  uint8_t* data;         // NULL: none
  float* scales;
  int64_t ld, stride_row, stride_col;
};

// What becomes of a product's sums.  Index 1: the second weight of a gated
// product, or the second of two products in one launch.
struct FfnOut {
  void* out[2];
  const void* add[2];    // addend (residual), NULL: none
  const void* bias;
  void* keep[2];         // sums as they are, NULL: not kept
  FfnCodes codes[2];
  int64_t ld_out[2], ld_add[2], ld_keep[2];
  int32_t bf16;          // the 16-bit type
  int32_t out_f32;
  int32_t bias_f32;
  int32_t act;
  int32_t vec;           // rows of out, add and keep are on boundaries of 32 bytes (2), 16 (1), or neither (0)
};

// A product: out[r][c] = sum over s of a[r][s] * b[c][s].
struct FfnProduct {
  int32_t op;
  const void* a[2];      // second ones: input gradient (more of the summed axis), weight gradient (a second product)
  const void* b[2];      // ... input gradient, or the second weight of a gated product
  int64_t lda[2], ldb[2];
  int64_t rows, cols, summed;
  int32_t count;
  FfnOut out;
  gp_plan plan;
  cudaStream_t stream;
  KernelCtl ctl;
};

// K blocks that one accumulator takes.
inline int ffn_restart(bool wide, bool bf16) { return wide ? kFfnRestart : (bf16 ? kFfnRestartBF16 : kFfnRestartF16); }
int ffn_plan_impl(int op, int64_t rows, int64_t cols, int64_t summed, int count, bool wide_sums, bool codes, bool bf16, int sms,
                  const gp_ffn_options* opts, gp_plan* p);
// Pairs must sit on one TPC each: where fewer fit at once than the plan counted on, launch those.
cudaError_t ffn_fit_pairs(gp_plan* plan, bool whole_groups);
cudaError_t launch_ffn_linear(FfnProduct& a, const void** kernel);
cudaError_t launch_ffn_gated(FfnProduct& a, const void** kernel);
cudaError_t launch_ffn_input_grad(FfnProduct& a, const void** kernel);
cudaError_t launch_ffn_weight_grad(FfnProduct& a, const void** kernel);
cudaError_t launch_ffn_few(FfnProduct& a, const void** kernel);
// Ring depth, stage bytes and shared memory of the kernel that a plan of this tile runs.
void ffn_few_shape(gp_plan* p, int rows, bool gated);
int ffn_few_most_ctas(int rows);   // that may share a tile's K blocks

// ---------------------------------------------------------------------------
// element by element
// ---------------------------------------------------------------------------
struct FfnActArgs {
  const void* dy;
  const void* z[2];      // [1]: the second of a gated product
  FfnCodes codes[2];
  int32_t e5m2;          // format of the codes
  void* dz[2];
  void* h;
  float* dbias;
  float* partials;       // parts x N sums of it
  int64_t ld_dy, ldz[2], ld_dz[2], ldh;
  int64_t M, N;
  int32_t type, act;
  int32_t vec;
};
// Rows of partial sums of dbias that a call of this size leaves (1: none, it adds them up itself).
int64_t ffn_act_parts(int64_t M, int64_t N, int sm_count);
cudaError_t launch_ffn_act_backward(const FfnActArgs& a, int sm_count, cudaStream_t stream, const void** kernel, gp_plan* plan);
cudaError_t launch_ffn_gated_backward(const FfnActArgs& a, int sm_count, cudaStream_t stream, const void** kernel,
                                      gp_plan* plan);
cudaError_t launch_ffn_pack(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int64_t rows, int64_t cols,
                            cudaStream_t stream, const void** kernel, gp_plan* plan);

}  // namespace gp
