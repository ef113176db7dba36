// fp8_internal.h -- declarations shared by the FP8 entry points and kernels.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "gemm_fp8.h"
#include "gp_internal.h"

namespace gp {

constexpr int kFp8Group = 128;   // values along the summed axis that share a scale

inline int real_bytes(int type) { return type == GP_REAL_F32 ? 4 : 2; }

// Whether every chunk of 8 values of a matrix starts on a 16-byte boundary.
inline bool vec16(const void* p, int64_t ld, int elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem % 16 == 0;
}

// Launch as a programmatic dependent of the work before it in the stream: the
// kernel touches no memory before its pdl_wait().
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Each launcher fills *kernel with the function launched and plan's kernel, threads and grid.
cudaError_t launch_fp8_quantize(const void* x, int64_t ldx, int64_t rows, int64_t cols, int type,
                                const gp_fp8_matrix* q, const gp_fp8_matrix* qt, cudaStream_t stream,
                                const void** kernel, gp_plan* plan);

struct NormArgs {
  const void *x, *residual, *weight;
  void *h, *y;
  float* rstd;
  gp_fp8_matrix q;       // data NULL: not written
  int64_t ldx, ld_res, ld_h, ld_y;
  int64_t rows, cols;
  float eps, fmax;
  int32_t type, weight_type, e5m2;
  int32_t vec, vec_w;    // the matrices' and the weight's chunks of 8 values are 16-byte aligned
};
cudaError_t launch_fp8_rmsnorm(const NormArgs& a, int sm_count, cudaStream_t stream, const void** kernel, gp_plan* plan);

// p[0 .. n - 1] = value.
cudaError_t launch_fp8_fill_f32(float* p, int64_t n, float value, cudaStream_t stream);

struct NormGradArgs {
  const void *dy, *h, *dres, *weight;
  const float* rstd;
  void* dx;
  float* dw;             // the weight's gradient; NULL: not computed
  float* partials;       // parts x cols sums of it (NULL where parts is 0)
  int64_t ld_dy, ld_h, ld_dres, ld_dx;
  int64_t rows, cols;
  int32_t type, weight_type;
  int32_t vec, vec_w;
  int32_t col_blocks;    // blocks that work out dw by columns (the launcher's)
};
// Rows of partial sums that a call of this size leaves (workspace: that many x cols floats).
int64_t fp8_rmsnorm_backward_parts(int64_t rows, int64_t cols, int sm_count);
cudaError_t launch_fp8_rmsnorm_backward(const NormGradArgs& a, int sm_count, cudaStream_t stream, const void** kernel,
                                        gp_plan* plan);

struct Fp8GemmArgs {
  gp_fp8_matrix A, B;
  void* C;
  const void* addend;
  int64_t ldc, ld_add;
  int32_t M, N, K;
  int32_t out_type;
  gp_plan plan;
  cudaStream_t stream;
  KernelCtl ctl;
};
int fp8_plan_impl(int64_t M, int64_t N, int64_t K, int a_group, int b_group, int sms, const gp_fp8_options* opts,
                  gp_plan* p);
// Pairs must sit on one TPC each: where fewer fit at once than the plan counted on, launch those.
cudaError_t fp8_fit_pairs(gp_plan* plan);
cudaError_t launch_fp8_gemm(Fp8GemmArgs& a, const void** kernel);
// C = addend, or zeros (K == 0).
cudaError_t launch_fp8_fill(void* C, int64_t ldc, const void* addend, int64_t ld_add, int64_t M, int64_t N,
                            int out_type, cudaStream_t stream);

// ---------------------------------------------------------------------------
// the library's per-call state (api.cu)
// ---------------------------------------------------------------------------
struct CallInfo {
  int device;
  int sm_count;
  KernelCtl ctl;
};
// Start this thread's last-call record.
void call_reset(cudaStream_t stream);
// Device, SM count and status slot of a call that is about to launch.
cudaError_t call_begin(uint64_t timeout_ns, CallInfo* info);
// What the record shows of the launch.
void call_launched(const gp_plan& plan, const void* kernel);
// Close the record; returns `status`.  A CUDA error's site defaults to the launch, or what a helper noted.
int call_finish(int status, cudaError_t error = cudaSuccess, int site = 0);

}  // namespace gp
