// fp8_api.cu -- the C ABI of the FP8 operators (include/gemm_fp8.h): argument
// checks and the per-thread last-call record.
#include <cstring>
#include <initializer_list>
#include <limits>

#include "fp8_internal.h"

namespace gp {
namespace {

bool real_ok(int type) { return type == GP_REAL_F16 || type == GP_REAL_BF16 || type == GP_REAL_F32; }

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

int check_sizes(int64_t a, int64_t b, int64_t c = 0) {
  if (a < 0 || b < 0 || c < 0) return GP_ERR_ARG;
  if (a > INT32_MAX || b > INT32_MAX || c > INT32_MAX) return GP_ERR_SIZE;
  return GP_OK;
}

// An 8-bit matrix with `cols` columns that the call reads or writes.
int check_fp8(const gp_fp8_matrix* m, int64_t cols) {
  if (!m || !m->data || !m->scales) return GP_ERR_ARG;
  if (m->format != GP_E4M3 && m->format != GP_E5M2) return GP_ERR_ARG;
  if (m->group != 1 && m->group != kFp8Group) return GP_ERR_ARG;
  if (m->ld < cols) return GP_ERR_ARG;
  if (!aligned(m->data, 16) || m->ld % 16 != 0 || !aligned(m->scales, 4)) return GP_ERR_UNSUPPORTED;
  return GP_OK;
}

// A row-major matrix of 16- or 32-bit values; p may be NULL where it is optional.
int check_real(const void* p, int64_t ld, int64_t cols, int type, bool optional) {
  if (!p) return optional ? GP_OK : GP_ERR_ARG;
  if (ld < cols) return GP_ERR_ARG;
  return aligned(p, real_bytes(type)) ? GP_OK : GP_ERR_UNSUPPORTED;
}

constexpr int64_t kMaxGemm = INT32_MAX - 255;        // a size rounded up to whole tiles stays below 2^31
constexpr int64_t kMaxNormCols = int64_t(1) << 30;   // column numbers plus a step stay below 2^31

int first_error(std::initializer_list<int> codes) {
  for (int c : codes)
    if (c != GP_OK) return c;
  return GP_OK;
}

int current_sms() {
  int ndev = 0, dev = 0, sms = 0;
  if (cudaGetDeviceCount(&ndev) == cudaSuccess && ndev > 0) {
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  } else {
    cudaGetLastError();   // clear the "no device" error of the probe
  }
  return sms;
}

int check_gemm(const gp_fp8_matrix* A, const gp_fp8_matrix* B, const void* C, int64_t ldc, const void* addend,
               int64_t ld_add, int64_t M, int64_t N, int64_t K, int out_type) {
  if (K > 0) {
    const int rc = first_error({check_fp8(A, K), check_fp8(B, K)});
    if (rc != GP_OK) return rc;
  }
  return first_error({check_real(C, ldc, N, out_type, false), check_real(addend, ld_add, N, out_type, true)});
}

}  // namespace
}  // namespace gp

using namespace gp;

extern "C" {

int gemm_fp8_plan(int64_t M, int64_t N, int64_t K, int a_group, int b_group, int sms, const gp_fp8_options* opts,
                  gp_plan* out) {
  if (!out || sms < 0) return GP_ERR_ARG;
  if ((a_group != 1 && a_group != kFp8Group) || (b_group != 1 && b_group != kFp8Group)) return GP_ERR_ARG;
  int rc = check_sizes(M, N, K);
  if (rc == GP_OK && (M > kMaxGemm || N > kMaxGemm || K > kMaxGemm)) rc = GP_ERR_SIZE;
  if (rc != GP_OK) return rc;
  return fp8_plan_impl(M, N, K, a_group, b_group, sms > 0 ? sms : current_sms(), opts, out);
}

int gemm_fp8(const gp_fp8_matrix* A, const gp_fp8_matrix* B, void* C, int64_t ldc, const void* addend, int64_t ld_add,
             int64_t M, int64_t N, int64_t K, int out_type, void* stream, const gp_fp8_options* opts) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st);
  int rc = check_sizes(M, N, K);
  if (rc == GP_OK && (M > kMaxGemm || N > kMaxGemm || K > kMaxGemm)) rc = GP_ERR_SIZE;
  if (rc == GP_OK && !real_ok(out_type)) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (M == 0 || N == 0) return call_finish(GP_OK);
  rc = check_gemm(A, B, C, ldc, addend, ld_add, M, N, K, out_type);
  if (rc != GP_OK) return call_finish(rc);
  gp_plan plan;
  if (K > 0) {
    rc = fp8_plan_impl(M, N, K, A->group, B->group, 0, opts, &plan);   // what needs no device
    if (rc != GP_OK) return call_finish(rc);
  }
  CallInfo info;
  cudaError_t e = call_begin(opts ? opts->timeout_ns : 0, &info);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
  if (K == 0) {
    e = launch_fp8_fill(C, ldc, addend, ld_add, M, N, out_type, st);
    return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
  }
  Fp8GemmArgs a = {};
  rc = fp8_plan_impl(M, N, K, A->group, B->group, info.sm_count, opts, &a.plan);
  if (rc != GP_OK) return call_finish(rc);
  e = fp8_fit_pairs(&a.plan);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_CAPACITY);
  a.A = *A;
  a.B = *B;
  a.C = C;
  a.addend = addend;
  a.ldc = ldc;
  a.ld_add = ld_add;
  a.M = static_cast<int32_t>(M);
  a.N = static_cast<int32_t>(N);
  a.K = static_cast<int32_t>(K);
  a.out_type = out_type;
  a.stream = st;
  a.ctl = info.ctl;
  a.ctl.inject_lost_load = opts ? opts->inject_lost_load : 0;
  const void* kernel = nullptr;
  e = launch_fp8_gemm(a, &kernel);
  call_launched(a.plan, kernel);
  return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
}

int fp8_quantize(const void* x, int64_t ldx, int64_t rows, int64_t cols, int type, const gp_fp8_matrix* q,
                 const gp_fp8_matrix* qt, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st);
  int rc = check_sizes(rows, cols);
  if (rc == GP_OK && (!real_ok(type) || (!q && !qt))) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (rows == 0 || cols == 0) return call_finish(GP_OK);
  rc = first_error({check_real(x, ldx, cols, type, false), q ? check_fp8(q, cols) : GP_OK,
                    qt ? check_fp8(qt, rows) : GP_OK});
  if (rc == GP_OK && q && qt && (q->format != qt->format || q->group != qt->group)) rc = GP_ERR_ARG;
  if (rc == GP_OK && ((rows + 127) / 128) * ((cols + 127) / 128) > INT32_MAX) rc = GP_ERR_SIZE;
  if (rc != GP_OK) return call_finish(rc);
  CallInfo info;
  cudaError_t e = call_begin(0, &info);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
  gp_plan plan = {};
  const void* kernel = nullptr;
  e = launch_fp8_quantize(x, ldx, rows, cols, type, q, qt, st, &kernel, &plan);
  call_launched(plan, kernel);
  return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
}

int fp8_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ld_res, const void* weight, int weight_type,
                float eps, int64_t rows, int64_t cols, int type, void* h_out, int64_t ld_h, float* rstd, void* y_out,
                int64_t ld_y, const gp_fp8_matrix* q, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st);
  int rc = check_sizes(rows, cols);
  if (rc == GP_OK && cols > kMaxNormCols) rc = GP_ERR_SIZE;
  if (rc == GP_OK && (!real_ok(type) || !real_ok(weight_type) || !(eps >= 0.f))) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (rows == 0 || (cols == 0 && !rstd)) return call_finish(GP_OK);
  if (cols == 0) {
    // the mean of no values is NaN
    if (!aligned(rstd, 4)) return call_finish(GP_ERR_UNSUPPORTED);
    CallInfo info;
    cudaError_t e = call_begin(0, &info);
    if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
    e = launch_fp8_fill_f32(rstd, rows, std::numeric_limits<float>::quiet_NaN(), st);
    return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
  }
  rc = first_error({check_real(x, ldx, cols, type, false), check_real(residual, ld_res, cols, type, true),
                    check_real(weight, cols, cols, weight_type, false), check_real(h_out, ld_h, cols, type, true),
                    check_real(y_out, ld_y, cols, type, true), q ? check_fp8(q, cols) : GP_OK,
                    aligned(rstd, 4) ? GP_OK : GP_ERR_UNSUPPORTED});
  if (rc == GP_OK && q && q->group != 1) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  CallInfo info;
  cudaError_t e = call_begin(0, &info);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.h = h_out;
  a.y = y_out;
  a.rstd = rstd;
  if (q) a.q = *q;
  a.ldx = ldx;
  a.ld_res = ld_res;
  a.ld_h = ld_h;
  a.ld_y = ld_y;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  a.type = type;
  a.weight_type = weight_type;
  a.e5m2 = q && q->format == GP_E5M2;
  a.fmax = a.e5m2 ? 57344.f : 448.f;
  const int w = real_bytes(type);
  a.vec = vec16(x, ldx, w) && (!residual || vec16(residual, ld_res, w)) && (!h_out || vec16(h_out, ld_h, w)) &&
          (!y_out || vec16(y_out, ld_y, w));
  a.vec_w = aligned(weight, 16);
  gp_plan plan = {};
  const void* kernel = nullptr;
  e = launch_fp8_rmsnorm(a, info.sm_count, st, &kernel, &plan);
  call_launched(plan, kernel);
  return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
}

int fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int sms, int64_t* bytes) {
  if (!bytes || sms < 0) return GP_ERR_ARG;
  const int rc = check_sizes(rows, cols);
  if (rc != GP_OK) return rc;
  if (cols > kMaxNormCols) return GP_ERR_SIZE;
  if (sms == 0) sms = current_sms();
  *bytes = rows == 0 || cols == 0 ? 0 : fp8_rmsnorm_backward_parts(rows, cols, sms > 0 ? sms : 152) * cols * 4;
  return GP_OK;
}

int fp8_rmsnorm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const void* dres, int64_t ld_dres,
                         const void* weight, int weight_type, const float* rstd, int64_t rows, int64_t cols, int type,
                         void* dx, int64_t ld_dx, float* dw, void* workspace, int64_t workspace_bytes, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st);
  int rc = check_sizes(rows, cols);
  if (rc == GP_OK && cols > kMaxNormCols) rc = GP_ERR_SIZE;
  if (rc == GP_OK && (!real_ok(type) || !real_ok(weight_type))) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (cols == 0 || (rows == 0 && !dw)) return call_finish(GP_OK);
  if (rows > 0)
    rc = first_error({check_real(dy, ld_dy, cols, type, false), check_real(h, ld_h, cols, type, false),
                      check_real(dres, ld_dres, cols, type, true), check_real(weight, cols, cols, weight_type, false),
                      check_real(rstd, 1, 1, GP_REAL_F32, false), check_real(dx, ld_dx, cols, type, false)});
  const bool parts = dw && rows > 0 && fp8_rmsnorm_backward_parts(rows, cols, 1) > 0;   // (whether, not how many)
  if (rc == GP_OK && parts && !workspace) rc = GP_ERR_ARG;
  if (rc == GP_OK && !(aligned(dw, 4) && aligned(workspace, 16))) rc = GP_ERR_UNSUPPORTED;
  if (rc != GP_OK) return call_finish(rc);
  CallInfo info;
  cudaError_t e = call_begin(0, &info);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
  NormGradArgs a = {};
  a.dy = dy;
  a.h = h;
  a.dres = dres;
  a.weight = weight;
  a.rstd = rstd;
  a.dx = dx;
  a.dw = dw;
  a.ld_dy = ld_dy;
  a.ld_h = ld_h;
  a.ld_dres = ld_dres;
  a.ld_dx = ld_dx;
  a.rows = rows;
  a.cols = cols;
  a.type = type;
  a.weight_type = weight_type;
  const int w = real_bytes(type);
  a.vec = vec16(dy, ld_dy, w) && vec16(h, ld_h, w) && (!dres || vec16(dres, ld_dres, w)) && vec16(dx, ld_dx, w);
  a.vec_w = aligned(weight, 16);
  gp_plan plan = {};
  if (parts) {
    plan.workspace_bytes = fp8_rmsnorm_backward_parts(rows, cols, info.sm_count) * cols * 4;
    if (workspace_bytes < plan.workspace_bytes) return call_finish(GP_ERR_ARG);
    a.partials = static_cast<float*>(workspace);
  }
  const void* kernel = nullptr;
  e = launch_fp8_rmsnorm_backward(a, info.sm_count, st, &kernel, &plan);
  call_launched(plan, kernel);
  return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
}

}  // extern "C"
