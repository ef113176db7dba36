// ffn_api.cu -- the C ABI of the feed-forward operators (include/gemm_ffn.h):
// argument checks and the per-thread last-call record.
#include <cstring>
#include <initializer_list>

#include "ffn_internal.h"

namespace gp {
namespace {

constexpr int64_t kMaxSize = INT32_MAX - 255;        // a size rounded up to whole tiles stays below 2^31

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

int first_error(std::initializer_list<int> codes) {
  for (int c : codes)
    if (c != GP_OK) return c;
  return GP_OK;
}

int check_sizes(int64_t a, int64_t b, int64_t c = 0) {
  if (a < 0 || b < 0 || c < 0) return GP_ERR_ARG;
  return a > kMaxSize || b > kMaxSize || c > kMaxSize ? GP_ERR_SIZE : GP_OK;
}

bool type_ok(int type) { return type == GP_REAL_F16 || type == GP_REAL_BF16; }
bool out_ok(int type, int out) { return out == type || out == GP_REAL_F32; }
bool act_ok(int act) { return act >= GP_ACT_NONE && act <= GP_ACT_SIGMOID; }

// An operand of a product: rows on 16-byte boundaries.
int check_operand(const void* p, int64_t ld, int64_t cols) {
  if (!p || ld < cols) return GP_ERR_ARG;
  return aligned(p, 16) && ld % 8 == 0 ? GP_OK : GP_ERR_UNSUPPORTED;
}

// Any other matrix; p may be NULL where it is optional.
int check_real(const void* p, int64_t ld, int64_t cols, int type, bool optional) {
  if (!p) return optional ? GP_OK : GP_ERR_ARG;
  if (ld < cols) return GP_ERR_ARG;
  return aligned(p, real_bytes(type)) ? GP_OK : GP_ERR_UNSUPPORTED;
}

// An 8-bit matrix with a scale for each row's 128 values; data NULL: none.
int check_codes(const gp_fp8_matrix& m, int64_t cols, bool e5m2) {
  if (!m.data) return GP_OK;
  if (!m.scales || m.ld < cols || m.group != 1) return GP_ERR_ARG;
  if (m.format != GP_E4M3 && !(e5m2 && m.format == GP_E5M2)) return GP_ERR_ARG;
  return aligned(m.data, 16) && m.ld % 16 == 0 && aligned(m.scales, 4) ? GP_OK : GP_ERR_UNSUPPORTED;
}

// Boundaries that the rows of a matrix begin on: 32 bytes (2), 16 (1), or neither; one that is not there, on any.
int align_of(const void* p, int64_t ld, int type) {
  if (!p) return 2;
  const int64_t at = reinterpret_cast<intptr_t>(p) | (ld * real_bytes(type));
  return at % 32 == 0 ? 2 : (at % 16 == 0 ? 1 : 0);
}

int least(std::initializer_list<int> v) {
  int m = 2;
  for (int x : v) m = x < m ? x : m;
  return m;
}

FfnCodes codes_of(const gp_fp8_matrix& m) {
  return FfnCodes{static_cast<uint8_t*>(m.data), m.scales, m.ld, m.stride_row, m.stride_col};
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

// Plan and launch a checked product.
int run_product(FfnProduct& p, const gp_ffn_options* opts) {
  const bool codes = p.out.codes[0].data != nullptr, wide = p.out.out_f32 || codes;
  int rc = ffn_plan_impl(p.op, p.rows, p.cols, p.summed, p.count, wide, codes, p.out.bf16, 0, opts, &p.plan);   // what needs no device
  if (rc != GP_OK) return call_finish(rc);
  CallInfo info;
  cudaError_t e = call_begin(opts ? opts->timeout_ns : 0, &info);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
  rc = ffn_plan_impl(p.op, p.rows, p.cols, p.summed, p.count, wide, codes, p.out.bf16, info.sm_count, opts, &p.plan);
  if (rc != GP_OK) return call_finish(rc);
  e = ffn_fit_pairs(&p.plan, codes && p.op == kFfnGated);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_CAPACITY);
  p.ctl = info.ctl;
  p.ctl.inject_lost_load = opts ? opts->inject_lost_load : 0;
  const void* kernel = nullptr;
  if (p.plan.layout)
    e = launch_ffn_few(p, &kernel);
  else if (p.op == kFfnLinear)
    e = launch_ffn_linear(p, &kernel);
  else if (p.op == kFfnGated)
    e = launch_ffn_gated(p, &kernel);
  else if (p.op == kFfnInputGrad)
    e = launch_ffn_input_grad(p, &kernel);
  else
    e = launch_ffn_weight_grad(p, &kernel);
  call_launched(p.plan, kernel);
  return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
}

}  // namespace
}  // namespace gp

using namespace gp;

extern "C" {

int gemm_ffn_plan(int op, int64_t M, int64_t N, int64_t K, int count, int kept, int sms, const gp_ffn_options* opts,
                  gp_plan* out) {
  if (!out || sms < 0 || op < kFfnLinear || op > kFfnWeightGrad || count < 1 || count > 2 || kept < 0 || kept > 7 ||
      (op == kFfnGated && (kept & 2)))
    return GP_ERR_ARG;
  const int rc = check_sizes(M, N, K);
  if (rc != GP_OK) return rc;
  const int64_t rows = op == kFfnWeightGrad ? N : M, cols = op == kFfnLinear || op == kFfnGated ? N : K;
  const int64_t summed = op == kFfnInputGrad ? N : (op == kFfnWeightGrad ? M : K);
  if (rows == 0 || cols == 0) return GP_ERR_ARG;
  return ffn_plan_impl(op, rows, cols, summed, count, (kept & 3) != 0, (kept & 1) != 0 && op <= kFfnGated, (kept & 4) == 0,
                       sms > 0 ? sms : current_sms(), opts, out);
}

int gemm_linear(const gp_linear* a, void* stream, const gp_ffn_options* opts) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st, opts && opts->continues);
  if (!a) return call_finish(GP_ERR_ARG);
  int rc = check_sizes(a->M, a->N, a->K);
  if (rc == GP_OK && (!type_ok(a->type) || !out_ok(a->type, a->out_type) || !act_ok(a->activation))) rc = GP_ERR_ARG;
  if (rc == GP_OK && a->bias && !out_ok(a->type, a->bias_type)) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (a->M == 0 || a->N == 0) return call_finish(GP_OK);
  if (a->K > 0) rc = first_error({check_operand(a->x, a->ldx, a->K), check_operand(a->weight, a->ldw, a->K)});
  if (rc == GP_OK)
    rc = first_error({check_real(a->y, a->ldy, a->N, a->out_type, false),
                      check_real(a->residual, a->ld_res, a->N, a->out_type, true),
                      check_real(a->z, a->ldz, a->N, a->type, true), check_codes(a->q, a->N, false),
                      a->bias && !aligned(a->bias, real_bytes(a->bias_type)) ? GP_ERR_UNSUPPORTED : GP_OK,
                      a->z && a->q.data ? GP_ERR_ARG : GP_OK});
  if (rc != GP_OK) return call_finish(rc);
  FfnProduct p = {};
  p.op = kFfnLinear;
  p.a[0] = a->x;
  p.b[0] = a->weight;
  p.lda[0] = a->ldx;
  p.ldb[0] = a->ldw;
  p.rows = a->M;
  p.cols = a->N;
  p.summed = a->K;
  p.count = 1;
  p.stream = st;
  FfnOut& o = p.out;
  o.out[0] = a->y;
  o.ld_out[0] = a->ldy;
  o.add[0] = a->residual;
  o.ld_add[0] = a->ld_res;
  o.bias = a->bias;
  o.keep[0] = a->z;
  o.ld_keep[0] = a->ldz;
  o.codes[0] = codes_of(a->q);
  o.bf16 = a->type == GP_REAL_BF16;
  o.out_f32 = a->out_type == GP_REAL_F32;
  o.bias_f32 = a->bias_type == GP_REAL_F32;
  o.act = a->activation;
  o.vec = least({align_of(a->y, a->ldy, a->out_type), align_of(a->residual, a->ld_res, a->out_type),
                 align_of(a->z, a->ldz, a->type)});
  return run_product(p, opts);
}

int gemm_gated(const gp_gated* a, void* stream, const gp_ffn_options* opts) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st, opts && opts->continues);
  if (!a) return call_finish(GP_ERR_ARG);
  int rc = check_sizes(a->M, a->N, a->K);
  if (rc == GP_OK && (!type_ok(a->type) || !act_ok(a->activation))) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (a->M == 0 || a->N == 0) return call_finish(GP_OK);
  if (a->K > 0)
    rc = first_error({check_operand(a->x, a->ldx, a->K), check_operand(a->gate, a->ld_gate, a->K),
                      check_operand(a->up, a->ld_up, a->K)});
  const bool real = a->z_gate || a->z_up, codes = a->q_gate.data || a->q_up.data;
  if (rc == GP_OK && ((real && (!a->z_gate || !a->z_up || a->z_gate == a->z_up)) || (codes && (!a->q_gate.data || !a->q_up.data)) || (real && codes)))
    rc = GP_ERR_ARG;
  if (rc == GP_OK)
    rc = first_error({check_real(a->h, a->ldh, a->N, a->type, false), check_real(a->z_gate, a->ld_zg, a->N, a->type, true),
                      check_real(a->z_up, a->ld_zu, a->N, a->type, true), check_codes(a->q_gate, a->N, false),
                      check_codes(a->q_up, a->N, false)});
  if (rc != GP_OK) return call_finish(rc);
  FfnProduct p = {};
  p.op = kFfnGated;
  p.a[0] = a->x;
  p.b[0] = a->gate;
  p.b[1] = a->up;
  p.lda[0] = a->ldx;
  p.ldb[0] = a->ld_gate;
  p.ldb[1] = a->ld_up;
  p.rows = a->M;
  p.cols = a->N;
  p.summed = a->K;
  p.count = 1;
  p.stream = st;
  FfnOut& o = p.out;
  o.out[0] = a->h;
  o.ld_out[0] = a->ldh;
  o.keep[0] = a->z_gate;
  o.keep[1] = a->z_up;
  o.ld_keep[0] = a->ld_zg;
  o.ld_keep[1] = a->ld_zu;
  o.codes[0] = codes_of(a->q_gate);
  o.codes[1] = codes_of(a->q_up);
  o.bf16 = a->type == GP_REAL_BF16;
  o.act = a->activation;
  o.vec = least({align_of(a->h, a->ldh, a->type), align_of(a->z_gate, a->ld_zg, a->type), align_of(a->z_up, a->ld_zu, a->type)});
  return run_product(p, opts);
}

int gemm_input_grad(const gp_input_grad* a, void* stream, const gp_ffn_options* opts) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st, opts && opts->continues);
  if (!a) return call_finish(GP_ERR_ARG);
  int rc = check_sizes(a->M, a->N, a->K);
  if (rc == GP_OK && (!type_ok(a->type) || !out_ok(a->type, a->out_type) || a->count < 1 || a->count > 2)) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (a->M == 0 || a->K == 0) return call_finish(GP_OK);
  for (int i = 0; rc == GP_OK && a->N > 0 && i < a->count; ++i)
    rc = first_error({check_operand(a->dz[i], a->ld_dz[i], a->N), check_operand(a->weight[i], a->ldw[i], a->K)});
  if (rc == GP_OK) rc = check_real(a->dx, a->ld_dx, a->K, a->out_type, false);
  if (rc != GP_OK) return call_finish(rc);
  FfnProduct p = {};
  p.op = kFfnInputGrad;
  for (int i = 0; i < a->count; ++i) {
    p.a[i] = a->dz[i];
    p.b[i] = a->weight[i];
    p.lda[i] = a->ld_dz[i];
    p.ldb[i] = a->ldw[i];
  }
  p.rows = a->M;
  p.cols = a->K;
  p.summed = a->N;
  p.count = a->count;
  p.stream = st;
  FfnOut& o = p.out;
  o.out[0] = a->dx;
  o.ld_out[0] = a->ld_dx;
  o.bf16 = a->type == GP_REAL_BF16;
  o.out_f32 = a->out_type == GP_REAL_F32;
  o.vec = align_of(a->dx, a->ld_dx, a->out_type);
  return run_product(p, opts);
}

int gemm_weight_grad(const gp_weight_grad* a, void* stream, const gp_ffn_options* opts) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st, opts && opts->continues);
  if (!a) return call_finish(GP_ERR_ARG);
  int rc = check_sizes(a->M, a->N, a->K);
  if (rc == GP_OK && (!type_ok(a->type) || !out_ok(a->type, a->out_type) || a->count < 1 || a->count > 2)) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (a->N == 0 || a->K == 0) return call_finish(GP_OK);
  if (a->M > 0) rc = check_operand(a->x, a->ldx, a->K);
  for (int i = 0; rc == GP_OK && i < a->count; ++i)
    rc = first_error({a->M > 0 ? check_operand(a->dz[i], a->ld_dz[i], a->N) : GP_OK,
                      check_real(a->dw[i], a->ld_dw[i], a->K, a->out_type, false),
                      check_real(a->addend[i], a->ld_add[i], a->K, a->out_type, true)});
  if (rc == GP_OK && a->count == 2 && (!a->addend[0] != !a->addend[1] || a->dw[0] == a->dw[1])) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  FfnProduct p = {};
  p.op = kFfnWeightGrad;
  FfnOut& o = p.out;
  o.vec = 2;
  for (int i = 0; i < a->count; ++i) {
    p.a[i] = a->dz[i];
    p.lda[i] = a->ld_dz[i];
    o.out[i] = a->dw[i];
    o.ld_out[i] = a->ld_dw[i];
    o.add[i] = a->addend[i];
    o.ld_add[i] = a->ld_add[i];
    o.vec = least({o.vec, align_of(a->dw[i], a->ld_dw[i], a->out_type), align_of(a->addend[i], a->ld_add[i], a->out_type)});
  }
  p.b[0] = a->x;
  p.ldb[0] = a->ldx;
  p.rows = a->N;
  p.cols = a->K;
  p.summed = a->M;
  p.count = a->count;
  p.stream = st;
  o.bf16 = a->type == GP_REAL_BF16;
  o.out_f32 = a->out_type == GP_REAL_F32;
  return run_product(p, opts);
}

int ffn_act_backward_workspace(int64_t M, int64_t N, int sms, int64_t* bytes) {
  if (!bytes || sms < 0) return GP_ERR_ARG;
  const int rc = check_sizes(M, N);
  if (rc != GP_OK) return rc;
  if (sms == 0) sms = current_sms();
  const int64_t parts = M == 0 || N == 0 ? 0 : ffn_act_parts(M, N, sms > 0 ? sms : 152);
  *bytes = parts > 1 ? parts * N * 4 : 0;
  return GP_OK;
}

int ffn_act_backward(const gp_act_backward* a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st);
  if (!a) return call_finish(GP_ERR_ARG);
  int rc = check_sizes(a->M, a->N);
  if (rc == GP_OK && (!type_ok(a->type) || !act_ok(a->activation))) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (a->N == 0 || (a->M == 0 && !a->dbias)) return call_finish(GP_OK);
  const bool act = a->activation != GP_ACT_NONE;
  if (!aligned(a->dbias, 4) || !aligned(a->workspace, 16)) rc = GP_ERR_UNSUPPORTED;
  if (rc == GP_OK && a->M > 0) {
    rc = first_error({check_real(a->dy, a->ld_dy, a->N, a->type, false), check_real(a->dz, a->ld_dz, a->N, a->type, true)});
    if (rc == GP_OK && act) {
      rc = first_error({check_real(a->z, a->ldz, a->N, a->type, true), check_codes(a->q, a->N, true)});
      if (rc == GP_OK && !a->z == !a->q.data) rc = GP_ERR_ARG;
    }
  }
  if (rc != GP_OK || (a->M > 0 && !a->dz && !a->dbias)) return call_finish(rc);
  CallInfo info;
  cudaError_t e = call_begin(0, &info);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
  if (a->M == 0) {
    e = launch_fp8_fill_f32(a->dbias, a->N, 0.f, st);
    return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
  }
  FfnActArgs g = {};
  g.dy = a->dy;
  g.ld_dy = a->ld_dy;
  if (act) {
    g.z[0] = a->z;
    g.ldz[0] = a->ldz;
    g.codes[0] = codes_of(a->q);
    g.e5m2 = a->q.data && a->q.format == GP_E5M2;
  }
  g.dz[0] = a->dz;
  g.ld_dz[0] = a->ld_dz;
  g.dbias = a->dbias;
  g.M = a->M;
  g.N = a->N;
  g.type = a->type;
  g.act = a->activation;
  g.vec = vec16(a->dy, a->ld_dy, 2) && (!a->dz || vec16(a->dz, a->ld_dz, 2)) && (!g.z[0] || vec16(a->z, a->ldz, 2));
  gp_plan plan = {};
  const int64_t parts = ffn_act_parts(a->M, a->N, info.sm_count);
  if (a->dbias && parts > 1) {
    plan.workspace_bytes = parts * a->N * 4;
    if (!a->workspace || a->workspace_bytes < plan.workspace_bytes) return call_finish(GP_ERR_ARG);
    g.partials = static_cast<float*>(a->workspace);
  }
  const void* kernel = nullptr;
  e = launch_ffn_act_backward(g, info.sm_count, st, &kernel, &plan);
  call_launched(plan, kernel);
  return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
}

int ffn_gated_backward(const gp_gated_backward* a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st);
  if (!a) return call_finish(GP_ERR_ARG);
  int rc = check_sizes(a->M, a->N);
  if (rc == GP_OK && (!type_ok(a->type) || !act_ok(a->activation))) rc = GP_ERR_ARG;
  if (rc != GP_OK) return call_finish(rc);
  if (a->M == 0 || a->N == 0) return call_finish(GP_OK);
  const bool real = a->z_gate && a->z_up, codes = a->q_gate.data && a->q_up.data;
  if (real == codes || (codes ? a->z_gate || a->z_up : a->q_gate.data || a->q_up.data)) return call_finish(GP_ERR_ARG);
  rc = first_error({check_real(a->dh, a->ld_dh, a->N, a->type, false), check_real(a->z_gate, a->ld_zg, a->N, a->type, true),
                    check_real(a->z_up, a->ld_zu, a->N, a->type, true), check_codes(a->q_gate, a->N, true),
                    check_codes(a->q_up, a->N, true), check_real(a->dgate, a->ld_dgate, a->N, a->type, false),
                    check_real(a->dup, a->ld_dup, a->N, a->type, false), check_real(a->h, a->ldh, a->N, a->type, true),
                    codes && a->q_gate.format != a->q_up.format ? GP_ERR_ARG : GP_OK,
                    a->dgate == a->dup ? GP_ERR_ARG : GP_OK});
  if (rc != GP_OK) return call_finish(rc);
  CallInfo info;
  cudaError_t e = call_begin(0, &info);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
  FfnActArgs g = {};
  g.dy = a->dh;
  g.ld_dy = a->ld_dh;
  g.z[0] = a->z_gate;
  g.z[1] = a->z_up;
  g.ldz[0] = a->ld_zg;
  g.ldz[1] = a->ld_zu;
  g.codes[0] = codes_of(a->q_gate);
  g.codes[1] = codes_of(a->q_up);
  g.e5m2 = codes && a->q_gate.format == GP_E5M2;
  g.dz[0] = a->dgate;
  g.dz[1] = a->dup;
  g.ld_dz[0] = a->ld_dgate;
  g.ld_dz[1] = a->ld_dup;
  g.h = a->h;
  g.ldh = a->ldh;
  g.M = a->M;
  g.N = a->N;
  g.type = a->type;
  g.act = a->activation;
  g.vec = vec16(a->dh, a->ld_dh, 2) && vec16(a->dgate, a->ld_dgate, 2) && vec16(a->dup, a->ld_dup, 2) &&
          (!a->h || vec16(a->h, a->ldh, 2)) && (!real || (vec16(a->z_gate, a->ld_zg, 2) && vec16(a->z_up, a->ld_zu, 2)));
  gp_plan plan = {};
  const void* kernel = nullptr;
  e = launch_ffn_gated_backward(g, info.sm_count, st, &kernel, &plan);
  call_launched(plan, kernel);
  return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
}

int ffn_pack_rows(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int64_t rows, int64_t cols, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  call_reset(st);
  int rc = check_sizes(rows, cols);
  if (rc != GP_OK) return call_finish(rc);
  if (rows == 0 || cols == 0) return call_finish(GP_OK);
  rc = first_error({check_real(src, ld_src, cols, GP_REAL_F16, false), check_operand(dst, ld_dst, cols)});
  if (rc != GP_OK) return call_finish(rc);
  CallInfo info;
  cudaError_t e = call_begin(0, &info);
  if (e != cudaSuccess) return call_finish(GP_ERR_CUDA, e, GP_SITE_DEVICE);
  gp_plan plan = {};
  const void* kernel = nullptr;
  e = launch_ffn_pack(src, ld_src, dst, ld_dst, rows, cols, st, &kernel, &plan);
  call_launched(plan, kernel);
  return e == cudaSuccess ? call_finish(GP_OK) : call_finish(GP_ERR_CUDA, e);
}

}  // extern "C"
