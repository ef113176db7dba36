// torch_ffn.cpp -- the feed-forward operators on torch tensors: argument checks,
// outputs and calls of the C ABI (include/gemm_ffn.h), as a CPython extension.
//
// Small calls take some microseconds on the GPU.  In Python the checks and the
// allocations around one took 12 us, here 4.  Nothing is computed in this file.
#include <Python.h>

#include <string>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <dlfcn.h>

#include "gemm_ffn.h"

namespace {

// ---------------------------------------------------------------------------
// errors
// ---------------------------------------------------------------------------
struct Refused {      // ValueError
  std::string what;
};
struct Wrong {        // TypeError
  std::string what;
};
struct Failed {       // GemmError
  int code;
  const char* where;
};

PyObject* g_failed = nullptr;   // called with (code, where): the exception to raise

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}
std::string type_of(const at::Tensor& t) { return std::string(c10::toString(t.scalar_type())); }

// ---------------------------------------------------------------------------
// the library
// ---------------------------------------------------------------------------
struct Library {
  decltype(&gemm_linear) linear;
  decltype(&gemm_gated) gated;
  decltype(&gemm_input_grad) input_grad;
  decltype(&gemm_weight_grad) weight_grad;
  decltype(&ffn_act_backward) act_backward;
  decltype(&ffn_act_backward_workspace) act_workspace;
  decltype(&ffn_gated_backward) gated_backward;
  decltype(&ffn_pack_rows) pack;
} lib;

void check(int rc, const char* where) {
  if (rc != GP_OK) throw Failed{rc, where};
}

// ---------------------------------------------------------------------------
// tensors
// ---------------------------------------------------------------------------
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Wrong{std::string(name) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

int real_of(at::ScalarType t) {
  return t == at::kHalf ? GP_REAL_F16 : (t == at::kBFloat16 ? GP_REAL_BF16 : (t == at::kFloat ? GP_REAL_F32 : -1));
}

// A matrix whose rows are contiguous: its sizes and row stride.
struct Matrix {
  int64_t rows, cols, ld;
  void* p;
};
Matrix matrix(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) throw Refused{std::string(name) + " must have two dimensions, got " + std::to_string(t.dim())};
  if (!t.is_cuda()) throw Refused{std::string(name) + " must be on a CUDA device"};
  const int64_t rows = t.size(0), cols = t.size(1), ld = t.stride(0);
  if (cols > 1 && t.stride(1) != 1)
    throw Refused{std::string(name) + " must have contiguous rows (stride 1 along the last dimension)"};
  return Matrix{rows, cols, rows > 1 || ld > cols ? ld : cols, t.data_ptr()};
}

// One that is read or written: its rows lie apart.
Matrix rows_apart(const at::Tensor& t, const char* name) {
  const Matrix m = matrix(t, name);
  if (m.rows > 1 && m.ld < m.cols) throw Refused{std::string("the rows of ") + name + " overlap"};
  return m;
}

// A matrix of given sizes, type and device.
Matrix shaped(const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, const at::Tensor& like, const char* name) {
  const Matrix m = rows_apart(t, name);
  if (m.rows != rows || m.cols != cols || t.scalar_type() != type || t.get_device() != like.get_device())
    throw Refused{std::string(name) + " must be " + std::to_string(rows) + " x " + std::to_string(cols) + " of " +
                  c10::toString(type) + " on " + like.device().str() + ": got " + shape_of(t) + " of " + type_of(t) + " on " +
                  t.device().str()};
  return m;
}

// Whether two matrices share a byte.  Rows of the same stride may lie side by side, as halves of one matrix do; where the
// strides differ, ranges that meet count.
bool meet(const Matrix& a, const at::Tensor& ta, const Matrix& b, const at::Tensor& tb) {
  if (a.rows == 0 || a.cols == 0 || b.rows == 0 || b.cols == 0) return false;
  const int64_t wa = a.cols * ta.element_size(), wb = b.cols * tb.element_size();
  const int64_t sa = a.ld * ta.element_size(), sb = b.ld * tb.element_size();
  const int64_t at = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);   // where b begins, from a
  if (at >= (a.rows - 1) * sa + wa || -at >= (b.rows - 1) * sb + wb) return false;
  if (a.rows > 1 && b.rows > 1 && sa != sb) return true;
  const int64_t s = a.rows > 1 ? sa : (b.rows > 1 ? sb : 0);
  if (s <= 0) return true;
  const int64_t in = (at % s + s) % s;
  return in < wa || in + wb > s;
}
// An output that a kernel writes while it reads another matrix: apart from it, or that matrix itself where it may be.
void apart(const at::Tensor& out, const at::Tensor& other, const char* name, bool may_be_it = false) {
  const Matrix a = matrix(out, "out"), b = matrix(other, name);
  if (may_be_it && a.p == b.p && (a.ld == b.ld || a.rows <= 1)) return;
  if (meet(a, out, b, other)) throw Refused{std::string("out overlaps ") + name};
}

// A tensor of the caller's that a kernel writes counts as changed, as after torch's own operations in place: autograd then
// refuses to use what it kept of the values before.
void changed(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

int type16(const at::Tensor& t, const char* name) {
  const int r = real_of(t.scalar_type());
  if (r != GP_REAL_F16 && r != GP_REAL_BF16)
    throw Refused{std::string(name) + " must be float16 or bfloat16, got " + type_of(t)};
  return r;
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// The device of a call made current, and its stream.
struct Call {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit Call(const at::Tensor& t) {
    const c10::DeviceIndex d = static_cast<c10::DeviceIndex>(t.get_device());
    if (d != c10::cuda::current_device()) guard.set_index(d);
    stream = c10::cuda::getCurrentCUDAStream(d).stream();
  }
};

// An operand of a product: rows on 16-byte boundaries, or `loose` until lay_out() has copied it.  Calls look at all of
// their arguments first, and lay out, allocate and launch then.
struct Operand : Matrix {
  bool loose = false;
  at::Tensor copy;
};
Operand operand(const at::Tensor& t, const char* name, const at::Tensor* like) {
  Operand m;
  static_cast<Matrix&>(m) = rows_apart(t, name);
  if (like && (t.scalar_type() != like->scalar_type() || t.get_device() != like->get_device()))
    throw Refused{std::string(name) + " is " + type_of(t) + " on " + t.device().str() + ": want " + type_of(*like) + " on " +
                  like->device().str()};
  if (m.rows <= 1) m.ld = up(m.cols, 8);   // the stride of a single row is never used
  m.loose = (reinterpret_cast<uintptr_t>(m.p) | static_cast<uintptr_t>(m.ld * 2)) % 16 != 0;
  return m;
}
void lay_out(Operand& m, const at::Tensor& like, const Call& call) {
  if (!m.loose) return;
  const int64_t ld = up(m.cols, 8);
  m.copy = at::empty_strided({m.rows, m.cols}, {ld, 1}, like.options());
  check(lib.pack(m.p, m.ld, m.copy.data_ptr(), ld, m.rows, m.cols, call.stream), "ffn_pack_rows");
  m.p = m.copy.data_ptr();
  m.ld = ld;
  m.loose = false;
}

// An output whose rows begin on 16-byte boundaries.
at::Tensor rows_of(int64_t rows, int64_t cols, at::ScalarType type, const at::Tensor& like) {
  const int64_t per16 = type == at::kFloat ? 4 : (type == at::kFloat8_e4m3fn ? 16 : 8);
  return at::empty_strided({rows, cols}, {up(cols, per16), 1}, like.options().dtype(type));
}

// Codes to be written: the scales of one group of columns side by side, as quantize_fp8 lays them out.
struct Codes {
  at::Tensor data, scales;
};
Codes new_codes(int64_t rows, int64_t cols, const at::Tensor& like, gp_fp8_matrix* q) {
  Codes c{rows_of(rows, cols, at::kFloat8_e4m3fn, like),
          at::empty_strided({rows, (cols + 127) / 128}, {1, rows > 0 ? rows : 1}, like.options().dtype(at::kFloat))};
  *q = gp_fp8_matrix{c.data.data_ptr(), c.scales.data_ptr<float>(), up(cols, 16), 1, rows > 0 ? rows : 1, GP_E4M3, 1};
  return c;
}

// Values kept by a forward call, of one product.
struct Kept {
  void* z = nullptr;
  int64_t ld = 0;
  gp_fp8_matrix q = {};
};
gp_fp8_matrix kept_codes(const at::Tensor& data, const at::Tensor& scales, int64_t rows, int64_t cols, const at::Tensor& like,
                         const char* name) {
  const Matrix m = rows_apart(data, name);
  const at::ScalarType t = data.scalar_type();
  if ((t != at::kFloat8_e4m3fn && t != at::kFloat8_e5m2) || m.rows != rows || m.cols != cols ||
      data.get_device() != like.get_device())
    throw Refused{std::string(name) + " must be an 8-bit " + std::to_string(rows) + " x " + std::to_string(cols) +
                  " matrix on " + like.device().str() + ": got " + shape_of(data) + " of " + type_of(data) + " on " +
                  data.device().str()};
  if (scales.scalar_type() != at::kFloat || scales.dim() != 2 || scales.size(0) != rows || scales.size(1) != (cols + 127) / 128 ||
      scales.get_device() != like.get_device())
    throw Refused{std::string("the scales of ") + name + " must be float32 (" + std::to_string(rows) + ", " +
                  std::to_string((cols + 127) / 128) + ") on its device"};
  const int64_t ld = rows <= 1 ? up(cols, 16) : m.ld;
  if (rows > 0 && cols > 0 && (reinterpret_cast<uintptr_t>(m.p) | static_cast<uintptr_t>(ld)) % 16 != 0)
    throw Refused{std::string("the rows of ") + name + " in 8 bits must begin on 16-byte boundaries, as quantize_fp8 lays them out"};
  return gp_fp8_matrix{m.p, scales.data_ptr<float>(), ld, scales.stride(0), scales.stride(1),
                       t == at::kFloat8_e5m2 ? GP_E5M2 : GP_E4M3, 1};
}
void read_kept(PyObject* o, int weights, int64_t rows, int64_t cols, const at::Tensor& like, Kept* kept) {
  PyObject* items[4];
  Py_ssize_t n = -1;
  if (THPVariable_Check(o)) {
    items[0] = o;
    n = 1;
  } else if (PyTuple_Check(o) || PyList_Check(o)) {
    n = PySequence_Fast_GET_SIZE(o);
    for (Py_ssize_t i = 0; i < n && i < 4; ++i) items[i] = PySequence_Fast_GET_ITEM(o, i);
  }
  if (n != weights && n != 2 * weights)
    throw Refused{"kept must be what the forward call returned: " + std::to_string(weights) + " matrices, or " +
                  std::to_string(weights) + " with their scales"};
  for (int i = 0; i < weights; ++i) {
    const char* name = i ? "the other kept values" : "the kept values";
    if (n == weights) {
      const Matrix m = shaped(tensor(items[i], "kept"), rows, cols, like.scalar_type(), like, name);
      kept[i].z = m.p;
      kept[i].ld = m.ld;
    } else {
      kept[i].q = kept_codes(tensor(items[2 * i], "kept"), tensor(items[2 * i + 1], "kept"), rows, cols, like, name);
    }
  }
}

// The type of an output that may be FP32: from what is asked for (None: the default).
at::ScalarType out_type(PyObject* dtype, at::ScalarType own, const char* name) {
  if (dtype == Py_None) return own;
  if (!THPDtype_Check(dtype)) throw Wrong{std::string(name) + " must be a torch.dtype"};
  const at::ScalarType t = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  if (t != own && t != at::kFloat)
    throw Refused{std::string(name) + " must be " + c10::toString(own) + " or float32, got " + c10::toString(t)};
  return t;
}

const gp_ffn_options* options(PyObject* o) {   // None, or the packed struct
  return o == Py_None ? nullptr : reinterpret_cast<const gp_ffn_options*>(PyBytes_AS_STRING(o));
}

// The options of one of the products that a call makes: `which` in the test hook's bits; one that `continues` shares the
// record of the product before, so that a wait that gave up in either is the call's status.
struct ProductOptions {
  gp_ffn_options own = {};
  const gp_ffn_options* p;
  ProductOptions(const gp_ffn_options* given, int which, bool continues) : p(given || continues ? &own : nullptr) {
    if (given) own = *given;
    own.inject_lost_load = own.inject_lost_load & which ? 1 : 0;
    own.continues = continues;
  }
};

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* tuple(std::initializer_list<at::Tensor> tensors) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  Py_ssize_t i = 0;
  for (const at::Tensor& t : tensors) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}
PyObject* with_kept(const at::Tensor& out, PyObject* kept) {
  PyObject* r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, wrap(out));
  PyTuple_SET_ITEM(r, 1, kept);
  return r;
}

enum Keep { kKeepNone = 0, kKeepReal = 1, kKeepCodes = 2 };

// ---------------------------------------------------------------------------
// the operators
// ---------------------------------------------------------------------------
// linear(x, weight, bias, activation, residual, keep, out, out_dtype, options)
PyObject* linear(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  if (!x.is_cuda()) throw Refused{"x must be on a CUDA device"};
  const int real = type16(x, "x");
  const Call call(x);
  gp_linear g = {};
  Operand mx = operand(x, "x", nullptr), mw = operand(tensor(a[1], "weight"), "weight", &x);
  if (mw.cols != mx.cols)
    throw Refused{"x has " + std::to_string(mx.cols) + " columns and weight " + std::to_string(mw.cols)};
  const int64_t M = mx.rows, N = mw.rows;
  g.M = M;
  g.N = N;
  g.K = mx.cols;
  g.type = g.bias_type = real;
  g.activation = static_cast<int32_t>(PyLong_AsLong(a[3]));
  if (a[2] != Py_None) {
    const at::Tensor& b = tensor(a[2], "bias");
    if (b.dim() != 1 || b.size(0) != N || b.get_device() != x.get_device() || (N > 1 && b.stride(0) != 1) ||
        (b.scalar_type() != at::kFloat && b.scalar_type() != x.scalar_type()))
      throw Refused{"bias must be " + std::to_string(N) + " contiguous values of " + type_of(x) + " or float32 on " +
                    x.device().str()};
    g.bias = b.data_ptr();
    g.bias_type = real_of(b.scalar_type());
  }
  at::Tensor y;
  at::ScalarType type;
  if (a[6] == Py_None) {
    type = out_type(a[7], x.scalar_type(), "out_dtype");
  } else {
    y = tensor(a[6], "out");
    if (a[7] != Py_None && (!THPDtype_Check(a[7]) || reinterpret_cast<THPDtype*>(a[7])->scalar_type != y.scalar_type()))
      throw Refused{"out is " + type_of(y) + ": out_dtype asks for another type"};
    type = y.scalar_type() == at::kFloat ? at::kFloat : x.scalar_type();
    g.ldy = shaped(y, M, N, type, x, "out").ld;
  }
  g.out_type = real_of(type);
  if (a[4] != Py_None) {
    const Matrix r = shaped(tensor(a[4], "residual"), M, N, type, x, "residual");
    g.residual = r.p;
    g.ld_res = r.ld;
    if (a[6] != Py_None) apart(y, tensor(a[4], "residual"), "residual", true);
  }
  if (a[6] != Py_None) {
    apart(y, x, "x");
    apart(y, tensor(a[1], "weight"), "weight");
    if (a[2] != Py_None) apart(y, tensor(a[2], "bias").unsqueeze(0), "bias");
  }
  lay_out(mx, x, call);
  lay_out(mw, x, call);
  g.x = mx.p;
  g.weight = mw.p;
  g.ldx = mx.ld;
  g.ldw = mw.ld;
  if (a[6] == Py_None) {
    y = rows_of(M, N, type, x);
    g.ldy = y.stride(0);
  }
  g.y = y.data_ptr();
  const long keep = PyLong_AsLong(a[5]);
  at::Tensor z;
  Codes codes;
  if (keep == kKeepReal) {
    z = rows_of(M, N, x.scalar_type(), x);
    g.z = z.data_ptr();
    g.ldz = z.stride(0);
  } else if (keep == kKeepCodes) {
    codes = new_codes(M, N, x, &g.q);
  }
  check(lib.linear(&g, call.stream, options(a[8])), "gemm_linear");
  if (a[6] != Py_None) changed(y);
  if (keep == kKeepNone) return wrap(y);
  return with_kept(y, keep == kKeepReal ? tuple({z}) : tuple({codes.data, codes.scales}));
}

// gated(x, w_gate, w_up, activation, keep, out, options)
PyObject* gated(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  if (!x.is_cuda()) throw Refused{"x must be on a CUDA device"};
  gp_gated g = {};
  g.type = type16(x, "x");
  const Call call(x);
  Operand mx = operand(x, "x", nullptr), mg = operand(tensor(a[1], "w_gate"), "w_gate", &x),
          mu = operand(tensor(a[2], "w_up"), "w_up", &x);
  const int64_t M = mx.rows, N = mg.rows;
  if (mg.cols != mx.cols || mu.cols != mx.cols || mu.rows != N)
    throw Refused{"x has " + std::to_string(mx.cols) + " columns: the weights are " + shape_of(tensor(a[1], "w_gate")) + " and " +
                  shape_of(tensor(a[2], "w_up"))};
  g.M = M;
  g.N = N;
  g.K = mx.cols;
  g.activation = static_cast<int32_t>(PyLong_AsLong(a[3]));
  at::Tensor h;
  if (a[5] != Py_None) {
    h = tensor(a[5], "out");
    g.ldh = shaped(h, M, N, x.scalar_type(), x, "out").ld;
    apart(h, x, "x");
    apart(h, tensor(a[1], "w_gate"), "w_gate");
    apart(h, tensor(a[2], "w_up"), "w_up");
  }
  for (Operand* m : {&mx, &mg, &mu}) lay_out(*m, x, call);
  g.x = mx.p;
  g.gate = mg.p;
  g.up = mu.p;
  g.ldx = mx.ld;
  g.ld_gate = mg.ld;
  g.ld_up = mu.ld;
  if (a[5] == Py_None) {
    h = rows_of(M, N, x.scalar_type(), x);
    g.ldh = h.stride(0);
  }
  g.h = h.data_ptr();
  const long keep = PyLong_AsLong(a[4]);
  at::Tensor zg, zu;
  Codes cg, cu;
  if (keep == kKeepReal) {
    zg = rows_of(M, N, x.scalar_type(), x);
    zu = rows_of(M, N, x.scalar_type(), x);
    g.z_gate = zg.data_ptr();
    g.z_up = zu.data_ptr();
    g.ld_zg = g.ld_zu = zg.stride(0);
  } else if (keep == kKeepCodes) {
    cg = new_codes(M, N, x, &g.q_gate);
    cu = new_codes(M, N, x, &g.q_up);
  }
  check(lib.gated(&g, call.stream, options(a[6])), "gemm_gated");
  if (a[5] != Py_None) changed(h);
  if (keep == kKeepNone) return wrap(h);
  return with_kept(h, keep == kKeepReal ? tuple({zg, zu}) : tuple({cg.data, cg.scales, cu.data, cu.scales}));
}

// dx of one product or of a pair.
at::Tensor input_gradient(int count, const Matrix* dz, const Operand* w, int64_t M, int64_t N, int64_t K, int real,
                          const at::Tensor& like, const Call& call, const gp_ffn_options* opts) {
  at::Tensor dx = rows_of(M, K, like.scalar_type(), like);
  gp_input_grad g = {};
  for (int i = 0; i < count; ++i) {
    g.dz[i] = dz[i].p;
    g.ld_dz[i] = dz[i].ld;
    g.weight[i] = w[i].p;
    g.ldw[i] = w[i].ld;
  }
  g.dx = dx.data_ptr();
  g.ld_dx = dx.stride(0);
  g.M = M;
  g.N = N;
  g.K = K;
  g.type = g.out_type = real;
  g.count = count;
  check(lib.input_grad(&g, call.stream, opts), "gemm_input_grad");
  return dx;
}

// Item i of an argument that is None, a tensor (count 1) or a sequence of `count`.
PyObject* item(PyObject* o, int i, int count, const char* name) {
  if (o == Py_None) return Py_None;
  if (THPVariable_Check(o) && count == 1) return o;
  if (!(PyTuple_Check(o) || PyList_Check(o)) || PySequence_Fast_GET_SIZE(o) != count)
    throw Refused{std::string(name) + " takes " + std::to_string(count) + (count == 1 ? " matrix" : " matrices")};
  return PySequence_Fast_GET_ITEM(o, i);
}

// Where the gradients of the weights of products that share x go, and what is added to them.
struct WeightGradients {
  gp_weight_grad g = {};
  at::ScalarType type;
  at::Tensor dw[2];      // those that are given
};
// x_given, dz_given (NULL: of the call's own): the operands as tensors.
WeightGradients look_at_weight_gradients(int count, int64_t N, int64_t K, PyObject* dtype, PyObject* addend, PyObject* out,
                                         const at::Tensor& like, const at::Tensor& x_given, const at::Tensor* dz_given) {
  WeightGradients r;
  gp_weight_grad& g = r.g;
  at::Tensor* const dw = r.dw;
  at::ScalarType& type = r.type;
  type = out_type(dtype, like.scalar_type(), "out_dtype");
  if (dtype == Py_None) {   // what is given says
    PyObject* first = out != Py_None ? item(out, 0, count, "out") : item(addend, 0, count, "addend");
    if (first != Py_None && tensor(first, "out").scalar_type() == at::kFloat) type = at::kFloat;
  }
  for (int i = 0; i < count; ++i) {
    PyObject* o = item(out, i, count, "out");
    PyObject* add = item(addend, i, count, "addend");
    if (o != Py_None) {
      dw[i] = tensor(o, "out");
      g.ld_dw[i] = shaped(dw[i], N, K, type, like, "out").ld;
    }
    if (add != Py_None) {
      const Matrix m = shaped(tensor(add, "addend"), N, K, type, like, "addend");
      g.addend[i] = m.p;
      g.ld_add[i] = m.ld;
    }
  }
  if (out != Py_None) {
    for (int i = 0; i < count; ++i) {
      if (!dw[i].defined()) continue;
      apart(dw[i], x_given, "x");
      if (dz_given) apart(dw[i], *dz_given, "dy");
      for (int j = 0; j < count; ++j) {
        PyObject* add = item(addend, j, count, "addend");
        if (add != Py_None) apart(dw[i], tensor(add, "addend"), "addend", i == j);
        if (j > i && dw[j].defined()) apart(dw[i], dw[j], "the other out");
      }
    }
  }
  return r;
}
void weight_gradients(int count, const Matrix* dz, const Operand& x, int64_t N, int real, WeightGradients& r,
                      const at::Tensor& like, const Call& call, const gp_ffn_options* opts) {
  gp_weight_grad& g = r.g;
  const int64_t K = x.cols;
  bool given[2] = {r.dw[0].defined(), r.dw[1].defined()};
  for (int i = 0; i < count; ++i) {
    g.dz[i] = dz[i].p;
    g.ld_dz[i] = dz[i].ld;
    if (!given[i]) {
      r.dw[i] = rows_of(N, K, r.type, like);
      g.ld_dw[i] = r.dw[i].stride(0);
    }
    g.dw[i] = r.dw[i].data_ptr();
  }
  g.x = x.p;
  g.ldx = x.ld;
  g.M = x.rows;
  g.N = N;
  g.K = K;
  g.type = real;
  g.out_type = real_of(r.type);
  g.count = count;
  check(lib.weight_grad(&g, call.stream, opts), "gemm_weight_grad");
  for (int i = 0; i < count; ++i)
    if (given[i]) changed(r.dw[i]);
}

// linear_backward(dy, x, weight, activation, kept, bias_grad, input_grad, weight_grad, out_dtype, addend, out, options)
PyObject* linear_backward(PyObject* const* a) {
  const at::Tensor& dy = tensor(a[0], "dy");
  if (!dy.is_cuda()) throw Refused{"dy must be on a CUDA device"};
  const int real = type16(dy, "dy");
  const Call call(dy);
  const int act = static_cast<int>(PyLong_AsLong(a[3]));
  const bool bias = a[5] == Py_True, want_x = a[6] == Py_True, want_w = a[7] == Py_True;
  const gp_ffn_options* opts = options(a[11]);
  if (act == GP_ACT_NONE && a[4] != Py_None) throw Refused{"without an activation nothing is kept"};
  if (!want_w && (a[9] != Py_None || a[10] != Py_None)) throw Refused{"addend and out are for dweight"};
  const Matrix md = rows_apart(dy, "dy");
  const int64_t M = md.rows, N = md.cols;
  const at::Tensor& w = tensor(a[2], "weight");
  const Matrix vw = matrix(w, "weight");
  if (vw.rows != N) throw Refused{"dy is " + shape_of(dy) + ": the weight is " + shape_of(w)};
  Operand mx, mw;
  if (want_w || a[1] != Py_None) {
    const at::Tensor& x = tensor(a[1], "x");
    const Matrix vx = matrix(x, "x");
    if (vx.rows != M || vw.cols != vx.cols)
      throw Refused{"dy is " + shape_of(dy) + " and x " + shape_of(x) + ": the weight is " + shape_of(w)};
    if (want_w) mx = operand(x, "x", &dy);
  }
  Kept kept;
  if (act != GP_ACT_NONE) read_kept(a[4], 1, M, N, dy, &kept);
  if (want_x) mw = operand(w, "weight", &dy);
  at::Tensor dz, dbias, work, dx;
  Operand md16;
  const bool own = act != GP_ACT_NONE && (want_x || want_w);    // dz in memory of its own
  if (!own && (want_x || want_w)) md16 = operand(dy, "dy", nullptr);
  WeightGradients dw;
  if (want_w)
    dw = look_at_weight_gradients(1, N, vw.cols, a[8], a[9], a[10], dy, tensor(a[1], "x"), own ? nullptr : &dy);
  for (Operand* m : {&mx, &mw, &md16}) lay_out(*m, dy, call);
  if (act != GP_ACT_NONE || bias) {
    gp_act_backward g = {};
    g.dy = md.p;
    g.ld_dy = md.ld;
    g.z = kept.z;
    g.ldz = kept.ld;
    g.q = kept.q;
    g.M = M;
    g.N = N;
    g.type = real;
    g.activation = act;
    if (own) {
      dz = rows_of(M, N, dy.scalar_type(), dy);
      g.dz = dz.data_ptr();
      g.ld_dz = dz.stride(0);
    }
    if (bias) {
      dbias = at::empty({N}, dy.options().dtype(at::kFloat));
      g.dbias = dbias.data_ptr<float>();
      check(lib.act_workspace(M, N, 0, &g.workspace_bytes), "ffn_act_backward_workspace");
      if (g.workspace_bytes > 0) {
        work = at::empty({g.workspace_bytes / 4}, dy.options().dtype(at::kFloat));   // (freed in the call's stream order)
        g.workspace = work.data_ptr();
      }
    }
    check(lib.act_backward(&g, call.stream), "ffn_act_backward");
  }
  if (want_x || want_w) {
    if (own) static_cast<Matrix&>(md16) = Matrix{M, N, dz.stride(0), dz.data_ptr()};
    if (want_x) dx = input_gradient(1, &md16, &mw, M, N, vw.cols, real, dy, call, ProductOptions(opts, 1, false).p);
    if (want_w) weight_gradients(1, &md16, mx, N, real, dw, dy, call, ProductOptions(opts, 2, want_x).p);
  }
  return tuple({dx, dw.dw[0], dbias});
}

// gated_backward(dh, x, w_gate, w_up, kept, activation, product, input_grad, weight_grad, out_dtype, addend, out, options)
PyObject* gated_backward(PyObject* const* a) {
  const at::Tensor& dh = tensor(a[0], "dh");
  if (!dh.is_cuda()) throw Refused{"dh must be on a CUDA device"};
  const int real = type16(dh, "dh");
  const Call call(dh);
  const bool product = a[6] == Py_True, want_x = a[7] == Py_True, want_w = a[8] == Py_True;
  const gp_ffn_options* opts = options(a[12]);
  if (!want_w && (a[10] != Py_None || a[11] != Py_None)) throw Refused{"addend and out are for the weights' gradients"};
  if ((a[10] != Py_None) && (item(a[10], 0, 2, "addend") == Py_None) != (item(a[10], 1, 2, "addend") == Py_None))
    throw Refused{"addend takes 2 matrices"};
  const Matrix md = rows_apart(dh, "dh");
  const int64_t M = md.rows, N = md.cols;
  const at::Tensor &wg = tensor(a[2], "w_gate"), &wu = tensor(a[3], "w_up");
  const Matrix vg = matrix(wg, "w_gate"), vu = matrix(wu, "w_up");
  if (vg.rows != N || vu.rows != N || vu.cols != vg.cols)
    throw Refused{"dh is " + shape_of(dh) + ": the weights are " + shape_of(wg) + " and " + shape_of(wu)};
  Operand mx, mw[2];
  if (want_w || a[1] != Py_None) {
    const at::Tensor& x = tensor(a[1], "x");
    const Matrix vx = matrix(x, "x");
    if (vx.rows != M || vx.cols != vg.cols)
      throw Refused{"dh is " + shape_of(dh) + " and x " + shape_of(x) + ": the weights are " + shape_of(wg) + " and " + shape_of(wu)};
    if (want_w) mx = operand(x, "x", &dh);
  }
  Kept kept[2];
  read_kept(a[4], 2, M, N, dh, kept);
  if (want_x) {
    mw[0] = operand(wg, "w_gate", &dh);
    mw[1] = operand(wu, "w_up", &dh);
  }
  WeightGradients dw;
  if (want_w) dw = look_at_weight_gradients(2, N, vg.cols, a[9], a[10], a[11], dh, tensor(a[1], "x"), nullptr);
  for (Operand* m : {&mx, &mw[0], &mw[1]}) lay_out(*m, dh, call);
  // the products' gradients, one after the other
  const int64_t ld = up(N, 8);
  at::Tensor both = at::empty_strided({2 * M, N}, {ld, 1}, dh.options()), h, dx;
  const Matrix dz[2] = {Matrix{M, N, ld, both.data_ptr()},
                        Matrix{M, N, ld, static_cast<char*>(both.data_ptr()) + 2 * M * ld}};
  gp_gated_backward g = {};
  g.dh = md.p;
  g.ld_dh = md.ld;
  g.z_gate = kept[0].z;
  g.z_up = kept[1].z;
  g.ld_zg = kept[0].ld;
  g.ld_zu = kept[1].ld;
  g.q_gate = kept[0].q;
  g.q_up = kept[1].q;
  g.dgate = dz[0].p;
  g.dup = dz[1].p;
  g.ld_dgate = g.ld_dup = ld;
  if (product) {
    h = rows_of(M, N, dh.scalar_type(), dh);
    g.h = h.data_ptr();
    g.ldh = h.stride(0);
  }
  g.M = M;
  g.N = N;
  g.type = real;
  g.activation = static_cast<int32_t>(PyLong_AsLong(a[5]));
  check(lib.gated_backward(&g, call.stream), "ffn_gated_backward");
  if (want_x) dx = input_gradient(2, dz, mw, M, N, vg.cols, real, dh, call, ProductOptions(opts, 1, false).p);
  if (want_w) weight_gradients(2, dz, mx, N, real, dw, dh, call, ProductOptions(opts, 2, want_x).p);
  return product ? tuple({dx, dw.dw[0], dw.dw[1], h}) : tuple({dx, dw.dw[0], dw.dw[1]});
}

// ---------------------------------------------------------------------------
// the module
// ---------------------------------------------------------------------------
// Errors of any kind become Python's.
template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS || !g_failed) {
    PyErr_SetString(PyExc_TypeError, g_failed ? "wrong number of arguments" : "the library is not loaded");
    return nullptr;
  }
  try {
    PyObject* r = F(args);
    if (PyErr_Occurred()) {
      Py_XDECREF(r);
      return nullptr;
    }
    return r;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Wrong& e) {
    PyErr_SetString(PyExc_TypeError, e.what.c_str());
  } catch (const Failed& e) {
    PyObject* x = PyObject_CallFunction(g_failed, "is", e.code, e.where);
    if (x) {
      PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(x)), x);
      Py_DECREF(x);
    }
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* cuda = PyImport_ImportModule("torch");
    PyObject* type = cuda ? PyObject_GetAttrString(cuda, "OutOfMemoryError") : nullptr;
    Py_XDECREF(cuda);
    if (!type) PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_RuntimeError, e.what_without_backtrace());
    Py_XDECREF(type);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// load(path of the library, exception maker)
PyObject* load(PyObject*, PyObject* const* args, Py_ssize_t n) {
  const char* path = n == 2 ? PyUnicode_AsUTF8(args[0]) : nullptr;
  if (!path) {
    PyErr_SetString(PyExc_TypeError, "load takes a path and a callable");
    return nullptr;
  }
  void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(h, name));
    return f != nullptr;
  };
  if (!(find(lib.linear, "gemm_linear") && find(lib.gated, "gemm_gated") && find(lib.input_grad, "gemm_input_grad") &&
        find(lib.weight_grad, "gemm_weight_grad") && find(lib.act_backward, "ffn_act_backward") &&
        find(lib.act_workspace, "ffn_act_backward_workspace") && find(lib.gated_backward, "ffn_gated_backward") &&
        find(lib.pack, "ffn_pack_rows"))) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks a function of gemm_ffn.h");
    return nullptr;
  }
  Py_INCREF(args[1]);
  Py_XSETREF(g_failed, args[1]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"load", fast(load), METH_FASTCALL, "load(path, exception): the library whose functions are called"},
    {"linear", fast(guarded<linear, 9>), METH_FASTCALL, nullptr},
    {"gated", fast(guarded<gated, 7>), METH_FASTCALL, nullptr},
    {"linear_backward", fast(guarded<linear_backward, 12>), METH_FASTCALL, nullptr},
    {"gated_backward", fast(guarded<gated_backward, 13>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_ffn", "The feed-forward operators on torch tensors (see ffn.py).", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ffn() { return PyModule_Create(&module); }
