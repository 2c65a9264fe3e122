// The operators around the expert layer on torch tensors: argument checks,
// output tensors from torch's allocator and the call of the C entry point on
// torch's current stream (include/qmoe.h defines what each computes).
//
// A CPython module because the smallest calls are bound by the host: checks and
// allocations in Python took 7 to 14 us of a call whose kernel takes 3.  The
// arguments are positional; ops.py gives them names, streams and automatic
// differentiation.  A refused argument raises QMoEError.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "../../include/qmoe.h"

namespace {

using at::Tensor;

// Python classes of ops.py, set once by setup().
PyObject *g_error = nullptr, *g_plan = nullptr, *g_mx4 = nullptr, *g_stats = nullptr, *g_grads = nullptr;

// A Python exception is set.
struct Refused {};

[[noreturn]] void raise(int status, const std::string& msg) {
  PyObject* args = Py_BuildValue("(is)", status, msg.c_str());
  if (args) {
    PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, args);
    Py_DECREF(args);
  }
  throw Refused{};
}
[[noreturn]] void refuse(const std::string& msg) { raise(QMOE_ERR_INVALID_ARG, msg); }
void check(qmoe_status st) {
  if (st != QMOE_OK) raise(st, qmoe_op_last_error());
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

int dtype_code(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return QMOE_F32;
  if (t == at::kHalf) return QMOE_F16;
  if (t == at::kBFloat16) return QMOE_BF16;
  refuse(std::string(name) + " is " + c10::toString(t) + ": float32, float16 or bfloat16");
}

// The tensor that decides the device, which has to be the current one.
const Tensor& first(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != c10::cuda::current_device()) refuse(std::string(name) + " is not on the current device");
  return t;
}
// A further one, on the same device and of a given type.
const Tensor& further(PyObject* o, const char* name, at::ScalarType type, const Tensor& like) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type) refuse(std::string(name) + " is " + c10::toString(t.scalar_type()) + ", not " + c10::toString(type));
  if (t.get_device() != like.get_device()) refuse(std::string(name) + " is not on the current device");
  return t;
}

// Rows of `width` values (the last axis), `n` of them, `ld` apart; a copy is
// made where the last axis is not contiguous or rows overlap.
struct Rows {
  Tensor held;
  const void* p = nullptr;
  int64_t n = 0, width = 0, ld = 0;
};
Rows rows_of(const Tensor& t) {
  Rows r;
  const auto sizes = t.sizes(), strides = t.strides();
  const int64_t d = t.dim();
  r.width = sizes[d - 1];
  r.n = 1;
  for (int64_t i = 0; i + 1 < d; ++i) r.n *= sizes[i];
  r.ld = r.width > 0 ? r.width : 1;
  if (!t.is_contiguous()) {
    const bool plain = d == 2 && (strides[1] == 1 || r.width <= 1) && (strides[0] >= r.width || r.n <= 1);
    if (!plain) {
      r.held = t.contiguous();
      r.p = r.held.const_data_ptr();
      return r;
    }
    if (r.n > 1) r.ld = strides[0];
  }
  r.p = t.const_data_ptr();
  return r;
}
Rows rows_2d(const Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(std::string(name) + " must be two-dimensional, not " + shape_of(t.sizes()));
  return rows_of(t);
}

// A tensor's elements in order.
struct Flat {
  Tensor held;
  void* p = nullptr;
};
Flat flat(const Tensor& t) {
  Flat f;
  if (t.is_contiguous()) {
    f.p = const_cast<void*>(t.const_data_ptr());
  } else {
    f.held = t.contiguous();
    f.p = const_cast<void*>(f.held.const_data_ptr());
  }
  return f;
}
// A further tensor of `numel` elements.
Flat flat(PyObject* o, const char* name, at::ScalarType type, int64_t numel, const Tensor& like) {
  const Tensor& t = further(o, name, type, like);
  if (t.numel() != numel) refuse(std::string(name) + " has " + std::to_string(t.numel()) + " elements, not " + std::to_string(numel));
  return flat(t);
}
// A value a route: [tokens, k], or flat.
Flat route_values(PyObject* o, const char* name, int64_t tokens, int64_t k, const Tensor& like) {
  const Tensor& t = further(o, name, at::kFloat, like);
  const auto s = t.sizes();
  if (!(s.size() == 2 && s[0] == tokens && s[1] == k) && !(s.size() == 1 && s[0] == tokens * k))
    refuse(std::string(name) + " is " + shape_of(s) + ", not " + shape_of({tokens, k}));
  return flat(t);
}
// A value a column: [width], or with leading axes of one.
Flat column_values(PyObject* o, const char* name, int64_t width, const Tensor& like) {
  const Tensor& t = further(o, name, like.scalar_type(), like);
  if (t.dim() < 1 || t.size(-1) != width || t.numel() != width)
    refuse(std::string(name) + " is " + shape_of(t.sizes()) + ", not " + shape_of({width}));
  return flat(t);
}

Tensor make(at::IntArrayRef size, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}
void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }
PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* wrap_or_none(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
void* ptr(const Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }

long to_long(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
double to_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

// An ExpertPlan.
struct Plan {
  Flat pos, offsets;
  int64_t tokens = 0;
  int k = 0, experts = 0;
};
Plan plan_of(PyObject* o, const Tensor& like, int64_t tokens = -1) {
  if (!g_plan || !PyObject_TypeCheck(o, reinterpret_cast<PyTypeObject*>(g_plan)) || PyTuple_GET_SIZE(o) != 5)
    refuse("plan must be an ExpertPlan");
  Plan p;
  p.k = (int)to_long(PyTuple_GET_ITEM(o, 3), "plan.k");
  p.experts = (int)to_long(PyTuple_GET_ITEM(o, 4), "plan.experts");
  PyObject* pos = PyTuple_GET_ITEM(o, 1);
  const int64_t n = THPVariable_Check(pos) ? THPVariable_Unpack(pos).numel() : 0;
  if (p.k < 1 || n % p.k) refuse("plan.pos does not hold whole tokens");
  p.tokens = n / p.k;
  if (tokens >= 0 && p.tokens != tokens)
    refuse("the plan is of " + std::to_string(p.tokens) + " tokens, not " + std::to_string(tokens));
  p.pos = flat(pos, "plan.pos", at::kInt, n, like);
  p.offsets = flat(PyTuple_GET_ITEM(o, 2), "plan.offsets", at::kInt, (int64_t)p.experts + 1, like);
  return p;
}

// Every entry: translate exceptions, never let one into the interpreter.
template <typename F>
PyObject* entry(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "takes %zd arguments (%zd given)", want, n);
    throw Refused{};
  }
}
#define ENTRY(name, count)                                              \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n_args) { \
    return entry([&]() -> PyObject* {                                \
      need_args(n_args, count);
#define END_ENTRY \
  });             \
  }

// setup(QMoEError, ExpertPlan, MX4Tensor, NormStats, NormGrads)
ENTRY(setup, 5)
PyObject** to[] = {&g_error, &g_plan, &g_mx4, &g_stats, &g_grads};
for (int i = 0; i < 5; ++i) {
  Py_INCREF(a[i]);
  Py_XDECREF(*to[i]);
  *to[i] = a[i];
}
Py_RETURN_NONE;
END_ENTRY

// ---- tokens sorted by expert and back ----

// (ids, experts) -> ExpertPlan
ENTRY(expert_sort, 2)
const Tensor& ids = first(a[0], "ids");
const auto type = ids.scalar_type();
if (type != at::kInt && type != at::kLong) refuse(std::string("ids is ") + c10::toString(type) + ": int32 or int64");
const long experts = to_long(a[1], "experts");
const Rows r = rows_2d(ids, "ids");
const int64_t R = r.n * r.width;
if (experts < 1 || experts > INT32_MAX) refuse("experts " + std::to_string(experts) + " is not positive");
if (r.width < 1) refuse("ids has no slots");
Tensor perm = make({R}, at::kInt, ids), pos = make({R}, at::kInt, ids), offsets = make({(int64_t)experts + 1}, at::kInt, ids);
check(qmoe_expert_sort(r.p, type == at::kInt ? 4 : 8, r.ld, r.n, (int)r.width, (int)experts, perm.mutable_data_ptr<int32_t>(),
                       pos.mutable_data_ptr<int32_t>(), offsets.mutable_data_ptr<int32_t>(), stream()));
PyObject *o0 = wrap(perm), *o1 = wrap(pos), *o2 = wrap(offsets), *o3 = PyLong_FromLong((long)r.width);
PyObject* out = o0 && o1 && o2 && o3 ? PyObject_CallFunctionObjArgs(g_plan, o0, o1, o2, o3, a[1], nullptr) : nullptr;
Py_XDECREF(o0);
Py_XDECREF(o1);
Py_XDECREF(o2);
Py_XDECREF(o3);
return out;
END_ENTRY

// (x, plan) -> xs
ENTRY(dispatch, 2)
const Tensor& x = first(a[0], "x");
const int dt = dtype_code(x.scalar_type(), "x");
const Rows r = rows_2d(x, "x");
const Plan p = plan_of(a[1], x, r.n);
Tensor xs = make({r.n * p.k, r.width}, x.scalar_type(), x);
check(qmoe_dispatch(r.p, r.ld, static_cast<int32_t*>(p.pos.p), static_cast<int32_t*>(p.offsets.p), r.n, p.k, p.experts, r.width,
                    dt, xs.mutable_data_ptr(), stream()));
return wrap(std::move(xs));
END_ENTRY

// (y, weights or None, plan) -> out; dispatch's gradient without weights
ENTRY(combine, 3)
const Tensor& y = first(a[0], "y");
const int dt = dtype_code(y.scalar_type(), "y");
const Rows r = rows_2d(y, "y");
const Plan p = plan_of(a[2], y);
if (r.n != p.tokens * p.k)
  refuse("y has " + std::to_string(r.n) + " rows, the plan " + std::to_string(p.tokens * p.k));
Flat w;
if (a[1] != Py_None) w = route_values(a[1], "weights", p.tokens, p.k, y);
Tensor out = make({p.tokens, r.width}, y.scalar_type(), y);
check(qmoe_combine(r.p, r.ld, static_cast<float*>(w.p), static_cast<int32_t*>(p.pos.p), p.tokens, p.k, r.width, dt,
                   out.mutable_data_ptr(), stream()));
return wrap(std::move(out));
END_ENTRY

// (dout, y, weights or None, plan, need dy, need dweights) -> (dy or None, dweights or None)
ENTRY(combine_grad, 6)
const Tensor& dout = first(a[0], "dout");
const int dt = dtype_code(dout.scalar_type(), "dout");
const Rows r = rows_2d(dout, "dout");
const Plan p = plan_of(a[3], dout, r.n);
const bool need_dy = PyObject_IsTrue(a[4]) == 1, need_dw = PyObject_IsTrue(a[5]) == 1;
Flat w;
if (a[2] != Py_None) w = route_values(a[2], "weights", r.n, p.k, dout);
Rows y;
if (need_dw) {
  y = rows_2d(further(a[1], "y", dout.scalar_type(), dout), "y");
  if (y.n != r.n * p.k || y.width != r.width)
    refuse("y is " + shape_of({y.n, y.width}) + ", not " + shape_of({r.n * p.k, r.width}));
}
Tensor dy, dw;
if (need_dy) dy = make({r.n * p.k, r.width}, dout.scalar_type(), dout);
if (need_dw) dw = make({r.n, (int64_t)p.k}, at::kFloat, dout);
check(qmoe_combine_grad(r.p, r.ld, y.p, need_dw ? y.ld : r.width, static_cast<float*>(w.p), static_cast<int32_t*>(p.pos.p),
                        static_cast<int32_t*>(p.offsets.p), r.n, p.k, p.experts, r.width, dt, ptr(dy),
                        static_cast<float*>(ptr(dw)), stream()));
PyObject *o0 = wrap_or_none(dy), *o1 = wrap_or_none(dw);
PyObject* out = o0 && o1 ? PyTuple_Pack(2, o0, o1) : nullptr;
Py_XDECREF(o0);
Py_XDECREF(o1);
return out;
END_ENTRY

// ---- microscaled 4-bit floating point ----

PyObject* make_mx4(Tensor codes, Tensor scales, int64_t cols) {
  PyObject *o0 = wrap(std::move(codes)), *o1 = wrap(std::move(scales)), *o2 = PyLong_FromLongLong(cols);
  PyObject* out = o0 && o1 && o2 ? PyObject_CallFunctionObjArgs(g_mx4, o0, o1, o2, nullptr) : nullptr;
  Py_XDECREF(o0);
  Py_XDECREF(o1);
  Py_XDECREF(o2);
  return out;
}

// (x, plan or None, QMOE_ACT_* or QMOE_ACT_NONE) -> MX4Tensor
ENTRY(mx4_quantize, 3)
const Tensor& x = first(a[0], "x");
const int dt = dtype_code(x.scalar_type(), "x");
const long act = to_long(a[2], "activation");
if (x.dim() < 2) refuse("x must have rows: two dimensions at least");
const Rows r = rows_of(x);
int64_t cols = r.width;
if (act != QMOE_ACT_NONE) {
  if (cols % 2) refuse("gate | up needs an even row length, not " + std::to_string(cols));
  cols /= 2;
}
if (cols < 1) refuse("x has rows without values");
Plan p;
p.k = p.experts = 1;
int64_t n = x.size(-2);
if (a[1] != Py_None) {
  if (x.dim() != 2) refuse("with a plan x is [T, K]");
  p = plan_of(a[1], x, r.n);
  n = r.n * p.k;
}
const int64_t nb = (cols + 31) / 32, nq = (nb + 3) / 4;
c10::SmallVector<int64_t, 6> cs(x.sizes().begin(), x.sizes().end() - 2), ss(cs);
cs.append({n, nb * 16});
ss.append({nq, n, 4});
Tensor codes = make(cs, at::kByte, x), scales = make(ss, at::kByte, x);
check(qmoe_mx4_quantize(r.p, r.ld, r.n, cols, dt, (int)act, static_cast<int32_t*>(p.pos.p), static_cast<int32_t*>(p.offsets.p),
                        p.k, p.experts, n, codes.mutable_data_ptr<uint8_t>(), scales.mutable_data_ptr<uint8_t>(), stream()));
return make_mx4(std::move(codes), std::move(scales), cols);
END_ENTRY

// An MX4Tensor.
struct Mx4 {
  const Tensor* codes_t = nullptr;
  Flat codes, scales;
  int64_t cols = 0, rows = 0;   // values a row, rows of a matrix
};
Mx4 mx4_of(PyObject* o, const char* name, const Tensor* like) {
  const std::string nm(name);
  if (!g_mx4 || !PyObject_TypeCheck(o, reinterpret_cast<PyTypeObject*>(g_mx4)) || PyTuple_GET_SIZE(o) != 3)
    refuse(nm + " must be an MX4Tensor");
  Mx4 m;
  m.cols = to_long(PyTuple_GET_ITEM(o, 2), "cols");
  const std::string nc = nm + ".codes", ns = nm + ".scales";
  const Tensor& c = like ? further(PyTuple_GET_ITEM(o, 0), nc.c_str(), at::kByte, *like) : first(PyTuple_GET_ITEM(o, 0), nc.c_str());
  const int64_t nb = (m.cols + 31) / 32, nq = (nb + 3) / 4, d = c.dim();
  if (m.cols < 1 || d < 2 || c.scalar_type() != at::kByte || c.size(-1) != nb * 16)
    refuse(nc + " " + shape_of(c.sizes()) + " does not hold rows of " + std::to_string(m.cols) + " values");
  m.codes_t = &c;
  m.rows = c.size(-2);
  m.codes = flat(PyTuple_GET_ITEM(o, 0), nc.c_str(), at::kByte, c.numel(), c);
  m.scales = flat(PyTuple_GET_ITEM(o, 1), ns.c_str(), at::kByte, c.numel() / (nb * 16) * nq * 4, c);
  const auto ss = THPVariable_Unpack(PyTuple_GET_ITEM(o, 1)).sizes();
  bool same = (int64_t)ss.size() == d + 1 && ss[d] == 4 && ss[d - 1] == m.rows && ss[d - 2] == nq;
  for (int64_t i = 0; same && i + 2 < d; ++i) same = ss[i] == c.size(i);
  if (!same) refuse(ns + " " + shape_of(ss) + " does not belong to codes " + shape_of(c.sizes()));
  return m;
}

// (q, dtype code) -> values
ENTRY(mx4_dequantize, 2)
const Mx4 q = mx4_of(a[0], "q", nullptr);
const long dt = to_long(a[1], "dtype");
const at::ScalarType type = dt == QMOE_F32 ? at::kFloat : dt == QMOE_F16 ? at::kHalf : at::kBFloat16;
c10::SmallVector<int64_t, 6> size(q.codes_t->sizes().begin(), q.codes_t->sizes().end());
size.back() = q.cols;
Tensor out = make(size, type, *q.codes_t);
check(qmoe_mx4_dequantize(static_cast<uint8_t*>(q.codes.p), static_cast<uint8_t*>(q.scales.p), out.numel() / q.cols, q.cols,
                          q.rows, (int)dt, out.mutable_data_ptr(), q.cols, stream()));
return wrap(std::move(out));
END_ENTRY

// (a, w, plan or None, dtype code) -> product
ENTRY(mx4_matmul, 4)
const Mx4 x = mx4_of(a[0], "a", nullptr), w = mx4_of(a[1], "w", x.codes_t);
const long dt = to_long(a[3], "out_dtype");
const at::ScalarType type = dt == QMOE_F32 ? at::kFloat : dt == QMOE_F16 ? at::kHalf : at::kBFloat16;
if (x.codes_t->dim() != 2) refuse("a must be [R, K]");
if (x.cols != w.cols) refuse("a has rows of " + std::to_string(x.cols) + " values, w of " + std::to_string(w.cols));
Plan p;
p.k = p.experts = 1;
if (a[2] != Py_None) {
  p = plan_of(a[2], *x.codes_t);
  if (p.tokens * p.k != x.rows)
    refuse("a has " + std::to_string(x.rows) + " rows, the plan " + std::to_string(p.tokens * p.k));
}
const int64_t d = w.codes_t->dim();
if (d > 3 || (d == 3 ? w.codes_t->size(0) : 1) != p.experts)
  refuse("w.codes " + shape_of(w.codes_t->sizes()) + " does not hold " + std::to_string(p.experts) + " expert(s)");
Tensor out = make({x.rows, w.rows}, type, *x.codes_t);
check(qmoe_mx4_matmul(static_cast<uint8_t*>(x.codes.p), static_cast<uint8_t*>(x.scales.p), x.rows, static_cast<uint8_t*>(w.codes.p),
                      static_cast<uint8_t*>(w.scales.p), static_cast<int32_t*>(p.offsets.p), p.experts, w.rows, x.cols, (int)dt,
                      out.mutable_data_ptr(), w.rows, stream()));
return wrap(std::move(out));
END_ENTRY

// ---- norms around a block ----

Rows norm_rows(PyObject* o, const char* name, const Tensor& x) {
  const Tensor& t = further(o, name, x.scalar_type(), x);
  if (t.sizes() != x.sizes()) refuse(std::string(name) + " must have the shape " + shape_of(x.sizes()) + ", not " + shape_of(t.sizes()));
  return rows_of(t);
}
struct Norm {
  const Tensor* x = nullptr;
  Rows rx, ro, rg;
  Flat g, wq, wp;
  const void* gate = nullptr;
  int kind = QMOE_GATE_NONE, dt = 0;
  bool has_o = false;
};
// x, o, gate, w_post, w_pre at a[0 .. 4]
Norm norm_of(PyObject* const* a) {
  Norm m;
  const Tensor& x = first(a[0], "x");
  m.x = &x;
  m.dt = dtype_code(x.scalar_type(), "x");
  if (x.dim() < 1 || x.size(-1) < 1) refuse("x must have rows of at least one value");
  m.rx = rows_of(x);
  m.has_o = a[1] != Py_None;
  if (m.has_o) m.ro = norm_rows(a[1], "o", x);
  if (a[2] != Py_None) {
    if (!m.has_o) refuse("gate needs o");
    const Tensor& g = further(a[2], "gate", x.scalar_type(), x);
    const auto gs = g.sizes(), xs = x.sizes();
    if (gs == xs) {
      m.kind = QMOE_GATE_FULL;
      m.rg = rows_of(g);
      m.gate = m.rg.p;
    } else if (gs.size() == 1 && gs[0] == m.rx.width) {
      m.kind = QMOE_GATE_CHANNEL;
      m.g = flat(a[2], "gate", x.scalar_type(), m.rx.width, x);
      m.gate = m.g.p;
    } else if (gs.size() == xs.size() && gs.back() == 1 && gs.slice(0, gs.size() - 1) == xs.slice(0, xs.size() - 1)) {
      m.kind = QMOE_GATE_TOKEN;
      m.g = flat(a[2], "gate", x.scalar_type(), m.rx.n, x);
      m.gate = m.g.p;
    } else {
      refuse("gate " + shape_of(gs) + " is not of the shape of x, of its last axis or of its rows");
    }
  }
  if (a[3] != Py_None) m.wq = column_values(a[3], "w_post", m.rx.width, x);
  if (a[4] != Py_None) m.wp = column_values(a[4], "w_pre", m.rx.width, x);
  return m;
}
PyObject* make_stats(const Tensor& s1, const Tensor& s2) {
  PyObject *o0 = wrap_or_none(s1), *o1 = wrap_or_none(s2);
  PyObject* out = o0 && o1 ? PyObject_CallFunctionObjArgs(g_stats, o0, o1, nullptr) : nullptr;
  Py_XDECREF(o0);
  Py_XDECREF(o1);
  return out;
}

// (x, o, gate, w_post, w_pre, residual_scale, eps, statistics wanted) -> (r, h), with statistics (r, h, NormStats)
ENTRY(block_norm, 8)
const Norm m = norm_of(a);
const Tensor& x = *m.x;
const float scale = (float)to_double(a[5]), eps = (float)to_double(a[6]);
const bool stats = PyObject_IsTrue(a[7]) == 1, post = a[3] != Py_None, pre = a[4] != Py_None;
Tensor r = make(x.sizes(), x.scalar_type(), x), h, s1, s2;
if (pre) h = make(x.sizes(), x.scalar_type(), x);
if (stats && post) s1 = make({m.rx.n}, at::kFloat, x);
if (stats && pre) s2 = make({m.rx.n}, at::kFloat, x);
check(qmoe_block_norm(m.rx.p, m.rx.ld, m.ro.p, m.ro.ld, m.gate, m.kind, m.rg.ld, m.wq.p, m.wp.p, scale, eps, m.rx.n, m.rx.width,
                      m.dt, r.mutable_data_ptr(), ptr(h), static_cast<float*>(ptr(s1)), static_cast<float*>(ptr(s2)), stream()));
PyObject *o0 = wrap(std::move(r)), *o1 = wrap_or_none(h), *o2 = stats ? make_stats(s1, s2) : nullptr;
PyObject* out = !o0 || !o1 || (stats && !o2) ? nullptr : stats ? PyTuple_Pack(3, o0, o1, o2) : PyTuple_Pack(2, o0, o1);
Py_XDECREF(o0);
Py_XDECREF(o1);
Py_XDECREF(o2);
return out;
END_ENTRY

// (x, o, gate, w_post, w_pre, dr, dh, rstd_post, rstd_pre, residual_scale) -> NormGrads
ENTRY(block_norm_grad, 10)
const Norm m = norm_of(a);
const Tensor& x = *m.x;
const auto type = x.scalar_type();
const int64_t T = m.rx.n, H = m.rx.width;
Rows dr, dh;
if (a[5] != Py_None) dr = norm_rows(a[5], "dr", x);
if (a[6] != Py_None) {
  if (a[4] == Py_None) refuse("dh needs w_pre");
  dh = norm_rows(a[6], "dh", x);
}
Flat s1, s2;
if (a[3] != Py_None) s1 = flat(a[7], "stats.rstd_post", at::kFloat, T, x);
if (a[4] != Py_None) s2 = flat(a[8], "stats.rstd_pre", at::kFloat, T, x);
const float scale = (float)to_double(a[9]);
Tensor dx = make(x.sizes(), type, x), d_o, dg, dwq, dwp;
if (m.has_o) d_o = make(x.sizes(), type, x);
if (m.gate || m.kind != QMOE_GATE_NONE) dg = make(THPVariable_Unpack(a[2]).sizes(), type, x);
if (a[3] != Py_None) dwq = make(THPVariable_Unpack(a[3]).sizes(), type, x);
if (a[4] != Py_None) dwp = make(THPVariable_Unpack(a[4]).sizes(), type, x);
const size_t bytes = qmoe_block_norm_grad_workspace(T, H, m.dt);
Tensor work = make({(int64_t)bytes}, at::kByte, x);
check(qmoe_block_norm_grad(dr.p, dr.ld, dh.p, dh.ld, m.rx.p, m.rx.ld, m.ro.p, m.ro.ld, m.gate, m.kind, m.rg.ld, m.wq.p, m.wp.p,
                           static_cast<float*>(s1.p), static_cast<float*>(s2.p), scale, T, H, m.dt, dx.mutable_data_ptr(), ptr(d_o),
                           ptr(dg), ptr(dwq), ptr(dwp), work.mutable_data_ptr(), bytes, stream()));
PyObject* o[] = {wrap(std::move(dx)), wrap_or_none(d_o), wrap_or_none(dg), wrap_or_none(dwq), wrap_or_none(dwp)};
PyObject* out = o[0] && o[1] && o[2] && o[3] && o[4]
                    ? PyObject_CallFunctionObjArgs(g_grads, o[0], o[1], o[2], o[3], o[4], nullptr)
                    : nullptr;
for (PyObject* q : o) Py_XDECREF(q);
return out;
END_ENTRY

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(setup),          METHOD(expert_sort),  METHOD(dispatch),   METHOD(combine),
                           METHOD(combine_grad),   METHOD(mx4_quantize), METHOD(mx4_dequantize), METHOD(mx4_matmul),
                           METHOD(block_norm),     METHOD(block_norm_grad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops_torch", "Operators around the expert layer on torch tensors", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_torch() { return PyModule_Create(&g_module); }
