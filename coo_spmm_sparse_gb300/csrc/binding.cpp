// Python binding of the dense operators: argument checks, output and scratch
// tensors, and the C calls.  The calls of a decode step take a few
// microseconds on the GPU; the same checks and allocations made from Python
// took 24 us (norm of one token) to 430 us (a list of 700 tensors).
//
// Every function takes positional arguments only; signatures, defaults and
// documentation are the Python functions' that call them.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <limits>
#include <memory>
#include <optional>
#include <string>
#include <vector>

#include "snack.h"

namespace {

PyObject *g_error = nullptr;  // SnackError

// A Python exception that is already set.
struct Raised {};

[[noreturn]] void type_error(const std::string &m) {
  PyErr_SetString(PyExc_TypeError, m.c_str());
  throw Raised{};
}
[[noreturn]] void value_error(const std::string &m) {
  PyErr_SetString(PyExc_ValueError, m.c_str());
  throw Raised{};
}

void check(snack_status st) {
  if (st == SNACK_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", (int)st, snack_last_error(nullptr));
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

std::string shape(const at::Tensor &t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

int type_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return SNACK_F32;
    case at::kBFloat16: return SNACK_BF16;
    case at::kHalf: return SNACK_F16;
    default: return -1;
  }
}

bool is_tensor(PyObject *o) { return THPVariable_Check(o); }

// A CUDA tensor of one of the three types.
const at::Tensor &dense(PyObject *o, const char *name) {
  if (is_tensor(o)) {
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.is_cuda() && type_code(t.scalar_type()) >= 0) return t;
  }
  type_error(std::string(name) + " must be a CUDA float32, bfloat16 or float16 tensor");
}

const at::Tensor *dense_or_none(PyObject *o, const char *name) {
  return o == Py_None ? nullptr : &dense(o, name);
}

const void *addr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

// Tells autograd that the call writes t, a tensor of the caller's: what kept
// it for a backward pass then raises rather than use the new values.
// (Inference tensors have no version.)
void written(const at::Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject *o) { written(THPVariable_Unpack(o)); }

// (rows, row stride) of t seen as [rows][last dimension].
struct Rows {
  int64_t n, step;
};
Rows rows_of(const at::Tensor &t, const char *name) {
  const int64_t d = t.dim() ? t.size(-1) : 1;
  if (t.is_contiguous()) return {d ? t.numel() / d : 0, d};
  if (t.dim() < 2 || (d > 1 && t.stride(-1) != 1))
    value_error(std::string(name) + " must be contiguous along its last dimension");
  int64_t n = 1, step = -1;
  for (int64_t i = t.dim() - 2; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (step < 0)
      step = t.stride(i);
    else if (t.stride(i) != step * n)
      value_error(std::string(name) + ": the rows of its leading dimensions are not evenly spaced");
    n *= t.size(i);
  }
  if (step < 0) step = d;
  if (step < d) value_error(std::string(name) + ": its rows overlap");
  return {n, step};
}

// All tensors of a call lie on the current device.
struct Device {
  c10::Device dev{c10::kCUDA, -1};
  void add(const at::Tensor *t) {
    if (!t) return;
    if (dev.index() < 0) {
      dev = t->device();
      const int cur = c10::cuda::current_device();
      if (dev.index() != cur)
        value_error("cuda:" + std::to_string(dev.index()) + " is not the current CUDA device");
    } else if (t->device() != dev) {
      value_error("all tensors must be on one device");
    }
  }
};

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
  return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
}

// The stream of a call.  One that is given is made current for the call: what
// it allocates and clears belongs to that stream, as under torch.cuda.stream().
struct Stream {
  void *raw;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  Stream(PyObject *o, c10::Device d) {
    if (o == Py_None) {
      raw = c10::cuda::getCurrentCUDAStream(d.index()).stream();
      return;
    }
    raw = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Raised{};
    guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), d.index()));
  }
  at::Tensor scratch(size_t bytes, c10::Device d) const {
    return bytes ? empty({(int64_t)bytes}, at::kByte, d) : at::Tensor();
  }
};

void *scratch_addr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("takes " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

template <typename F>
PyObject *guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *same(PyObject *o) {
  Py_INCREF(o);
  return o;
}

// ------------------------------------------------------------------ residual norm

// The options both calls share, from `o`: gate, post_weight, post_bias,
// next_weight, next_bias, kind, post_norm, next_norm, residual_scale,
// branch_scale, eps, branch_dtype.
constexpr int kNormOptions = 12;
struct Norm {
  snack_norm_args a{};
  Device dev;
  const at::Tensor *x, *y, *gate, *param[4];
  at::ScalarType branch;

  Norm(PyObject *x_, PyObject *y_, PyObject *const *o) {
    static const char *const names[4] = {"post_weight", "post_bias", "next_weight", "next_bias"};
    a.norm_kind = (int)PyLong_AsLong(o[5]);
    a.post_norm = truth(o[6]);
    a.next_norm = truth(o[7]);
    a.residual_scale = (float)number(o[8]);
    a.branch_scale = (float)number(o[9]);
    a.eps = (float)number(o[10]);
    x = &dense(x_, "x");
    y = dense_or_none(y_, "y");
    gate = o[0] == Py_None ? nullptr : &dense(o[0], "gate");
    if (x->dim() < 1 || x->size(-1) < 1) value_error("x must have a last dimension of at least 1");
    if (y) {
      if (y->sizes() != x->sizes()) value_error("y " + shape(*y) + " must have x's shape " + shape(*x));
      branch = y->scalar_type();
    } else if (a.post_norm || gate) {
      value_error("post_norm and gate need y");
    } else if (o[11] == Py_None) {
      branch = x->scalar_type();
    } else {
      if (!THPDtype_Check(o[11]) || type_code(reinterpret_cast<THPDtype *>(o[11])->scalar_type) < 0)
        type_error("branch_dtype must be float32, bfloat16 or float16");
      branch = reinterpret_cast<THPDtype *>(o[11])->scalar_type;
    }
    a.stream_type = type_code(x->scalar_type());
    a.branch_type = type_code(branch);
    if (a.stream_type != a.branch_type && a.stream_type != SNACK_F32)
      type_error("x must be float32 or have the branch's type");
    a.width = x->size(-1);
    a.param_type = -1;
    for (int i = 0; i < 4; ++i) {
      param[i] = dense_or_none(o[1 + i], names[i]);
      if (!param[i]) continue;
      const std::string name = names[i];
      if (!(i < 2 ? a.post_norm : a.next_norm)) value_error(name + " without its norm");
      const int k = type_code(param[i]->scalar_type());
      if (k != SNACK_F32 && k != a.branch_type) type_error(name + " must be float32 or have the branch's type");
      if (a.param_type >= 0 && k != a.param_type) type_error("weights and biases must have one type");
      if (param[i]->dim() != 1 || param[i]->numel() != a.width || !param[i]->is_contiguous())
        value_error(name + " must be a contiguous vector of " + std::to_string(a.width));
      a.param_type = k;
    }
    if (a.param_type < 0) a.param_type = SNACK_F32;
    const Rows xr = rows_of(*x, "x");
    a.rows = xr.n;
    a.x_stride = xr.step;
    if (y) a.y_stride = rows_of(*y, "y").step;
    if (gate) set_gate();
    dev.add(x);
    dev.add(y);
    dev.add(gate);
    for (auto *p : param) dev.add(p);
    a.x = addr(x);
    a.y = addr(y);
    a.gate = addr(gate);
    a.post_weight = addr(param[0]);
    a.post_bias = addr(param[1]);
    a.next_weight = addr(param[2]);
    a.next_bias = addr(param[3]);
  }

  void set_gate() {
    if (gate->scalar_type() != branch) type_error("gate must have y's type");
    const auto xs = x->sizes(), gs = gate->sizes();
    const int64_t n = x->dim();
    if (gs.size() == 1 && gs[0] == a.width) {
      a.gate_kind = SNACK_GATE_CHANNEL;
    } else if (gs == xs) {
      a.gate_kind = SNACK_GATE_FULL;
      a.gate_stride = rows_of(*gate, "gate").step;
      return;
    } else if ((int64_t)gs.size() == n && gs[n - 1] == 1 && gs.slice(0, n - 1) == xs.slice(0, n - 1)) {
      a.gate_kind = SNACK_GATE_TOKEN;
    } else if (n >= 3 && (int64_t)gs.size() == n && gs[n - 1] == a.width && gs[n - 2] == 1 &&
               gs.slice(0, n - 2) == xs.slice(0, n - 2)) {
      a.gate_kind = SNACK_GATE_SEQUENCE;
      a.group_rows = xs[n - 2];
      if (a.group_rows == 0) a.group_rows = 1;  // no rows at all
    } else {
      value_error("gate of shape " + shape(*gate) + " does not fit x " + shape(*x) +
                  ": it is [d], [..., 1], [sequences, 1, d] or x's shape");
    }
    if (!gate->is_contiguous()) value_error("gate must be contiguous");
  }
};

PyObject *norm_forward(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 2 + kNormOptions + 1);
    Norm m(o[0], o[1], o + 2);
    const Stream s(o[2 + kNormOptions], m.dev.dev);
    const bool bare = !m.y && m.a.residual_scale == 1.f;
    at::Tensor r, h, stats = empty({m.a.rows, 4}, at::kFloat, m.dev.dev);
    if (!bare) r = empty(m.x->sizes(), m.x->scalar_type(), m.dev.dev);
    if (m.a.next_norm) h = empty(m.x->sizes(), m.branch, m.dev.dev);
    m.a.stats = static_cast<float *>(stats.data_ptr());
    check(snack_residual_norm_forward(&m.a, bare ? nullptr : r.data_ptr(), h.defined() ? h.data_ptr() : nullptr,
                                      s.raw));
    return Py_BuildValue("(NNN)", bare ? same(o[0]) : wrap(r), h.defined() ? wrap(h) : same(Py_None), wrap(stats));
  });
}

PyObject *norm_backward(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 5 + kNormOptions + 1);
    Norm m(o[2], o[3], o + 5);
    const Stream s(o[5 + kNormOptions], m.dev.dev);
    const auto grad = [&](PyObject *g, at::ScalarType type, const char *name, int64_t *stride) -> const void * {
      if (g == Py_None) return nullptr;
      const at::Tensor &t = dense(g, name);
      if (t.scalar_type() != type) type_error(std::string(name) + " has another type than its output");
      if (t.sizes() != m.x->sizes())
        value_error(std::string(name) + " " + shape(t) + " must have x's shape " + shape(*m.x));
      *stride = rows_of(t, name).step;
      m.dev.add(&t);
      return t.data_ptr();
    };
    snack_norm_grads g{};
    g.dr = grad(o[0], m.x->scalar_type(), "dr", &g.dr_stride);
    if (o[1] != Py_None && !m.a.next_norm) value_error("dh without next_norm");
    g.dh = grad(o[1], m.branch, "dh", &g.dh_stride);
    if (!is_tensor(o[4])) type_error("stats must be a tensor");
    const at::Tensor &stats = THPVariable_Unpack(o[4]);
    if (stats.scalar_type() != at::kFloat || !stats.is_contiguous() || stats.numel() != 4 * m.a.rows)
      value_error("stats must be " + std::to_string(m.a.rows) + " x 4 contiguous float32");
    m.dev.add(&stats);
    m.a.stats = static_cast<float *>(stats.data_ptr());
    PyObject *out = PyDict_New();
    if (!out) throw Raised{};
    std::unique_ptr<PyObject, void (*)(PyObject *)> hold(out, [](PyObject *p) { Py_DECREF(p); });
    const auto put = [&](const char *name, const at::Tensor *like, at::ScalarType type) -> void * {
      if (!like) return nullptr;
      at::Tensor t = empty(like->sizes(), type, m.dev.dev);
      // without rows every sum is zero, and the C call writes no gate of a group that has none
      if (m.a.rows == 0) t.zero_();
      PyObject *w = wrap(t);
      const int bad = w ? PyDict_SetItemString(out, name, w) : -1;
      Py_XDECREF(w);
      if (bad) throw Raised{};
      return t.data_ptr();
    };
    g.dx = put("dx", m.x, m.x->scalar_type());
    if (m.y) g.dy = put("dy", m.y, m.branch);
    g.dgate = put("dgate", m.gate, m.branch);
    const auto param = [&](const char *name, int i) {
      return put(name, m.param[i], m.param[i] ? m.param[i]->scalar_type() : at::kFloat);
    };
    g.dpost_weight = param("dpost_weight", 0);
    g.dpost_bias = param("dpost_bias", 1);
    g.dnext_weight = param("dnext_weight", 2);
    g.dnext_bias = param("dnext_bias", 3);
    const at::Tensor ws = s.scratch(snack_residual_norm_workspace(&m.a), m.dev.dev);
    check(snack_residual_norm_backward(&m.a, &g, scratch_addr(ws), s.raw));
    return hold.release();
  });
}

// ------------------------------------------------------------------ adapters

// X, A, B, offsets, adapter, scale
struct Adapter {
  snack_adapter_args a{};
  Device dev;
  const at::Tensor *X, *A, *B;

  Adapter(PyObject *x, PyObject *const *o) {
    X = &dense(x, "X");
    A = &dense(o[0], "A");
    B = &dense(o[1], "B");
    const at::Tensor *const ab[2] = {A, B};
    for (int i = 0; i < 2; ++i) {
      const std::string name = i ? "B" : "A";
      if (ab[i]->scalar_type() != X->scalar_type()) type_error(name + " must have X's type");
      if (ab[i]->dim() != 3 || !ab[i]->is_contiguous())
        value_error(name + " must be contiguous with three dimensions");
    }
    a.adapters = A->size(0);
    a.rank = A->size(1);
    a.in = A->size(2);
    a.out = B->size(1);
    if (B->size(0) != a.adapters || B->size(2) != a.rank)
      value_error("A is [adapters][rank][in] " + shape(*A) + ", B [adapters][out][rank] " + shape(*B) +
                  ": they do not fit");
    if (X->dim() < 1 || X->size(-1) != a.in)
      value_error("X must be [..., " + std::to_string(a.in) + "], got " + shape(*X));
    const at::Tensor &off = ints(o[2], "offsets"), &which = ints(o[3], "adapter");
    if (off.numel() != which.numel() + 1) value_error("offsets must have one element more than adapter");
    a.uniform_scale = 1.f;
    const at::Tensor *scale = nullptr;
    if (is_tensor(o[4])) {
      scale = &THPVariable_Unpack(o[4]);
      if (!scale->is_cuda() || scale->scalar_type() != at::kFloat || !scale->is_contiguous() ||
          scale->numel() != a.adapters)
        value_error("scale must be a number or " + std::to_string(a.adapters) + " contiguous CUDA float32");
    } else {
      a.uniform_scale = (float)number(o[4]);
    }
    const Rows r = rows_of(*X, "X");
    a.tokens = r.n;
    a.x_stride = r.step;
    a.requests = which.numel();
    a.type = type_code(X->scalar_type());
    dev.add(X);
    for (const at::Tensor *t : {A, B, &off, &which, scale}) dev.add(t);
    a.X = addr(X);
    a.A = addr(A);
    a.B = addr(B);
    a.offsets = static_cast<const int32_t *>(off.data_ptr());
    a.adapter = static_cast<const int32_t *>(which.data_ptr());
    a.scale = static_cast<const float *>(addr(scale));
  }

  static const at::Tensor &ints(PyObject *o, const char *name) {
    if (is_tensor(o)) {
      const at::Tensor &t = THPVariable_Unpack(o);
      if (t.is_cuda() && t.scalar_type() == at::kInt && t.dim() == 1 && t.is_contiguous()) return t;
    }
    type_error(std::string(name) + " must be a contiguous CUDA int32 vector");
  }

  // A tensor of X's type with X's rows and `width` columns; its row stride.
  const at::Tensor &like(PyObject *o, int64_t width, const char *name, int64_t *stride) {
    if (!is_tensor(o) || !THPVariable_Unpack(o).is_cuda() ||
        THPVariable_Unpack(o).scalar_type() != X->scalar_type())
      type_error(std::string(name) + " must be a CUDA tensor of X's type");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() < 1 || t.size(-1) != width)
      value_error(std::string(name) + " must be [..., " + std::to_string(width) + "], got " + shape(t));
    const Rows r = rows_of(t, name);
    if (r.n != a.tokens)
      value_error(std::string(name) + " has " + std::to_string(r.n) + " rows, X has " + std::to_string(a.tokens));
    *stride = r.step;
    dev.add(&t);
    return t;
  }

  float *hidden(PyObject *o) {
    if (is_tensor(o)) {
      const at::Tensor &t = THPVariable_Unpack(o);
      if (t.is_cuda() && t.scalar_type() == at::kFloat && t.is_contiguous() && t.numel() == a.tokens * a.rank) {
        dev.add(&t);
        return static_cast<float *>(t.data_ptr());
      }
    }
    value_error("H must be " + std::to_string(a.tokens) + " x " + std::to_string(a.rank) + " contiguous float32");
  }
};

// X, A, B, offsets, adapter, scale, Y, H, stream
PyObject *adapter_forward(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 9);
    Adapter m(o[0], o + 1);
    int64_t ys = 0;
    const at::Tensor &Y = m.like(o[6], m.a.out, "Y", &ys);
    const Stream s(o[8], m.dev.dev);
    at::Tensor fresh;
    float *H;
    if (o[7] == Py_None) {
      fresh = empty({m.a.tokens, m.a.rank}, at::kFloat, m.dev.dev);
      H = static_cast<float *>(fresh.data_ptr());
    } else {
      H = m.hidden(o[7]);
    }
    const at::Tensor ws = s.scratch(snack_adapter_forward_workspace(&m.a), m.dev.dev);
    check(snack_adapter_forward(&m.a, Y.data_ptr(), ys, H, scratch_addr(ws), s.raw));
    written(Y);
    if (!fresh.defined()) written(o[7]);
    return Py_BuildValue("(NN)", same(o[6]), fresh.defined() ? wrap(fresh) : same(o[7]));
  });
}

// X, dY, A, B, offsets, adapter, scale, H, dX, need_dx, need_dw, stream
PyObject *adapter_backward(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 12);
    Adapter m(o[0], o + 2);
    int64_t dys = 0, dxs = m.a.in;
    const at::Tensor &dY = m.like(o[1], m.a.out, "dY", &dys);
    const float *H = m.hidden(o[7]);
    const Stream s(o[11], m.dev.dev);
    const bool need_dx = truth(o[9]), need_dw = truth(o[10]);
    at::Tensor fresh, dA, dB;
    void *dX = nullptr;
    if (need_dx) {
      if (o[8] == Py_None) {
        fresh = at::zeros(m.X->sizes(), m.X->options());
        dX = fresh.data_ptr();
      } else {
        dX = m.like(o[8], m.a.in, "dX", &dxs).data_ptr();
      }
    }
    if (need_dw) {
      dA = empty(m.A->sizes(), m.A->scalar_type(), m.dev.dev);
      dB = empty(m.B->sizes(), m.B->scalar_type(), m.dev.dev);
    }
    const at::Tensor ws = s.scratch(snack_adapter_backward_workspace(&m.a), m.dev.dev);
    check(snack_adapter_backward(&m.a, dY.data_ptr(), dys, H, dX, dxs, need_dw ? dA.data_ptr() : nullptr,
                                 need_dw ? dB.data_ptr() : nullptr, scratch_addr(ws), s.raw));
    if (need_dx && !fresh.defined()) written(o[8]);
    return Py_BuildValue("(NNN)", !need_dx ? same(Py_None) : (fresh.defined() ? wrap(fresh) : same(o[8])),
                         need_dw ? wrap(dA) : same(Py_None), need_dw ? wrap(dB) : same(Py_None));
  });
}

// ------------------------------------------------------------------ gradient norm

// Addresses, sizes and types of a list's tensors.
struct List {
  std::vector<void *> ptr;
  std::vector<int64_t> size;
  std::vector<int32_t> type;
  c10::Device dev{c10::kCUDA, -1};
  // What holds the tensors: nobody else may (those of a generator), and their
  // memory must not be handed out before the call's work is in the stream.
  std::unique_ptr<PyObject, void (*)(PyObject *)> hold{nullptr, [](PyObject *p) { Py_DECREF(p); }};

  explicit List(PyObject *seq) {
    PyObject *fast = PySequence_Fast(seq, "a list of tensors, or a SnackTensorList");
    if (!fast) throw Raised{};
    hold.reset(fast);
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
    PyObject *const *items = PySequence_Fast_ITEMS(fast);
    ptr.reserve(n);
    size.reserve(n);
    type.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor *t = is_tensor(items[i]) ? &THPVariable_Unpack(items[i]) : nullptr;
      const int k = t && t->is_cuda() ? type_code(t->scalar_type()) : -1;
      if (k < 0) type_error("tensor " + std::to_string(i) + " must be a CUDA float32, bfloat16 or float16 tensor");
      if (!t->is_contiguous()) value_error("tensor " + std::to_string(i) + " must be contiguous");
      if (i == 0)
        dev = t->device();
      else if (t->device() != dev)
        value_error("all tensors must be on one device");
      ptr.push_back(t->data_ptr());
      size.push_back(t->numel());
      type.push_back(k);
    }
    if (n == 0) dev = c10::Device(c10::kCUDA, c10::cuda::current_device());
  }

  // Whether the tensors lie where they were found: `.data = `, set_(),
  // resize_() and Module.to() give a tensor other memory, type or size.
  bool current() const {
    PyObject *const *items = PySequence_Fast_ITEMS(hold.get());
    const size_t n = ptr.size();
    for (size_t i = 0; i < n; ++i) {
      const c10::TensorImpl *t = THPVariable_Unpack(items[i]).unsafeGetTensorImpl();
      if (t->data() != ptr[i] || t->numel() != size[i] || !t->is_contiguous() ||
          type_code(c10::typeMetaToScalarType(t->dtype())) != type[i])
        return false;
    }
    return true;
  }
};

constexpr const char *kListName = "snack tensor list";

PyObject *tensor_list(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 1);
    auto l = std::make_unique<List>(o[0]);
    PyObject *c = PyCapsule_New(l.get(), kListName, [](PyObject *p) {
      delete static_cast<List *>(PyCapsule_GetPointer(p, kListName));
    });
    if (c) l.release();
    return c;
  });
}

// A kept list, or one made for this call.
struct ListArg {
  std::unique_ptr<List> own;
  const List *l;
  explicit ListArg(PyObject *o) {
    if (PyCapsule_IsValid(o, kListName)) {
      // a kept list means its tensors, wherever they lie by now: if one has
      // moved all are checked again, and the memory of before is not touched
      List *kept = static_cast<List *>(PyCapsule_GetPointer(o, kListName));
      if (!kept->current()) *kept = List(kept->hold.get());
      l = kept;
    } else {
      own = std::make_unique<List>(o);
      l = own.get();
    }
    if (l->dev.index() != c10::cuda::current_device())
      value_error("cuda:" + std::to_string(l->dev.index()) + " is not the current CUDA device");
  }
  // (Not of a kept list: 96 tensors of one add 1 us to a call of 9.)
  void written_all() const {
    if (!own) return;
    PyObject *const *items = PySequence_Fast_ITEMS(own->hold.get());
    for (size_t i = 0; i < own->ptr.size(); ++i) written(items[i]);
  }
};

int norm_kind(PyObject *o) {
  const double v = number(o);
  if (v == 2.0) return 0;
  if (v == std::numeric_limits<double>::infinity()) return 1;
  value_error("norm_type must be 2.0 or inf");
}

at::Tensor norm_out(PyObject *o, c10::Device dev) {
  if (o == Py_None) return empty({}, at::kFloat, dev);
  if (is_tensor(o)) {
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() == at::kFloat && t.numel() == 1 && t.device() == dev) return t;
  }
  value_error("norm must be one float32 on the gradients' device");
}

// grads, norm_type, norm, stream
PyObject *grad_norm(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 4);
    const ListArg g(o[0]);
    const int kind = norm_kind(o[1]);
    const Stream s(o[3], g.l->dev);
    const at::Tensor norm = norm_out(o[2], g.l->dev);
    const int64_t c = (int64_t)g.l->ptr.size();
    const at::Tensor ws = s.scratch(snack_grad_norm_workspace(c), g.l->dev);
    check(snack_grad_norm(c, const_cast<const void *const *>(g.l->ptr.data()), g.l->size.data(), g.l->type.data(),
                          kind, static_cast<float *>(norm.data_ptr()), scratch_addr(ws), s.raw));
    if (o[2] != Py_None) written(o[2]);
    return o[2] == Py_None ? wrap(norm) : same(o[2]);
  });
}

// grads, max_norm, norm_type, out, eps, norm, stream
PyObject *clip_grad_norm(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 7);
    const ListArg g(o[0]);
    const double max_norm = number(o[1]);
    if (!(max_norm >= 0.0)) value_error("max_norm must be >= 0");
    const int kind = norm_kind(o[2]);
    std::unique_ptr<ListArg> out;
    if (o[3] != Py_None) {
      out = std::make_unique<ListArg>(o[3]);
      if (out->l->size != g.l->size) value_error("out must hold as many elements as grads, tensor by tensor");
      if (out->l->dev != g.l->dev) value_error("all tensors must be on one device");
    }
    const Stream s(o[6], g.l->dev);
    const at::Tensor norm = norm_out(o[5], g.l->dev);
    const int64_t c = (int64_t)g.l->ptr.size();
    const at::Tensor ws = s.scratch(snack_grad_norm_workspace(c), g.l->dev);
    check(snack_clip_grad_norm(c, const_cast<const void *const *>(g.l->ptr.data()),
                               out ? out->l->ptr.data() : nullptr, g.l->size.data(), g.l->type.data(),
                               out ? out->l->type.data() : nullptr, kind, (float)max_norm, (float)number(o[4]),
                               static_cast<float *>(norm.data_ptr()), scratch_addr(ws), s.raw));
    (out ? *out : g).written_all();
    if (o[5] != Py_None) written(o[5]);
    return o[5] == Py_None ? wrap(norm) : same(o[5]);
  });
}

// ------------------------------------------------------------------ attention and dropout

// A number of the dropout's seed, or a device tensor that holds it.
struct Seed {
  uint64_t value = 0;
  const uint64_t *at = nullptr;
  const at::Tensor *tensor = nullptr;
  explicit Seed(PyObject *o) {
    if (is_tensor(o)) {
      const at::Tensor &t = THPVariable_Unpack(o);
      if (!t.is_cuda() || t.scalar_type() != at::kLong || t.numel() != 1)
        type_error("seed must be a number or one CUDA int64");
      tensor = &t;
      at = static_cast<const uint64_t *>(t.data_ptr());
      return;
    }
    value = PyLong_AsUnsignedLongLongMask(o);
    if (PyErr_Occurred()) throw Raised{};
  }
};

// q, k, v, then kAttentionOptions: causal, scale, q_offsets, k_offsets,
// q_lengths, k_lengths, dropout, seed.
constexpr int kAttentionOptions = 8;
struct Attention {
  snack_attention_args a{};
  Device dev;
  const at::Tensor *q, *k, *v;
  bool q_ragged, k_ragged;

  static const at::Tensor *ints(PyObject *o, const char *name) {
    return o == Py_None ? nullptr : &Adapter::ints(o, name);
  }

  // Strides of t, which is [sequences][tokens][heads][d], or [tokens][heads][d] where ragged.
  static void strides(const at::Tensor &t, int64_t (&s)[3], const char *name) {
    const int64_t n = t.dim();
    if (t.size(n - 1) > 1 && t.stride(n - 1) != 1)
      value_error(std::string(name) + " must be contiguous along its last dimension");
    s[0] = n == 4 ? t.stride(0) : 0;
    s[1] = t.stride(n - 3);
    s[2] = t.stride(n - 2);
  }

  // Whether the rows of a 16-bit tensor of t's shape begin on 16 bytes and repeat no memory.  A
  // gradient whose do not is copied: it is the only operand that the plan does not know, and without
  // room for it in the workspace its call would leave the tensor cores' fast path.  (Of head sizes
  // that do not fill 16 bytes every tensor is copied in the call.)
  static bool even(const at::Tensor &t, const void *p, const int64_t (&s)[3]) {
    if (t.element_size() != 2 || t.size(-1) % 8 || t.numel() == 0) return true;
    for (int64_t i = 0; i < t.dim() - 1; ++i) {
      const int64_t stride = s[3 - (t.dim() - 1) + i];
      if (t.size(i) > 1 && (stride == 0 || stride % 8)) return false;
    }
    return reinterpret_cast<uintptr_t>(p) % 16 == 0;
  }

  const at::Tensor &like_q(PyObject *o, const char *name, int64_t (&s)[3]) { return like(o, *q, name, "q", s); }
  const at::Tensor &like(PyObject *o, const at::Tensor &other, const char *name, const char *of, int64_t (&s)[3]) {
    const at::Tensor &t = dense(o, name);
    if (t.scalar_type() != other.scalar_type()) type_error(std::string(name) + " must have " + of + "'s type");
    if (t.sizes() != other.sizes())
      value_error(std::string(name) + " " + shape(t) + " must have " + of + "'s shape " + shape(other));
    strides(t, s, name);
    dev.add(&t);
    return t;
  }

  Attention(PyObject *q_, PyObject *k_, PyObject *v_, PyObject *const *o) {
    q = &dense(q_, "q");
    k = &dense(k_, "k");
    v = &dense(v_, "v");
    a.causal = truth(o[0]);
    const at::Tensor *const qo = ints(o[2], "q_offsets"), *const ko = ints(o[3], "k_offsets");
    const at::Tensor *const ql = ints(o[4], "q_lengths"), *const kl = ints(o[5], "k_lengths");
    a.dropout = (float)number(o[6]);
    if (!(a.dropout >= 0.f && a.dropout < 1.f)) value_error("dropout must be at least 0 and below 1");
    const Seed seed(o[7]);
    a.seed = seed.value;
    a.seed_at = seed.at;
    q_ragged = qo != nullptr;
    k_ragged = ko != nullptr;
    if (k->scalar_type() != q->scalar_type() || v->scalar_type() != q->scalar_type())
      type_error("q, k and v must have one type");
    if (q->dim() != (q_ragged ? 3 : 4))
      value_error(q_ragged ? "q must be [tokens][heads][d] with q_offsets, got " + shape(*q)
                           : "q must be [sequences][tokens][heads][d], got " + shape(*q));
    if (k->dim() != (k_ragged ? 3 : 4))
      value_error(k_ragged ? "k must be [tokens][heads][d] with k_offsets, got " + shape(*k)
                           : "k must be [sequences][tokens][heads][d], got " + shape(*k));
    if (v->sizes() != k->sizes()) value_error("v " + shape(*v) + " must have k's shape " + shape(*k));
    const int64_t d = q->size(-1), heads = q->size(-2), key_heads = k->size(-2);
    if (k->size(-1) != d) value_error("q and k must have one head size");
    if (d < 1 || d > 128) value_error("the head size must be 1 to 128, got " + std::to_string(d));
    if (key_heads < 1 || heads < 1 || heads % key_heads || heads > 65536)
      value_error(std::to_string(heads) + " heads are not a multiple of " + std::to_string(key_heads) +
                  " key heads (at most 65536)");
    if ((q_ragged && ql) || (k_ragged && kl)) value_error("a side has offsets or lengths, not both");
    const auto count_of = [&](const at::Tensor *off, const at::Tensor &t, const char *name) {
      if (off && off->numel() < 1) value_error(std::string(name) + " must have at least one element");
      return off ? off->numel() - 1 : t.size(0);
    };
    a.sequences = count_of(qo, *q, "q_offsets");
    if (count_of(ko, *k, "k_offsets") != a.sequences) value_error("q and k must have the same number of sequences");
    for (const at::Tensor *l : {ql, kl})
      if (l && l->numel() != a.sequences) value_error("lengths must have one element for each sequence");
    a.q_tokens = q->size(q_ragged ? 0 : 1);
    a.k_tokens = k->size(k_ragged ? 0 : 1);
    a.heads = (int32_t)heads;
    a.key_heads = (int32_t)key_heads;
    a.head_size = (int32_t)d;
    a.type = type_code(q->scalar_type());
    a.scale = o[1] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)number(o[1]);
    if (!std::isfinite(a.scale)) value_error("scale must be finite");
    for (const at::Tensor *t : {q, k, v, qo, ko, ql, kl, seed.tensor}) dev.add(t);
    a.q = addr(q);
    a.k = addr(k);
    a.v = addr(v);
    strides(*q, a.q_stride, "q");
    strides(*k, a.k_stride, "k");
    strides(*v, a.v_stride, "v");
    const auto at_ = [](const at::Tensor *t) { return static_cast<const int32_t *>(addr(t)); };
    a.q_offsets = at_(qo);
    a.k_offsets = at_(ko);
    a.q_lengths = at_(ql);
    a.k_lengths = at_(kl);
  }

  std::vector<int64_t> lse_shape() const {
    if (q_ragged) return {a.heads, a.q_tokens};
    return {a.heads, a.sequences, a.q_tokens};
  }
};

// q, k, v, options, stream
PyObject *attention_forward(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 3 + kAttentionOptions + 1);
    Attention m(o[0], o[1], o[2], o + 3);
    const Stream s(o[3 + kAttentionOptions], m.dev.dev);
    const at::Tensor out = empty(m.q->sizes(), m.q->scalar_type(), m.dev.dev);
    const at::Tensor lse = empty(m.lse_shape(), at::kFloat, m.dev.dev);
    int64_t stride[3];
    Attention::strides(out, stride, "out");
    const at::Tensor ws = s.scratch(snack_attention_forward_workspace(&m.a), m.dev.dev);
    check(snack_attention_forward(&m.a, out.data_ptr(), stride, static_cast<float *>(lse.data_ptr()),
                                  scratch_addr(ws), s.raw));
    return Py_BuildValue("(NN)", wrap(out), wrap(lse));
  });
}

// dout, q, k, v, out, lse, options, dq, dk, dv, need_dq, need_dkv, stream
PyObject *attention_backward(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 6 + kAttentionOptions + 6);
    Attention m(o[1], o[2], o[3], o + 6);
    PyObject *const *const r = o + 6 + kAttentionOptions;
    snack_attention_grads g{};
    g.dout = m.like_q(o[0], "dout", g.dout_stride).data_ptr();
    g.out = m.like_q(o[4], "out", g.out_stride).data_ptr();
    const at::Tensor &lse = dense(o[5], "lse");
    if (lse.scalar_type() != at::kFloat || !lse.is_contiguous() || lse.numel() != m.q->numel() / m.a.head_size)
      value_error("lse must be the forward call's: " + std::to_string(m.q->numel() / m.a.head_size) +
                  " contiguous float32");
    m.dev.add(&lse);
    g.lse = static_cast<const float *>(lse.data_ptr());
    const bool need_dq = truth(r[3]), need_dkv = truth(r[4]);
    const Stream s(r[5], m.dev.dev);
    at::Tensor even_dout;
    if (!Attention::even(*m.q, g.dout, g.dout_stride)) {
      even_dout = THPVariable_Unpack(o[0]).detach().clone(at::MemoryFormat::Contiguous);
      g.dout = even_dout.data_ptr();
      Attention::strides(even_dout, g.dout_stride, "dout");
    }
    at::Tensor fresh[3];
    PyObject *res[3] = {Py_None, Py_None, Py_None};
    const auto result = [&](int i, const at::Tensor &like, const char *name, const char *of, int64_t (&st)[3],
                            bool need) -> void * {
      if (!need) return nullptr;
      if (r[i] != Py_None) {
        const at::Tensor &t = m.like(r[i], like, name, of, st);
        for (int64_t k = 0; k < t.dim() - 1; ++k)
          if (t.size(k) > 1 && t.stride(k) == 0) value_error(std::string(name) + ": its elements overlap");
        res[i] = r[i];
        return t.data_ptr();
      }
      fresh[i] = empty(like.sizes(), like.scalar_type(), m.dev.dev);
      Attention::strides(fresh[i], st, name);
      return fresh[i].data_ptr();
    };
    g.dq = result(0, *m.q, "dq", "q", g.dq_stride, need_dq);
    g.dk = result(1, *m.k, "dk", "k", g.dk_stride, need_dkv);
    g.dv = result(2, *m.v, "dv", "v", g.dv_stride, need_dkv);
    const at::Tensor ws = s.scratch(snack_attention_backward_workspace(&m.a), m.dev.dev);
    check(snack_attention_backward(&m.a, &g, scratch_addr(ws), s.raw));
    for (int i = 0; i < 3; ++i)
      if (res[i] != Py_None) written(res[i]);
    const auto give = [&](int i) { return fresh[i].defined() ? wrap(fresh[i]) : same(res[i]); };
    return Py_BuildValue("(NNN)", give(0), give(1), give(2));
  });
}

// x, residual, dtype of y, p, seed, stream
PyObject *dropout(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 6);
    const at::Tensor &x = dense(o[0], "x");
    const at::Tensor *const res = dense_or_none(o[1], "residual");
    if (!x.is_contiguous() || (res && !res->is_contiguous())) value_error("x and residual must be contiguous");
    if (res && res->sizes() != x.sizes())
      value_error("residual " + shape(*res) + " must have x's shape " + shape(x));
    at::ScalarType type = res ? res->scalar_type() : x.scalar_type();
    if (o[2] != Py_None) {
      if (!THPDtype_Check(o[2]) || type_code(reinterpret_cast<THPDtype *>(o[2])->scalar_type) < 0)
        type_error("dtype must be float32, bfloat16 or float16");
      type = reinterpret_cast<THPDtype *>(o[2])->scalar_type;
      if (res && type != res->scalar_type()) type_error("the result has the residual's type");
    }
    const double p = number(o[3]);
    if (!(p >= 0.0 && p < 1.0)) value_error("p must be at least 0 and below 1");
    const Seed seed(o[4]);
    Device dev;
    for (const at::Tensor *t : {&x, res, seed.tensor}) dev.add(t);
    const Stream s(o[5], dev.dev);
    const at::Tensor y = empty(x.sizes(), type, dev.dev);
    check(snack_dropout(x.numel(), x.data_ptr(), type_code(x.scalar_type()), addr(res), y.data_ptr(), type_code(type),
                        (float)p, seed.value, seed.at, s.raw));
    return wrap(y);
  });
}

PyObject *set_error(PyObject *, PyObject *e) {
  Py_INCREF(e);
  Py_XSETREF(g_error, e);
  Py_RETURN_NONE;
}

#define SNACK_FN(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SNACK_FN(norm_forward),    SNACK_FN(norm_backward), SNACK_FN(adapter_forward),
                         SNACK_FN(adapter_backward), SNACK_FN(tensor_list),   SNACK_FN(grad_norm),
                         SNACK_FN(clip_grad_norm),   SNACK_FN(attention_forward), SNACK_FN(attention_backward),
                         SNACK_FN(dropout),          {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dense() { return PyModule_Create(&module); }
