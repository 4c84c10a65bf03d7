// Compiled half of newton_schulz_05_gb300/layers.py: checks the tensors of a
// call, allocates its outputs and calls libmuon's C ABI.  These operators run
// many times a training step on tensors that may be small, and the host side
// of a call through ctypes (15 to 33 us on the GB300 node's cores, mostly
// argument checks and allocations in Python) exceeded the kernel's time for
// anything below a few tens of MB.  No arithmetic happens here.
//
// Every function takes its arguments by position and returns the tensors of
// the result, or the muon_status (an int) of a call that libmuon refused.
// Wrong arguments raise TypeError or ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "muon.h"

namespace {

decltype(&muon_layer_norm) p_layer_norm;
decltype(&muon_layer_norm_backward) p_layer_norm_backward;
decltype(&muon_layer_norm_workspace_bytes) p_layer_norm_workspace_bytes;
decltype(&muon_dropout) p_dropout;
decltype(&muon_route) p_route;
decltype(&muon_route_workspace_bytes) p_route_workspace_bytes;
decltype(&muon_route_backward) p_route_backward;

// a Python error to raise
struct Raise {
  PyObject* type;
  std::string what;
};
[[noreturn]] void value_error(std::string s) { throw Raise{PyExc_ValueError, std::move(s)}; }
[[noreturn]] void type_error(std::string s) { throw Raise{PyExc_TypeError, std::move(s)}; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}
// null for None
const at::Tensor* maybe(PyObject* o, const char* what) {
  return o == Py_None ? nullptr : &tensor(o, what);
}

int dtype_of(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return MUON_BF16;
  if (t.scalar_type() == at::kFloat) return MUON_F32;
  type_error(std::string(what) + " must be bf16 or fp32, got " + c10::toString(t.scalar_type()));
}

struct Rows { int64_t rows, cols, ld; };

// t as rows at one stride with a dense last dimension; the reason it is not,
// or null
const char* rows_of(const at::Tensor& t, Rows* r) {
  if (!t.is_cuda()) return " is not on a CUDA device";
  const int64_t nd = t.dim();
  if (nd == 0) return " needs at least one dimension";
  const auto size = t.sizes();
  const int64_t cols = size[nd - 1];
  if (t.is_contiguous()) {
    *r = {cols ? t.numel() / cols : 0, cols, cols};
    return nullptr;
  }
  const auto stride = t.strides();
  if (cols > 1 && stride[nd - 1] != 1) return " has a last dimension that is not dense";
  int64_t rows = 1, ld = -1;
  for (int64_t d = nd - 2; d >= 0; --d) {      // innermost first
    if (size[d] == 1) continue;
    if (ld < 0) ld = stride[d];
    else if (stride[d] != ld * rows) return " has leading dimensions that are not rows at one stride";
    rows *= size[d];
  }
  *r = {rows, cols, ld < 0 ? cols : ld};
  return nullptr;
}

Rows rows_or_raise(const at::Tensor& t, const char* what) {
  Rows r;
  if (const char* why = rows_of(t, &r)) value_error(std::string(what) + why);
  return r;
}

// the stream of a call: the current one of the tensor's device, which must be
// the current device
void* stream_of(const at::Tensor& t) {
  const auto current = c10::cuda::current_device();
  if (t.get_device() != current)
    value_error("tensors are on cuda:" + std::to_string((int)t.get_device()) +
                ", the current device is cuda:" + std::to_string((int)current));
  return c10::cuda::getCurrentCUDAStream(current).stream();
}

const void* vector_of(const at::Tensor* t, int64_t cols, const at::Tensor& like, const char* what) {
  if (!t) return nullptr;
  if (t->dim() != 1 || t->size(0) != cols || !t->is_contiguous())
    value_error(std::string(what) + " must be a dense vector of " + std::to_string(cols) + " elements");
  if (t->device() != like.device()) value_error(std::string(what) + " is not on the device of the rows");
  return t->const_data_ptr();
}

// row stride of t, which must match `like` in shape, type and device
int64_t same_rows(const at::Tensor& t, const at::Tensor& like, const char* what) {
  if (t.sizes() != like.sizes() || t.device() != like.device())
    value_error(std::string(what) + " must have the rows' shape and device");
  if (t.scalar_type() != like.scalar_type())
    type_error(std::string(what) + " must be of the rows' type, got " + c10::toString(t.scalar_type()));
  return rows_or_raise(t, what).ld;
}

void check_flat(const at::Tensor& t, int64_t numel, at::ScalarType type, const at::Tensor& like,
                const char* what) {
  if (t.scalar_type() != type)
    type_error(std::string(what) + " must be " + c10::toString(type) + ", got " +
               c10::toString(t.scalar_type()));
  if (t.numel() != numel || !t.is_contiguous() || t.device() != like.device())
    value_error(std::string(what) + " must be dense with " + std::to_string(numel) +
                " elements on the device of the rows");
}

// Whether two shapes of as many elements list them alike: the first is one
// dimension, or both are the same but for dimensions of one.
bool listed_alike(at::IntArrayRef a, at::IntArrayRef b) {
  size_t i = 0, j = 0;
  if (a.size() == 1) return true;
  for (;;) {
    while (i < a.size() && a[i] == 1) ++i;
    while (j < b.size() && b[j] == 1) ++j;
    if (i == a.size() || j == b.size()) return i == a.size() && j == b.size();
    if (a[i++] != b[j++]) return false;
  }
}

// t has one element for each row of `like`, in the order of its leading
// dimensions.  Other shapes of as many elements are refused: a transposed one would
// be read in the wrong order.
void check_each_row(const at::Tensor& t, int64_t rows, at::ScalarType type, const at::Tensor& like,
                    const char* what) {
  check_flat(t, rows, type, like, what);
  if (!listed_alike(t.sizes(), like.sizes().slice(0, like.dim() - 1)))
    value_error(std::string(what) + " must have the shape of the rows' leading dimensions, or one dimension");
}

// A dense tensor on the current device (stream_of has checked that it is the inputs').
// Every result has memory of its own: results that shared an allocation would be
// resized, saved and kept alive together.  Straight from the caching allocator, as
// at::detail::empty_cuda takes 0.3 us more host time a tensor.
at::Tensor empty(at::IntArrayRef size, at::ScalarType type) {
  c10::Allocator* const allocator = c10::cuda::CUDACachingAllocator::get();
  size_t bytes = c10::elementSize(type);
  for (const int64_t n : size) bytes *= (size_t)n;
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                         allocator->allocate(bytes), allocator, true)),
      c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(size);
  return t;
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* none() { Py_RETURN_NONE; }

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raise{nullptr, ""};
  return v;
}
uint64_t word(PyObject* o) {
  const uint64_t v = PyLong_AsUnsignedLongLongMask(o);
  if (v == (uint64_t)-1 && PyErr_Occurred()) throw Raise{nullptr, ""};
  return v;
}
int small(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raise{nullptr, ""};
  return v > 0x7fffffff ? 0x7fffffff : v < -0x7fffffff ? -0x7fffffff : (int)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raise{nullptr, ""};
  return v != 0;
}

// Gives up the interpreter lock for its lifetime: allocation and launch may block (a
// full queue, a device allocation), and other Python threads run meanwhile.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs f, which returns a new reference, and turns C++ errors into Python ones
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raise& r) {
    if (r.type) PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  } catch (const std::exception&) {      // an allocation that failed, and the like
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// a tuple of the n objects, whose references it takes
PyObject* tuple_of(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  bool ok = t != nullptr;
  for (PyObject* o : items) {
    if (!o) ok = false;
    if (t) PyTuple_SET_ITEM(t, i++, o);
    else Py_XDECREF(o);
  }
  if (ok) return t;
  Py_XDECREF(t);
  return nullptr;
}

// (x, weight, bias, eps, residual, p, seed, offset) -> (y, sum or None, mean, rstd)
PyObject* layer_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor *w = maybe(a[1], "weight"), *b = maybe(a[2], "bias");
    const at::Tensor* res = maybe(a[4], "residual");
    const double eps = number(a[3]), p = number(a[5]);
    const uint64_t seed = word(a[6]), offset = word(a[7]);
    const int dt = dtype_of(x, "x");
    const Rows r = rows_or_raise(x, "x");
    int wdt = MUON_F32;
    if (w || b) wdt = dtype_of(w ? *w : *b, "weight and bias");
    if (w && b && w->scalar_type() != b->scalar_type()) type_error("weight and bias must be of one type");
    const void* pw = vector_of(w, r.cols, x, "weight");
    const void* pb = vector_of(b, r.cols, x, "bias");
    void* stream = stream_of(x);
    const int64_t ldr = res ? same_rows(*res, x, "residual") : 0;
    const at::ScalarType type = x.scalar_type();
    at::Tensor total, y, mean, rstd;
    muon_status st;
    {
      const Unlocked unlocked;
      if (res || p != 0.0) total = empty(x.sizes(), type);
      y = empty(x.sizes(), type);
      const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
      mean = empty(lead, at::kFloat);
      rstd = empty(lead, at::kFloat);
      st = p_layer_norm(
          r.rows, r.cols, dt, wdt, x.const_data_ptr(), r.ld, res ? res->const_data_ptr() : nullptr, ldr,
          pw, pb, (float)eps, (float)p, seed, offset,
          total.defined() ? total.mutable_data_ptr() : nullptr, y.mutable_data_ptr(),
          static_cast<float*>(mean.mutable_data_ptr()), static_cast<float*>(rstd.mutable_data_ptr()),
          stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({wrap(std::move(y)), total.defined() ? wrap(std::move(total)) : none(),
                     wrap(std::move(mean)), wrap(std::move(rstd))});
  });
}

// (dy, sum, mean, rstd, weight, dsum, p, seed, offset, need_weight, need_bias)
// -> (dx, dresidual or None, dweight or None, dbias or None)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &dy = tensor(a[0], "dy"), &sum = tensor(a[1], "sum");
    const at::Tensor &mean = tensor(a[2], "mean"), &rstd = tensor(a[3], "rstd");
    const at::Tensor *w = maybe(a[4], "weight"), *ds = maybe(a[5], "dsum");
    const double p = number(a[6]);
    const uint64_t seed = word(a[7]), offset = word(a[8]);
    const bool need_w = truth(a[9]), need_b = truth(a[10]);
    const int dt = dtype_of(dy, "dy");
    const Rows r = rows_or_raise(dy, "dy");
    const int64_t lds = same_rows(sum, dy, "sum");
    check_each_row(mean, r.rows, at::kFloat, dy, "mean");
    check_each_row(rstd, r.rows, at::kFloat, dy, "rstd");
    const int wdt = w ? dtype_of(*w, "weight") : MUON_F32;
    const at::ScalarType wtype = w ? w->scalar_type() : at::kFloat, type = dy.scalar_type();
    const void* pw = vector_of(w, r.cols, dy, "weight");
    void* stream = stream_of(dy);
    const int64_t ldd = ds ? same_rows(*ds, dy, "dsum") : 0;
    at::Tensor dx, dres, dw, db, ws;
    size_t bytes = 0;
    muon_status st = MUON_OK;
    if (need_w || need_b) st = p_layer_norm_workspace_bytes(r.rows, r.cols, &bytes);
    if (st != MUON_OK) return PyLong_FromLong(st);
    {
      const Unlocked unlocked;
      dx = empty(dy.sizes(), type);
      if (p != 0.0) dres = empty(dy.sizes(), type);
      if (need_w) dw = empty({r.cols}, wtype);
      if (need_b) db = empty({r.cols}, wtype);
      if (need_w || need_b) ws = empty({(int64_t)bytes}, at::kByte);
      auto ptr = [](at::Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; };
      st = p_layer_norm_backward(
          r.rows, r.cols, dt, wdt, dy.const_data_ptr(), r.ld, sum.const_data_ptr(), lds,
          static_cast<const float*>(mean.const_data_ptr()),
          static_cast<const float*>(rstd.const_data_ptr()), pw, ds ? ds->const_data_ptr() : nullptr, ldd,
          (float)p, seed, offset, ptr(dx), ptr(dres), ptr(dw), ptr(db), ptr(ws), bytes, stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    auto out = [](at::Tensor& t) { return t.defined() ? wrap(std::move(t)) : none(); };
    return tuple_of({out(dx), out(dres), out(dw), out(db)});
  });
}

// (x, p, seed, offset, residual, out) -> y
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const double p = number(a[1]);
    const uint64_t seed = word(a[2]), offset = word(a[3]);
    const at::Tensor *res = maybe(a[4], "residual"), *given = maybe(a[5], "out");
    const int dt = dtype_of(x, "x");
    if (!x.is_cuda()) value_error("x is not on a CUDA device");
    const at::ScalarType type = x.scalar_type();
    check_flat(x, x.numel(), type, x, "x");
    void* stream = stream_of(x);
    if (res) {
      if (res->sizes() != x.sizes()) value_error("residual must have the shape of x");
      check_flat(*res, x.numel(), type, x, "residual");
    }
    at::Tensor y;
    if (given) {
      if (given->sizes() != x.sizes()) value_error("out must have the shape of x");
      check_flat(*given, x.numel(), type, x, "out");
      if (c10::GradMode::is_enabled() && given->requires_grad())
        throw Raise{PyExc_RuntimeError, "out requires grad, and the call is not differentiable"};
      // what autograd has saved of it is no longer what it saw
      given->unsafeGetTensorImpl()->bump_version();
      y = *given;
    }
    muon_status st;
    {
      const Unlocked unlocked;
      if (!given) y = empty(x.sizes(), type);
      st = p_dropout(x.numel(), dt, x.const_data_ptr(), res ? res->const_data_ptr() : nullptr, (float)p,
                     seed, offset, y.mutable_data_ptr(), stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    if (given) {
      Py_INCREF(a[5]);
      return a[5];
    }
    return wrap(std::move(y));
  });
}

const uint8_t* mask_of(const at::Tensor* m, int64_t tokens, const at::Tensor& like) {
  if (!m) return nullptr;
  if (m->scalar_type() != at::kBool && m->scalar_type() != at::kByte)
    type_error(std::string("token_mask must be bool or uint8, got ") + c10::toString(m->scalar_type()));
  check_each_row(*m, tokens, m->scalar_type(), like, "token_mask");
  return static_cast<const uint8_t*>(m->const_data_ptr());
}

// (logits, k, token_mask, normalize) -> (weights, index, counts, mean_prob, loss)
PyObject* route_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const at::Tensor& l = tensor(a[0], "logits");
    const int k = small(a[1]);
    const at::Tensor* mask = maybe(a[2], "token_mask");
    const bool normalize = truth(a[3]);
    const int dt = dtype_of(l, "logits");
    const Rows r = rows_or_raise(l, "logits");
    void* stream = stream_of(l);
    const uint8_t* pm = mask_of(mask, r.rows, l);
    if (r.cols > 0x7fffffff) return PyLong_FromLong(MUON_ERR_UNSUPPORTED_SHAPE);
    const int experts = (int)r.cols;
    size_t bytes = 0;
    muon_status st = k < 1 ? MUON_ERR_INVALID_ARG : k > experts ? MUON_ERR_UNSUPPORTED_SHAPE
                           : p_route_workspace_bytes(r.rows, experts, &bytes);
    if (st != MUON_OK) return PyLong_FromLong(st);
    c10::SmallVector<int64_t, 6> shape(l.sizes().begin(), l.sizes().end());
    shape.back() = k;
    at::Tensor ws, weights, index, counts, mean_prob, loss;
    {
      const Unlocked unlocked;
      ws = empty({(int64_t)bytes}, at::kByte);
      weights = empty(shape, at::kFloat);
      index = empty(shape, at::kInt);
      counts = empty({experts + 1}, at::kInt);
      mean_prob = empty({experts}, at::kFloat);
      loss = empty({}, at::kFloat);
      st = p_route(r.rows, experts, k, dt, l.const_data_ptr(), r.ld, pm, normalize,
                   static_cast<float*>(weights.mutable_data_ptr()),
                   static_cast<int32_t*>(index.mutable_data_ptr()),
                   static_cast<int32_t*>(counts.mutable_data_ptr()),
                   static_cast<float*>(mean_prob.mutable_data_ptr()),
                   static_cast<float*>(loss.mutable_data_ptr()), ws.mutable_data_ptr(), bytes, stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({wrap(std::move(weights)), wrap(std::move(index)), wrap(std::move(counts)),
                     wrap(std::move(mean_prob)), wrap(std::move(loss))});
  });
}

// (logits, index, counts, dweights, dloss, token_mask, normalize) -> dlogits
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor &l = tensor(a[0], "logits"), &index = tensor(a[1], "index"),
                     &counts = tensor(a[2], "counts");
    const at::Tensor *dw = maybe(a[3], "dweights"), *dl = maybe(a[4], "dloss"),
                     *mask = maybe(a[5], "token_mask");
    const bool normalize = truth(a[6]);
    const int dt = dtype_of(l, "logits");
    const Rows r = rows_or_raise(l, "logits");
    void* stream = stream_of(l);
    const int64_t nd = l.dim();
    if (index.dim() != nd || index.sizes().slice(0, nd - 1) != l.sizes().slice(0, nd - 1))
      value_error("index must have one row of picks a token");
    const int64_t k = index.size(nd - 1);
    if (r.cols > 0x7fffffff || k > 0x7fffffff) return PyLong_FromLong(MUON_ERR_UNSUPPORTED_SHAPE);
    check_flat(index, r.rows * k, at::kInt, l, "index");
    check_flat(counts, r.cols + 1, at::kInt, l, "counts");
    if (dw) {
      check_flat(*dw, r.rows * k, at::kFloat, l, "dweights");
      const int64_t two[2] = {r.rows, k};
      if (!listed_alike(dw->sizes(), index.sizes()) && !listed_alike(dw->sizes(), two))
        value_error("dweights must have the shape of index, or its rows in two dimensions or one");
    }
    const uint8_t* pm = mask_of(mask, r.rows, l);
    at::Tensor out;
    muon_status st;
    {
      const Unlocked unlocked;
      out = empty(l.sizes(), l.scalar_type());
      st = p_route_backward(
          r.rows, (int)r.cols, (int)k, dt, l.const_data_ptr(), r.ld, pm, normalize,
          static_cast<const int32_t*>(index.const_data_ptr()),
          static_cast<const int32_t*>(counts.const_data_ptr()),
          dw ? static_cast<const float*>(dw->const_data_ptr()) : nullptr,
          dl ? static_cast<const float*>(dl->const_data_ptr()) : nullptr, out.mutable_data_ptr(), stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return wrap(std::move(out));
  });
}

// whether a tensor can be passed as rows without a copy
PyObject* is_rows(PyObject*, PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a tensor");
    return nullptr;
  }
  Rows r;
  return PyBool_FromLong(rows_of(THPVariable_Unpack(o), &r) == nullptr);
}

// bind({name: address}): the library's entry points
PyObject* bind(PyObject*, PyObject* names) {
  auto get = [&](const char* name, auto& to) {
    PyObject* v = PyDict_Check(names) ? PyDict_GetItemString(names, name) : nullptr;
    void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
    to = reinterpret_cast<std::decay_t<decltype(to)>>(p);
    return p != nullptr;
  };
  if (!get("muon_layer_norm", p_layer_norm) ||
      !get("muon_layer_norm_backward", p_layer_norm_backward) ||
      !get("muon_layer_norm_workspace_bytes", p_layer_norm_workspace_bytes) ||
      !get("muon_dropout", p_dropout) || !get("muon_route", p_route) ||
      !get("muon_route_workspace_bytes", p_route_workspace_bytes) ||
      !get("muon_route_backward", p_route_backward)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point of libmuon is missing");
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FAST(layer_norm_forward), FAST(layer_norm_backward), FAST(dropout), FAST(route_forward),
    FAST(route_backward), {"is_rows", is_rows, METH_O, nullptr}, {"bind", bind, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) {
  return PyModule_Create(&module);
}
