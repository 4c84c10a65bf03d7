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

#include <cstring>
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
decltype(&muon_gated_scan) p_gated_scan;
decltype(&muon_gated_scan_backward) p_gated_scan_backward;
decltype(&muon_norm_rotate_heads) p_norm_rotate_heads;
decltype(&muon_norm_rotate_heads_backward) p_norm_rotate_heads_backward;
decltype(&muon_norm_rotate_heads_workspace_bytes) p_norm_rotate_heads_workspace_bytes;
decltype(&muon_token_log_probs) p_token_log_probs;
decltype(&muon_token_log_probs_backward) p_token_log_probs_backward;
decltype(&muon_policy_loss) p_policy_loss;
decltype(&muon_policy_loss_backward) p_policy_loss_backward;
decltype(&muon_policy_loss_workspace_bytes) p_policy_loss_workspace_bytes;

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

// ------------------------------------------------------- operators over sequences

// the data of a tensor that may be absent
template <typename T> const T* data(const at::Tensor* t) {
  return t ? static_cast<const T*>(t->const_data_ptr()) : nullptr;
}
template <typename T> T* data(at::Tensor& t) {
  return t.defined() ? static_cast<T*>(t.mutable_data_ptr()) : nullptr;
}
PyObject* wrapped(at::Tensor& t) { return t.defined() ? wrap(std::move(t)) : none(); }

// bytes, one for each of `shape`, of a bool or uint8 tensor that lists its elements
// like them
const uint8_t* flags_of(const at::Tensor* t, at::IntArrayRef shape, int64_t numel,
                        const at::Tensor& like, const char* what) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kBool && t->scalar_type() != at::kByte)
    type_error(std::string(what) + " must be bool or uint8, got " + c10::toString(t->scalar_type()));
  check_flat(*t, numel, t->scalar_type(), like, what);
  if (!listed_alike(t->sizes(), shape))
    value_error(std::string(what) + " must have the shape of the tokens, or one dimension");
  return data<uint8_t>(t);
}

// Sequences of rows: [..., length, dim]
struct Sequences { int64_t batch, length, dim; };
Sequences sequences_of(const at::Tensor& t, const char* what) {
  const int64_t nd = t.dim();
  if (nd < 2) value_error(std::string(what) + " needs at least two dimensions, tokens and channels");
  int64_t batch = 1;
  for (int64_t d = 0; d < nd - 2; ++d) batch *= t.size(d);
  return {batch, t.size(nd - 2), t.size(nd - 1)};
}
// the dense fp32 state of each sequence and channel
const float* state_of(const at::Tensor* t, const Sequences& q, const at::Tensor& like, const char* what) {
  if (!t) return nullptr;
  check_flat(*t, q.batch * q.dim, at::kFloat, like, what);
  c10::SmallVector<int64_t, 6> shape(like.sizes().begin(), like.sizes().end() - 2);
  shape.push_back(q.dim);
  const int64_t two[2] = {q.batch, q.dim};
  if (t->sizes() != at::IntArrayRef(shape) && t->sizes() != at::IntArrayRef(two))
    value_error(std::string(what) + " must have the shape of x without the tokens' dimension");
  return data<float>(t);
}
at::Tensor empty_state(const at::Tensor& like, const Sequences& q) {
  c10::SmallVector<int64_t, 6> shape(like.sizes().begin(), like.sizes().end() - 2);
  shape.push_back(q.dim);
  return empty(shape, at::kFloat);
}

// (gate, x, state, starts, token_mask, mix) -> (h, state)
PyObject* gated_scan_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor &gate = tensor(a[0], "gate"), &x = tensor(a[1], "x");
    const at::Tensor *state = maybe(a[2], "state"), *starts = maybe(a[3], "starts"),
                     *mask = maybe(a[4], "token_mask");
    const bool mix = truth(a[5]);
    const int dt = dtype_of(x, "x");
    const Rows r = rows_or_raise(x, "x");
    const Sequences q = sequences_of(x, "x");
    const int64_t ldg = same_rows(gate, x, "gate");
    void* stream = stream_of(x);
    const at::IntArrayRef tokens = x.sizes().slice(0, x.dim() - 1);
    const uint8_t* ps = flags_of(starts, tokens, q.batch * q.length, x, "starts");
    const uint8_t* pm = flags_of(mask, tokens, q.batch * q.length, x, "token_mask");
    const float* p0 = state_of(state, q, x, "state");
    at::Tensor h, last;
    muon_status st;
    {
      const Unlocked unlocked;
      h = empty(x.sizes(), x.scalar_type());
      last = empty_state(x, q);
      st = p_gated_scan(q.batch, q.length, q.dim, dt, gate.const_data_ptr(), ldg, x.const_data_ptr(), r.ld,
                        p0, ps, pm, mix, h.mutable_data_ptr(), data<float>(last), stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({wrap(std::move(h)), wrap(std::move(last))});
  });
}

// (dh, gate, x, h, state, dstate, starts, token_mask, mix, need_gate, need_x,
// need_state) -> (dgate or None, dx or None, dstate or None)
PyObject* gated_scan_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor &dh = tensor(a[0], "dh"), &gate = tensor(a[1], "gate"), &h = tensor(a[3], "h");
    const at::Tensor *x = maybe(a[2], "x"), *state = maybe(a[4], "state"), *dlast = maybe(a[5], "dstate"),
                     *starts = maybe(a[6], "starts"), *mask = maybe(a[7], "token_mask");
    const bool mix = truth(a[8]), need_g = truth(a[9]), need_x = truth(a[10]), need_s = truth(a[11]);
    const int dt = dtype_of(dh, "dh");
    const Rows r = rows_or_raise(dh, "dh");
    const Sequences q = sequences_of(dh, "dh");
    const int64_t ldg = same_rows(gate, dh, "gate"), ldh = same_rows(h, dh, "h");
    const int64_t ldx = x ? same_rows(*x, dh, "x") : 0;
    void* stream = stream_of(dh);
    const at::IntArrayRef tokens = dh.sizes().slice(0, dh.dim() - 1);
    const uint8_t* ps = flags_of(starts, tokens, q.batch * q.length, dh, "starts");
    const uint8_t* pm = flags_of(mask, tokens, q.batch * q.length, dh, "token_mask");
    const float *p0 = state_of(state, q, dh, "state"), *pl = state_of(dlast, q, dh, "dstate");
    at::Tensor dg, dx, ds;
    muon_status st;
    {
      const Unlocked unlocked;
      if (need_g) dg = empty(dh.sizes(), dh.scalar_type());
      if (need_x) dx = empty(dh.sizes(), dh.scalar_type());
      if (need_s) ds = empty_state(dh, q);
      st = p_gated_scan_backward(q.batch, q.length, q.dim, dt, dh.const_data_ptr(), r.ld,
                                 gate.const_data_ptr(), ldg, data<void>(x), ldx, h.const_data_ptr(), ldh, p0,
                                 pl, ps, pm, mix, data<void>(dg), data<void>(dx), data<float>(ds), stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({wrapped(dg), wrapped(dx), wrapped(ds)});
  });
}

// Heads of tokens: [..., heads, dim] with a dense last dimension, heads at one
// stride, tokens at one stride
struct HeadRows { int64_t tokens, heads, dim, ld, step; };
const char* heads_of(const at::Tensor& t, HeadRows* r) {
  if (!t.is_cuda()) return " is not on a CUDA device";
  const int64_t nd = t.dim();
  if (nd < 2) return " needs at least two dimensions, heads and their elements";
  const auto size = t.sizes(), stride = t.strides();
  *r = {1, size[nd - 2], size[nd - 1], -1, size[nd - 2] > 1 ? stride[nd - 2] : size[nd - 1]};
  if (r->dim > 1 && stride[nd - 1] != 1) return " has a last dimension that is not dense";
  const bool none = t.numel() == 0;
  for (int64_t d = nd - 3; d >= 0; --d) {
    if (size[d] != 1 && !none) {
      if (r->ld < 0) r->ld = stride[d];
      else if (stride[d] != r->ld * r->tokens) return " has leading dimensions that are not tokens at one stride";
    }
    r->tokens *= size[d];
  }
  if (r->ld < 0) r->ld = r->heads * r->dim;
  return nullptr;
}
HeadRows heads_or_raise(const at::Tensor& t, const char* what) {
  HeadRows r;
  if (const char* why = heads_of(t, &r)) value_error(std::string(what) + why);
  return r;
}
// laid out like `like` but for its strides
HeadRows same_heads(const at::Tensor& t, const at::Tensor& like, const char* what) {
  if (t.sizes() != like.sizes() || t.device() != like.device())
    value_error(std::string(what) + " must have its heads' shape and device");
  if (t.scalar_type() != like.scalar_type())
    type_error(std::string(what) + " must be of its heads' type, got " + c10::toString(t.scalar_type()));
  return heads_or_raise(t, what);
}

// What the two passes over heads share: (q, k or None, q_weight, k_weight, cos, sin, positions,
// eps, neighbours) from a[0] on
struct HeadCall {
  const at::Tensor *q, *k, *qw, *kw, *cos, *sin, *pos;
  HeadRows rq{}, rk{};
  int dt, wdt, rotary = 0;
  int64_t table = 0, period = 1;
  float eps;
  bool neighbours;
  at::ScalarType wtype = at::kFloat;
  const void *pqw, *pkw;
  explicit HeadCall(PyObject* const* a)
      : q(&tensor(a[0], "q")), k(maybe(a[1], "k")), qw(maybe(a[2], "q_weight")), kw(maybe(a[3], "k_weight")),
        cos(maybe(a[4], "cos")), sin(maybe(a[5], "sin")), pos(maybe(a[6], "positions")),
        eps((float)number(a[7])), neighbours(truth(a[8])) {
    dt = dtype_of(*q, "q");
    rq = heads_or_raise(*q, "q");
    if (k) {
      if (k->scalar_type() != q->scalar_type())
        type_error(std::string("k must be of q's type, got ") + c10::toString(k->scalar_type()));
      rk = heads_or_raise(*k, "k");
      const int64_t nd = q->dim();
      if (k->device() != q->device() || k->dim() != nd ||
          k->sizes().slice(0, nd - 2) != q->sizes().slice(0, nd - 2) || rk.dim != rq.dim)
        value_error("k must have q's tokens, head width and device");
    }
    wdt = MUON_F32;
    if (qw || kw) {
      wdt = dtype_of(qw ? *qw : *kw, "q_weight and k_weight");
      wtype = (qw ? *qw : *kw).scalar_type();
    }
    if (qw && kw && qw->scalar_type() != kw->scalar_type())
      type_error("q_weight and k_weight must be of one type");
    pqw = vector_of(qw, rq.dim, *q, "q_weight");
    pkw = vector_of(kw, rq.dim, *q, "k_weight");
    if (!cos != !sin) value_error("cos and sin go together");
    if (cos) {
      if (cos->dim() != 2 || cos->sizes() != sin->sizes()) value_error("cos and sin must be of one shape [table, pairs]");
      check_flat(*cos, cos->numel(), at::kFloat, *q, "cos");
      check_flat(*sin, sin->numel(), at::kFloat, *q, "sin");
      table = cos->size(0);
      if (2 * cos->size(1) > rq.dim) value_error("cos and sin have more pairs than a head");
      rotary = (int)(2 * cos->size(1));
    }
    const at::IntArrayRef tokens = q->sizes().slice(0, q->dim() - 2);
    if (pos) {
      check_flat(*pos, rq.tokens, at::kLong, *q, "positions");
      if (!listed_alike(pos->sizes(), tokens))
        value_error("positions must have the shape of the tokens, or one dimension");
    } else if (!tokens.empty() && tokens.back() > 0) {
      period = tokens.back();
    }
    if (rq.heads > 65536 || rk.heads > 65536) value_error("more than 65536 heads");
    if (rq.dim > 1024) value_error("heads of more than 1024 elements");
  }
};

// (q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours) -> (q, k or None)
PyObject* norm_rotate_heads_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const HeadCall c(a);
    void* stream = stream_of(*c.q);
    at::Tensor yq, yk;
    muon_status st;
    {
      const Unlocked unlocked;
      yq = empty(c.q->sizes(), c.q->scalar_type());
      if (c.k) yk = empty(c.k->sizes(), c.q->scalar_type());
      st = p_norm_rotate_heads(c.rq.tokens, (int)c.rq.heads, (int)c.rk.heads, (int)c.rq.dim, c.rotary, c.dt,
                               c.wdt, c.q->const_data_ptr(), c.rq.ld, c.rq.step, data<void>(c.k), c.rk.ld,
                               c.rk.step, c.pqw, c.pkw, c.eps, data<float>(c.cos), data<float>(c.sin),
                               c.table, data<int64_t>(c.pos), c.period, c.neighbours, data<void>(yq),
                               data<void>(yk), stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({wrapped(yq), wrapped(yk)});
  });
}

// (q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours, dq, dk, need_q, need_k,
// need_q_weight, need_k_weight) -> (dq, dk, dq_weight, dk_weight), each or None
PyObject* norm_rotate_heads_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const HeadCall c(a);
    const at::Tensor &dq = tensor(a[9], "dq"), *dk = maybe(a[10], "dk");
    const bool nq = truth(a[11]), nk = truth(a[12]), nqw = truth(a[13]), nkw = truth(a[14]);
    if (!c.k != !dk) value_error("k and dk go together");
    const HeadRows rdq = same_heads(dq, *c.q, "dq"), rdk = c.k ? same_heads(*dk, *c.k, "dk") : HeadRows{};
    void* stream = stream_of(*c.q);
    size_t bytes = 0;
    muon_status st = MUON_OK;
    if (nqw || nkw)
      st = p_norm_rotate_heads_workspace_bytes(c.rq.tokens, (int)c.rq.heads, (int)c.rk.heads, (int)c.rq.dim,
                                               &bytes);
    if (st != MUON_OK) return PyLong_FromLong(st);
    at::Tensor gq, gk, gqw, gkw, ws;
    {
      const Unlocked unlocked;
      if (nq) gq = empty(c.q->sizes(), c.q->scalar_type());
      if (nk && c.k) gk = empty(c.k->sizes(), c.q->scalar_type());
      if (nqw) gqw = empty({c.rq.dim}, c.wtype);
      if (nkw) gkw = empty({c.rq.dim}, c.wtype);
      if (nqw || nkw) ws = empty({(int64_t)bytes}, at::kByte);
      st = p_norm_rotate_heads_backward(
          c.rq.tokens, (int)c.rq.heads, (int)c.rk.heads, (int)c.rq.dim, c.rotary, c.dt, c.wdt,
          dq.const_data_ptr(), rdq.ld, rdq.step, data<void>(dk), rdk.ld, rdk.step, c.q->const_data_ptr(),
          c.rq.ld, c.rq.step, data<void>(c.k), c.rk.ld, c.rk.step, c.pqw, c.pkw, c.eps, data<float>(c.cos),
          data<float>(c.sin), c.table, data<int64_t>(c.pos), c.period, c.neighbours, data<void>(gq),
          data<void>(gk), data<void>(gqw), data<void>(gkw), data<void>(ws), bytes, stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({wrapped(gq), wrapped(gk), wrapped(gqw), wrapped(gkw)});
  });
}

// the tokens whose log probabilities are asked for
const int64_t* tokens_of(const at::Tensor& t, int64_t rows, const at::Tensor& logits) {
  check_each_row(t, rows, at::kLong, logits, "tokens");
  return data<int64_t>(&t);
}

// (logits, tokens, scale) -> (log_probs, lse)
PyObject* token_log_probs_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    const at::Tensor &l = tensor(a[0], "logits"), &tokens = tensor(a[1], "tokens");
    const float scale = (float)number(a[2]);
    const int dt = dtype_of(l, "logits");
    const Rows r = rows_or_raise(l, "logits");
    void* stream = stream_of(l);
    const int64_t* index = tokens_of(tokens, r.rows, l);
    at::Tensor lp, lse;
    muon_status st;
    {
      const Unlocked unlocked;
      const at::IntArrayRef lead = l.sizes().slice(0, l.dim() - 1);
      lp = empty(lead, at::kFloat);
      lse = empty(lead, at::kFloat);
      st = p_token_log_probs(r.rows, r.cols, dt, l.const_data_ptr(), r.ld, index, scale, data<float>(lp),
                             data<float>(lse), stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({wrap(std::move(lp)), wrap(std::move(lse))});
  });
}

// (dlog_probs, logits, tokens, lse, scale, out) -> dlogits
PyObject* token_log_probs_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor &d = tensor(a[0], "dlog_probs"), &l = tensor(a[1], "logits"),
                     &tokens = tensor(a[2], "tokens"), &lse = tensor(a[3], "lse");
    const float scale = (float)number(a[4]);
    const at::Tensor* given = maybe(a[5], "out");
    const int dt = dtype_of(l, "logits");
    const Rows r = rows_or_raise(l, "logits");
    void* stream = stream_of(l);
    const int64_t* index = tokens_of(tokens, r.rows, l);
    check_each_row(d, r.rows, at::kFloat, l, "dlog_probs");
    check_each_row(lse, r.rows, at::kFloat, l, "lse");
    at::Tensor out;
    if (given) {
      if (given->sizes() != l.sizes()) value_error("out must have the shape of logits");
      check_flat(*given, l.numel(), l.scalar_type(), l, "out");
      if (c10::GradMode::is_enabled() && given->requires_grad())
        throw Raise{PyExc_RuntimeError, "out requires grad, and the call is not differentiable"};
      given->unsafeGetTensorImpl()->bump_version();
      out = *given;
    }
    muon_status st;
    {
      const Unlocked unlocked;
      if (!given) out = empty(l.sizes(), l.scalar_type());
      st = p_token_log_probs_backward(r.rows, r.cols, dt, data<float>(&d), l.const_data_ptr(), r.ld, index,
                                      data<float>(&lse), scale, out.mutable_data_ptr(), stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    if (given) {
      Py_INCREF(a[5]);
      return a[5];
    }
    return wrap(std::move(out));
  });
}

// What the two passes of the policy loss share: (log_probs, old, advantages, ref, token_mask,
// clip_low, clip_high, kl) from a[0] on
struct PolicyCall {
  const at::Tensor *lp, *old, *adv, *ref, *mask;
  double low, high;
  float kl;
  int64_t batch, length, ldl, ldo, lda, ldr;
  const uint8_t* pm;
  explicit PolicyCall(PyObject* const* a)
      : lp(&tensor(a[0], "log_probs")), old(&tensor(a[1], "old_log_probs")), adv(&tensor(a[2], "advantages")),
        ref(maybe(a[3], "ref_log_probs")), mask(maybe(a[4], "token_mask")), low(number(a[5])),
        high(number(a[6])), kl((float)number(a[7])) {
    if (lp->scalar_type() != at::kFloat)
      type_error(std::string("log_probs must be fp32, got ") + c10::toString(lp->scalar_type()));
    const Rows r = rows_or_raise(*lp, "log_probs");
    length = r.cols;
    batch = 1;
    for (int64_t d = 0; d + 1 < lp->dim(); ++d) batch *= lp->size(d);
    ldl = r.ld;
    ldo = same_rows(*old, *lp, "old_log_probs");
    ldr = ref ? same_rows(*ref, *lp, "ref_log_probs") : 0;
    const at::IntArrayRef lead = lp->sizes().slice(0, lp->dim() - 1);
    if (adv->sizes() == lp->sizes()) {
      lda = same_rows(*adv, *lp, "advantages");
    } else {
      check_flat(*adv, batch, at::kFloat, *lp, "advantages");
      const int64_t one[1] = {batch};
      if (adv->sizes() != lead && adv->sizes() != at::IntArrayRef(one))
        value_error("advantages must be one a token or one a sequence");
      lda = -1;
    }
    pm = flags_of(mask, lp->sizes(), batch * length, *lp, "token_mask");
  }
};

// (log_probs, old, advantages, ref, token_mask, clip_low, clip_high, kl, by_sequence)
// -> (loss, kl, clipped, weights)
PyObject* policy_loss_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const PolicyCall c(a);
    const bool by_sequence = truth(a[8]);
    void* stream = stream_of(*c.lp);
    size_t bytes = 0;
    muon_status st = p_policy_loss_workspace_bytes(c.batch, c.length, &bytes);
    if (st != MUON_OK) return PyLong_FromLong(st);
    at::Tensor loss, kl, clipped, weights, ws;
    {
      const Unlocked unlocked;
      loss = empty({}, at::kFloat);
      kl = empty({}, at::kFloat);
      clipped = empty({}, at::kFloat);
      weights = empty(c.lp->sizes().slice(0, c.lp->dim() - 1), at::kFloat);
      ws = empty({(int64_t)bytes}, at::kByte);
      st = p_policy_loss(c.batch, c.length, data<float>(c.lp), c.ldl, data<float>(c.old), c.ldo,
                         data<float>(c.adv), c.lda, data<float>(c.ref), c.ldr, c.pm, c.low, c.high, c.kl,
                         by_sequence, data<float>(loss), data<float>(kl), data<float>(clipped),
                         data<float>(weights), data<void>(ws), bytes, stream);
    }
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({wrapped(loss), wrapped(kl), wrapped(clipped), wrapped(weights)});
  });
}

// (log_probs, old, advantages, ref, token_mask, clip_low, clip_high, kl, weights, dloss) -> dlog_probs
PyObject* policy_loss_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const PolicyCall c(a);
    const at::Tensor &weights = tensor(a[8], "weights"), *dloss = maybe(a[9], "dloss");
    check_each_row(weights, c.batch, at::kFloat, *c.lp, "weights");
    if (dloss) check_flat(*dloss, 1, at::kFloat, *c.lp, "dloss");
    void* stream = stream_of(*c.lp);
    at::Tensor out;
    muon_status st;
    {
      const Unlocked unlocked;
      out = empty(c.lp->sizes(), at::kFloat);
      st = p_policy_loss_backward(c.batch, c.length, data<float>(c.lp), c.ldl, data<float>(c.old), c.ldo,
                                  data<float>(c.adv), c.lda, data<float>(c.ref), c.ldr, c.pm, c.low, c.high,
                                  c.kl, data<float>(&weights), data<float>(dloss), data<float>(out), stream);
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

// whether a tensor can be passed as heads of tokens without a copy
PyObject* is_heads(PyObject*, PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a tensor");
    return nullptr;
  }
  HeadRows r;
  return PyBool_FromLong(heads_of(THPVariable_Unpack(o), &r) == nullptr);
}

// bind({name: address}): the library's entry points.  Those of the training operators are all
// there, those over sequences all or, once they are bound, none; no other name is.  What
// is refused binds nothing.
struct Entry { const char* name; void* to; };
#define ENTRY(f) Entry{"muon_" #f, &p_##f}
const Entry training_entries[] = {ENTRY(layer_norm), ENTRY(layer_norm_backward), ENTRY(layer_norm_workspace_bytes),
                                  ENTRY(dropout), ENTRY(route), ENTRY(route_workspace_bytes), ENTRY(route_backward)};
const Entry sequence_entries[] = {
    ENTRY(gated_scan), ENTRY(gated_scan_backward), ENTRY(norm_rotate_heads), ENTRY(norm_rotate_heads_backward),
    ENTRY(norm_rotate_heads_workspace_bytes), ENTRY(token_log_probs), ENTRY(token_log_probs_backward),
    ENTRY(policy_loss), ENTRY(policy_loss_backward), ENTRY(policy_loss_workspace_bytes)};
#undef ENTRY

PyObject* bind(PyObject*, PyObject* names) {
  return guarded(0, 0, [&]() -> PyObject* {
    if (!PyDict_Check(names)) type_error("entry points must be a dict of names and addresses");
    auto given = [&](const Entry& e) { return PyDict_GetItemString(names, e.name); };
    auto address = [&](const Entry& e) {
      PyObject* v = given(e);
      void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
      if (PyErr_Occurred()) throw Raise{nullptr, ""};
      if (!p) value_error(std::string("the entry point ") + e.name + " of libmuon is missing");
      return p;
    };
    bool sequences = !p_gated_scan;
    Py_ssize_t known = 0;
    for (const Entry& e : sequence_entries) sequences = sequences || given(e);
    for (const Entry& e : training_entries) known += address(e) != nullptr;
    if (sequences)
      for (const Entry& e : sequence_entries) known += address(e) != nullptr;
    if (PyDict_Size(names) != known) value_error("a name that is no entry point of libmuon");
    auto put = [&](const Entry& e) {
      void* const p = address(e);
      std::memcpy(e.to, &p, sizeof(p));
    };
    for (const Entry& e : training_entries) put(e);
    if (sequences)
      for (const Entry& e : sequence_entries) put(e);
    Py_RETURN_NONE;
  });
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FAST(layer_norm_forward), FAST(layer_norm_backward), FAST(dropout), FAST(route_forward),
    FAST(route_backward), FAST(gated_scan_forward), FAST(gated_scan_backward),
    FAST(norm_rotate_heads_forward), FAST(norm_rotate_heads_backward), FAST(token_log_probs_forward),
    FAST(token_log_probs_backward), FAST(policy_loss_forward), FAST(policy_loss_backward),
    {"is_rows", is_rows, METH_O, nullptr}, {"is_heads", is_heads, METH_O, nullptr}, {"bind", bind, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) {
  return PyModule_Create(&module);
}
