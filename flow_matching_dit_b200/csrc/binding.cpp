// The operators' Python calls: argument checks, outputs and the call of the C
// entry point (include/gdit.h).  In C++ because a call is a few microseconds of
// GPU time: the same checks in Python took 6 to 10.
//
// The entry points come as addresses from the loaded library (init), so this
// module is not linked against it; torch supplies the tensors' memory and the
// current stream.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cmath>
#include <cstring>
#include <string>

#include "gdit.h"

namespace {

int (*fn_linear)(const gdit_linear_args*, void*);
int (*fn_norm)(const gdit_norm_args*, void*);
int (*fn_attention)(const gdit_attention_args*, void*);
PyObject* on_error;   // called with a negative status code; raises

// A Python exception that is already set, on its way out.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised();
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool is_none(PyObject* o) { return o == Py_None; }

// Every tensor of a call goes through here.
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (at::GradMode::is_enabled() && t.requires_grad())
    raise(PyExc_RuntimeError, std::string(name) + " requires a gradient, which this operator does not have: call it under torch.no_grad() or with " +
                                  name + ".detach()");
  return t;
}

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t n : t.sizes()) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
  return s + ")";
}

std::string name_of(int device) { return "cuda:" + std::to_string(device); }

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
  return t.get_device();
}

bool on(const at::Tensor& t, int device) { return t.is_cuda() && t.get_device() == device; }

int code_of(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return GDIT_F32;
  if (t == at::kBFloat16) return GDIT_BF16;
  raise(PyExc_TypeError, std::string(name) + " must be float32 or bfloat16, got " + c10::toString(t));
}

at::ScalarType dtype(PyObject* o, const char* name) {
  if (!THPDtype_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be float32 or bfloat16");
  const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  code_of(t, name);
  return t;
}

// One of the names; None is the first.
int choice(PyObject* o, const char* what, const char* const* names, int n) {
  if (is_none(o)) return 0;
  if (PyUnicode_Check(o))
    for (int i = 0; i < n; ++i)
      if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return i;
  std::string all;
  for (int i = 0; i < n; ++i) all += (i ? ", '" : "'") + std::string(names[i]) + "'";
  PyErr_Format(PyExc_ValueError, "%s is %R, expected one of [%s]", what, o, all.c_str());
  throw Raised();
}

const char* const kActivations[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};
const char* const kNorms[] = {"none", "layer", "rms"};

int whole(PyObject* o, const char* name) {
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (overflow || v != (int)v) raise(PyExc_ValueError, std::string(name) + " is out of range");
  return (int)v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return (float)v;
}

// Row stride of a [rows, cols] matrix with dense rows.
int64_t rows_of(const at::Tensor& t, const char* name, int device, int64_t rows, int64_t cols) {
  const std::string n(name);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    raise(PyExc_ValueError, n + " has shape " + shape_of(t) + ", expected (" + std::to_string(rows) + ", " + std::to_string(cols) + ")");
  if (!on(t, device)) raise(PyExc_ValueError, n + " is on " + t.device().str() + ", expected " + name_of(device));
  const int64_t s0 = t.stride(0), s1 = t.stride(1);
  if (s1 != 1 && cols > 1) raise(PyExc_ValueError, "the rows of " + n + " must be dense");
  if (s0 < cols) {
    if (rows > 1) raise(PyExc_ValueError, "the rows of " + n + " overlap");
    return (cols + 7) / 8 * 8;   // one row: its stride addresses nothing
  }
  return s0;
}

// Address of an optional contiguous vector [n], or table [groups, n] if groups >= 0.
template <typename T>
const T* vector(PyObject* o, const char* name, int device, int64_t n, int64_t groups = -1) {
  if (is_none(o)) return nullptr;
  const at::Tensor& t = tensor(o, name);
  const at::ScalarType want = std::is_same<T, float>::value ? at::kFloat : at::kInt;
  if (t.scalar_type() != want || !on(t, device) || !t.is_contiguous())
    raise(PyExc_TypeError, std::string(name) + " must be a contiguous " + (want == at::kFloat ? "torch.float32" : "torch.int32") +
                               " tensor on " + name_of(device));
  if (groups < 0 ? t.dim() != 1 || t.size(0) != n : t.dim() != 2 || t.size(0) != groups || t.size(1) != n)
    raise(PyExc_ValueError, std::string(name) + " has shape " + shape_of(t) + ", expected (" +
                                (groups < 0 ? std::to_string(n) + ",)" : std::to_string(groups) + ", " + std::to_string(n) + ")"));
  return static_cast<const T*>(t.data_ptr());
}

// The same for a [n] or [groups, n] table; groups is 1 without one.
const float* table(PyObject* o, const char* name, int device, int64_t n, int64_t& groups) {
  groups = 1;
  if (is_none(o)) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.dim() == 1) return vector<float>(o, name, device, n);
  groups = t.dim() > 0 ? t.size(0) : 0;
  if (groups < 1) raise(PyExc_ValueError, std::string(name) + " has no group");
  if (groups > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " has too many groups");
  return vector<float>(o, name, device, n, groups);
}

at::Tensor fresh(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}

// Where a call runs: the tensors' device and its current stream, or the stream given by
// its handle.  That is the current stream while this lives, so that outputs made
// meanwhile come from what the allocator keeps for it: a block of another stream's may
// still have a reader there, and may be handed out again there before the call has run.
struct Place {
  c10::cuda::CUDAStream stream;
  c10::cuda::OptionalCUDAStreamGuard guard;

  Place(PyObject* handle, int device) : stream(of(handle, (c10::DeviceIndex)device)) {
    if (!is_none(handle) || c10::cuda::current_device() != device) guard.reset_stream(stream);
  }

 private:
  static c10::cuda::CUDAStream of(PyObject* handle, c10::DeviceIndex device) {
    if (is_none(handle)) return c10::cuda::getCurrentCUDAStream(device);
    void* s = PyLong_AsVoidPtr(handle);
    if (s == nullptr && PyErr_Occurred()) throw Raised();
    if (s == nullptr || s == cudaStreamLegacy) return c10::cuda::getDefaultCUDAStream(device);
    return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), device);
  }
};

template <typename Args>
void call(int (*fn)(const Args*, void*), const Args& a, const Place& place) {
  void* s = place.stream.stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = fn(&a, s);
  Py_END_ALLOW_THREADS
  if (rc < 0) {
    PyObject* r = PyObject_CallFunction(on_error, "i", rc);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the call failed");
    throw Raised();
  }
}

void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
  if (fn_linear == nullptr) raise(PyExc_RuntimeError, "the library's entry points are not set");
}

// An output: the tensor given, whose version counts the write (so that autograd sees that a
// tensor which it has kept is no longer what it was), or the one made here.
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (is_none(given)) return THPVariable_Wrap(made);
  const at::Tensor& t = THPVariable_Unpack(given);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return Py_NewRef(given);
}

// linear(x, w, bias, activation, residual, out, out_dtype, stream)
PyObject* linear(PyObject*, PyObject* const* p, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect(n_args, 8);
    const at::Tensor &x = tensor(p[0], "x"), &w = tensor(p[1], "w");
    const int d = device_of(x, "x");
    if (x.scalar_type() != at::kBFloat16 || w.scalar_type() != at::kBFloat16)
      raise(PyExc_TypeError, "x and w must be bfloat16");
    if (x.dim() != 2 || w.dim() != 2) raise(PyExc_ValueError, "x must be [m, k] and w [n, k]");
    const int64_t m = x.size(0), k = x.size(1), n = w.size(0);
    if (k > INT32_MAX || n > INT32_MAX) raise(PyExc_ValueError, "x or w is too wide");
    gdit_linear_args a = {};
    a.ldx = rows_of(x, "x", d, m, k);
    a.ldw = rows_of(w, "w", d, n, k);
    if (m <= 1) a.ldx = k;   // one row: its stride addresses nothing, and need not be the multiple of 8 that k is
    if (n <= 1) a.ldw = k;
    const at::Tensor *res = is_none(p[4]) ? nullptr : &tensor(p[4], "residual"), *out = is_none(p[5]) ? nullptr : &tensor(p[5], "out");
    const at::ScalarType type = !is_none(p[6]) ? dtype(p[6], "out_dtype") : out ? out->scalar_type() : res ? res->scalar_type() : at::kBFloat16;
    a.out_dtype = code_of(type, "out_dtype");
    a.ldr = a.ldo = n;
    if (res != nullptr) {
      if (res->scalar_type() != type)
        raise(PyExc_TypeError, std::string("residual is ") + c10::toString(res->scalar_type()) + ", the output " + c10::toString(type) + ": they must be the same");
      a.ldr = rows_of(*res, "residual", d, m, n);
      a.residual = res->data_ptr();
    }
    a.activation = choice(p[3], "activation", kActivations, 5);
    a.bias = vector<float>(p[2], "bias", d, n);
    const Place place(p[7], d);
    at::Tensor made;
    if (out != nullptr) {
      if (out->scalar_type() != type)
        raise(PyExc_TypeError, std::string("out is ") + c10::toString(out->scalar_type()) + ", expected " + c10::toString(type));
      a.ldo = rows_of(*out, "out", d, m, n);
    } else {
      made = fresh({m, n}, type, d);
    }
    a.x = x.data_ptr(), a.w = w.data_ptr(), a.out = (out ? *out : made).data_ptr();
    a.m = m, a.n = (int)n, a.k = (int)k;
    call(fn_linear, a, place);
    return result(p[5], made);
  });
}

// norm_residual(h, y, post, post_gain, post_bias, gate, residual_scale, pre, pre_gain, pre_bias, scale, shift, row_group,
//               eps, out_h, out_u, u_dtype, stream)
PyObject* norm_residual(PyObject*, PyObject* const* p, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect(n_args, 18);
    const at::Tensor& h = tensor(p[0], "h");
    const int d = device_of(h, "h");
    if (h.dim() != 2) raise(PyExc_ValueError, "h must be [rows, dim]");
    const int64_t rows = h.size(0), dim = h.size(1);
    if (dim > INT32_MAX) raise(PyExc_ValueError, "h is too wide");
    gdit_norm_args a = {};
    a.rows = rows, a.dim = (int)dim;
    a.h_dtype = code_of(h.scalar_type(), "h");
    a.pre = choice(p[7], "pre", kNorms, 3);
    a.post = choice(p[2], "post", kNorms, 3);
    a.ldh = rows_of(h, "h", d, rows, dim);
    a.h = h.data_ptr();
    a.ldy = a.ldoh = a.ldou = dim;
    a.y_dtype = a.u_dtype = GDIT_BF16;
    const at::Tensor* y = is_none(p[1]) ? nullptr : &tensor(p[1], "y");
    if (y != nullptr) {
      a.ldy = rows_of(*y, "y", d, rows, dim);
      a.y = y->data_ptr();
      a.y_dtype = code_of(y->scalar_type(), "y");
    } else if (a.post != 0 || !is_none(p[3]) || !is_none(p[4]) || !is_none(p[5])) {
      raise(PyExc_ValueError, "post and gate act on y, which is not given");
    }
    int64_t gate_groups, g1, g2;
    a.gate = table(p[5], "gate", d, dim, gate_groups);
    a.scale = table(p[10], "scale", d, dim, g1);
    a.shift = table(p[11], "shift", d, dim, g2);
    const bool scaled = !is_none(p[10]), shifted = !is_none(p[11]);
    if (scaled && shifted && g1 != g2)
      raise(PyExc_ValueError, "scale has " + std::to_string(g1) + " groups, shift " + std::to_string(g2));
    a.gate_groups = (int)gate_groups;
    a.mod_groups = (int)(scaled ? g1 : g2);
    if (!is_none(p[12])) a.row_group = vector<int32_t>(p[12], "row_group", d, rows);
    else if (a.gate_groups > 1 || a.mod_groups > 1)
      raise(PyExc_ValueError, "row_group is needed: gate, scale or shift have several groups");
    if (a.post == 0 && (!is_none(p[3]) || !is_none(p[4]))) raise(PyExc_ValueError, "post_gain and post_bias need post");
    if (a.pre == 0 && (!is_none(p[8]) || !is_none(p[9]))) raise(PyExc_ValueError, "pre_gain and pre_bias need pre");
    a.post_gain = vector<float>(p[3], "post_gain", d, dim);
    a.post_bias = vector<float>(p[4], "post_bias", d, dim);
    a.pre_gain = vector<float>(p[8], "pre_gain", d, dim);
    a.pre_bias = vector<float>(p[9], "pre_bias", d, dim);
    a.residual_scale = number(p[6]);
    a.eps = number(p[13]);
    const bool want_h = y != nullptr || a.residual_scale != 1.f || !is_none(p[14]);
    const bool want_u = a.pre != 0 || scaled || shifted || !is_none(p[15]) || !is_none(p[16]);
    if (!want_h && !want_u)
      raise(PyExc_ValueError, "nothing to compute: give y, a residual_scale, pre, scale or shift");
    const Place place(p[17], d);
    at::Tensor made_h, made_u;
    if (!is_none(p[14])) {
      const at::Tensor& t = tensor(p[14], "out_h");
      if (t.scalar_type() != h.scalar_type())
        raise(PyExc_TypeError, std::string("out_h is ") + c10::toString(t.scalar_type()) + ", h is " + c10::toString(h.scalar_type()) + ": they must be the same");
      a.ldoh = rows_of(t, "out_h", d, rows, dim);
      a.out_h = t.data_ptr();
    }
    if (want_u) {
      const at::Tensor* u = is_none(p[15]) ? nullptr : &tensor(p[15], "out_u");
      const at::ScalarType type = !is_none(p[16]) ? dtype(p[16], "u_dtype") : u ? u->scalar_type() : y ? y->scalar_type() : at::kBFloat16;
      a.u_dtype = code_of(type, "u_dtype");
      if (u != nullptr) {
        if (u->scalar_type() != type)
          raise(PyExc_TypeError, std::string("out_u is ") + c10::toString(u->scalar_type()) + ", expected " + c10::toString(type));
        a.ldou = rows_of(*u, "out_u", d, rows, dim);
        a.out_u = u->data_ptr();
      } else {
        made_u = fresh({rows, dim}, type, d);
        a.out_u = made_u.data_ptr();
      }
    }
    if (want_h && is_none(p[14])) {
      made_h = fresh({rows, dim}, h.scalar_type(), d);
      a.out_h = made_h.data_ptr();
    }
    call(fn_norm, a, place);
    PyObject* first = want_h ? result(p[14], made_h) : Py_NewRef(p[0]);
    PyObject* second = want_u ? result(p[15], made_u) : Py_NewRef(Py_None);
    PyObject* both = PyTuple_Pack(2, first, second);
    Py_DECREF(first);
    Py_DECREF(second);
    return both;
  });
}

struct Heads {
  int64_t n, heads, dim, token, head;
};

Heads heads_of(const at::Tensor& t, const char* name, int device) {
  if (t.scalar_type() != at::kBFloat16 || !on(t, device))
    raise(PyExc_TypeError, std::string(name) + " must be a bfloat16 tensor on " + name_of(device));
  if (t.dim() != 3)
    raise(PyExc_ValueError, std::string(name) + " must be [tokens, heads, head_dim], got " + shape_of(t));
  Heads r = {t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
  if (t.stride(2) != 1 && r.dim > 1) raise(PyExc_ValueError, std::string("the last dimension of ") + name + " must be dense");
  if (r.heads > INT32_MAX || r.dim > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is too wide");
  // the stride of a dimension of one element addresses nothing
  if (r.n <= 1) r.token = r.heads * r.dim;
  if (r.heads <= 1) r.head = r.dim;
  return r;
}

// attention(q, k, v, cu_q, cu_k, max_q, max_k, causal, scale, k_len, out, return_lse, stream)
PyObject* attention(PyObject*, PyObject* const* p, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect(n_args, 13);
    const at::Tensor &q = tensor(p[0], "q"), &k = tensor(p[1], "k"), &v = tensor(p[2], "v");
    const int d = device_of(q, "q");
    const Heads hq = heads_of(q, "q", d), hk = heads_of(k, "k", d), hv = heads_of(v, "v", d);
    if (hk.dim != hq.dim || v.sizes() != k.sizes())
      raise(PyExc_ValueError, "q " + shape_of(q) + ", k " + shape_of(k) + " and v " + shape_of(v) + " do not fit together");
    const at::Tensor& cq = tensor(p[3], "cu_q");
    if (cq.dim() != 1 || cq.size(0) < 1) raise(PyExc_ValueError, "cu_q must be [batch + 1]");
    if (cq.size(0) > INT32_MAX) raise(PyExc_ValueError, "cu_q is too long");
    const int64_t batch = cq.size(0) - 1;
    gdit_attention_args a = {};
    a.out_token_stride = hq.heads * hq.dim, a.out_head_stride = hq.dim;
    if (!is_none(p[10])) {
      const at::Tensor& out = tensor(p[10], "out");
      const Heads ho = heads_of(out, "out", d);
      if (out.sizes() != q.sizes())
        raise(PyExc_ValueError, "out has shape " + shape_of(out) + ", expected " + shape_of(q));
      a.out_token_stride = ho.token, a.out_head_stride = ho.head;
      a.out = out.data_ptr();
    }
    a.cu_q = vector<int32_t>(p[3], "cu_q", d, batch + 1);
    a.cu_k = vector<int32_t>(p[4], "cu_k", d, batch + 1);
    a.k_len = vector<int32_t>(p[9], "k_len", d, batch);
    a.q = q.data_ptr(), a.k = k.data_ptr(), a.v = v.data_ptr();
    a.total_q = hq.n, a.total_k = hk.n;
    a.q_token_stride = hq.token, a.q_head_stride = hq.head, a.k_token_stride = hk.token, a.k_head_stride = hk.head;
    a.v_token_stride = hv.token, a.v_head_stride = hv.head;
    a.batch = (int)batch, a.heads = (int)hq.heads, a.kv_heads = (int)hk.heads, a.head_dim = (int)hq.dim;
    a.max_q = whole(p[5], "max_q"), a.max_k = whole(p[6], "max_k");
    a.causal = PyObject_IsTrue(p[7]);
    if (a.causal < 0) throw Raised();
    a.scale = is_none(p[8]) ? (float)(1.0 / std::sqrt((double)(hq.dim > 0 ? hq.dim : 1))) : number(p[8]);
    const int with_lse = PyObject_IsTrue(p[11]);
    if (with_lse < 0) throw Raised();
    const Place place(p[12], d);
    at::Tensor made, lse;
    if (is_none(p[10])) {
      made = fresh({hq.n, hq.heads, hq.dim}, at::kBFloat16, d);
      a.out = made.data_ptr();
    }
    if (with_lse) {
      lse = fresh({hq.n, hq.heads}, at::kFloat, d);
      a.lse = static_cast<float*>(lse.data_ptr());
    }
    call(fn_attention, a, place);
    PyObject* first = result(p[10], made);
    if (!with_lse) return first;
    PyObject* second = THPVariable_Wrap(lse);
    PyObject* both = PyTuple_Pack(2, first, second);
    Py_DECREF(first);
    Py_DECREF(second);
    return both;
  });
}

// init(address of gdit_linear, of gdit_norm_residual, of gdit_attention, on_error)
PyObject* init(PyObject*, PyObject* const* p, Py_ssize_t n_args) {
  if (n_args != 4) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  void* f[3];
  for (int i = 0; i < 3; ++i) {
    f[i] = PyLong_AsVoidPtr(p[i]);
    if (f[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is NULL");
      return nullptr;
    }
  }
  fn_linear = reinterpret_cast<decltype(fn_linear)>(f[0]);
  fn_norm = reinterpret_cast<decltype(fn_norm)>(f[1]);
  fn_attention = reinterpret_cast<decltype(fn_attention)>(f[2]);
  Py_XDECREF(on_error);
  on_error = Py_NewRef(p[3]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(linear), FAST(norm_residual), FAST(attention), FAST(init), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr) PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION);
  return m;
}
