// CPython binding of the operators beside the expert layer (include/moe_ops_gb300.h): takes torch
// tensors, checks shapes, types and devices, and calls the C entry points. The same checks written
// in Python took 4 to 8 us a call, more than the small operators' kernels; here they take a few
// hundred ns. ops.py holds the signatures and documents them.
// Every function takes its arguments by position and returns the C status; a wrong tensor raises
// ValueError (TypeError where a tensor or number is something else) before anything is enqueued.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/moe_ops_gb300.h"

namespace {

struct Raised {};  // a Python exception is set

[[noreturn]] void fail(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised();
}

std::string list(at::IntArrayRef dims) {
  std::string s = "[";
  for (size_t i = 0; i < dims.size(); ++i) s += (i ? ", " : "") + std::to_string(dims[i]);
  return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

// The device of a call's first tensor, which has to be the current one.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) fail(PyExc_ValueError, std::string(name) + ": expected a CUDA tensor");
  const int dev = t.get_device();
  if (dev != c10::cuda::current_device())
    fail(PyExc_ValueError, std::string(name) + ": expected a tensor on the current device, got cuda:" + std::to_string(dev));
  return dev;
}

// Shape, type and device; the innermost dimension contiguous.
void expect(const at::Tensor& t, const char* name, at::IntArrayRef dims, at::ScalarType type, int dev) {
  if (t.sizes() != dims || t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev)
    fail(PyExc_ValueError, std::string(name) + ": expected " + at::toString(type) + " " + list(dims) + " on cuda:" +
                               std::to_string(dev) + ", got " + at::toString(t.scalar_type()) + " " + list(t.sizes()) + " on " +
                               t.device().str());
  if (dims.size() && dims.back() > 1 && t.stride(-1) != 1)
    fail(PyExc_ValueError, std::string(name) + ": expected a contiguous innermost dimension");
}

void* ptr(const at::Tensor& t) { return t.data_ptr(); }

template <typename T = int32_t>
T* ints(PyObject* o, const char* name, int64_t n, int dev) {
  const at::Tensor& t = tensor(o, name);
  expect(t, name, {n}, at::kInt, dev);
  return static_cast<T*>(ptr(t));
}

uint32_t* err_word(PyObject* o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "err");
  if (t.numel() != 1 || t.element_size() != 4 || !t.is_cuda() || t.get_device() != dev)
    fail(PyExc_ValueError, "err: expected one 4-byte word on the device");
  return static_cast<uint32_t*>(ptr(t));
}

void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Raised();
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw Raised();
  return s;
}

int32_t int32(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, std::string(name) + ": out of range");
  return static_cast<int32_t>(v);
}
int32_t int32(int64_t v, const char* name) {
  if (v > INT32_MAX) fail(PyExc_ValueError, std::string(name) + ": too large");
  return static_cast<int32_t>(v);
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}

int dtype16(const at::Tensor& t, const char* name, int64_t dims, const char* form) {
  const at::ScalarType s = t.scalar_type();
  if ((s != at::kBFloat16 && s != at::kHalf) || t.dim() != dims)
    fail(PyExc_ValueError, std::string(name) + ": expected bf16 or f16 " + form + ", got " + at::toString(s) + " " + list(t.sizes()));
  return s == at::kBFloat16 ? MOE_DT_BF16 : MOE_DT_F16;
}

// A row tensor [T][H]; returns its row stride (a single row's is its width).
int64_t rows(const at::Tensor& t, const char* name, at::IntArrayRef dims, at::ScalarType type, int dev) {
  expect(t, name, dims, type, dev);
  return dims[0] > 1 ? t.stride(0) : dims[1];
}

int norm(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const int dev = device_of(x, "x");
  moe_rmsnorm_args p = {};
  p.dtype = dtype16(x, "x", 2, "[T][H]");
  const at::ScalarType type = x.scalar_type();
  const int64_t T = x.size(0), H = x.size(1);
  const at::IntArrayRef dims = x.sizes();
  p.x_stride = rows(x, "x", dims, type, dev);
  p.x = ptr(x);
  const at::Tensor& w = tensor(a[1], "weight");
  p.weight_f32 = w.scalar_type() == at::kFloat;
  expect(w, "weight", {H}, p.weight_f32 ? at::kFloat : type, dev);
  p.weight = ptr(w);
  p.eps = number(a[2]);
  if (a[3] != Py_None) {
    const at::Tensor& t = tensor(a[3], "out");
    p.out_stride = rows(t, "out", dims, type, dev);
    p.out = ptr(t);
  }
  if (a[4] != Py_None) {
    const at::Tensor& t = tensor(a[4], "residual");
    p.residual_stride = rows(t, "residual", dims, type, dev);
    p.residual = ptr(t);
  }
  if (a[5] != Py_None) {
    const at::Tensor& t = tensor(a[5], "residual_out");
    p.residual_out_stride = rows(t, "residual_out", dims, type, dev);
    p.residual_out = ptr(t);
  }
  p.group = int32(a[8], "group");
  if (a[6] != Py_None) {
    const at::Tensor& t = tensor(a[6], "out8");
    if (t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte)
      fail(PyExc_ValueError, std::string("out8: expected float8_e4m3fn or uint8, got ") + at::toString(t.scalar_type()));
    p.out8_stride = rows(t, "out8", dims, t.scalar_type(), dev);
    p.out8 = static_cast<uint8_t*>(ptr(t));
    if (a[7] == Py_None) fail(PyExc_ValueError, "scales: out8 needs scales");
    const at::Tensor& s = tensor(a[7], "scales");
    expect(s, "scales", {T, p.group > 0 ? (H + p.group - 1) / p.group : 1}, at::kFloat, dev);
    if (!s.is_contiguous()) fail(PyExc_ValueError, "scales: expected a contiguous tensor");
    p.scales = static_cast<float*>(ptr(s));
  } else if (a[7] != Py_None) {
    fail(PyExc_ValueError, "scales: only with out8");
  }
  p.err = err_word(a[9], dev);
  p.T = int32(T, "x");
  p.H = int32(H, "x");
  return moe_add_rmsnorm(stream_of(a[10], dev), &p);
}

int plan(PyObject* const* a) {
  const at::Tensor& ctx = tensor(a[0], "ctx_lens");
  const int dev = device_of(ctx, "ctx_lens");
  const int64_t B = ctx.numel();
  moe_paged_plan_args p = {};
  p.ctx_lens = ints(a[0], "ctx_lens", B, dev);
  p.new_lens = ints(a[1], "new_lens", B, dev);
  const at::Tensor& table = tensor(a[2], "block_table");
  if (table.dim() != 2) fail(PyExc_ValueError, "block_table: expected [B][W]");
  const int64_t W = table.size(1);
  p.table_stride = rows(table, "block_table", {B, W}, at::kInt, dev);
  p.block_table = static_cast<int32_t*>(ptr(table));
  const int64_t F = tensor(a[3], "free_pages").numel(), N = tensor(a[8], "positions").numel();
  p.free_pages = ints(a[3], "free_pages", F, dev);
  p.free_head = ints(a[4], "free_head", 1, dev);
  p.page_size = int32(a[5], "page_size");
  p.q_start = ints(a[6], "q_start", B + 1, dev);
  p.kv_lens = ints(a[7], "kv_lens", B, dev);
  p.positions = ints(a[8], "positions", N, dev);
  p.slots = ints(a[9], "slots", N, dev);
  p.free_head_out = ints(a[10], "free_head_out", 1, dev);
  p.err = err_word(a[11], dev);
  p.B = int32(B, "ctx_lens");
  p.W = int32(W, "block_table");
  p.F = int32(F, "free_pages");
  p.N = int32(N, "positions");
  return moe_paged_plan(stream_of(a[12], dev), &p);
}

struct Caches {
  const at::Tensor& k;
  const at::Tensor& v;
  Caches(PyObject* ko, PyObject* vo, at::ScalarType type, int dev, int64_t D, int64_t heads /* or -1 */)
      : k(tensor(ko, "k_cache")), v(tensor(vo, "v_cache")) {
    if (k.dim() != 4 || k.size(3) != D || (heads >= 0 && k.size(2) != heads) || v.sizes() != k.sizes())
      fail(PyExc_ValueError, "k_cache, v_cache: expected [pages][page_size][" + (heads < 0 ? "Hkv" : std::to_string(heads)) +
                                 "][" + std::to_string(D) + "], got " + list(k.sizes()) + ", " + list(v.sizes()));
    expect(k, "k_cache", k.sizes(), type, dev);
    expect(v, "v_cache", k.sizes(), type, dev);
  }
  template <typename Args>
  void fill(Args& p) const {
    p.num_pages = int32(k.size(0), "k_cache");
    p.page_size = int32(k.size(1), "k_cache");
    p.Hkv = int32(k.size(2), "k_cache");
    p.kc_page = k.stride(0);
    p.kc_row = k.stride(1);
    p.kc_head = k.stride(2);
    p.vc_page = v.stride(0);
    p.vc_row = v.stride(1);
    p.vc_head = v.stride(2);
    p.k_cache = ptr(k);
    p.v_cache = ptr(v);
  }
};

int rotary(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const int dev = device_of(q, "q");
  moe_rotary_args p = {};
  p.dtype = dtype16(q, "q", 3, "[N][Hq][D]");
  const at::ScalarType type = q.scalar_type();
  const at::Tensor& k = tensor(a[1], "k");
  const at::Tensor& v = tensor(a[2], "v");
  if (k.dim() != 3) fail(PyExc_ValueError, "k: expected [N][Hkv][D], got " + list(k.sizes()));
  const int64_t N = q.size(0), D = q.size(2);
  expect(q, "q", q.sizes(), type, dev);
  expect(k, "k", {N, k.size(1), D}, type, dev);
  expect(v, "v", {N, k.size(1), D}, type, dev);
  const at::Tensor& o = a[8] == Py_None ? q : tensor(a[8], "q_out");
  expect(o, "q_out", q.sizes(), type, dev);
  Caches(a[6], a[7], type, dev, D, k.size(1)).fill(p);
  const at::Tensor& f = tensor(a[5], "inv_freq");
  const int64_t half = f.numel();
  expect(f, "inv_freq", {half}, at::kDouble, dev);
  p.q = ptr(q);
  p.k = ptr(k);
  p.v = ptr(v);
  p.q_out = ptr(o);
  p.positions = ints(a[3], "positions", N, dev);
  p.slots = ints(a[4], "slots", N, dev);
  p.inv_freq = static_cast<const double*>(ptr(f));
  p.q_tok = q.stride(0);
  p.q_head = q.stride(1);
  p.k_tok = k.stride(0);
  p.k_head = k.stride(1);
  p.v_tok = v.stride(0);
  p.v_head = v.stride(1);
  p.qo_tok = o.stride(0);
  p.qo_head = o.stride(1);
  p.N = int32(N, "q");
  p.Hq = int32(q.size(1), "q");
  p.D = int32(D, "q");
  p.rot = int32(2 * half, "inv_freq");
  const int on = PyObject_IsTrue(a[9]);
  if (on < 0) throw Raised();
  p.interleaved = on;
  p.mscale = number(a[10]);
  p.err = err_word(a[11], dev);
  return moe_rotary_append(stream_of(a[12], dev), &p);
}

int attention(PyObject* const* a) {
  moe_attn_ctx* ctx = static_cast<moe_attn_ctx*>(PyLong_AsVoidPtr(a[0]));
  if (PyErr_Occurred()) throw Raised();
  const int dev = int32(a[1], "device");  // the handle's
  const at::Tensor& q = tensor(a[2], "q");
  moe_attn_args p = {};
  p.dtype = dtype16(q, "q", 3, "[N][Hq][D]");
  const at::ScalarType type = q.scalar_type();
  expect(q, "q", q.sizes(), type, dev);
  const at::Tensor& o = tensor(a[8], "out");
  expect(o, "out", q.sizes(), type, dev);
  Caches(a[3], a[4], type, dev, q.size(2), -1).fill(p);
  const int64_t B = tensor(a[7], "kv_lens").numel();
  const at::Tensor& table = tensor(a[5], "block_table");
  if (table.dim() != 2) fail(PyExc_ValueError, "block_table: expected [B][W]");
  p.table_stride = rows(table, "block_table", {B, table.size(1)}, at::kInt, dev);
  p.block_table = static_cast<const int32_t*>(ptr(table));
  p.q_start = ints(a[6], "q_start", B + 1, dev);
  p.kv_lens = ints(a[7], "kv_lens", B, dev);
  p.scale = number(a[9]);
  if (a[10] != Py_None) {
    const at::Tensor& l = tensor(a[10], "lse");
    expect(l, "lse", {q.size(0), q.size(1)}, at::kFloat, dev);
    if (!l.is_contiguous()) fail(PyExc_ValueError, "lse: expected a contiguous tensor");
    p.lse = static_cast<float*>(ptr(l));
  }
  p.max_new = int32(a[11], "max_new");
  p.q = ptr(q);
  p.out = ptr(o);
  p.q_tok = q.stride(0);
  p.q_head = q.stride(1);
  p.out_tok = o.stride(0);
  p.out_head = o.stride(1);
  p.N = int32(q.size(0), "q");
  p.B = int32(B, "kv_lens");
  p.Hq = int32(q.size(1), "q");
  p.D = int32(q.size(2), "q");
  p.W = int32(table.size(1), "block_table");
  return moe_attn_forward(ctx, stream_of(a[12], dev), &p);
}

// No C++ exception leaves a function.
template <int (*F)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define ENTRY(f, n) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>))
PyMethodDef methods[] = {{"norm", ENTRY(norm, 11), METH_FASTCALL, nullptr},
                         {"plan", ENTRY(plan, 13), METH_FASTCALL, nullptr},
                         {"rotary", ENTRY(rotary, 13), METH_FASTCALL, nullptr},
                         {"attention", ENTRY(attention, 13), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_binding() { return PyModule_Create(&module); }
