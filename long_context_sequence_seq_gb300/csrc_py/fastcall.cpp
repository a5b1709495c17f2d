// Marshalling of the strided calls (rotary positions, paged cache, single-token
// attention) in C++: what ulysses.py does for them in Python, without the
// interpreter.  A kernel of these takes 3 to 8 us at decode sizes and the
// Python marshalling around it 18 to 24, so the calls that a decode loop makes
// go through here.
//
// Only plain calls are taken: tensors that are torch.Tensor itself, on the
// current CUDA device, of the shapes, types and strides that the call wants,
// on the current stream.  Anything else returns None and the Python function
// goes on with its own checks, which say what is wrong; so a refusal has one
// place.  A call that was made returns its results, or the library's status
// code where that is not 0.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ulysses.h"

namespace {

using at::Tensor;

decltype(&ulysses_rope_fwd) g_rope_fwd = nullptr;
decltype(&ulysses_rope_bwd) g_rope_bwd = nullptr;
decltype(&ulysses_cache_write) g_cache_write = nullptr;
decltype(&ulysses_cache_read) g_cache_read = nullptr;
decltype(&ulysses_attn_decode) g_attn_decode = nullptr;
decltype(&ulysses_attn_decode_workspace) g_attn_decode_workspace = nullptr;

struct NotPlain {};   // thrown where the Python function has to look at the call

void plain(bool ok) { if (!ok) throw NotPlain(); }

const Tensor& tensor(PyObject* o) {
  plain(THPVariable_CheckExact(o));
  return THPVariable_Unpack(o);
}

int code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return ULYSSES_BF16;
    case at::kFloat: return ULYSSES_FP32;
    case at::kFloat8_e4m3fn: return ULYSSES_E4M3;
    default: throw NotPlain();
  }
}

// The device of the call: the first tensor's, which has to be the current one;
// every other tensor is checked against it.
struct Call {
  int dev;
  explicit Call(const Tensor& t) : dev(t.is_cuda() ? t.get_device() : -1) {
    plain(dev >= 0 && dev == c10::cuda::current_device());
  }
  const Tensor& on(const Tensor& t) const {
    plain(t.is_cuda() && t.get_device() == dev);
    return t;
  }
  // data of a contiguous tensor of one type
  template <typename T>
  T* flat(const Tensor& t, at::ScalarType type) const {
    on(t);
    plain(t.scalar_type() == type && t.is_contiguous());
    return static_cast<T*>(t.data_ptr());
  }
  Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

bool is_head(PyObject* layout) {
  plain(PyUnicode_Check(layout));
  if (PyUnicode_CompareWithASCIIString(layout, "head") == 0) return true;
  plain(PyUnicode_CompareWithASCIIString(layout, "seq") == 0);
  return false;
}

// Tokens and heads of a tensor of rows in either layout.
struct Rows { int64_t ts, hs, T, H, D; };
Rows rows(const Tensor& t, bool head, int dims = 3) {
  plain(t.dim() == dims && t.numel() > 0 && t.stride(dims - 1) == 1);
  const int a = dims - 3, tok = head ? a + 1 : a, hd = head ? a : a + 1;
  return Rows{t.stride(tok), t.stride(hd), t.size(tok), t.size(hd), t.size(dims - 1)};
}

struct Cache {
  void *k, *v;
  float *ks = nullptr, *vs = nullptr;
  int64_t pages;
  int H, page, D, type;
  Cache(const Call& c, PyObject* pk, PyObject* pv, PyObject* pks, PyObject* pvs) {
    const Tensor &tk = tensor(pk), &tv = tensor(pv);
    plain(tk.dim() == 4 && tk.sizes() == tv.sizes());
    k = c.flat<void>(tk, tk.scalar_type());
    v = c.flat<void>(tv, tk.scalar_type());
    pages = tk.size(0);
    H = (int)tk.size(1);
    page = (int)tk.size(2);
    D = (int)tk.size(3);
    plain(tk.size(1) <= INT32_MAX && tk.size(2) <= INT32_MAX && tk.size(3) <= INT32_MAX);
    type = code(tk.scalar_type());
    if (pks != Py_None) ks = scale(c, tensor(pks), tk);
    if (pvs != Py_None) vs = scale(c, tensor(pvs), tk);
  }
  static float* scale(const Call& c, const Tensor& s, const Tensor& of) {
    plain(s.sizes() == of.sizes().slice(0, 3));
    return c.flat<float>(s, at::kFloat);
  }
};

struct Table {
  int32_t* p;
  int cols;
  Table(const Call& c, PyObject* o, int64_t B) {
    const Tensor& t = tensor(o);
    plain(t.dim() == 2 && t.size(0) == B && t.size(1) <= INT32_MAX);
    p = c.flat<int32_t>(t, at::kInt);
    cols = (int)t.size(1);
  }
};

PyObject* status(int rc) { return PyLong_FromLong(rc); }

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
  return r;
}

// The library call, without the interpreter's lock (a launch can wait).
template <typename F>
int unlocked(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

// inverse, q, k, positions, inv_freq, axes, layout, pairs, dtype, out
PyObject* rope(PyObject* const* a) {
  const bool inverse = a[0] == Py_True, head = is_head(a[6]);
  PyObject* const objs[2] = {a[1] != Py_None ? a[1] : a[2], a[1] != Py_None ? a[2] : Py_None};
  const int n = objs[1] == Py_None ? 1 : 2;
  const Tensor& first = tensor(objs[0]);
  const Call c(first);
  const int dims = (int)first.dim();
  plain(dims == 3 || dims == 4);
  at::ScalarType out_type = first.scalar_type();
  if (a[8] != Py_None) {
    plain(THPDtype_Check(a[8]));
    out_type = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
  }
  PyObject* outs[2] = {nullptr, nullptr};
  if (a[9] != Py_None) {
    if (n == 1 && THPVariable_CheckExact(a[9])) {
      outs[0] = a[9];
    } else {
      plain(PyTuple_CheckExact(a[9]) && PyTuple_GET_SIZE(a[9]) == n);
      for (int i = 0; i < n; ++i) outs[i] = PyTuple_GET_ITEM(a[9], i);
    }
  }
  ulysses_rope_item items[2];
  Tensor result[2];
  Rows r0{};
  int64_t B = 1;
  for (int i = 0; i < n; ++i) {
    const Tensor& t = c.on(tensor(objs[i]));
    const Rows r = rows(t, head, dims);
    const int64_t b = dims == 4 ? t.size(0) : 1;
    if (i == 0) { r0 = r; B = b; }
    plain(r.T == r0.T && b == B && r.D == r0.D && t.scalar_type() == first.scalar_type());
    if (outs[i]) {
      const Tensor& o = c.on(tensor(outs[i]));
      plain(o.sizes() == t.sizes() && o.scalar_type() == out_type);
      result[i] = o;
    } else {
      result[i] = c.empty(t.sizes(), out_type);
    }
    const Rows o = rows(result[i], head, dims);
    plain(r.H <= INT32_MAX);
    items[i] = ulysses_rope_item{t.data_ptr(), result[i].data_ptr(), (int)r.H, dims == 4 ? t.stride(0) : 0, r.ts, r.hs,
                                 dims == 4 ? result[i].stride(0) : 0, o.ts, o.hs};
  }
  const Tensor& pos = tensor(a[3]);
  const int extra = (int)pos.dim() - (dims - 2);
  plain(extra == 0 || extra == 1);
  plain(dims == 3 ? pos.size(extra) == r0.T : pos.size(extra) == B && pos.size(extra + 1) == r0.T);
  const Tensor& inv = tensor(a[4]);
  plain(inv.is_cpu() && inv.scalar_type() == at::kDouble && inv.is_contiguous() && inv.numel() <= 64);
  const int32_t* axes = nullptr;
  if (a[5] != Py_None) {
    const Tensor& x = tensor(a[5]);
    plain(x.is_cpu() && x.scalar_type() == at::kInt && x.is_contiguous() && x.numel() == inv.numel());
    axes = static_cast<const int32_t*>(x.data_ptr());
  }
  plain(PyUnicode_Check(a[7]));
  const bool half = PyUnicode_CompareWithASCIIString(a[7], "half") == 0;
  plain(half || PyUnicode_CompareWithASCIIString(a[7], "adjacent") == 0);
  plain(B <= INT32_MAX && r0.D <= INT32_MAX);
  const int32_t* p = c.flat<int32_t>(pos, at::kInt);
  const int ci = code(first.scalar_type()), co = code(out_type), axn = extra ? (int)pos.size(0) : 1;
  const double* f = static_cast<const double*>(inv.data_ptr());
  const int rot = 2 * (int)inv.numel();
  const int rc = unlocked([&] {
    return (inverse ? g_rope_bwd : g_rope_fwd)(items, n, p, axn, f, axes, rot, half ? ULYSSES_PAIRS_HALF : ULYSSES_PAIRS_ADJACENT,
                                               r0.T, (int)B, (int)r0.D, ci, co, c.stream());
  });
  if (rc) return status(rc);
  if (n == 2) return pair(result[0], result[1]);
  return THPVariable_Wrap(result[0]);
}

// k, v, k_cache, v_cache, page_table, seq_lens, cu_new, k_scale, v_scale, layout
PyObject* cache_write(PyObject* const* a) {
  const Tensor &k = tensor(a[0]), &v = tensor(a[1]), &lens = tensor(a[5]);
  const Call c(k);
  c.on(v);
  const bool head = is_head(a[9]);
  const Rows rk = rows(k, head), rv = rows(v, head);
  plain(k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type());
  const Cache cache(c, a[2], a[3], a[7], a[8]);
  plain(rk.H == cache.H && rk.D == cache.D);
  const int64_t B = lens.numel();
  plain(B <= INT32_MAX);
  const Table table(c, a[4], B);
  const int32_t* cu = nullptr;
  if (a[6] != Py_None) {
    const Tensor& t = tensor(a[6]);
    plain(t.numel() == B + 1);
    cu = c.flat<int32_t>(t, at::kInt);
  }
  const int32_t* ln = c.flat<int32_t>(lens, at::kInt);
  const int type = code(k.scalar_type());
  const int rc = unlocked([&] {
    return g_cache_write(k.data_ptr(), v.data_ptr(), rk.ts, rk.hs, rv.ts, rv.hs, rk.T, (int)B, cu, table.p, table.cols, ln,
                         cache.k, cache.v, cache.ks, cache.vs, cache.pages, cache.page, cache.H, cache.D, type, cache.type,
                         c.stream());
  });
  return status(rc);
}

// k_cache, v_cache, page_table, cu_seqlens, T, first, k_scale, v_scale, dtype, layout, out
PyObject* cache_read(PyObject* const* a) {
  const Tensor &kc = tensor(a[0]), &cu = tensor(a[3]);
  const Call c(kc);
  const Cache cache(c, a[0], a[1], a[6], a[7]);
  const bool head = is_head(a[9]);
  plain(PyLong_CheckExact(a[4]) && cu.numel() > 0);
  const int64_t T = PyLong_AsLongLong(a[4]), B = cu.numel() - 1;
  plain(T > 0 && B <= INT32_MAX);
  const Table table(c, a[2], B);
  const int32_t* first = nullptr;
  if (a[5] != Py_None) {
    const Tensor& t = tensor(a[5]);
    plain(t.numel() == B);
    first = c.flat<int32_t>(t, at::kInt);
  }
  at::ScalarType type = kc.scalar_type() == at::kFloat8_e4m3fn ? at::kBFloat16 : kc.scalar_type();
  Tensor k, v;
  const int64_t size[3] = {head ? cache.H : T, head ? T : cache.H, cache.D};
  if (a[10] != Py_None) {
    plain(PyTuple_CheckExact(a[10]) && PyTuple_GET_SIZE(a[10]) == 2);
    k = c.on(tensor(PyTuple_GET_ITEM(a[10], 0)));
    v = c.on(tensor(PyTuple_GET_ITEM(a[10], 1)));
    type = k.scalar_type();
  }
  if (a[8] != Py_None) {
    plain(THPDtype_Check(a[8]));
    type = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
  }
  const int32_t* pcu = c.flat<int32_t>(cu, at::kInt);
  const int out_code = code(type);
  if (!k.defined()) {
    k = c.empty(size, type);
    v = c.empty(size, type);
  }
  plain(k.sizes() == at::IntArrayRef(size, 3) && v.sizes() == k.sizes() && k.scalar_type() == type && v.scalar_type() == type);
  const Rows rk = rows(k, head), rv = rows(v, head);
  const int rc = unlocked([&] {
    return g_cache_read(cache.k, cache.v, cache.ks, cache.vs, table.p, table.cols, pcu, first, k.data_ptr(), v.data_ptr(), rk.ts,
                        rk.hs, rv.ts, rv.hs, T, (int)B, cache.pages, cache.page, cache.H, cache.D, out_code, cache.type,
                        c.stream());
  });
  return rc ? status(rc) : pair(k, v);
}

// q, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, scale, layout, workspace, out, lse
PyObject* attn_decode(PyObject* const* a) {
  const Tensor &q = tensor(a[0]), &lens = tensor(a[4]);
  const Call c(q);
  const bool head = is_head(a[8]);
  const Rows rq = rows(q, head);
  const Cache cache(c, a[1], a[2], a[5], a[6]);
  const int64_t B = rq.T;
  plain(rq.D == cache.D && lens.numel() == B && B <= INT32_MAX && rq.H <= INT32_MAX);
  const Table table(c, a[3], B);
  const int32_t* ln = c.flat<int32_t>(lens, at::kInt);
  double scale = 0.0;
  if (a[7] != Py_None) {
    plain(PyFloat_CheckExact(a[7]));
    scale = PyFloat_AS_DOUBLE(a[7]);
  }
  const int dq = code(q.scalar_type());
  Tensor o, lse, ws;
  if (a[10] != Py_None) {
    o = c.on(tensor(a[10]));
    plain(o.sizes() == q.sizes() && o.scalar_type() == q.scalar_type());
  } else {
    o = c.empty(q.sizes(), q.scalar_type());
  }
  const Rows ro = rows(o, head);
  const int64_t ls[2] = {B, rq.H};
  if (a[11] != Py_None) {
    lse = tensor(a[11]);
    plain(lse.sizes() == at::IntArrayRef(ls, 2));
  } else {
    lse = c.empty(ls, at::kFloat);
  }
  float* pl = c.flat<float>(lse, at::kFloat);
  if (a[9] != Py_None) {
    ws = tensor(a[9]);
  } else {
    const int64_t n = (int64_t)g_attn_decode_workspace((int)B, (int)rq.H, cache.H, cache.D, table.cols, cache.page, dq, cache.type);
    if (n) ws = c.empty(n, at::kByte);
  }
  void* pw = nullptr;
  size_t nw = 0;
  if (ws.defined()) {
    pw = c.flat<void>(ws, at::kByte);
    nw = (size_t)ws.numel();
  }
  const int rc = unlocked([&] {
    return g_attn_decode(q.data_ptr(), rq.ts, rq.hs, cache.k, cache.v, cache.ks, cache.vs, table.p, table.cols, ln, o.data_ptr(),
                         ro.ts, ro.hs, pl, (int)B, (int)rq.H, cache.H, cache.D, cache.pages, cache.page, (float)scale, dq,
                         cache.type, pw, nw, c.stream());
  });
  return rc ? status(rc) : pair(o, lse);
}

template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return kFn(args);
  } catch (...) {
    // not a plain call, or torch refused something (memory): the Python function looks
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// Addresses of the library's functions, in this order.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[6];
  if (!PyArg_ParseTuple(args, "KKKKKK", p, p + 1, p + 2, p + 3, p + 4, p + 5)) return nullptr;
  g_rope_fwd = reinterpret_cast<decltype(g_rope_fwd)>(p[0]);
  g_rope_bwd = reinterpret_cast<decltype(g_rope_bwd)>(p[1]);
  g_cache_write = reinterpret_cast<decltype(g_cache_write)>(p[2]);
  g_cache_read = reinterpret_cast<decltype(g_cache_read)>(p[3]);
  g_attn_decode = reinterpret_cast<decltype(g_attn_decode)>(p[4]);
  g_attn_decode_workspace = reinterpret_cast<decltype(g_attn_decode_workspace)>(p[5]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"rope", (PyCFunction)(void*)entry<rope, 10>, METH_FASTCALL, nullptr},
    {"cache_write", (PyCFunction)(void*)entry<cache_write, 10>, METH_FASTCALL, nullptr},
    {"cache_read", (PyCFunction)(void*)entry<cache_read, 11>, METH_FASTCALL, nullptr},
    {"attn_decode", (PyCFunction)(void*)entry<attn_decode, 12>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
