// The marshalling of the calls that a decode step makes eagerly, in their usual
// form: every output allocated here, the current stream, tensors on the current
// device.  What a call of a few microseconds waits for is its arguments' way
// from Python to C: 20 to 35 us through ctypes, 3 to 9 here.
//
// Each function checks what the Python binding checks and returns NotImplemented
// where anything is out of the ordinary; the caller then takes the Python way,
// which says what is wrong or carries the call out.  A status other than DSA_OK
// comes back as an int.  The C entry points are handed over once by `bind`.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "dsa_prep.h"

namespace {

decltype(&dsa_rms_norm) g_rms_norm = nullptr;
decltype(&dsa_kv_append) g_kv_append = nullptr;
decltype(&dsa_tree_attention) g_tree_attention = nullptr;
decltype(&dsa_paged_attention_workspace_bytes) g_attention_workspace = nullptr;
decltype(&dsa_cache_keep) g_cache_keep = nullptr;
decltype(&dsa_cache_keep_workspace_bytes) g_keep_workspace = nullptr;

PyObject* out_of_the_ordinary() {
  PyErr_Clear();
  Py_INCREF(Py_NotImplemented);
  return Py_NotImplemented;
}

PyObject* status_of(dsa_status st) { return PyLong_FromLong(static_cast<long>(st)); }

// The arguments of one call, taken one after the other; `ok` falls with the first
// that is not as it should be.
struct Args {
  PyObject* const* at;
  bool ok = true;
  c10::Device device{c10::kCUDA, -1};
  at::ScalarType type = at::kFloat;

  const at::Tensor* tensor(int64_t dim) {  // the first one sets the device
    PyObject* o = *at++;
    if (!ok || !THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.dim() != dim ||
        (dim > 0 && t.stride(dim - 1) != 1 && t.size(dim - 1) > 1)) {
      ok = false;
      return nullptr;
    }
    if (device.index() < 0)
      device = t.device();
    else if (t.device() != device)
      ok = false;
    return &t;
  }
  const at::Tensor* tensor(int64_t dim, at::ScalarType want) {
    const at::Tensor* t = tensor(dim);
    if (t && t->scalar_type() != want) ok = false;
    return t;
  }
  const at::Tensor* maybe(int64_t dim, at::ScalarType want) {  // or None
    if (*at == Py_None) {
      ++at;
      return nullptr;
    }
    return tensor(dim, want);
  }
  const at::Tensor* rows16(int64_t dim) {  // bf16 or fp16, which sets the type
    const at::Tensor* t = tensor(dim);
    if (!t) return nullptr;
    type = t->scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf) ok = false;
    return t;
  }
  int64_t integer() {
    PyObject* o = *at++;
    if (!PyLong_Check(o)) {
      ok = false;
      return 0;
    }
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  int32_t int32() {
    const int64_t v = integer();
    if (v < INT32_MIN || v > INT32_MAX) ok = false;
    return static_cast<int32_t>(v);
  }
  double number() {
    PyObject* o = *at++;
    if (!PyFloat_Check(o) && !PyLong_Check(o)) {
      ok = false;
      return 0;
    }
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return v;
  }
  bool truth() {
    const int v = PyObject_IsTrue(*at++);
    if (v < 0) ok = false;
    return v == 1;
  }
  int32_t* error_word() {
    PyObject* o = *at++;
    if (o == Py_None) return nullptr;
    if (!ok || !THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.device() != device || t.scalar_type() != at::kInt || t.numel() < 1 ||
        (t.dim() && t.stride(-1) != 1 && t.size(-1) > 1))
      ok = false;
    return ok ? static_cast<int32_t*>(t.data_ptr()) : nullptr;
  }
  // Whether the call may be carried out here.
  bool usual() {
    if (!ok || PyErr_Occurred() || device.index() < 0 ||
        c10::cuda::current_device() != device.index())
      return false;
    return true;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
  // As at::empty, but not through the dispatcher, which takes 0.2 us for each.
  at::Tensor fresh(at::IntArrayRef shape, at::ScalarType t) const {
    return at::Tensor(at::detail::empty_cuda(shape, t, device, std::nullopt));
  }
  int32_t dtype() const { return type == at::kBFloat16 ? DSA_DTYPE_BF16 : DSA_DTYPE_FP16; }
};

// Lets other Python threads run while memory is allocated and kernels are launched:
// both may wait for the GPU, and what it waits for may need them.
struct NoGil {
  PyThreadState* const state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <class T>
T* ptr_of(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
int64_t stride0(const at::Tensor* t) { return t ? t->stride(0) : 0; }

PyObject* pack(const at::Tensor& a) { return THPVariable_Wrap(a); }

// (x, gamma, eps, residual, group or 0 for 16 bits, 8-bit scales?, pdl) -> out,
// (out, residual_out), (codes, scales) or (codes, scales, residual_out)
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 7 || !g_rms_norm) return out_of_the_ordinary();
  Args a{args};
  const at::Tensor* x = a.rows16(2);
  const at::Tensor* gamma = a.tensor(1, at::kFloat);
  const double eps = a.number();
  const at::Tensor* res = a.maybe(2, a.type);
  const int32_t group = a.int32();
  const bool bytes = a.truth(), pdl = a.truth();
  if (!a.usual() || gamma->size(0) != x->size(1) || (res && res->sizes() != x->sizes()) ||
      (group != 0 && group != 32 && group != 128) || x->size(0) > INT32_MAX ||
      x->size(1) > INT32_MAX)
    return out_of_the_ordinary();
  const int64_t T = x->size(0), N = x->size(1);
  at::Tensor out, codes, scales, z;
  dsa_status st;
  {
    const NoGil free;
    if (group) {
      codes = a.fresh({T, N}, at::kFloat8_e4m3fn);
      scales = a.fresh({T, (N + group - 1) / group}, bytes ? at::kFloat8_e8m0fnu : at::kFloat);
    } else {
      out = a.fresh({T, N}, a.type);
    }
    if (res) z = a.fresh({T, N}, a.type);
    st = g_rms_norm(
        x->data_ptr(), x->stride(0), ptr(res), stride0(res), res ? z.data_ptr() : nullptr,
        res ? N : 0, ptr_of<const float>(gamma), static_cast<float>(eps),
        group ? nullptr : out.data_ptr(), N, group ? codes.data_ptr() : nullptr, N,
        group ? scales.data_ptr() : nullptr, group ? scales.size(1) : 0,
        bytes ? DSA_SCALE_UE8M0 : DSA_SCALE_FP32, group ? group : 128, static_cast<int32_t>(T),
        static_cast<int32_t>(N), a.dtype(), pdl ? DSA_FLAG_PDL : 0u, a.stream());
  }
  if (st != DSA_OK) return status_of(st);
  if (!group && !res) return pack(out);
  PyObject* got = PyTuple_New((group ? 2 : 1) + (res ? 1 : 0));
  if (!got) return nullptr;
  Py_ssize_t i = 0;
  if (group) {
    PyTuple_SET_ITEM(got, i++, pack(codes));
    PyTuple_SET_ITEM(got, i++, pack(scales));
  } else {
    PyTuple_SET_ITEM(got, i++, pack(out));
  }
  if (res) PyTuple_SET_ITEM(got, i++, pack(z));
  return got;
}

// (k, v, k_cache, v_cache, positions, slots, q, cos, sin, rope_dim, rope_style,
// q_gamma, k_gamma, eps, err, pdl) -> q_out
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 16 || !g_kv_append) return out_of_the_ordinary();
  Args a{args};
  const at::Tensor* k = a.rows16(3);
  const at::ScalarType t16 = a.type;
  const at::Tensor *v = a.tensor(3, t16), *kc = a.tensor(4, t16), *vc = a.tensor(4, t16);
  const at::Tensor *pos = a.tensor(1, at::kLong), *slots = a.tensor(1, at::kLong);
  const at::Tensor* q = a.maybe(3, t16);
  const at::Tensor *cos = a.maybe(2, at::kFloat), *sin = a.maybe(2, at::kFloat);
  const int32_t rope = a.int32(), style = a.int32();
  const at::Tensor *qg = a.maybe(1, at::kFloat), *kg = a.maybe(1, at::kFloat);
  const double eps = a.number();
  int32_t* err = a.error_word();
  const bool pdl = a.truth();
  if (!a.usual()) return out_of_the_ordinary();
  const int64_t T = k->size(0), Hkv = k->size(1), D = k->size(2), H = q ? q->size(1) : 0;
  if (v->size(0) < T || v->size(1) != Hkv || v->size(2) != D || kc->size(2) != Hkv ||
      kc->size(3) != D || vc->sizes() != kc->sizes() || pos->size(0) < T || slots->size(0) < T ||
      (q && (q->size(0) < T || q->size(2) != D)) || (qg && qg->size(0) != D) ||
      (kg && kg->size(0) != D) || T > INT32_MAX || H > INT32_MAX || Hkv > INT32_MAX ||
      D > INT32_MAX || kc->size(1) > INT32_MAX)
    return out_of_the_ordinary();
  int64_t cs_stride = 0, rows = 1LL << 62;
  if (rope) {
    if (!cos || !sin || cos->stride(0) != sin->stride(0) || cos->size(0) != sin->size(0) ||
        rope < 0 || cos->size(1) < rope / 2 || sin->size(1) < rope / 2)
      return out_of_the_ordinary();
    cs_stride = cos->stride(0);
    rows = cos->size(0);
  }
  at::Tensor out;
  dsa_status st;
  {
    const NoGil free;
    if (q) out = a.fresh({T, H, D}, t16);
    st = g_kv_append(
        ptr(q), q ? q->stride(0) : 0, q ? q->stride(1) : 0, k->data_ptr(), k->stride(0),
        k->stride(1), v->data_ptr(), v->stride(0), v->stride(1), ptr_of<const int64_t>(pos),
        ptr_of<const int64_t>(slots), rope ? ptr_of<const float>(cos) : nullptr,
        rope ? ptr_of<const float>(sin) : nullptr, cs_stride, rows, ptr_of<const float>(qg),
        ptr_of<const float>(kg), static_cast<float>(eps), q ? out.data_ptr() : nullptr, H * D, D,
        kc->data_ptr(), vc->data_ptr(), kc->stride(0), kc->stride(1), kc->stride(2), vc->stride(0),
        vc->stride(1), vc->stride(2), kc->size(0), static_cast<int32_t>(kc->size(1)),
        static_cast<int32_t>(T), static_cast<int32_t>(H), static_cast<int32_t>(Hkv),
        static_cast<int32_t>(D), rope, style, a.dtype(), pdl ? DSA_FLAG_PDL : 0u, err, a.stream());
  }
  if (st != DSA_OK) return status_of(st);
  if (!q) Py_RETURN_NONE;
  return pack(out);
}

// A number of tokens: no context is longer than the largest int32.
int32_t span(int64_t n) {
  return n < 0 ? -1 : n > INT32_MAX ? INT32_MAX : static_cast<int32_t>(n);
}

// (q, k_cache, v_cache, table, start, lens, max_context, mask, scale, window,
// sinks, err, pdl) -> (out, lse)
PyObject* tree_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 13 || !g_tree_attention) return out_of_the_ordinary();
  Args a{args};
  const at::Tensor* q = a.rows16(3);
  const at::Tensor *kc = a.tensor(4, a.type), *vc = a.tensor(4, a.type);
  const at::Tensor *table = a.tensor(2, at::kInt), *start = a.tensor(1, at::kInt);
  const at::Tensor* lens = a.tensor(1, at::kInt);
  const int32_t most = a.int32();
  const at::Tensor* mask = a.tensor(2, at::kInt);
  const bool own_scale = *a.at == Py_None;
  double scale = 0;
  if (own_scale)
    ++a.at;
  else
    scale = a.number();
  const int32_t window = span(a.integer()), sinks = span(a.integer());
  int32_t* err = a.error_word();
  const bool pdl = a.truth();
  if (!a.usual()) return out_of_the_ordinary();
  const int64_t T = q->size(0), H = q->size(1), D = q->size(2), B = start->size(0) - 1;
  const int64_t page = kc->size(1), Hkv = kc->size(2), cols = table->size(1);
  if (vc->sizes() != kc->sizes() || kc->size(3) != D || Hkv < 1 || H % Hkv || B < 0 ||
      table->size(0) < B || cols * page < most || lens->size(0) < B || mask->size(0) < T ||
      T > INT32_MAX || H > INT32_MAX || D > INT32_MAX || B > INT32_MAX || page > INT32_MAX ||
      mask->size(1) > INT32_MAX)
    return out_of_the_ordinary();
  const int32_t t = static_cast<int32_t>(T), b = static_cast<int32_t>(B),
                h = static_cast<int32_t>(H), hkv = static_cast<int32_t>(Hkv),
                d = static_cast<int32_t>(D);
  if (own_scale) scale = std::pow(static_cast<double>(D), -0.5);
  at::Tensor out, lse, ws;
  dsa_status st;
  {
    const NoGil free;
    out = a.fresh({T, H, D}, a.type);
    lse = a.fresh({T, H}, at::kFloat);
    const size_t need = g_attention_workspace(t, b, h, hkv, d, most);
    if (need) ws = a.fresh({static_cast<int64_t>(need)}, at::kByte);
    const int64_t ts = table->stride(0);
    st = g_tree_attention(
        q->data_ptr(), q->stride(0), q->stride(1), kc->data_ptr(), vc->data_ptr(), kc->stride(0),
        kc->stride(1), kc->stride(2), vc->stride(0), vc->stride(1), vc->stride(2), kc->size(0),
        static_cast<int32_t>(page), ptr_of<const int32_t>(table),
        ts > cols || table->size(0) > 1 ? ts : cols, ptr_of<const int32_t>(start),
        ptr_of<const int32_t>(lens), most, ptr_of<const uint32_t>(mask),
        static_cast<int32_t>(mask->size(1)), mask->size(0) > 1 ? mask->stride(0) : mask->size(1),
        static_cast<float>(scale), window, sinks, out.data_ptr(), H * D, D,
        static_cast<float*>(lse.data_ptr()), t, b, h, hkv, d, a.dtype(), pdl ? DSA_FLAG_PDL : 0u,
        need ? ws.data_ptr() : nullptr, need, err, a.stream());
  }
  if (st != DSA_OK) return status_of(st);
  PyObject* got = PyTuple_New(2);
  if (!got) return nullptr;
  PyTuple_SET_ITEM(got, 0, pack(out));
  PyTuple_SET_ITEM(got, 1, pack(lse));
  return got;
}

// (bases, shapes, views, their pages, page size and device, page_refs, table, lens, page
// size, rows, drafted, kept, n_kept, err) -> 0
PyObject* cache_keep(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 15 || !g_cache_keep) return out_of_the_ordinary();
  Args a{args};
  const int64_t bases = a.integer(), shapes = a.integer();
  const int32_t views = a.int32();
  const int64_t view_pages = a.integer(), view_page = a.integer(), view_device = a.integer();
  const at::Tensor* refs = a.tensor(1, at::kInt);
  const at::Tensor *table = a.tensor(2, at::kInt), *lens = a.tensor(1, at::kInt);
  const int32_t page = a.int32();
  const at::Tensor *rows = a.tensor(1, at::kInt), *drafted = a.tensor(1, at::kInt);
  const at::Tensor *kept = a.tensor(2, at::kInt), *n_kept = a.tensor(1, at::kInt);
  int32_t* err = a.error_word();
  if (!a.usual()) return out_of_the_ordinary();
  const int64_t table_rows = table->size(0), cols = table->size(1), count = kept->size(0);
  if (refs->size(0) < 1 || lens->size(0) < table_rows ||
      (table_rows > 1 && table->stride(0) < cols) || table_rows > INT32_MAX || cols > INT32_MAX ||
      rows->size(0) != count || drafted->size(0) != count || n_kept->size(0) != count ||
      count > INT32_MAX || kept->size(1) > INT32_MAX ||
      (views && (view_pages != refs->size(0) || view_page != page ||
                 view_device != a.device.index())))
    return out_of_the_ordinary();
  const int32_t c = static_cast<int32_t>(count), most = static_cast<int32_t>(kept->size(1));
  const size_t need = g_keep_workspace(c, most);
  dsa_status st;
  {
    const NoGil free;
    const at::Tensor ws = a.fresh({static_cast<int64_t>(need ? need : 1)}, at::kByte);
    st = g_cache_keep(
        reinterpret_cast<void* const*>(bases), reinterpret_cast<const int64_t*>(shapes), views,
        refs->size(0), ptr_of<int32_t>(refs), ptr_of<int32_t>(table), static_cast<int32_t>(cols),
        table->stride(0) > cols ? table->stride(0) : cols, ptr_of<int32_t>(lens),
        static_cast<int32_t>(table_rows), page, ptr_of<const int32_t>(rows),
        ptr_of<const int32_t>(drafted), ptr_of<const int32_t>(kept),
        count > 1 ? kept->stride(0) : most, most, ptr_of<const int32_t>(n_kept), c, 0,
        ws.data_ptr(), need, err, a.stream());
  }
  return status_of(st);
}

// The addresses of the C entry points, in the order of the pointers above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 6) return out_of_the_ordinary();
  void* at[6];
  for (int i = 0; i < 6; ++i) at[i] = PyLong_AsVoidPtr(args[i]);
  if (PyErr_Occurred()) return nullptr;
  g_rms_norm = reinterpret_cast<decltype(g_rms_norm)>(at[0]);
  g_kv_append = reinterpret_cast<decltype(g_kv_append)>(at[1]);
  g_tree_attention = reinterpret_cast<decltype(g_tree_attention)>(at[2]);
  g_attention_workspace = reinterpret_cast<decltype(g_attention_workspace)>(at[3]);
  g_cache_keep = reinterpret_cast<decltype(g_cache_keep)>(at[4]);
  g_keep_workspace = reinterpret_cast<decltype(g_keep_workspace)>(at[5]);
  Py_RETURN_NONE;
}

// C++ exceptions (an allocation that fails) become Python's.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (const c10::OutOfMemoryError& e) {
    // the Python way runs out of memory too, with torch's own exception
    return out_of_the_ordinary();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<F>)), METH_FASTCALL,
          nullptr};
}

PyMethodDef g_methods[] = {method<rms_norm>("rms_norm"), method<kv_append>("kv_append"),
                           method<tree_attention>("tree_attention"),
                           method<cache_keep>("cache_keep"), method<bind>("bind"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
