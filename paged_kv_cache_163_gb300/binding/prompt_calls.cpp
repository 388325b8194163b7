// The argument checks of the binding's prompt-side calls in native code.
//
// Checking a dozen tensors' device, type, shape and density, and marshalling
// some thirty arguments, takes the interpreter 9 to 12 us a call, more than the
// kernels of small batches run.  Each function here checks what the Python
// function of the same call checks and, when all is in order, makes the C ABI
// call and returns its status.  When anything is not (or is unusual: another
// current device, a raw pointer), it returns None and has done nothing: the
// Python code then finds the words, or makes the call itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "pkv.h"

namespace {

decltype(&paged_kv_append_rope) call_append_rope;
decltype(&paged_kv_gather) call_gather;
decltype(&paged_attention_extend) call_extend;

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const at::Tensor *t, int dev) { return t && t->is_cuda() && t->get_device() == dev; }

// A dense tensor of this type and shape on the device.
bool dense(const at::Tensor *t, int dev, at::ScalarType type, at::IntArrayRef shape) {
  return on(t, dev) && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
}

// pkv_dtype of a 16-bit type, -1 for others.
int pair_type(at::ScalarType t) {
  return t == at::kHalf ? static_cast<int>(PKV_F16) : t == at::kBFloat16 ? static_cast<int>(PKV_BF16) : -1;
}

bool small(int64_t x) { return x >= 0 && x <= INT_MAX; }

bool integer(PyObject *o, int32_t *out) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  if (over || v < INT_MIN || v > INT_MAX) return false;
  *out = static_cast<int32_t>(v);
  return true;
}

bool error_word(PyObject *o, int dev, int32_t **out) {
  *out = nullptr;
  if (o == Py_None) return true;
  const at::Tensor *t = tensor(o);
  if (!on(t, dev) || t->numel() != 1 || t->scalar_type() != at::kInt) return false;
  *out = static_cast<int32_t *>(t->data_ptr());
  return true;
}

// The caller's stream handle, or torch's current stream.
bool stream_of(PyObject *o, int dev, pkv_stream_t *out) {
  if (o == Py_None) {
    *out = reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    return true;
  }
  if (!PyLong_Check(o)) return false;
  *out = reinterpret_cast<pkv_stream_t>(PyLong_AsVoidPtr(o));
  return !PyErr_Occurred();
}

struct Pool {
  int32_t nb, hkv, bs, d;
  pkv_dtype type;
  void *k, *v;
  float *ks = nullptr, *vs = nullptr;
};

// args: k_cache, v_cache, k_scale, v_scale; type -1: by the tensors' own
bool pool_of(PyObject *const *args, int32_t type, int dev, Pool &p) {
  const at::Tensor *k = tensor(args[0]), *v = tensor(args[1]);
  if (!on(k, dev) || k->dim() != 4 || !k->is_contiguous()) return false;
  if (type < 0) type = pair_type(k->scalar_type());
  if (type < 0 || type == PKV_F32) return false;
  const bool scaled = type != PKV_F16 && type != PKV_BF16;
  if (k->element_size() != (scaled ? 1 : 2)) return false;
  const auto s = k->sizes();
  for (const int64_t x : s)
    if (!small(x)) return false;
  const int64_t v_row = type == PKV_FP8_E4M3_INT4 ? s[3] / 2 : s[3];
  if (!dense(v, dev, k->scalar_type(), {s[0], s[1], s[2], v_row})) return false;
  p.nb = static_cast<int32_t>(s[0]);
  p.hkv = static_cast<int32_t>(s[1]);
  p.bs = static_cast<int32_t>(s[2]);
  p.d = static_cast<int32_t>(s[3]);
  p.type = static_cast<pkv_dtype>(type);
  p.k = k->data_ptr();
  p.v = v->data_ptr();
  if (scaled) {
    const int64_t shape[3] = {s[0], s[1], s[2]}, strides[3] = {2 * s[1] * s[2], 2 * s[2], 1};
    for (int i = 0; i < 2; ++i) {
      const at::Tensor *t = tensor(args[2 + i]);
      if (!on(t, dev) || t->scalar_type() != at::kFloat || t->sizes() != at::IntArrayRef(shape, 3) ||
          t->strides() != at::IntArrayRef(strides, 3))
        return false;
      (i ? p.vs : p.ks) = static_cast<float *>(t->data_ptr());
    }
  }
  return true;
}

// Rows [tokens, heads, d] of `type` whose tokens' rows are dense; the elements from token to token.
bool rows_of(const at::Tensor *t, int dev, at::ScalarType type, int64_t n, int64_t h, int64_t d, int64_t *step) {
  if (!on(t, dev) || t->scalar_type() != type || t->dim() != 3) return false;
  const auto z = t->sizes();
  if (z[0] != n || z[1] != h || z[2] != d) return false;
  const auto s = t->strides();
  if (n && h && (s[2] != 1 || (h > 1 && s[1] != d))) return false;
  *step = n > 1 ? s[0] : h * d;
  return true;
}

int32_t *ints(const at::Tensor *t) { return static_cast<int32_t *>(t->data_ptr()); }

#define OR_PYTHON(ok) \
  if (!(ok)) Py_RETURN_NONE

// q_out, q, k, v, positions, slots, cos_sin, k_cache, v_cache, k_scale, v_scale, interleaved, d_error, stream, type
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  OR_PYTHON(n == 15 && call_append_rope);
  try {
    const at::Tensor *k = tensor(a[2]), *v = tensor(a[3]), *cs = tensor(a[6]);
    OR_PYTHON(k && k->is_cuda() && k->dim() == 3);
    const int dev = k->get_device();
    OR_PYTHON(dev == c10::cuda::current_device());
    const auto type = k->scalar_type();
    const int dt = pair_type(type);
    int32_t cdt, *err;
    pkv_stream_t stream;
    Pool p;
    OR_PYTHON(dt >= 0 && integer(a[14], &cdt) && pool_of(a + 7, cdt, dev, p) && error_word(a[12], dev, &err) &&
              stream_of(a[13], dev, &stream));
    const int64_t t = k->size(0);
    int64_t qs = 0, ks, vs, hq = 0;
    OR_PYTHON(small(t) && rows_of(k, dev, type, t, p.hkv, p.d, &ks) && rows_of(v, dev, type, t, p.hkv, p.d, &vs));
    void *qp = nullptr, *qo = nullptr;
    if (a[1] != Py_None) {
      const at::Tensor *q = tensor(a[1]), *out = tensor(a[0]);
      OR_PYTHON(q && q->dim() == 3);
      hq = q->size(1);
      OR_PYTHON(small(hq) && rows_of(q, dev, type, t, hq, p.d, &qs) && dense(out, dev, type, {t, hq, p.d}));
      if (hq) {
        qp = q->data_ptr();
        qo = out->data_ptr();
      }
    }
    const at::Tensor *pos = tensor(a[4]), *slots = tensor(a[5]);
    OR_PYTHON(dense(pos, dev, at::kInt, {t}) && dense(slots, dev, at::kInt, {t}) && on(cs, dev) && cs->dim() == 3 &&
              cs->size(1) == 2 && cs->scalar_type() == at::kFloat && cs->is_contiguous() && small(cs->size(0)) &&
              small(2 * cs->size(2)));
    const int il = PyObject_IsTrue(a[11]);
    OR_PYTHON(il >= 0);
    return PyLong_FromLong(call_append_rope(
        qo, qp, k->data_ptr(), v->data_ptr(), static_cast<pkv_dtype>(dt), qs, ks, vs, static_cast<int32_t>(t),
        static_cast<int32_t>(hq), p.hkv, p.d, ints(pos), ints(slots), static_cast<const float *>(cs->data_ptr()),
        static_cast<int32_t>(cs->size(0)), static_cast<int32_t>(2 * cs->size(2)), il, p.k, p.v, p.type, p.ks, p.vs,
        p.nb, p.bs, err, stream));
  } catch (...) {
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

// k_out, v_out, k_cache, v_cache, k_scale, v_scale, tables, lens, starts, token_starts, d_error, stream, type
PyObject *gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
  OR_PYTHON(n == 13 && call_gather);
  try {
    const at::Tensor *ko = tensor(a[0]), *vo = tensor(a[1]), *tab = tensor(a[6]), *lens = tensor(a[7]),
                     *starts = tensor(a[8]);
    OR_PYTHON(ko && ko->is_cuda() && ko->dim() == 3);
    const int dev = ko->get_device();
    OR_PYTHON(dev == c10::cuda::current_device());
    const auto type = ko->scalar_type();
    const int dt = type == at::kFloat ? static_cast<int>(PKV_F32) : pair_type(type);
    int32_t cdt, *err;
    pkv_stream_t stream;
    Pool p;
    OR_PYTHON(dt >= 0 && integer(a[12], &cdt) && pool_of(a + 2, cdt, dev, p) && error_word(a[10], dev, &err) &&
              stream_of(a[11], dev, &stream));
    const int64_t rows = ko->size(0);
    OR_PYTHON(small(rows) && dense(ko, dev, type, {rows, p.hkv, p.d}) && dense(vo, dev, type, {rows, p.hkv, p.d}));
    OR_PYTHON(on(tab, dev) && tab->dim() == 2 && tab->scalar_type() == at::kInt && tab->is_contiguous());
    const int64_t b = tab->size(0), mb = tab->size(1);
    OR_PYTHON(small(b) && small(mb) && dense(lens, dev, at::kInt, {b}) && dense(starts, dev, at::kInt, {b + 1}));
    const int32_t *first = nullptr;
    if (a[9] != Py_None) {
      const at::Tensor *f = tensor(a[9]);
      OR_PYTHON(dense(f, dev, at::kInt, {b}));
      first = ints(f);
    }
    return PyLong_FromLong(call_gather(ko->data_ptr(), vo->data_ptr(), static_cast<pkv_dtype>(dt),
                                       static_cast<int32_t>(rows), p.k, p.v, p.type, p.ks, p.vs, ints(tab),
                                       static_cast<int32_t>(mb), first, ints(lens), ints(starts),
                                       static_cast<int32_t>(b), p.hkv, p.d, p.nb, p.bs, err, stream));
  } catch (...) {
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

// out, q, k_cache, v_cache, k_scale, v_scale, tables, lens, starts, scale, workspace, window, sinks, d_error, stream, type
PyObject *extend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  OR_PYTHON(n == 16 && call_extend);
  try {
    const at::Tensor *out = tensor(a[0]), *q = tensor(a[1]), *tab = tensor(a[6]), *lens = tensor(a[7]),
                     *starts = tensor(a[8]), *ws = tensor(a[10]);
    OR_PYTHON(q && q->is_cuda() && q->dim() == 3 && out);
    const int dev = q->get_device();
    OR_PYTHON(dev == c10::cuda::current_device());
    const auto type = q->scalar_type(), out_type = out->scalar_type();
    const int dt = pair_type(type);
    int32_t cdt, window, sinks, *err;
    pkv_stream_t stream;
    Pool p;
    OR_PYTHON(dt >= 0 && integer(a[15], &cdt) && pool_of(a + 2, cdt, dev, p) && error_word(a[13], dev, &err) &&
              stream_of(a[14], dev, &stream) && integer(a[11], &window) && integer(a[12], &sinks));
    const int64_t rows = q->size(0), hq = q->size(1);
    OR_PYTHON(q->size(2) == p.d && q->is_contiguous() && small(rows) && small(hq) &&
              (out_type == at::kFloat || out_type == type) && dense(out, dev, out_type, q->sizes()));
    OR_PYTHON(on(tab, dev) && tab->dim() == 2 && tab->scalar_type() == at::kInt && tab->is_contiguous());
    const int64_t b = tab->size(0), mb = tab->size(1);
    OR_PYTHON(small(b) && small(mb) && dense(lens, dev, at::kInt, {b}) && dense(starts, dev, at::kInt, {b + 1}) &&
              on(ws, dev) && ws->is_contiguous());
    const double scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    return PyLong_FromLong(call_extend(
        out->data_ptr(), out_type == at::kFloat ? PKV_F32 : static_cast<pkv_dtype>(dt), q->data_ptr(),
        static_cast<pkv_dtype>(dt), static_cast<int32_t>(rows), p.k, p.v, p.type, p.ks, p.vs, ints(tab),
        static_cast<int32_t>(mb), ints(lens), ints(starts), static_cast<int32_t>(b), static_cast<int32_t>(hq), p.hkv,
        p.d, p.nb, p.bs, static_cast<float>(scale), window, sinks, ws->data_ptr(), ws->nbytes(), err, stream));
  } catch (...) {
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

// The addresses of the library's calls: append_rope, gather, extend.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *f[3] = {};
  for (Py_ssize_t i = 0; i < n && i < 3; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  call_append_rope = reinterpret_cast<decltype(call_append_rope)>(f[0]);
  call_gather = reinterpret_cast<decltype(call_gather)>(f[1]);
  call_extend = reinterpret_cast<decltype(call_extend)>(f[2]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"append_rope", fast(append_rope), METH_FASTCALL, nullptr},
                         {"gather", fast(gather), METH_FASTCALL, nullptr},
                         {"extend", fast(extend), METH_FASTCALL, nullptr},
                         {"bind", fast(bind), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_prompt_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__prompt_calls() { return PyModule_Create(&module); }
