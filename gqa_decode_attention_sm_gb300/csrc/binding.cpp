// Native binding of the cache write and read-back calls, and of gqa_decode_fp4kv,
// gqa_decode_verify and gqa_decode_paged (caches of every format) and a prepared
// 4-bit launch with everything given (output, split count, workspace): the argument
// checks and the call of the C ABI without the interpreter between them (writing 256
// tokens costs the host 4 us a call so, 16 us through ctypes).
//
// Each function checks exactly what api.py checks.  Arguments in any other form
// than the plain one (wrong types, shapes or devices, tensor subclasses, another
// current device) are not judged here: the function returns None, and api.py
// takes its own path, which says what is wrong.  Else it returns the output
// tensor, or the C call's status if that is not GQA_OK.  No C++ exception leaves
// a function.
#include <Python.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gqa_decode.h"

namespace {

constexpr int64_t kHq = GQA_NUM_Q_HEADS, kHkv = GQA_NUM_KV_HEADS, kD = GQA_HEAD_DIM;

const at::Tensor* plain(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == at::kStrided && t.is_cuda() ? &t : nullptr;
}

// A dense tensor on `dev` of one type and these sizes (none: any sizes).
const at::Tensor* dense(PyObject* o, c10::Device dev, at::ScalarType type, at::IntArrayRef sizes = {}) {
  const at::Tensor* t = plain(o);
  return t && t->device() == dev && t->scalar_type() == type && (sizes.empty() || t->sizes() == sizes) &&
                 t->is_contiguous()
             ? t
             : nullptr;
}

bool half_type(at::ScalarType t, int* code) {
  *code = t == at::kBFloat16 ? GQA_BF16 : GQA_F16;
  return t == at::kBFloat16 || t == at::kHalf;
}

// A cache (or page pool) and its scales.
struct Cache {
  void* kv = nullptr;
  const void* scales = nullptr;
  int format = -1;
  int64_t units = 0, rows = 0;
  c10::Device dev = c10::Device(c10::kCPU);
};

bool cache_of(PyObject* kv, PyObject* scales, Cache& c) {
  const at::Tensor* t = plain(kv);
  if (!t || t->dim() != 5 || t->size(1) != 2 || t->size(2) != kHkv || !t->is_contiguous()) return false;
  c.dev = t->device();
  c.units = t->size(0);
  c.rows = t->size(3);
  const at::ScalarType s = t->scalar_type();
  if (t->size(4) == kD) {
    c.format = s == at::kHalf ? GQA_KV_F16
               : s == at::kBFloat16 ? GQA_KV_BF16
               : s == at::kByte || s == at::kFloat8_e4m3fn ? GQA_KV_E4M3
               : s == at::kChar ? GQA_KV_I8
                                : -1;
  } else if (t->size(4) == kD / 2 && s == at::kByte) {
    c.format = GQA_KV_E2M1;
  }
  if (c.format < 0) return false;
  c.kv = t->data_ptr();
  const at::Tensor* sc = nullptr;
  if (c.format == GQA_KV_I8) {
    if (!(sc = dense(scales, c.dev, at::kBFloat16, {c.units, 2, kHkv, c.rows}))) return false;
  } else if (c.format == GQA_KV_E2M1) {
    sc = dense(scales, c.dev, at::kByte, {c.units, 2, kHkv, c.rows, 8});
    if (!sc) sc = dense(scales, c.dev, at::kFloat8_e4m3fn, {c.units, 2, kHkv, c.rows, 8});
    if (!sc) return false;
  }
  if (sc) c.scales = sc->data_ptr();
  return true;
}

// A projection [n, heads, 128] whose tokens may lie apart; its stride, or 0.
int64_t token_stride(PyObject* o, c10::Device dev, at::ScalarType type, int64_t n, int64_t heads, const void** ptr) {
  const at::Tensor* t = plain(o);
  if (!t || t->device() != dev || t->scalar_type() != type || t->dim() != 3 || t->size(0) != n || t->size(1) != heads ||
      t->size(2) != kD)
    return 0;
  *ptr = t->data_ptr();
  if (t->is_contiguous()) return heads * kD;
  return t->stride(2) == 1 && t->stride(1) == kD ? t->stride(0) : 0;
}

bool as_float(PyObject* o, float* x) {
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *x = (float)d;
  return true;
}

// An optional workspace; false if it is not one.
bool workspace_of(PyObject* o, c10::Device dev, void** ptr, size_t* bytes) {
  *ptr = nullptr;
  *bytes = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = dense(o, dev, at::kByte);
  if (!t) return false;
  *ptr = t->data_ptr();
  *bytes = (size_t)t->numel();
  return true;
}

bool fits(int64_t x) { return x >= 0 && x <= INT32_MAX; }

// write(address, paged, q_proj, k_proj, v_proj, q_norm_w, k_norm_w, positions, rows,
//       slots, kv, block_table, q_out, mrope_section, mrope_interleaved, eps,
//       rope_theta, k_scale, v_scale, kv_scales, workspace)
PyObject* write(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 21) return nullptr;
  void* fn = PyLong_AsVoidPtr(a[0]);
  const bool paged = a[1] == Py_True;
  const at::Tensor* q = plain(a[2]);
  int dtype;
  if (!fn || !q || q->dim() != 3 || !half_type(q->scalar_type(), &dtype)) return nullptr;
  const int64_t n = q->size(0);
  const c10::Device dev = q->device();
  const at::ScalarType type = q->scalar_type();
  if (n < 1 || !fits(n) || c10::cuda::current_device() != dev.index()) return nullptr;
  const void *qp, *kp, *vp;
  const int64_t qs = token_stride(a[2], dev, type, n, kHq, &qp), ks = token_stride(a[3], dev, type, n, kHkv, &kp),
                vs = token_stride(a[4], dev, type, n, kHkv, &vp);
  if (!qs || !ks || !vs) return nullptr;
  const void *qw = nullptr, *kw = nullptr;
  if (a[5] != Py_None || a[6] != Py_None) {
    const at::Tensor *wq = dense(a[5], dev, type, {kD}), *wk = dense(a[6], dev, type, {kD});
    if (!wq || !wk) return nullptr;
    qw = wq->data_ptr();
    kw = wk->data_ptr();
  }
  int section[3];
  const bool axes = a[13] != Py_None;
  if (axes) {
    if (!PyTuple_Check(a[13]) || PyTuple_GET_SIZE(a[13]) != 3) return nullptr;
    for (int i = 0; i < 3; ++i) {
      const long x = PyLong_Check(PyTuple_GET_ITEM(a[13], i)) ? PyLong_AsLong(PyTuple_GET_ITEM(a[13], i)) : -1;
      if (x < 0 || x > 64) {
        PyErr_Clear();
        return nullptr;
      }
      section[i] = (int)x;
    }
  }
  const at::Tensor* pos = axes ? dense(a[7], dev, at::kInt, {3, n}) : dense(a[7], dev, at::kInt, {n});
  const at::Tensor *rows = dense(a[8], dev, at::kInt, {n}), *slots = dense(a[9], dev, at::kInt, {n});
  Cache c;
  if (!pos || !rows || !slots || !cache_of(a[10], a[19], c) || c.dev != dev || !fits(c.units) || !fits(c.rows))
    return nullptr;
  const at::Tensor* table = nullptr;
  if (paged && (!(table = dense(a[11], dev, at::kInt)) || table->dim() != 2 || !fits(table->size(0)) ||
                !fits(table->size(1))))
    return nullptr;
  at::Tensor made;
  const at::Tensor* out = nullptr;
  if (a[12] == Py_None) {
    made = at::empty({n, kHq, kD}, q->options());
    out = &made;
  } else {
    out = dense(a[12], dev, type, {n, kHq, kD});
  }
  float eps, theta, k_scale, v_scale;
  void* ws;
  size_t ws_bytes;
  const int interleaved = PyObject_IsTrue(a[14]);
  if (!out || interleaved < 0 || !as_float(a[15], &eps) || !as_float(a[16], &theta) || !as_float(a[17], &k_scale) ||
      !as_float(a[18], &v_scale) || !workspace_of(a[20], dev, &ws, &ws_bytes))
    return nullptr;
  void* const q_out = out->data_ptr();
  void* const stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  const auto i32 = [](const at::Tensor* t) { return static_cast<const int32_t*>(t->data_ptr()); };
  const auto dt = static_cast<gqa_dtype_t>(dtype);
  const auto fmt = static_cast<gqa_kv_format_t>(c.format);
  gqa_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  if (paged)
    st = reinterpret_cast<decltype(&gqa_write_kv_paged)>(fn)(
        qp, kp, vp, qs, ks, vs, qw, kw, dt, i32(pos), axes ? section : nullptr, interleaved, i32(rows), i32(slots), (int)n,
        q_out, c.kv, fmt, const_cast<void*>(c.scales), i32(table), (int)table->size(0), (int)table->size(1), (int)c.units,
        (int)c.rows, eps, theta, k_scale, v_scale, ws, ws_bytes, stream);
  else
    st = reinterpret_cast<decltype(&gqa_write_kv)>(fn)(
        qp, kp, vp, qs, ks, vs, qw, kw, dt, i32(pos), axes ? section : nullptr, interleaved, i32(rows), i32(slots), (int)n,
        q_out, c.kv, fmt, const_cast<void*>(c.scales), (int)c.units, (int)c.rows, eps, theta, k_scale, v_scale, ws,
        ws_bytes, stream);
  Py_END_ALLOW_THREADS;
  if (st != GQA_OK) return PyLong_FromLong(st);
  return a[12] == Py_None ? THPVariable_Wrap(made) : Py_NewRef(a[12]);
}

// read(address, paged, kv, block_table, sequence_lengths, starts, out, dtype, k_scale,
//      v_scale, kv_scales, workspace)
PyObject* read(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 12 || a[6] == Py_None || a[7] != Py_None) return nullptr;  // (an output given)
  void* fn = PyLong_AsVoidPtr(a[0]);
  const bool paged = a[1] == Py_True;
  Cache c;
  if (!fn || !cache_of(a[2], a[10], c) || !fits(c.units) || !fits(c.rows) ||
      c10::cuda::current_device() != c.dev.index())
    return nullptr;
  const at::Tensor* table = nullptr;
  if (paged && (!(table = dense(a[3], c.dev, at::kInt)) || table->dim() != 2 || !fits(table->size(0)) ||
                !fits(table->size(1))))
    return nullptr;
  const int64_t batch = paged ? table->size(0) : c.units;
  const at::Tensor* lens = dense(a[4], c.dev, at::kInt, {batch});
  const at::Tensor* starts = a[5] == Py_None ? nullptr : dense(a[5], c.dev, at::kInt, {batch});
  const at::Tensor* out = plain(a[6]);
  int dtype;
  if (!lens || (a[5] != Py_None && !starts) || !out || out->device() != c.dev ||
      !half_type(out->scalar_type(), &dtype) || out->dim() != 5 || out->size(0) != batch || out->size(1) != 2 ||
      out->size(2) != kHkv || out->size(4) != kD || !fits(out->size(3)) || !out->is_contiguous())
    return nullptr;
  float k_scale, v_scale;
  void* ws;
  size_t ws_bytes;
  if (!as_float(a[8], &k_scale) || !as_float(a[9], &v_scale) || !workspace_of(a[11], c.dev, &ws, &ws_bytes))
    return nullptr;
  void* const stream = c10::cuda::getCurrentCUDAStream(c.dev.index()).stream();
  const auto i32 = [](const at::Tensor* t) { return t ? static_cast<const int32_t*>(t->data_ptr()) : nullptr; };
  const auto dt = static_cast<gqa_dtype_t>(dtype);
  const auto fmt = static_cast<gqa_kv_format_t>(c.format);
  void* const to = out->data_ptr();
  const int cap = (int)out->size(3);
  gqa_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  if (paged)
    st = reinterpret_cast<decltype(&gqa_read_kv_paged)>(fn)(c.kv, fmt, c.scales, i32(table), (int)table->size(1),
                                                            (int)c.units, (int)c.rows, i32(lens), i32(starts), to, dt,
                                                            (int)batch, cap, k_scale, v_scale, ws, ws_bytes, stream);
  else
    st = reinterpret_cast<decltype(&gqa_read_kv)>(fn)(c.kv, fmt, c.scales, i32(lens), i32(starts), to, dt, (int)batch,
                                                      (int)c.rows, cap, k_scale, v_scale, ws, ws_bytes, stream);
  Py_END_ALLOW_THREADS;
  return st == GQA_OK ? Py_NewRef(a[6]) : PyLong_FromLong(st);
}

// attend(address, kind, q, kv, block_table, sequence_lengths, out, kv_scales,
//        workspace, num_splits, q_scale, k_scale, v_scale)
// kind: 0 gqa_decode_fp4kv, 1 gqa_decode_verify, 2 gqa_decode_paged
PyObject* attend(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 13 || a[6] == Py_None || a[8] == Py_None || !PyLong_Check(a[9])) return nullptr;
  void* fn = PyLong_AsVoidPtr(a[0]);
  const long kind = PyLong_AsLong(a[1]), splits = PyLong_AsLong(a[9]);
  const at::Tensor* q = plain(a[2]);
  int dtype;
  if (!fn || !q || !half_type(q->scalar_type(), &dtype) || !q->is_contiguous() || splits < 1 ||
      splits > GQA_MAX_SPLITS)
    return nullptr;
  const c10::Device dev = q->device();
  const bool window = q->dim() == 4;
  if ((!window && (q->dim() != 3 || kind == 1)) || (window && kind == 0) || q->size(-2) != kHq || q->size(-1) != kD)
    return nullptr;
  const int64_t batch = q->size(0), q_len = window ? q->size(1) : 1;
  Cache c;
  if (!fits(batch) || q_len < 1 || q_len > 4 || !cache_of(a[3], a[7], c) || c.dev != dev || !fits(c.units) ||
      !fits(c.rows) || c10::cuda::current_device() != dev.index())
    return nullptr;
  const at::Tensor* table = nullptr;
  if (kind == 2) {
    if (!(table = dense(a[4], dev, at::kInt)) || table->dim() != 2 || table->size(0) != batch || !fits(table->size(1)))
      return nullptr;
  } else if (c.units != batch || (kind == 0 && c.format != GQA_KV_E2M1)) {
    return nullptr;
  }
  const at::Tensor *lens = dense(a[5], dev, at::kInt, {batch}), *out = dense(a[6], dev, q->scalar_type(), q->sizes());
  float q_scale, k_scale, v_scale;
  void* ws;
  size_t ws_bytes;
  if (!lens || !out || !as_float(a[10], &q_scale) || !as_float(a[11], &k_scale) || !as_float(a[12], &v_scale) ||
      !workspace_of(a[8], dev, &ws, &ws_bytes))
    return nullptr;
  void* const stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  const auto i32 = [](const at::Tensor* t) { return static_cast<const int32_t*>(t->data_ptr()); };
  const auto dt = static_cast<gqa_dtype_t>(dtype);
  const auto fmt = static_cast<gqa_kv_format_t>(c.format);
  const void* const qp = q->data_ptr();
  void* const to = out->data_ptr();
  gqa_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  if (kind == 0)
    st = reinterpret_cast<decltype(&gqa_decode_fp4kv)>(fn)(
        qp, static_cast<const uint8_t*>(c.kv), static_cast<const uint8_t*>(c.scales), i32(lens), to, (int)batch,
        (int)c.rows, dt, q_scale, k_scale, v_scale, (int)splits, ws, ws_bytes, stream);
  else if (kind == 1)
    st = reinterpret_cast<decltype(&gqa_decode_verify)>(fn)(qp, dt, c.kv, fmt, c.scales, i32(lens), to, (int)batch,
                                                            (int)c.rows, (int)q_len, q_scale, k_scale, v_scale,
                                                            (int)splits, ws, ws_bytes, stream);
  else
    st = reinterpret_cast<decltype(&gqa_decode_paged)>(fn)(
        qp, dt, c.kv, fmt, c.scales, i32(table), (int)table->size(1), (int)c.units, (int)c.rows, i32(lens), to, (int)batch,
        (int)q_len, q_scale, k_scale, v_scale, (int)splits, ws, ws_bytes, stream);
  Py_END_ALLOW_THREADS;
  return st == GQA_OK ? Py_NewRef(a[6]) : PyLong_FromLong(st);
}

// Runs f; None where it does not judge its arguments or something threw.
template <PyObject* (*f)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  PyObject* r = nullptr;
  try {
    r = f(a, n);
  } catch (...) {
  }
  if (r) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<attend>)), METH_FASTCALL, nullptr},
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<write>)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<read>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) {
  PyObject* m = PyModule_Create(&kModule);
  // the torch and the C interface it was compiled against: api.py takes it only
  // with the same ones (and the build looks for built_for in the file)
  if (m && (PyModule_AddStringConstant(m, "torch_version", GQA_TORCH_VERSION) < 0 ||
            PyModule_AddStringConstant(m, "interface", GQA_INTERFACE) < 0 ||
            PyModule_AddStringConstant(m, "built_for", GQA_BUILT_FOR) < 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
