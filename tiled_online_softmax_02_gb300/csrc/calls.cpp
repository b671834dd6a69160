// calls.cpp -- the Python entry points of the 4-bit cache and of the rotary
// positions, marshalled natively: what a decode step calls once a layer, with
// kernels of two to ten microseconds, where sixteen more for reading tensors'
// shapes from Python would be most of the call.
//
// Each function looks over ordinary arguments (plain CUDA tensors of the right
// types and shapes on the current device), makes what outputs are not given, and
// calls the C ABI on torch's current stream.  It returns the entry point's result;
// an int, the C ABI's status, where that is not ATTN_OK; and None, having done
// nothing, where an argument is anything else.  The Python code then looks at the
// arguments one by one, and says what is wrong or makes the call itself.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/attn.h"

namespace {

decltype(&attn_cache_append_fp4) g_append;
decltype(&attn_cache_read_fp4) g_read;
decltype(&attn_fwd_paged_fp4) g_attend;
decltype(&attn_paged_fp4_workspace_bytes) g_workspace;
decltype(&attn_rope) g_rope;

constexpr int64_t kGroup = 16;  // values that share a scale

// A plain tensor, or nullptr (None among them: *none).
const at::Tensor* tensor(PyObject* o, bool* none = nullptr) {
  if (none) *none = o == Py_None;
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? ATTN_F32 : t == at::kHalf ? ATTN_F16 : t == at::kBFloat16 ? ATTN_BF16 : -1;
}

// Whether t is a contiguous tensor of this type and shape on CUDA device `index`.
bool is(const at::Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape, int index) {
  return t && t->is_cuda() && t->get_device() == index && t->scalar_type() == type &&
         t->sizes() == at::IntArrayRef(shape.begin(), shape.size()) && t->is_contiguous();
}

// Elements from one token of a [T, H, D] tensor to the next; false unless its heads are dense.
bool token_stride(const at::Tensor& t, int64_t* stride) {
  const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
  if ((t.stride(2) != 1 && D > 1) || (t.stride(1) != D && H > 1)) return false;
  *stride = T > 1 ? t.stride(0) : H * D;
  return true;
}

struct Cache {
  const at::Tensor *k, *v, *ks, *vs;
  const float *kh = nullptr, *vh = nullptr;
  int64_t blocks, Hkv, block_size, D;
};

// The six tensors of a 4-bit cache (o[0 .. 3] caches and scales, o[4], o[5] head scales or None) on device `index`.
bool cache(PyObject* const* o, PyObject* kh, PyObject* vh, int index, Cache* c) {
  c->k = tensor(o[0]); c->v = tensor(o[1]); c->ks = tensor(o[2]); c->vs = tensor(o[3]);
  if (!c->k || !c->ks || c->k->dim() != 4) return false;
  c->blocks = c->k->size(0); c->Hkv = c->k->size(1); c->block_size = c->k->size(2);
  const int64_t half = c->k->size(3), groups = half * 2 / kGroup;
  c->D = half * 2;
  const at::ScalarType st = c->ks->scalar_type();
  if (st != at::kFloat8_e4m3fn && st != at::kByte) return false;
  if (!is(c->k, at::kByte, {c->blocks, c->Hkv, c->block_size, half}, index) ||
      !is(c->v, at::kByte, {c->blocks, c->Hkv, c->block_size, half}, index) ||
      !is(c->ks, st, {c->blocks, c->Hkv, c->block_size, groups}, index) ||
      !is(c->vs, st, {c->blocks, c->Hkv, c->block_size, groups}, index))
    return false;
  bool none;
  const at::Tensor* t = tensor(kh, &none);
  if (!none && !is(t, at::kFloat, {c->Hkv}, index)) return false;
  c->kh = none ? nullptr : static_cast<const float*>(t->data_ptr());
  t = tensor(vh, &none);
  if (!none && !is(t, at::kFloat, {c->Hkv}, index)) return false;
  c->vh = none ? nullptr : static_cast<const float*>(t->data_ptr());
  return true;
}

// The current device's number if t lies on it, else -1.
int device_of(const at::Tensor* t) {
  if (!t || !t->is_cuda()) return -1;
  const int index = t->get_device();
  return index == c10::cuda::current_device() ? index : -1;
}

bool fits(std::initializer_list<int64_t> sizes) {  // the C ABI's ints
  for (int64_t n : sizes)
    if (n > INT32_MAX) return false;
  return true;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)index)));
}

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }

template <typename F>
int without_gil(F&& call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  return rc;
}

// append(k, v, slot_map, k_cache, v_cache, k_scales, v_scales, k_heads, v_heads) -> int status or None
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 9 || !g_append) Py_RETURN_NONE;
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *map = tensor(a[2]);
  const int index = device_of(k);
  Cache c;
  if (index < 0 || !v || k->dim() != 3 || !v->is_cuda() || v->get_device() != index || v->sizes() != k->sizes() ||
      v->scalar_type() != k->scalar_type() || !cache(a + 3, a[7], a[8], index, &c))
    Py_RETURN_NONE;
  const int code = dtype_code(k->scalar_type());
  const int64_t T = k->size(0), Hkv = k->size(1), D = k->size(2);
  int64_t ks, vs;
  if (code < 0 || Hkv != c.Hkv || D != c.D || !is(map, at::kLong, {T}, index) || !token_stride(*k, &ks) || !token_stride(*v, &vs) ||
      !fits({T, Hkv, D, c.blocks, c.block_size}))
    Py_RETURN_NONE;
  void* stream = stream_of(index);
  return PyLong_FromLong(without_gil([&] {
    return g_append(k->data_ptr(), v->data_ptr(), static_cast<const int64_t*>(map->data_ptr()), c.k->data_ptr(), c.v->data_ptr(),
                    c.ks->data_ptr(), c.vs->data_ptr(), c.kh, c.vh, (int)T, (int)Hkv, (int)D, ks, vs, (int)c.blocks,
                    (int)c.block_size, code, stream);
  }));
} catch (...) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// read(k_cache, v_cache, k_scales, v_scales, slot_map, dtype, k_heads, v_heads) -> (k, v), int status or None
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 8 || !g_read || !THPDtype_Check(a[5])) Py_RETURN_NONE;
  const at::Tensor* map = tensor(a[4]);
  const int index = device_of(map);
  const at::ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
  const int code = dtype_code(type);
  Cache c;
  if (index < 0 || code < 0 || map->dim() != 1 || !cache(a, a[6], a[7], index, &c)) Py_RETURN_NONE;
  const int64_t T = map->size(0);
  if (!is(map, at::kLong, {T}, index) || !fits({T, c.Hkv, c.D, c.blocks, c.block_size})) Py_RETURN_NONE;
  const at::Tensor k = make({T, c.Hkv, c.D}, type, index), v = make({T, c.Hkv, c.D}, type, index);
  void* stream = stream_of(index);
  const int64_t ts = c.Hkv * c.D;
  const int rc = without_gil([&] {
    return g_read(c.k->data_ptr(), c.v->data_ptr(), c.ks->data_ptr(), c.vs->data_ptr(), c.kh, c.vh,
                  static_cast<const int64_t*>(map->data_ptr()), k.data_ptr(), v.data_ptr(), (int)T, (int)c.Hkv, (int)c.D, ts, c.D,
                  ts, c.D, (int)c.blocks, (int)c.block_size, code, stream);
  });
  if (rc != ATTN_OK) return PyLong_FromLong(rc);
  return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
} catch (...) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// attend(q, k_cache, v_cache, k_scales, v_scales, tables, q_starts, totals, k_heads, v_heads, causal, window, scale, softcap,
//        out) -> out, int status or None.  The workspace comes from torch's allocator.
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 15 || !g_attend || !PyLong_Check(a[11])) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[0]), *tables = tensor(a[5]), *starts = tensor(a[6]), *totals = tensor(a[7]);
  const int index = device_of(q);
  Cache c;
  if (index < 0 || !tables || q->dim() != 3 || tables->dim() != 2 || !cache(a + 1, a[8], a[9], index, &c)) Py_RETURN_NONE;
  const at::ScalarType type = q->scalar_type();
  const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), B = tables->size(0), width = tables->size(1);
  int64_t stride;
  if ((type != at::kHalf && type != at::kBFloat16) || D != c.D || !is(tables, at::kInt, {B, width}, index) ||
      !is(starts, at::kInt, {B + 1}, index) || !is(totals, at::kInt, {B}, index) || !token_stride(*q, &stride) ||
      !fits({T, Hq, D, B, width, c.blocks, c.Hkv, c.block_size}))
    Py_RETURN_NONE;
  bool none;
  const at::Tensor* given = tensor(a[14], &none);
  if (!none && !is(given, type, {T, Hq, D}, index)) Py_RETURN_NONE;
  const int causal = PyObject_IsTrue(a[10]);
  const long window = PyLong_AsLong(a[11]);
  const double scale = a[12] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AsDouble(a[12]), softcap = PyFloat_AsDouble(a[13]);
  if (PyErr_Occurred() || causal < 0 || window > INT32_MAX || window < INT32_MIN) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const at::Tensor out = none ? make({T, Hq, D}, type, index) : *given;
  const size_t need = g_workspace((int)T, (int)B, (int)Hq, (int)c.Hkv, (int)D);
  const at::Tensor ws = make({(int64_t)need}, at::kByte, index);
  void* stream = stream_of(index);
  const int rc = without_gil([&] {
    return g_attend(q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), c.ks->data_ptr(), c.vs->data_ptr(), c.kh, c.vh,
                    static_cast<const int32_t*>(tables->data_ptr()), static_cast<const int32_t*>(starts->data_ptr()),
                    static_cast<const int32_t*>(totals->data_ptr()), out.data_ptr(), nullptr, (int)T, (int)B, (int)Hq, (int)c.Hkv,
                    (int)D, stride, (int)c.blocks, (int)c.block_size, (int)width, causal, (int)window, (float)scale,
                    (float)softcap, type == at::kHalf ? ATTN_F16 : ATTN_BF16, ws.data_ptr(), need, stream);
  });
  if (rc != ATTN_OK) return PyLong_FromLong(rc);
  if (!none) {
    Py_INCREF(a[14]);
    return a[14];
  }
  return THPVariable_Wrap(out);
} catch (...) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// rope(q, k, inv_freq, positions, q_starts, totals, interleaved, inverse, scale, q_out, k_out) -> (q_out, k_out), int status or
// None
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 11 || !g_rope) Py_RETURN_NONE;
  bool no_k, no_pos, no_starts, no_totals, no_out[2];
  const at::Tensor *x[2] = {tensor(a[0]), tensor(a[1], &no_k)}, *freq = tensor(a[2]), *pos = tensor(a[3], &no_pos);
  const at::Tensor *starts = tensor(a[4], &no_starts), *totals = tensor(a[5], &no_totals);
  const at::Tensor* given[2] = {tensor(a[9], &no_out[0]), tensor(a[10], &no_out[1])};
  const int index = device_of(x[0]);
  if (index < 0 || x[0]->dim() != 3 || !freq || freq->dim() != 1) Py_RETURN_NONE;
  const at::ScalarType type = x[0]->scalar_type();
  const int code = dtype_code(type);
  const int64_t T = x[0]->size(0), D = x[0]->size(2), pairs = freq->size(0);
  int64_t B = 0;
  if (code < 0 || !is(freq, at::kDouble, {pairs}, index)) Py_RETURN_NONE;
  if (!no_pos) {
    if (!no_starts || !no_totals || !is(pos, at::kInt, {T}, index)) Py_RETURN_NONE;
  } else {
    if (!totals || totals->dim() != 1) Py_RETURN_NONE;
    B = totals->size(0);
    if (!is(totals, at::kInt, {B}, index) || !is(starts, at::kInt, {B + 1}, index)) Py_RETURN_NONE;
  }
  if (no_k && !no_out[1]) Py_RETURN_NONE;
  int64_t H[2] = {0, 0}, in[2] = {0, 0}, to[2] = {0, 0};
  at::Tensor out[2];
  for (int i = 0; i < (no_k ? 1 : 2); ++i) {
    if (!x[i] || !x[i]->is_cuda() || x[i]->get_device() != index || x[i]->dim() != 3 || x[i]->size(0) != T || x[i]->size(2) != D ||
        x[i]->scalar_type() != type || !token_stride(*x[i], &in[i]))
      Py_RETURN_NONE;
    if (c10::GradMode::is_enabled() && x[i]->requires_grad()) Py_RETURN_NONE;  // recorded by the Python code
    H[i] = x[i]->size(1);
    if (!no_out[i] && (!given[i] || !given[i]->is_cuda() || given[i]->get_device() != index || given[i]->sizes() != x[i]->sizes() ||
                       given[i]->scalar_type() != type || !token_stride(*given[i], &to[i])))
      Py_RETURN_NONE;
  }
  const int inter = PyObject_IsTrue(a[6]), inverse = PyObject_IsTrue(a[7]);
  const double scale = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred() || inter < 0 || inverse < 0 || !fits({T, B, H[0], H[1], D, 2 * pairs})) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  for (int i = 0; i < (no_k ? 1 : 2); ++i) {
    if (no_out[i]) {
      out[i] = make(x[i]->sizes(), type, index);
      to[i] = H[i] * D;
    } else {
      out[i] = *given[i];
    }
  }
  void* stream = stream_of(index);
  const int rc = without_gil([&] {
    return g_rope(x[0]->data_ptr(), no_k ? nullptr : x[1]->data_ptr(), out[0].data_ptr(), no_k ? nullptr : out[1].data_ptr(),
                  static_cast<const double*>(freq->data_ptr()), no_pos ? nullptr : static_cast<const int32_t*>(pos->data_ptr()),
                  no_pos ? static_cast<const int32_t*>(starts->data_ptr()) : nullptr,
                  no_pos ? static_cast<const int32_t*>(totals->data_ptr()) : nullptr, (int)T, (int)B, (int)H[0], (int)H[1], (int)D,
                  (int)(2 * pairs), in[0], in[1], to[0], to[1], inter, inverse, (float)scale, code, stream);
  });
  if (rc != ATTN_OK) return PyLong_FromLong(rc);
  PyObject* made[2];
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && no_k) {
      Py_INCREF(Py_None);
      made[i] = Py_None;
    } else if (!no_out[i]) {
      Py_INCREF(a[9 + i]);
      made[i] = a[9 + i];
    } else {
      made[i] = THPVariable_Wrap(out[i]);
    }
  }
  return Py_BuildValue("NN", made[0], made[1]);
} catch (...) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// bind(append, read, attend, workspace, rope): the addresses of the C ABI's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[5];
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind takes five addresses");
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_append = reinterpret_cast<decltype(g_append)>(p[0]);
  g_read = reinterpret_cast<decltype(g_read)>(p[1]);
  g_attend = reinterpret_cast<decltype(g_attend)>(p[2]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[3]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[4]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(bind), ""}, {"append", FAST(append), ""}, {"read", FAST(read), ""},
                         {"attend", FAST(attend), ""}, {"rope", FAST(rope), ""}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
