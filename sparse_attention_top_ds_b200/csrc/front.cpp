// front.cpp -- the usual call of the 8-bit cache's front end, marshalled natively.
//
// A decode step calls these operators once per layer, and the smallest of them run
// for 2 to 7 us: reading shapes, types and addresses of ten tensors through Python
// takes longer than that.  Each function here takes the arguments of the Python
// function of the same name, checks them and calls the library, if the call is the
// usual one: plain contiguous CUDA tensors on the current device, on its current
// stream, with the documented shapes and types.  For anything else, a refusal by the
// library included, it returns None without having enqueued anything, and the Python
// function marshals the call (or says what is wrong with it) by itself.  Nothing is
// computed or kept here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <cmath>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ds_topk.h"

namespace {

using at::Tensor;

struct {
  decltype(&ds_cache_quantize) quantize;
  decltype(&ds_sparse_attention_q8) attention;
  decltype(&ds_attention_mass) mass;
  decltype(&ds_cache_evict) evict;
  decltype(&ds_cache_compact) compact;
} g_lib;

constexpr at::ScalarType kI32 = at::kInt, kF32 = at::kFloat, kBf16 = at::kBFloat16;

// The tensor of an argument, or null if it is none (or of a class of its own).
const Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous tensor of this type and shape on device dev?
bool is(const Tensor* t, at::ScalarType type, int dev, at::IntArrayRef shape) {
  return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->sizes() == shape && t->is_contiguous();
}

// The same for an argument that may be None; *p: its address, or null.
template <class T>
bool opt(PyObject* o, at::ScalarType type, int dev, at::IntArrayRef shape, T** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const Tensor* t = tensor(o);
  if (!is(t, type, dev, shape)) return false;
  *p = static_cast<T*>(t->data_ptr());
  return true;
}

template <class T>
T* data(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// The device that the call runs on, if that is the current one; -1 otherwise.
int device_of(const Tensor* t, int64_t dims) {
  if (!t || !t->is_cuda() || t->dim() != dims || t->numel() == 0) return -1;
  const int dev = t->get_device();
  return c10::cuda::current_device() == dev ? dev : -1;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

bool whole(PyObject* o, int* v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &over);
  *v = (int)x;
  return over == 0 && x >= 0 && x <= INT32_MAX;
}

bool number(PyObject* o, double fallback, float* v) {
  if (o == Py_None) {
    *v = (float)fallback;
    return true;
  }
  if (!PyFloat_CheckExact(o)) return false;
  *v = (float)PyFloat_AS_DOUBLE(o);
  return true;
}

bool small(at::IntArrayRef shape) {
  for (const int64_t n : shape)
    if (n > INT32_MAX) return false;
  return true;
}

// An 8-bit cache: codes [batch, T, heads, d] or [T, heads, d] with their scales.
struct Cache8 {
  int dtype, T, heads, d;
  int64_t codes_step, scales_step;
};
bool cache8(const Tensor* codes, const Tensor* scales, int block, int64_t batch, int dev, Cache8* c) {
  if (!codes || block < 1) return false;
  const auto type = codes->scalar_type();
  if (type != at::kFloat8_e4m3fn && type != at::kChar) return false;
  const int64_t lead = codes->dim() == 4 ? 1 : 0;
  if (codes->dim() != 3 + lead || (lead && codes->size(0) != batch) || !small(codes->sizes())) return false;
  const int64_t T = codes->size(lead), nb = (T + block - 1) / block, heads = codes->size(lead + 1);
  if (!is(codes, type, dev, codes->sizes())) return false;
  if (!(lead ? is(scales, kF32, dev, {batch, nb, heads}) : is(scales, kF32, dev, {nb, heads}))) return false;
  *c = {type == at::kChar ? DS_I8 : DS_E4M3, (int)T, (int)heads, (int)codes->size(lead + 2), lead ? T : 0, lead ? nb : 0};
  return true;
}

PyObject* none() { Py_RETURN_NONE; }

// (rows, codes, scales, block, pos, length)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const Tensor *rows = n == 6 ? tensor(a[0]) : nullptr, *codes, *scales;
  const int dev = device_of(rows, 4);
  int block;
  int32_t *pos, *length;
  Cache8 c;
  if (dev < 0 || !whole(a[3], &block)) return none();
  codes = tensor(a[1]), scales = tensor(a[2]);
  const auto s = rows->sizes();
  if (!small(s) || !cache8(codes, scales, block, s[0], dev, &c) || codes->dim() != 4 || c.heads != s[2] || c.d != s[3] ||
      !is(rows, kBf16, dev, s) || !opt(a[4], kI32, dev, {s[0]}, &pos) || !opt(a[5], kI32, dev, {s[0]}, &length))
    return none();
  const int64_t width = s[2] * s[3];
  if (g_lib.quantize(rows->data_ptr(), s[1] * width, width, (int)s[0], (int)s[1], c.heads, c.d, c.dtype, block, pos, length,
                     codes->data_ptr(), c.codes_step, data<float>(*scales), c.scales_step, c.T, stream_of(dev)) != DS_OK)
    return none();
  return PyTuple_Pack(2, a[1], a[2]);
}

// (q, codes, scales, idx, block, scale, win, win_len, sink, return_lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const Tensor* q = n == 10 ? tensor(a[0]) : nullptr;
  const int dev = device_of(q, 3);
  int block, k = 0, W = 0;
  float scale, *sink;
  int32_t *idx = nullptr, *win_len;
  void* win = nullptr;
  Cache8 c;
  if (dev < 0 || !whole(a[4], &block)) return none();
  const auto s = q->sizes();
  const Tensor *codes = tensor(a[1]), *scales = tensor(a[2]);
  if (!small(s) || !is(q, kBf16, dev, s) || !cache8(codes, scales, block, s[0], dev, &c) || c.d != s[2] ||
      !number(a[5], 1.0 / std::sqrt((double)s[2]), &scale) || !opt(a[7], kI32, dev, {s[0]}, &win_len) ||
      !opt(a[8], kF32, dev, {s[1]}, &sink))
    return none();
  if (a[3] != Py_None) {
    const Tensor* t = tensor(a[3]);
    if (!t || t->dim() != 2 || !small(t->sizes()) || !is(t, kI32, dev, {s[0], t->size(1)}) || t->size(1) == 0) return none();
    k = (int)t->size(1), idx = data<int32_t>(*t);
  }
  if (a[6] != Py_None) {
    const Tensor* t = tensor(a[6]);
    if (!t || t->dim() != 4 || !small(t->sizes()) || !is(t, kBf16, dev, {s[0], t->size(1), c.heads, s[2]}) || t->size(1) == 0)
      return none();
    W = (int)t->size(1), win = t->data_ptr();
  }
  const bool want_lse = a[9] == Py_True;
  Tensor out = at::empty(s, q->options()), lse;
  if (want_lse) lse = at::empty({s[0], s[1]}, q->options().dtype(kF32));
  if (g_lib.attention(q->data_ptr(), codes->data_ptr(), c.codes_step, data<float>(*scales), c.scales_step, c.dtype, block, c.T,
                      idx, k, win, W, win_len, sink, (int)s[0], (int)s[1], c.heads, c.d, scale, out.data_ptr(),
                      want_lse ? data<float>(lse) : nullptr, stream_of(dev)) != DS_OK)
    return none();
  PyObject* o = THPVariable_Wrap(std::move(out));
  if (!want_lse || !o) return o;
  PyObject* l = THPVariable_Wrap(std::move(lse));
  if (!l) {
    Py_DECREF(o);
    return nullptr;
  }
  PyObject* r = PyTuple_New(2);
  if (!r) {
    Py_DECREF(o);
    Py_DECREF(l);
    return nullptr;
  }
  PyTuple_SET_ITEM(r, 0, o);
  PyTuple_SET_ITEM(r, 1, l);
  return r;
}

// (q, cache, idx, lse, mass, scales, block, scale)
PyObject* mass(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const Tensor* q = n == 8 ? tensor(a[0]) : nullptr;
  const int dev = device_of(q, 3);
  int block;
  float scale;
  Cache8 c;
  if (dev < 0 || !whole(a[6], &block)) return none();
  const auto s = q->sizes();
  const Tensor *cache = tensor(a[1]), *idx = tensor(a[2]), *lse = tensor(a[3]), *acc = tensor(a[4]), *scales = nullptr;
  if (!small(s) || !is(q, kBf16, dev, s) || !cache) return none();
  if (a[5] != Py_None) {
    scales = tensor(a[5]);
    if (!cache8(cache, scales, block, s[0], dev, &c)) return none();
  } else {
    const int64_t dims = cache->dim();
    if (dims < 2 || dims > 4 || (dims > 2 && cache->size(0) != s[0]) || !small(cache->sizes()) ||
        !is(cache, kBf16, dev, cache->sizes()))
      return none();
    const int64_t T = cache->size(dims == 2 ? 0 : 1);
    c = {DS_BF16, (int)T, dims == 4 ? (int)cache->size(2) : 1, (int)cache->size(dims - 1), dims == 2 ? 0 : T, 0};
    block = 1;
  }
  if (c.d != s[2] || !idx || idx->dim() != 2 || !small(idx->sizes()) || idx->size(1) == 0 || !is(idx, kI32, dev, {s[0], idx->size(1)}) ||
      !is(lse, kF32, dev, {s[0], s[1]}) || !is(acc, kF32, dev, {s[0], c.T}) ||
      !number(a[7], 1.0 / std::sqrt((double)s[2]), &scale))
    return none();
  if (g_lib.mass(q->data_ptr(), cache->data_ptr(), c.codes_step, scales ? data<float>(*scales) : nullptr, c.scales_step, c.dtype,
                 block, c.T, data<int32_t>(*idx), (int)idx->size(1), data<float>(*lse), (int)s[0], (int)s[1], c.heads, c.d,
                 scale, data<float>(*acc), c.T, stream_of(dev)) != DS_OK)
    return none();
  Py_INCREF(a[4]);
  return a[4];
}

// (mass, budget, block, length, keep_first, keep_last)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const Tensor* acc = n == 6 ? tensor(a[0]) : nullptr;
  const int dev = device_of(acc, 2);
  int budget, block, first, last;
  int32_t* length;
  if (dev < 0 || !whole(a[1], &budget) || !whole(a[2], &block) || !whole(a[4], &first) || !whole(a[5], &last)) return none();
  const auto s = acc->sizes();
  // (a budget that no cache has is refused before its list is allocated)
  if (!small(s) || !is(acc, kF32, dev, s) || !opt(a[3], kI32, dev, {s[0]}, &length) || budget > s[1]) return none();
  Tensor kept = at::empty({s[0], budget}, acc->options().dtype(kI32)), len = at::empty({s[0]}, acc->options().dtype(kI32));
  if (g_lib.evict(data<float>(*acc), s[1], (int)s[0], (int)s[1], length, block, budget, first, last, data<int32_t>(kept),
                  data<int32_t>(len), stream_of(dev)) != DS_OK)
    return none();
  PyObject* o = THPVariable_Wrap(std::move(kept));
  PyObject* l = o ? THPVariable_Wrap(std::move(len)) : nullptr;
  PyObject* r = l ? PyTuple_Pack(2, o, l) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(l);
  return r;
}

// (kept, block, length, rows, blocks): True if done
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const Tensor* kept = n == 5 ? tensor(a[0]) : nullptr;
  const int dev = device_of(kept, 2);
  int block;
  int32_t* length;
  if (dev < 0 || !whole(a[1], &block) || block < 1) return none();
  const auto s = kept->sizes();
  if (!small(s) || !is(kept, kI32, dev, s) || !opt(a[2], kI32, dev, {s[0]}, &length)) return none();
  ds_cache_array arrays[DS_CACHE_MAX_ARRAYS];
  int count = 0;
  int64_t T = 0;
  for (int per_block = 0; per_block < 2; ++per_block) {
    PyObject* list = a[3 + per_block];
    if (!PyList_CheckExact(list) && !PyTuple_CheckExact(list)) return none();
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(list); ++i) {
      PyObject* pair = PySequence_Fast_GET_ITEM(list, i);
      if (!PyTuple_CheckExact(pair) || PyTuple_GET_SIZE(pair) != 2 || count == DS_CACHE_MAX_ARRAYS) return none();
      const Tensor *src = tensor(PyTuple_GET_ITEM(pair, 0)), *dst = tensor(PyTuple_GET_ITEM(pair, 1));
      if (!src || !dst || src->dim() < 2 || dst->dim() != src->dim() || src->numel() == 0 || !small(src->sizes())) return none();
      if (count == 0) T = src->size(1) * (per_block ? block : 1);
      const int64_t items = per_block ? (T + block - 1) / block : T, least = per_block ? s[1] : std::min(T, s[1] * block);
      if (T > INT32_MAX || src->size(0) != s[0] || src->size(1) != items || dst->size(0) != s[0] || dst->size(1) < least ||
          src->sizes().slice(2) != dst->sizes().slice(2) || !is(src, src->scalar_type(), dev, src->sizes()) ||
          !is(dst, src->scalar_type(), dev, dst->sizes()))
        return none();
      const int64_t size = src->element_size(), item = src->numel() / (s[0] * items) * size;
      arrays[count++] = {src->data_ptr(), dst->data_ptr(), items * item, dst->size(1) * item, item, per_block};
    }
  }
  if (count == 0 || g_lib.compact(arrays, count, data<int32_t>(*kept), (int)s[1], length, (int)s[0], (int)T, block,
                                  stream_of(dev)) != DS_OK)
    return none();
  Py_RETURN_TRUE;
}

// Addresses of the library's five functions, in this order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "five addresses are wanted");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_lib = {(decltype(g_lib.quantize))p[0], (decltype(g_lib.attention))p[1], (decltype(g_lib.mass))p[2],
           (decltype(g_lib.evict))p[3], (decltype(g_lib.compact))p[4]};
  Py_RETURN_NONE;
}

// No C++ exception may pass into the interpreter: the macros turn it into Python's.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(self, a, n);
  END_HANDLE_TH_ERRORS
}

#define DS_FRONT(name) {#name, (PyCFunction)(void (*)(void))guarded<name>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {DS_FRONT(bind),  DS_FRONT(quantize), DS_FRONT(attention), DS_FRONT(mass),
                          DS_FRONT(evict), DS_FRONT(compact),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front(void) { return PyModule_Create(&kModule); }
