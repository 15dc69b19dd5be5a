// pa_bind.cpp -- Python's way into the calls of rotated append and sparse
// attention where every argument fits: the checks of the binding in
// ../__init__.py and the C call, in C++ (a call from Python took 7 to 11 us with
// these checks in Python and the arguments converted by ctypes, of which the C
// call is 2).  What does not fit is left to the checks there, which name it: each
// function returns the call's status, or -1 for that.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/detail/CUDAHooksInterface.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <limits>

#include "../../include/pa.h"

namespace {

constexpr long kNoFit = -1;
enum Kind { k16 = 0, kFp8 = 1, kFp4 = 2 };  // of a cache

PyObject *g_raw_stream = nullptr;  // of a device: the current stream's handle

// The arguments of a call.  `ok` is false once one did not fit; nothing is looked
// at after that.
struct Args {
  PyObject *const *a;
  bool ok = true;
  int64_t dev = -1;

  void want(bool yes) { ok = ok && yes; }

  // Argument i, a tensor of `dim` dimensions (-1: any) on the current device.
  const at::Tensor *tensor(int i, at::ScalarType type, int dim, bool dense = true) {
    if (!ok) return nullptr;
    ok = THPVariable_Check(a[i]);
    if (!ok) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(a[i]);
    ok = t.is_cuda() && t.scalar_type() == type && (dim < 0 || t.dim() == dim);
    if (!ok) return nullptr;
    if (dev < 0) {
      dev = t.get_device();
      ok = dev == at::detail::getCUDAHooks().getCurrentDevice();
    }
    ok = ok && t.get_device() == dev && (!dense || t.is_contiguous());
    return ok ? &t : nullptr;
  }
  bool none(int i) const { return a[i] == Py_None; }
  // The type of the 16-bit tensor argument i.
  at::ScalarType half_type(int i) {
    ok = ok && THPVariable_Check(a[i]);
    if (!ok) return at::kHalf;
    const at::ScalarType t = THPVariable_Unpack(a[i]).scalar_type();
    ok = t == at::kHalf || t == at::kBFloat16;
    return t;
  }
  int32_t integer(int i) {
    if (!ok || !PyLong_Check(a[i])) {
      ok = false;
      return 0;
    }
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(a[i], &over);
    ok = !over && v >= std::numeric_limits<int32_t>::min() && v <= std::numeric_limits<int32_t>::max();
    return ok ? static_cast<int32_t>(v) : 0;
  }
  float number(int i) {
    if (!ok || !(PyFloat_Check(a[i]) || PyLong_Check(a[i]))) {
      ok = false;
      return 0.f;
    }
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return static_cast<float>(v);
  }
  bool truth(int i) {
    if (!ok) return false;
    const int v = PyObject_IsTrue(a[i]);
    ok = v >= 0;
    return v > 0;
  }
  // A stream: None (the current one), an object with a handle, or the handle.
  void *stream(int i) {
    if (!ok) return nullptr;
    PyObject *o = nullptr;
    if (a[i] == Py_None) {
      PyObject *d = PyLong_FromLongLong(dev);
      o = d ? PyObject_CallOneArg(g_raw_stream, d) : nullptr;
      Py_XDECREF(d);
    } else if (PyLong_Check(a[i])) {
      o = a[i];
      Py_INCREF(o);
    } else {
      o = PyObject_GetAttrString(a[i], "cuda_stream");
    }
    void *s = o && PyLong_Check(o) ? PyLong_AsVoidPtr(o) : nullptr;
    ok = o && PyLong_Check(o) && !PyErr_Occurred();
    Py_XDECREF(o);
    return s;
  }
  // Blocks, heads and block size of a cache for heads of d.
  void cache(const at::Tensor *t, int kind, int64_t d, int64_t &blocks, int64_t &heads, int64_t &bs) {
    if (!ok) return;
    blocks = t->size(0);
    heads = t->size(1);
    if (kind == kFp4) {
      ok = d > 0 && t->size(2) * 16 % (9 * d) == 0;
      bs = ok ? t->size(2) * 16 / (9 * d) : 0;
    } else {
      ok = t->size(3) == d;
      bs = t->size(2);
    }
  }
};

at::ScalarType cache_type(int kind, at::ScalarType rows) { return kind == k16 ? rows : at::kByte; }
int cache_dim(int kind) { return kind == kFp4 ? 3 : 4; }
int32_t code_of(at::ScalarType t) { return t == at::kHalf ? PA_FP16 : PA_BF16; }
bool fits32(int64_t v) { return v <= std::numeric_limits<int32_t>::max(); }

// f(Args): the call, or nothing if an argument does not fit.
template <typename F> PyObject *call(PyObject *const *a, Py_ssize_t n, Py_ssize_t want, F &&f) {
  long st = kNoFit;
  try {
    Args args{a};
    args.want(n == want);
    if (args.ok) st = f(args);
  } catch (...) {  // (a tensor without storage, say)
    st = kNoFit;
  }
  PyErr_Clear();
  return PyLong_FromLong(st);
}

// The GIL is given up for its life, and taken again however that ends.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The C call.  Its arguments are values by now: what asks a tensor for something
// (its address: a tensor without memory of its own throws) is done by the caller,
// with the GIL.
template <typename... P, typename... A> long launch(pa_status (*f)(P...), A... args) {
  const Unlocked unlocked;
  return static_cast<long>(f(args...));
}

// kind, query_out, query, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin,
// k_scale, v_scale, interleaved, stream
PyObject *rope(PyObject *, PyObject *const *argv, Py_ssize_t n) {
  return call(argv, n, 14, [](Args &a) -> long {
    const int kind = a.integer(0);
    const at::ScalarType type = a.half_type(2);
    const at::Tensor *q = a.tensor(2, type, 3, false), *qo = a.tensor(1, type, 3, false);
    const at::Tensor *k = a.tensor(3, type, 3, false), *v = a.tensor(4, type, 3, false);
    const at::Tensor *kc = a.tensor(5, cache_type(kind, type), cache_dim(kind));
    const at::Tensor *vc = a.tensor(6, cache_type(kind, type), cache_dim(kind));
    const at::Tensor *slots = a.tensor(7, at::kLong, -1), *pos = a.tensor(8, at::kLong, -1);
    const at::Tensor *table = a.tensor(9, at::kFloat, 2);
    const float ks = a.number(10), vs = a.number(11);
    const bool inter = a.truth(12);
    void *stream = a.stream(13);
    if (!a.ok) return kNoFit;
    const int64_t T = q->size(0), hq = q->size(1), d = q->size(2), hkv = k->size(1);
    int64_t nb = 0, heads = 0, bs = 0;
    a.cache(kc, kind, d, nb, heads, bs);
    for (const at::Tensor *t : {q, qo, k, v}) a.want(t->stride(2) == 1 && t->stride(1) == d);
    a.want(qo->sizes() == q->sizes() && v->sizes() == k->sizes() && k->size(0) == T &&
           k->size(2) == d && heads == hkv && vc->sizes() == kc->sizes() && slots->numel() == T &&
           pos->numel() == T && fits32(T) && fits32(hq) && fits32(hkv) && fits32(table->size(1)) &&
           fits32(bs));
    if (!a.ok) return kNoFit;
    // (the stride of a single row is not looked at)
    auto stride = [&](const at::Tensor *t) { return T > 1 ? t->stride(0) : t->size(1) * d; };
    auto with = [&](auto f, auto... scales) {
      return launch(f, qo->data_ptr(), q->data_ptr(), k->data_ptr(), v->data_ptr(), stride(qo),
                    stride(q), stride(k), stride(v), kc->data_ptr(), vc->data_ptr(),
                    static_cast<const int64_t *>(slots->data_ptr()),
                    static_cast<const int64_t *>(pos->data_ptr()),
                    static_cast<const float *>(table->data_ptr()), T, hq, hkv, d, table->size(1),
                    inter ? 1 : 0, bs, nb, table->size(0), code_of(type), scales..., stream);
    };
    return kind == k16 ? with(pa_rope_and_cache)
                       : with(kind == kFp8 ? pa_rope_and_cache_fp8 : pa_rope_and_cache_fp4, ks, vs);
  });
}

// kind, bounds, bound_scales, k_cache, block_tables, context_lens, query_start, max_q_len, stream
PyObject *key_bounds(PyObject *, PyObject *const *argv, Py_ssize_t n) {
  return call(argv, n, 9, [](Args &a) -> long {
    const int kind = a.integer(0);
    const at::ScalarType type = kind == k16 ? a.half_type(3) : at::kByte;
    const at::Tensor *kc = a.tensor(3, type, cache_dim(kind));
    const at::Tensor *bounds = a.tensor(1, at::kChar, 4), *scales = a.tensor(2, at::kFloat, 2);
    const at::Tensor *tables = a.tensor(4, at::kInt, 2), *lens = a.tensor(5, at::kInt, -1);
    const at::Tensor *start = a.none(6) ? nullptr : a.tensor(6, at::kInt, -1);
    const int32_t max_q = a.integer(7);
    void *stream = a.stream(8);
    if (!a.ok) return kNoFit;
    const int64_t d = bounds->size(3), B = lens->numel();
    int64_t nb = 0, heads = 0, bs = 0;
    a.cache(kc, kind, d, nb, heads, bs);
    a.want(bounds->size(0) == nb && bounds->size(1) == heads && bounds->size(2) == 2 &&
           scales->size(0) == nb && scales->size(1) == heads && tables->size(0) == B &&
           (!start || start->numel() == B + 1) && fits32(B) && fits32(heads) && fits32(d) &&
           fits32(bs) && fits32(tables->size(1)));
    if (!a.ok) return kNoFit;
    auto with = [&](auto f, auto... type_code) {
      return launch(f, static_cast<int8_t *>(bounds->data_ptr()),
                    static_cast<float *>(scales->data_ptr()), kc->data_ptr(),
                    static_cast<const int32_t *>(tables->data_ptr()), tables->size(1),
                    static_cast<const int32_t *>(lens->data_ptr()),
                    start ? static_cast<const int32_t *>(start->data_ptr()) : nullptr, B, max_q,
                    heads, d, bs, nb, type_code..., stream);
    };
    return kind == k16 ? with(pa_update_key_bounds, code_of(type))
                       : with(kind == kFp8 ? pa_update_key_bounds_fp8 : pa_update_key_bounds_fp4);
  });
}

// selected_tables, selected_lens, query, bounds, bound_scales, block_tables, context_lens,
// block_size, max_context_len, num_sink, num_recent, query_start, max_q_len, stream
PyObject *select(PyObject *, PyObject *const *argv, Py_ssize_t n) {
  return call(argv, n, 14, [](Args &a) -> long {
    const at::ScalarType type = a.half_type(2);
    const at::Tensor *q = a.tensor(2, type, 3);
    const at::Tensor *picked = a.tensor(0, at::kInt, 3), *plens = a.tensor(1, at::kInt, 2);
    const at::Tensor *bounds = a.tensor(3, at::kChar, 4), *scales = a.tensor(4, at::kFloat, 2);
    const at::Tensor *tables = a.tensor(5, at::kInt, 2), *lens = a.tensor(6, at::kInt, -1);
    const int32_t bs = a.integer(7), most = a.integer(8), sink = a.integer(9), recent = a.integer(10);
    const at::Tensor *start = a.none(11) ? nullptr : a.tensor(11, at::kInt, -1);
    int32_t max_q = a.integer(12);
    void *stream = a.stream(13);
    if (!a.ok) return kNoFit;
    const int64_t R = q->size(0), hq = q->size(1), d = q->size(2), B = lens->numel();
    const int64_t nb = bounds->size(0), hkv = bounds->size(1), K = picked->size(2);
    if (R == 0) max_q = 0;  // no rows: empty tensors have no address
    a.want(bounds->size(2) == 2 && bounds->size(3) == d && scales->size(0) == nb &&
           scales->size(1) == hkv && picked->size(0) == R && picked->size(1) == hkv &&
           plens->size(0) == R && plens->size(1) == hkv && tables->size(0) == B &&
           (start ? start->numel() == B + 1 : R == B) && fits32(B) && fits32(hq) && fits32(hkv) &&
           fits32(d) && fits32(K) && fits32(tables->size(1)));
    if (!a.ok) return kNoFit;
    return launch(pa_select_blocks, static_cast<int32_t *>(picked->data_ptr()),
                  static_cast<int32_t *>(plens->data_ptr()), q->data_ptr(),
                  static_cast<const int8_t *>(bounds->data_ptr()),
                  static_cast<const float *>(scales->data_ptr()),
                  static_cast<const int32_t *>(tables->data_ptr()), tables->size(1),
                  static_cast<const int32_t *>(lens->data_ptr()),
                  start ? static_cast<const int32_t *>(start->data_ptr()) : nullptr, B, max_q, hq,
                  hkv, d, bs, nb, most, K, sink, recent, code_of(type), stream);
  });
}

// kind, out, query, k_cache, v_cache, selected_tables, selected_lens, scale, k_scale, v_scale,
// stream
PyObject *sparse(PyObject *, PyObject *const *argv, Py_ssize_t n) {
  return call(argv, n, 11, [](Args &a) -> long {
    const int kind = a.integer(0);
    const at::ScalarType type = a.half_type(2);
    const at::Tensor *q = a.tensor(2, type, 3), *out = a.tensor(1, type, 3);
    const at::Tensor *kc = a.tensor(3, cache_type(kind, type), cache_dim(kind));
    const at::Tensor *vc = a.tensor(4, cache_type(kind, type), cache_dim(kind));
    const at::Tensor *picked = a.tensor(5, at::kInt, 3), *plens = a.tensor(6, at::kInt, 2);
    const float scale = a.number(7), ks = a.number(8), vs = a.number(9);
    void *stream = a.stream(10);
    if (!a.ok) return kNoFit;
    const int64_t R = q->size(0), hq = q->size(1), d = q->size(2), K = picked->size(2);
    int64_t nb = 0, hkv = 0, bs = 0;
    a.cache(kc, kind, d, nb, hkv, bs);
    a.want(out->sizes() == q->sizes() && vc->sizes() == kc->sizes() && picked->size(0) == R &&
           picked->size(1) == hkv && plens->size(0) == R && plens->size(1) == hkv && fits32(R) &&
           fits32(hq) && fits32(hkv) && fits32(d) && fits32(K) && fits32(bs));
    if (!a.ok) return kNoFit;
    auto with = [&](auto f, auto... scales) {
      return launch(f, out->data_ptr(), q->data_ptr(), kc->data_ptr(), vc->data_ptr(),
                    static_cast<const int32_t *>(picked->data_ptr()),
                    static_cast<const int32_t *>(plens->data_ptr()), R, K, hq, hkv, d, bs, nb,
                    scale, scales..., code_of(type), stream);
    };
    return kind == k16 ? with(pa_decode_sparse)
                       : with(kind == kFp8 ? pa_decode_sparse_fp8 : pa_decode_sparse_fp4, ks, vs);
  });
}

// The function that gives the current stream's handle on a device.
PyObject *set_raw_stream(PyObject *, PyObject *f) {
  Py_INCREF(f);
  Py_XSETREF(g_raw_stream, f);
  Py_RETURN_NONE;
}

#define PA_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {{"rope", PA_FAST(rope), nullptr},
                          {"key_bounds", PA_FAST(key_bounds), nullptr},
                          {"select", PA_FAST(select), nullptr},
                          {"sparse", PA_FAST(sparse), nullptr},
                          {"set_raw_stream", set_raw_stream, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "pa_bind", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit_pa_bind(void) { return PyModule_Create(&kModule); }
