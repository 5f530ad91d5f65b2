// swa_torch.cpp — the binding's short way to the library: SwaCache and swa_cache_attn, and swa_attn_fwd
// and swa_attn_bwd with sinks, for arguments as they should be.
//
// A step of one token is a few microseconds of GPU work, less than Python takes to look at a call's
// tensors.  This module looks at them, allocates what the call returns and its workspace from torch's
// allocator, and calls the library on the current stream.  Whatever is not plainly in order (another type,
// shape, device, layout; an int that is none; a subclass of Tensor) gets None for an answer, and the Python
// code, which checks the same and says what is wrong, takes the call.
//
// One Grace core, time of a call on the host, of which the launches are 4 us: a token over one sequence
// 8.9 us (23.8 in Python), a forward with sinks 6.5 (20.7), its backward 17 (37).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "swa_attn.h"
#include "swa_cache.h"

namespace {

// The library's functions, by the addresses that the binding loaded.
struct Library {
  decltype(&swa_cache_attn) attn;
  decltype(&swa_cache_attn_sinks) attn_sinks;
  decltype(&swa_cache_attn_shared) attn_shared;
  decltype(&swa_cache_attn_shared_workspace_bytes) attn_space;
  decltype(&swa_attn_fwd_sinks) fwd;
  decltype(&swa_attn_bwd_sinks) bwd;
  decltype(&swa_attn_sinks_workspace_bytes) space;
} lib;

const at::Tensor* tensor(PyObject* x) {
  if (!THPVariable_CheckExact(x)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(x);
  return t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}
bool good(const at::Tensor* t, at::IntArrayRef shape, at::ScalarType type, int gpu) {
  return t && t->scalar_type() == type && t->get_device() == gpu && t->sizes() == shape &&
         t->is_contiguous();
}
// The C int nearest to a Python int.
bool as_int(PyObject* x, int* out) {
  if (!PyLong_CheckExact(x)) return false;
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(x, &over);
  *out = over > 0 || v > INT_MAX ? INT_MAX : over < 0 || v < INT_MIN ? INT_MIN : static_cast<int>(v);
  return true;
}
bool fits(at::IntArrayRef shape) {
  for (int64_t n : shape)
    if (n > INT_MAX) return false;
  return true;
}
bool as_scale(PyObject* x, int64_t D, float* out) {
  if (x == Py_None) {
    *out = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
    return true;
  }
  if (!PyFloat_CheckExact(x)) return false;
  *out = static_cast<float>(PyFloat_AS_DOUBLE(x));
  return true;
}
int kind_of(at::ScalarType type) {
  return type == at::kBFloat16 ? SWA_BF16 : type == at::kHalf ? SWA_FP16 : type == at::kFloat ? SWA_FP32 : -1;
}
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int gpu) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, gpu));
}

// A tensor that the call writes: the caller's, or a new one.
struct Out {
  at::Tensor made;
  const at::Tensor* t = nullptr;
  PyObject* given = nullptr;
  bool set(PyObject* x, at::IntArrayRef shape, at::ScalarType type, int gpu) {
    if (x != Py_None) {
      given = x;
      t = tensor(x);
      return good(t, shape, type, gpu);
    }
    made = make(shape, type, gpu);
    t = &made;
    return true;
  }
  void* data() const { return t->data_ptr(); }
  PyObject* give() const { return given ? Py_NewRef(given) : THPVariable_Wrap(made); }
};

// The workspace: all bytes of the caller's tensor, or `need` new ones.
struct Space {
  at::Tensor made;
  void* at = nullptr;
  size_t bytes = 0;
  template <typename Need>
  bool set(PyObject* x, int gpu, Need need) {
    if (x != Py_None) {
      const at::Tensor* t = tensor(x);
      if (!t || t->get_device() != gpu || !t->is_contiguous()) return false;
      at = t->data_ptr();
      bytes = t->nbytes();
      return true;
    }
    bytes = need();
    if (bytes == 0) return true;
    made = make({static_cast<int64_t>(bytes)}, at::kByte, gpu);
    at = made.data_ptr();
    return true;
  }
};

// What a call returns: made before it is launched, since a call that fails afterwards must not be taken for
// one that has not been made.
template <size_t N>
PyObject* pack(const Out (&outs)[N]) {
  PyObject* all = PyTuple_New(N);
  for (size_t i = 0; all && i < N; ++i) {
    PyObject* t = outs[i].give();
    if (!t) {
      Py_DECREF(all);
      return nullptr;
    }
    PyTuple_SET_ITEM(all, i, t);
  }
  return all;
}
// `all`, or the library's status where that is not SWA_OK.
PyObject* answer(int status, PyObject* all) {
  if (status == SWA_OK) return all;
  Py_DECREF(all);
  return PyLong_FromLong(status);
}

template <typename Body>
PyObject* guarded(Body body) {
  try {
    if (PyObject* r = body()) return r;
  } catch (...) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// k, v, k_scale, v_scale, weight: SwaCache.held, the tensors with their device and k's shape.
PyObject* pool(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) return nullptr;
    const at::Tensor* k = tensor(x[0]);
    if (!k || k->dim() != 4) return nullptr;
    const at::IntArrayRef shape = k->sizes();
    const int gpu = static_cast<int>(k->get_device());
    if (!good(k, shape, at::kFloat8_e4m3fn, gpu) || !good(tensor(x[1]), shape, at::kFloat8_e4m3fn, gpu) ||
        !good(tensor(x[2]), shape.slice(0, 2), at::kFloat, gpu) ||
        !good(tensor(x[3]), shape.slice(0, 2), at::kFloat, gpu) ||
        (x[4] != Py_None && !good(tensor(x[4]), shape.slice(0, 3), at::kFloat, gpu)))
      return nullptr;
    PyObject* device = PyObject_GetAttrString(x[0], "device");
    PyObject* sizes = device ? Py_BuildValue("(LLLL)", static_cast<long long>(shape[0]),
                                             static_cast<long long>(shape[1]), static_cast<long long>(shape[2]),
                                             static_cast<long long>(shape[3]))
                             : nullptr;
    PyObject* held = sizes ? PyTuple_Pack(7, x[0], x[1], x[2], x[3], x[4], device, sizes) : nullptr;
    Py_XDECREF(device);
    Py_XDECREF(sizes);
    return held;
  });
}

// held (SwaCache.held), q, table, lens, new, out, lse, workspace, window, scale, accumulate, sinks, shared
PyObject* cache_attn(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13 || !PyTuple_CheckExact(x[0]) || PyTuple_GET_SIZE(x[0]) != 7) return nullptr;
    auto held = [&](int i) { return PyTuple_GET_ITEM(x[0], i); };
    const at::Tensor* pool[5];
    for (int i = 0; i < 5; ++i) {
      pool[i] = tensor(held(i));
      if (!pool[i] && (i < 4 || held(i) != Py_None)) return nullptr;
    }
    int size[4];  // pages, Hkv, page, D
    if (!PyTuple_CheckExact(held(6)) || PyTuple_GET_SIZE(held(6)) != 4) return nullptr;
    for (int i = 0; i < 4; ++i)
      if (!as_int(PyTuple_GET_ITEM(held(6), i), &size[i]) || size[i] == INT_MAX) return nullptr;
    const int gpu = static_cast<int>(pool[0]->get_device()), D = size[3];
    if (gpu != c10::cuda::current_device()) return nullptr;
    const at::Tensor *q = tensor(x[1]), *table = tensor(x[2]), *lens = tensor(x[3]);
    if (!q || !table || !lens || q->dim() != 4 || table->dim() != 2) return nullptr;
    const int64_t B = table->size(0), width = table->size(1), Hq = q->size(1), T = q->size(2);
    if (!fits({B, width, Hq, T})) return nullptr;
    const at::ScalarType type = q->scalar_type();
    const int kind = kind_of(type);
    if (kind != SWA_BF16 && kind != SWA_FP16) return nullptr;
    if (!good(q, {B, Hq, T, D}, type, gpu) || !good(table, {B, width}, at::kInt, gpu) ||
        !good(lens, {B}, at::kInt, gpu))
      return nullptr;
    const at::Tensor* fresh = nullptr;
    if (x[4] != Py_None && !good(fresh = tensor(x[4]), {B}, at::kInt, gpu)) return nullptr;
    int window, sinks, shared;
    float scale;
    if (!as_int(x[8], &window) || !as_scale(x[9], D, &scale) || !as_int(x[11], &sinks) ||
        !as_int(x[12], &shared))
      return nullptr;
    if (!PyBool_Check(x[10])) return nullptr;
    const int accumulate = x[10] == Py_True;
    const int b = static_cast<int>(B), hq = static_cast<int>(Hq), t = static_cast<int>(T),
              w = static_cast<int>(width);
    Out outs[2];
    Space space;
    if (!outs[0].set(x[5], q->sizes(), type, gpu) || !outs[1].set(x[6], {B, Hq, T}, at::kFloat, gpu) ||
        !space.set(x[7], gpu, [&] {
          return lib.attn_space(b, hq, size[1], t, D, w, size[2], window, sinks, shared, accumulate);
        }))
      return nullptr;
    auto ptr = [](const at::Tensor* v) { return v ? v->data_ptr() : nullptr; };
    swa_cache c;
    c.k = ptr(pool[0]);
    c.v = ptr(pool[1]);
    c.k_scale = static_cast<float*>(ptr(pool[2]));
    c.v_scale = static_cast<float*>(ptr(pool[3]));
    c.weight = static_cast<float*>(ptr(pool[4]));
    c.pages = size[0];
    c.Hkv = size[1];
    c.page = size[2];
    c.D = D;
    const int* tab = static_cast<const int*>(ptr(table));
    const int* len = static_cast<const int*>(ptr(lens));
    const int* add = static_cast<const int*>(ptr(fresh));
    const void* qp = ptr(q);
    void* op = outs[0].data();
    float* lp = static_cast<float*>(outs[1].data());
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(gpu).stream();
    PyObject* all = pack(outs);
    if (!all) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    if (shared)
      rc = lib.attn_shared(&c, tab, w, len, add, qp, op, lp, b, hq, t, window, sinks, shared, scale,
                           accumulate, kind, space.at, space.bytes, stream);
    else if (sinks)
      rc = lib.attn_sinks(&c, tab, w, len, add, qp, op, lp, b, hq, t, window, sinks, scale, accumulate,
                          kind, space.at, space.bytes, stream);
    else
      rc = lib.attn(&c, tab, w, len, add, qp, op, lp, b, hq, t, window, scale, accumulate, kind, space.at,
                    space.bytes, stream);
    Py_END_ALLOW_THREADS
    return answer(rc, all);
  });
}

// What fwd and bwd share: the tensors of a layer, its sizes and the window.
struct Layer {
  const at::Tensor *q, *k, *v;
  int gpu, B, Hq, Hkv, Lq, Lk, D, kind, window, causal, sinks;
  at::ScalarType type;
  float scale;
  int64_t rows[4], keys[4];
  bool set(PyObject* const* qkv, PyObject* win, PyObject* sc, PyObject* caus, PyObject* snk) {
    q = tensor(qkv[0]);
    k = tensor(qkv[1]);
    v = tensor(qkv[2]);
    if (!q || !k || !v || q->dim() != 4 || k->dim() != 4 || !fits(q->sizes()) || !fits(k->sizes()))
      return false;
    gpu = static_cast<int>(q->get_device());
    if (gpu != c10::cuda::current_device()) return false;
    type = q->scalar_type();
    kind = kind_of(type);
    if (kind < 0) return false;
    const int64_t d = q->size(3);
    const int64_t r[4] = {q->size(0), q->size(1), q->size(2), d};
    const int64_t e[4] = {q->size(0), k->size(1), k->size(2), d};
    for (int i = 0; i < 4; ++i) rows[i] = r[i], keys[i] = e[i];
    if (!good(q, rows, type, gpu) || !good(k, keys, type, gpu) || !good(v, keys, type, gpu)) return false;
    B = static_cast<int>(r[0]);
    Hq = static_cast<int>(r[1]);
    Lq = static_cast<int>(r[2]);
    D = static_cast<int>(d);
    Hkv = static_cast<int>(e[1]);
    Lk = static_cast<int>(e[2]);
    if (!PyBool_Check(caus)) return false;
    causal = caus == Py_True;
    return as_int(win, &window) && as_int(snk, &sinks) && as_scale(sc, d, &scale);
  }
  at::IntArrayRef stats() const { return at::IntArrayRef(rows, 3); }
  size_t need(int backward) const {
    return lib.space(B, Hq, Hkv, Lq, Lk, D, window, sinks, causal, kind, backward);
  }
};

// q, k, v, out, lse, workspace, window, scale, causal, sinks
PyObject* fwd(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Layer y;
    if (n != 10 || !y.set(x, x[6], x[7], x[8], x[9])) return nullptr;
    Out outs[2];
    Space space;
    if (!outs[0].set(x[3], y.rows, y.type, y.gpu) || !outs[1].set(x[4], y.stats(), at::kFloat, y.gpu) ||
        !space.set(x[5], y.gpu, [&] { return y.need(0); }))
      return nullptr;
    const void *q = y.q->data_ptr(), *k = y.k->data_ptr(), *v = y.v->data_ptr();
    void* o = outs[0].data();
    float* lse = static_cast<float*>(outs[1].data());
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(y.gpu).stream();
    PyObject* all = pack(outs);
    if (!all) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = lib.fwd(q, k, v, o, lse, y.B, y.Hq, y.Hkv, y.Lq, y.Lk, y.D, y.window, y.sinks, y.causal, y.scale,
                 y.kind, space.at, space.bytes, stream);
    Py_END_ALLOW_THREADS
    return answer(rc, all);
  });
}

// q, k, v, o, do, lse, dq, dk, dv, workspace, window, scale, causal, sinks
PyObject* bwd(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Layer y;
    if (n != 14 || !y.set(x, x[10], x[11], x[12], x[13])) return nullptr;
    const at::Tensor *o = tensor(x[3]), *dO = tensor(x[4]), *lse = tensor(x[5]);
    if (!good(o, y.rows, y.type, y.gpu) || !good(dO, y.rows, y.type, y.gpu) ||
        !good(lse, y.stats(), at::kFloat, y.gpu))
      return nullptr;
    Out outs[3];
    Space space;
    if (!outs[0].set(x[6], y.rows, y.type, y.gpu) || !outs[1].set(x[7], y.keys, y.type, y.gpu) ||
        !outs[2].set(x[8], y.keys, y.type, y.gpu) || !space.set(x[9], y.gpu, [&] { return y.need(1); }))
      return nullptr;
    const void *q = y.q->data_ptr(), *k = y.k->data_ptr(), *v = y.v->data_ptr();
    const void *op = o->data_ptr(), *gp = dO->data_ptr();
    const float* lp = static_cast<const float*>(lse->data_ptr());
    void *dq = outs[0].data(), *dk = outs[1].data(), *dv = outs[2].data();
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(y.gpu).stream();
    PyObject* all = pack(outs);
    if (!all) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = lib.bwd(q, k, v, op, gp, lp, dq, dk, dv, y.B, y.Hq, y.Hkv, y.Lq, y.Lk, y.D, y.window, y.sinks,
                 y.causal, y.scale, y.kind, space.at, space.bytes, stream);
    Py_END_ALLOW_THREADS
    return answer(rc, all);
  });
}

// The addresses of Library's members, in their order.
PyObject* use(PyObject*, PyObject* const* x, Py_ssize_t n) {
  void* at[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "use() takes the library's seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    at[i] = PyLong_AsVoidPtr(x[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
  }
  lib.attn = reinterpret_cast<decltype(lib.attn)>(at[0]);
  lib.attn_sinks = reinterpret_cast<decltype(lib.attn_sinks)>(at[1]);
  lib.attn_shared = reinterpret_cast<decltype(lib.attn_shared)>(at[2]);
  lib.attn_space = reinterpret_cast<decltype(lib.attn_space)>(at[3]);
  lib.fwd = reinterpret_cast<decltype(lib.fwd)>(at[4]);
  lib.bwd = reinterpret_cast<decltype(lib.bwd)>(at[5]);
  lib.space = reinterpret_cast<decltype(lib.space)>(at[6]);
  Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* ready(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  if (!lib.space) Py_RETURN_NONE;
  return f(self, x, n);
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"use", fast<use>(), METH_FASTCALL, nullptr},
    {"pool", fast<pool>(), METH_FASTCALL, nullptr},
    {"cache_attn", fast<ready<cache_attn>>(), METH_FASTCALL, nullptr},
    {"fwd", fast<ready<fwd>>(), METH_FASTCALL, nullptr},
    {"bwd", fast<ready<bwd>>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_swa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr,
                      nullptr};

}  // namespace

// `built_for` names the torch and the Python whose objects the module reads; the binding uses it with those
// alone.
PyMODINIT_FUNC PyInit__swa_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", SWA_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
