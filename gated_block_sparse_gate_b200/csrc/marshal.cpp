// marshal.cpp — argument checks and calls of the Python binding, on the tensors themselves.
//
// A call of a few microseconds on the GPU is otherwise outweighed by its argument checks:
// one to two microseconds a tensor in Python, some fifty nanoseconds here. fits and heads
// only answer whether a tensor plainly has what is asked of it, and the calls below make a
// call only where all of its arguments plainly have; anything else (another type, a view
// with a layout of its own, another device, a mistake) is left to the binding's own checks,
// which accept or refuse it in words.
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "gbs.h"

namespace {

// The tensor in t if it is plainly one on CUDA device `device` with one of the dtypes (a
// tuple) and that shape (None: any); else null.
const at::Tensor* plain(PyObject* t, PyObject* dtypes, PyObject* device, PyObject* shape) {
  if (!THPVariable_CheckExact(t) || !PyLong_Check(device)) return nullptr;
  const at::Tensor& x = THPVariable_Unpack(t);
  if (!x.defined() || x.layout() != at::kStrided || x.get_device() != PyLong_AsLong(device)) return nullptr;
  bool known = false;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(dtypes) && !known; ++i) {
    PyObject* d = PyTuple_GET_ITEM(dtypes, i);
    known = THPDtype_Check(d) && reinterpret_cast<THPDtype*>(d)->scalar_type == x.scalar_type();
  }
  if (!known) return nullptr;
  if (shape == Py_None) return &x;
  const auto sizes = x.sizes();
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != (Py_ssize_t)sizes.size()) return nullptr;
  for (size_t i = 0; i < sizes.size(); ++i)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)) != sizes[i]) return nullptr;
  return &x;
}

// fits(t, dtypes, device_index, shape): plainly so and contiguous?
PyObject* fits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4 || !PyTuple_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "fits(t, dtypes, device_index, shape)");
    return nullptr;
  }
  try {
    const at::Tensor* x = plain(a[0], a[1], a[2], a[3]);
    if (PyErr_Occurred()) return nullptr;
    return PyBool_FromLong(x && x->is_contiguous());
  } catch (...) {  // a tensor without sizes or storage of its own: not plain
    Py_RETURN_FALSE;
  }
}

// heads(t, dtypes, device_index, shape, token_major, written): gbs_heads of a 4-D tensor
// as bytes; None if it is not plainly so, its channels are not contiguous or, where it is
// written, it is not contiguous.
PyObject* heads(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !PyTuple_Check(a[1]) || !PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 4) {
    PyErr_SetString(PyExc_TypeError, "heads(t, dtypes, device_index, shape, token_major, written)");
    return nullptr;
  }
  try {
    const at::Tensor* x = plain(a[0], a[1], a[2], a[3]);
    if (PyErr_Occurred()) return nullptr;
    if (!x || (a[5] == Py_True && !x->is_contiguous())) Py_RETURN_NONE;
    int64_t step[4];
    for (int i = 0; i < 4; ++i) step[i] = i < 3 && x->size(i) == 1 ? 0 : x->stride(i);  // (that of one is never followed)
    if (step[3] != 1) Py_RETURN_NONE;
    const int h_at = a[4] == Py_True ? 2 : 1;
    const gbs_heads h = {x->data_ptr(), step[0], step[h_at], step[3 - h_at]};
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&h), sizeof h);
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// ---------------------------------------------------------------- whole calls
// The first argument is a Library as bytes, the others are those of the binding's functions
// of the same names, up to `stream`. Each returns None (the binding's own path takes the
// call), or (status, results...).

struct Library {  // entry points of a loaded library
  decltype(&gbs_qkv_rope_fwd) rope_fwd;
  decltype(&gbs_qkv_rope_bwd) rope_bwd;
  decltype(&gbs_qkv_rope_workspace_bytes) rope_bytes;
  decltype(&gbs_kv4_append) append;
  decltype(&gbs_kv4_read) read;
  decltype(&gbs_kv4_decode) decode;
  decltype(&gbs_kv4_workspace_bytes) decode_bytes;
};

using Sizes = at::IntArrayRef;
struct NotPlain {};  // thrown where an argument is left to the binding's own path
void need(bool ok) {
  if (!ok) throw NotPlain();
}

// The tensor that decides a call's device, which is the current one.
const at::Tensor& anchor(PyObject* o) {
  need(THPVariable_CheckExact(o));
  const at::Tensor& x = THPVariable_Unpack(o);
  need(x.defined() && x.is_cuda() && x.layout() == at::kStrided && x.get_device() == c10::cuda::current_device());
  return x;
}
const at::Tensor& on_device(PyObject* o, int device) {
  need(THPVariable_CheckExact(o));
  const at::Tensor& x = THPVariable_Unpack(o);
  need(x.defined() && x.is_cuda() && x.layout() == at::kStrided && x.get_device() == device);
  return x;
}
const at::Tensor& dense(PyObject* o, int device, at::ScalarType type, Sizes shape) {
  const at::Tensor& x = on_device(o, device);
  need(x.scalar_type() == type && x.sizes() == shape && x.is_contiguous());
  return x;
}
void* dense_ptr(PyObject* o, int device, at::ScalarType type, Sizes shape) {
  return dense(o, device, type, shape).data_ptr();
}
void* optional_ptr(PyObject* o, int device, at::ScalarType type, Sizes shape) {
  return o == Py_None ? nullptr : dense_ptr(o, device, type, shape);
}
gbs_heads heads_of(const at::Tensor& x, bool token_major) {
  int64_t step[4];
  for (int i = 0; i < 4; ++i) step[i] = i < 3 && x.size(i) == 1 ? 0 : x.stride(i);
  need(step[3] == 1);
  const int h_at = token_major ? 2 : 1;
  return {x.data_ptr(), step[0], step[h_at], step[3 - h_at]};
}
gbs_heads heads_in(PyObject* o, int device, at::ScalarType type, Sizes shape, bool token_major) {
  const at::Tensor& x = on_device(o, device);
  need(x.scalar_type() == type && x.sizes() == shape);
  return heads_of(x, token_major);
}
bool listed(PyObject* o, Py_ssize_t n) {
  return (PyTuple_CheckExact(o) || PyList_CheckExact(o)) && PySequence_Fast_GET_SIZE(o) == n;
}
// What a call returns where it is not given: a new tensor, or the given one (contiguous).
at::Tensor result(PyObject* o, const at::Tensor& like, at::ScalarType type, Sizes shape) {
  if (o == Py_None) return at::empty(shape, like.options().dtype(type));
  return dense(o, like.get_device(), type, shape);
}
// The same of four dimensions, the given one strided too: in the order of their steps,
// each has to pass all that lies in the ones before, so that no two elements share memory.
at::Tensor result4(PyObject* o, const at::Tensor& like, Sizes shape) {
  if (o == Py_None) return at::empty(shape, like.options());
  const at::Tensor& x = on_device(o, like.get_device());
  need(x.scalar_type() == like.scalar_type() && x.sizes() == shape && x.stride(3) == 1);
  if (x.is_contiguous()) return x;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int i, int j) { return x.stride(i) < x.stride(j); });
  int64_t least = shape[3];
  for (int i : order)
    if (shape[i] > 1) {
      need(x.stride(i) >= least);
      least = x.stride(i) * shape[i];
    }
  return x;
}
// The three of a tuple of outputs; all None where there is none.
void three(PyObject* o, bool third, PyObject** out) {
  out[0] = out[1] = out[2] = Py_None;
  if (o == Py_None) return;
  need(listed(o, 3));
  for (int i = 0; i < 3; ++i) {
    out[i] = PySequence_Fast_GET_ITEM(o, i);
    need((out[i] == Py_None) == (i == 2 && !third));
  }
}
int whole(PyObject* o) {
  need(PyLong_CheckExact(o));
  int overflow;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  need(!overflow && v == (int)v);
  return (int)v;
}
int whole(int64_t v) {
  need(v == (int)v);
  return (int)v;
}
float real(PyObject* o) {
  need(PyFloat_CheckExact(o) || PyLong_CheckExact(o));
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    throw NotPlain();
  }
  need(std::isfinite(v) && std::fabs(v) < 3e38);
  return (float)v;
}
int yes(PyObject* o) {
  need(PyBool_Check(o));
  return o == Py_True;
}
int act(const at::Tensor& x) {
  need(x.scalar_type() == at::kBFloat16 || x.scalar_type() == at::kFloat);
  return x.scalar_type() == at::kBFloat16 ? GBS_BF16 : GBS_F32;
}
void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

// (status, tensors...); an undefined one is None.
PyObject* returned(int status, std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(1 + (Py_ssize_t)ts.size());
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const at::Tensor& t : ts) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// A call: C++ exceptions end here, as the binding's own path or as Python's error.
template <Py_ssize_t N, PyObject* (*CALL)(const Library&, PyObject* const*)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Library lib;
  if (n != N + 1) {
    PyErr_SetString(PyExc_TypeError, "the library's entry points and the call's arguments");
    return nullptr;
  }
  if (!PyBytes_CheckExact(a[0]) || PyBytes_GET_SIZE(a[0]) != sizeof lib) Py_RETURN_NONE;  // a stand-in for the library
  memcpy(static_cast<void*>(&lib), PyBytes_AS_STRING(a[0]), sizeof lib);
  try {
    return CALL(lib, a + 1);
  } catch (const NotPlain&) {
    Py_RETURN_NONE;
  } catch (...) {  // torch's errors (no memory, a tensor without storage): found again by the binding's own path
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

struct RopeCall {
  gbs_rope_params p{};
  int64_t B, N, Hq, Hkv, d;
  int device;
  at::ScalarType type;
  void *cos, *sin, *pos, *wq = nullptr, *wk = nullptr;
  gbs_heads q, k;

  RopeCall(PyObject* q_, PyObject* k_, PyObject* cos_, PyObject* sin_, PyObject* pos_, PyObject* wq_, PyObject* wk_,
           PyObject* eps, PyObject* axes, PyObject* interleaved) {
    const at::Tensor& x = anchor(q_);
    device = x.get_device();
    type = x.scalar_type();
    p.dtype = act(x);
    const at::Tensor& y = on_device(k_, device);
    need(x.dim() == 4 && y.dim() == 4);
    B = x.size(0); N = x.size(1); Hq = x.size(2); d = x.size(3); Hkv = y.size(2);
    q = heads_of(x, true);
    k = heads_in(k_, device, type, {B, N, Hkv, d}, true);
    const at::Tensor& table = on_device(cos_, device);
    need(table.dim() == 2);
    const int64_t max_pos = table.size(0), half = table.size(1);
    cos = dense_ptr(cos_, device, at::kFloat, {max_pos, half});
    sin = dense_ptr(sin_, device, at::kFloat, {max_pos, half});
    const at::Tensor& at_ = on_device(pos_, device);
    need((at_.dim() == 2 || at_.dim() == 3) && half <= 64);
    const int64_t n_axes = at_.dim() == 2 ? 1 : at_.size(2);
    pos = at_.dim() == 2 ? dense_ptr(pos_, device, at::kInt, {B, N}) : dense_ptr(pos_, device, at::kInt, {B, N, n_axes});
    if (axes != Py_None) {
      need(listed(axes, half));
      for (int i = 0; i < half; ++i) {
        const int v = whole(PySequence_Fast_GET_ITEM(axes, i));
        need(v >= 0 && v < n_axes);
        p.axis[i] = (unsigned char)v;
      }
    }
    need((wq_ == Py_None) == (wk_ == Py_None));
    p.w_dtype = GBS_F32;
    if (wq_ != Py_None) {
      const at::Tensor& w = on_device(wq_, device);
      p.w_dtype = act(w);
      wq = dense_ptr(wq_, device, w.scalar_type(), {d});
      wk = dense_ptr(wk_, device, w.scalar_type(), {d});
    }
    p.B = whole(B); p.N = whole(N); p.Hq = whole(Hq); p.Hkv = whole(Hkv); p.d = whole(d);
    p.rot = (int)(2 * half); p.interleaved = yes(interleaved); p.n_axes = whole(n_axes); p.max_pos = whole(max_pos);
    p.eps = real(eps);
  }
};

// qkv_rope(q, k, v, cos, sin, pos, wq, wk, eps, axes, interleaved, out, ws)
PyObject* qkv_rope(const Library& lib, PyObject* const* a) {
  const RopeCall c(a[0], a[1], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10]);
  const at::Tensor& q = THPVariable_Unpack(a[0]);
  const bool values = a[2] != Py_None;
  gbs_heads v{}, oq, ok, ov{};
  if (values) v = heads_in(a[2], c.device, c.type, {c.B, c.N, c.Hkv, c.d}, true);
  void* ws = nullptr;
  if (a[12] != Py_None) {
    const at::Tensor& w = on_device(a[12], c.device);
    need(w.scalar_type() == at::kByte && w.is_contiguous() && w.numel() >= 256);
    ws = w.data_ptr();
  }
  PyObject* out[3];
  three(a[11], values, out);
  at::Tensor Q = result4(out[0], q, {c.B, c.Hq, c.N, c.d}), K = result4(out[1], q, {c.B, c.Hkv, c.N, c.d}), V;
  oq = heads_of(Q, false);
  ok = heads_of(K, false);
  if (values) ov = heads_of(V = result4(out[2], q, {c.B, c.Hkv, c.N, c.d}), false);
  return returned(lib.rope_fwd(&c.p, &c.q, &c.k, values ? &v : nullptr, c.wq, c.wk, (const float*)c.cos,
                               (const float*)c.sin, (const int32_t*)c.pos, &oq, &ok, values ? &ov : nullptr, ws,
                               stream_of(c.device)),
                  {Q, K, V});
}

// qkv_rope_backward(q, k, cos, sin, pos, dQ, dK, dV, wq, wk, eps, axes, interleaved, grads, ws)
PyObject* qkv_rope_backward(const Library& lib, PyObject* const* a) {
  const RopeCall c(a[0], a[1], a[2], a[3], a[4], a[8], a[9], a[10], a[11], a[12]);
  const at::Tensor& q = THPVariable_Unpack(a[0]);
  const bool values = a[7] != Py_None;
  const gbs_heads zq = heads_in(a[5], c.device, c.type, {c.B, c.Hq, c.N, c.d}, false);
  const gbs_heads zk = heads_in(a[6], c.device, c.type, {c.B, c.Hkv, c.N, c.d}, false);
  gbs_heads zv{}, oq, ok, ov{};
  if (values) zv = heads_in(a[7], c.device, c.type, {c.B, c.Hkv, c.N, c.d}, false);
  PyObject* out[3];
  three(a[13], values, out);
  at::Tensor ws;
  if (a[14] != Py_None) {
    ws = on_device(a[14], c.device);
    need(ws.scalar_type() == at::kByte && ws.is_contiguous());
  }
  at::Tensor dq = result4(out[0], q, {c.B, c.N, c.Hq, c.d}), dk = result4(out[1], q, {c.B, c.N, c.Hkv, c.d}), dv;
  oq = heads_of(dq, true);
  ok = heads_of(dk, true);
  if (values) ov = heads_of(dv = result4(out[2], q, {c.B, c.N, c.Hkv, c.d}), true);
  at::Tensor dwq, dwk;
  if (c.wq) {
    dwq = at::empty({c.d}, q.options().dtype(at::kFloat));
    dwk = at::empty({c.d}, q.options().dtype(at::kFloat));
  }
  if (!ws.defined()) {
    const size_t bytes = lib.rope_bytes(&c.p);
    ws = at::empty({(int64_t)(bytes ? bytes : 256)}, q.options().dtype(at::kByte));
  }
  return returned(lib.rope_bwd(&c.p, &c.q, &c.k, c.wq, c.wk, (const float*)c.cos, (const float*)c.sin,
                               (const int32_t*)c.pos, &zq, &zk, values ? &zv : nullptr, &oq, &ok,
                               values ? &ov : nullptr, c.wq ? dwq.data_ptr<float>() : nullptr,
                               c.wq ? dwk.data_ptr<float>() : nullptr, ws.data_ptr(), (size_t)ws.numel(),
                               stream_of(c.device)),
                  {dq, dk, dv, dwq, dwk});
}

struct CacheCall {
  gbs_kv4_cache c{};
  int64_t Hkv, d, most;  // most: the longest length that fits

  CacheCall(PyObject* cache, int64_t B, int device, int block, PyObject* table) {
    need(listed(cache, 4) && block > 0);
    PyObject* const* t = PySequence_Fast_ITEMS(cache);
    const at::Tensor& kc = on_device(t[0], device);
    need(kc.dim() == 4);
    const int64_t first = kc.size(0), rows = kc.size(2);
    Hkv = kc.size(1);
    d = 2 * kc.size(3);
    need(table == Py_None ? first == B && rows % block == 0 : rows == block);
    c.kc = dense_ptr(t[0], device, at::kByte, {first, Hkv, rows, d / 2});
    c.kp = dense_ptr(t[1], device, at::kHalf, {first, Hkv, rows, d / 32, 2});
    c.vc = dense_ptr(t[2], device, at::kByte, {first, Hkv, rows, d / 2});
    c.vp = dense_ptr(t[3], device, at::kHalf, {first, Hkv, rows, d / 32, 2});
    c.cap = whole(rows);
    most = rows;
    if (table != Py_None) {
      const at::Tensor& x = on_device(table, device);
      need(x.dim() == 2 && x.size(0) == B && x.scalar_type() == at::kInt && x.is_contiguous());
      c.block_table = x.data_ptr<int32_t>();
      c.max_blocks = whole(x.size(1));
      c.num_pages = whole(first);
      most = std::min<int64_t>(x.size(1) * block, INT32_MAX);  // positions are int32
    }
  }
};

// What append and read share, from their tensors on.
int rows_call(decltype(&gbs_kv4_append) fn, const at::Tensor& K, const at::Tensor& V, PyObject* cache, PyObject* start,
              PyObject* table, PyObject* count, PyObject* block_, PyObject* ws_) {
  const int device = K.get_device(), block = whole(block_);
  const int64_t B = K.size(0), T = K.size(2);
  const CacheCall c(cache, B, device, block, table);
  const int64_t shape[4] = {B, c.Hkv, T, c.d};
  need(K.sizes() == Sizes(shape) && V.sizes() == Sizes(shape) && V.scalar_type() == K.scalar_type() && T > 0);
  const gbs_heads hk = heads_of(K, false), hv = heads_of(V, false);
  void* ws = nullptr;
  if (ws_ != Py_None) {
    const at::Tensor& w = on_device(ws_, device);
    need(w.scalar_type() == at::kByte && w.is_contiguous() && w.numel() >= 256);
    ws = w.data_ptr();
  }
  const int h = whole(c.Hkv);
  const gbs_params p = {whole(B), h, h, whole(c.most), whole(c.d), block, 0, 0, act(K), 0.f, 0.f};
  return fn(&p, &c.c, &hk, &hv, whole(T), (const int32_t*)dense_ptr(start, device, at::kInt, {B}),
            (const int32_t*)optional_ptr(count, device, at::kInt, {B}), ws, stream_of(device));
}

// kv4_append(K, V, cache, start, block_table, count, block, ws)
PyObject* kv4_append(const Library& lib, PyObject* const* a) {
  const at::Tensor& K = anchor(a[0]);
  const at::Tensor& V = on_device(a[1], K.get_device());
  need(K.dim() == 4);
  return returned(rows_call(lib.append, K, V, a[2], a[3], a[4], a[5], a[6], a[7]), {});
}

// kv4_read(cache, start, T, block_table, count, dtype, block, out, ws), out None
PyObject* kv4_read(const Library& lib, PyObject* const* a) {
  const at::Tensor& start = anchor(a[1]);
  need(a[7] == Py_None && THPDtype_Check(a[5]) && listed(a[0], 4));
  const auto type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
  const at::Tensor& kc = on_device(PySequence_Fast_GET_ITEM(a[0], 0), start.get_device());
  const int T = whole(a[2]);
  need(kc.dim() == 4 && start.dim() == 1 && T > 0 && (type == at::kBFloat16 || type == at::kFloat));
  const int64_t shape[4] = {start.size(0), kc.size(1), T, 2 * kc.size(3)};
  const at::Tensor K = at::empty(shape, start.options().dtype(type)), V = at::empty(shape, start.options().dtype(type));
  return returned(rows_call(lib.read, K, V, a[0], a[1], a[3], a[4], a[6], a[8]), {K, V});
}

// kv4_decode(q, cache, S, L, block, topk, scale, num_splits, block_table, seq_lens,
//            group_shared, out, lse, ws, tau)
PyObject* kv4_decode(const Library& lib, PyObject* const* a) {
  const at::Tensor& q = anchor(a[0]);
  need(q.dim() == 3 && q.is_contiguous());
  const int device = q.get_device(), L = whole(a[3]), block = whole(a[4]), dtype = act(q), shared = yes(a[10]);
  const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2);
  const CacheCall c(a[1], B, device, block, a[8]);
  need(c.d == d && L >= 1 && L <= c.most);
  const void* S = dense_ptr(a[2], device, at::kFloat, {B, shared ? c.Hkv : Hq, (L + (int64_t)block - 1) / block});
  const void* lens = optional_ptr(a[9], device, at::kInt, {B});
  const gbs_params p = {whole(B), whole(Hq), whole(c.Hkv), L, whole(d), block, whole(a[5]),
                        a[14] == Py_None ? GBS_SPARSE : GBS_THRESHOLD, dtype, real(a[6]), a[14] == Py_None ? 0.f : real(a[14])};
  const int splits = whole(a[7]);
  at::Tensor ws;
  if (a[13] != Py_None) {
    ws = on_device(a[13], device);
    need(ws.scalar_type() == at::kByte && ws.is_contiguous());
  }
  const at::Tensor O = result(a[11], q, q.scalar_type(), {B, Hq, d}), lse = result(a[12], q, at::kFloat, {B, Hq});
  if (!ws.defined()) {
    const size_t bytes = lib.decode_bytes(&p);
    ws = at::empty({(int64_t)(bytes ? bytes : 256)}, q.options().dtype(at::kByte));
  }
  return returned(lib.decode(&p, &c.c, (const int32_t*)lens, shared, q.data_ptr(), (const float*)S, O.data_ptr(),
                             lse.data_ptr<float>(), splits, ws.data_ptr(), (size_t)ws.numel(), stream_of(device)),
                  {O, lse});
}

template <typename F>
PyCFunction method(F* f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"fits", method(fits), METH_FASTCALL, "whether a tensor plainly has a device, dtype and shape"},
    {"heads", method(heads), METH_FASTCALL, "gbs_heads of a tensor as bytes, or None"},
    {"qkv_rope", method(guarded<13, qkv_rope>), METH_FASTCALL, "the call, or None"},
    {"qkv_rope_backward", method(guarded<15, qkv_rope_backward>), METH_FASTCALL, "the call, or None"},
    {"kv4_append", method(guarded<8, kv4_append>), METH_FASTCALL, "the call, or None"},
    {"kv4_read", method(guarded<9, kv4_read>), METH_FASTCALL, "the call, or None"},
    {"kv4_decode", method(guarded<15, kv4_decode>), METH_FASTCALL, "the call, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
