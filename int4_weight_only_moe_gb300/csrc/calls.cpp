// Python calls of the order, gather, combine, gradients and adapters without ctypes: tensors'
// types, shapes and devices are read where they stand, and the C entry is called. A call that
// is not plainly right (a wrong type, another device, a subclass of tensors, a function
// transform's tensor without storage) returns None: the Python code that calls this checks it
// step by step and says what is wrong. A small call takes 4 us, 3 of them the launch; 8 to 11
// with the checks in Python.
//
// A tensor's methods may throw (its address, where it has no storage). They are called with
// the interpreter's lock held, all of them in front of the C entry, which alone runs without it.
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/moe_w4a16.h"

namespace {

struct Call {
  long dev;
  void* stream;
  bool ok = true;

  // The tensor of a strided tensor on the device, or null.
  const at::Tensor* tensor(PyObject* o) {
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev) return fail();
    // (a null address would stand for an optional tensor that is not given)
    if (!t.data_ptr() && t.numel() > 0) return fail();
    return &t;
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  bool need(bool right) { return ok = ok && right; }

  // Address of a contiguous tensor of this type and shape.
  template <typename T>
  T* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(o);
    if (!t || !need(t->scalar_type() == type && t->is_contiguous() && t->sizes() == at::IntArrayRef(shape))) return nullptr;
    return static_cast<T*>(t->data_ptr());
  }
  template <typename T>
  T* dense_or_none(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return o == Py_None ? nullptr : dense<T>(o, type, shape);
  }
  // Element type of the C interface, -1 for others.
  static int type_of(const at::Tensor& t, bool moved = false) {
    switch (t.scalar_type()) {
      case at::kFloat: return MOE_W4A16_F32;
      case at::kBFloat16: return MOE_W4A16_BF16;
      case at::kByte:
      case at::kFloat8_e4m3fn: return moved ? MOE_W4A16_E4M3 : -1;
      default: return -1;
    }
  }
  // A matrix whose rows are contiguous and do not overlap.
  const at::Tensor* rows(PyObject* o, long long* stride) {
    const at::Tensor* t = tensor(o);
    if (!t || !need(t->dim() == 2)) return nullptr;
    *stride = t->stride(0);
    if (!need((t->stride(1) == 1 || t->size(1) <= 1) && (*stride >= t->size(1) || t->size(0) <= 1))) return nullptr;
    *stride = std::max<long long>(*stride, t->size(1));
    return t;
  }
  const at::Tensor* matrix(PyObject* o) {
    const at::Tensor* t = tensor(o);
    return t && need(t->dim() == 2 && t->is_contiguous() && type_of(*t) >= 0) ? t : fail();
  }
};

constexpr int64_t kInt = 0x7FFFFFFF;

// `run` with the device and stream of the first two arguments; None where it is not `ok`.
template <typename F>
PyObject* with(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F&& run) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  const long dev = PyLong_AsLong(args[0]);
  void* stream = PyLong_AsVoidPtr(args[1]);
  if (PyErr_Occurred()) return nullptr;
  Call c{dev, stream};
  int rc = 0;
  try {
    rc = run(c);
  } catch (...) {
    c.ok = false;
  }
  if (PyErr_Occurred()) return nullptr;
  if (!c.ok) Py_RETURN_NONE;
  return PyLong_FromLong(rc);
}

// `entry`, a C entry that knows nothing of Python, without the interpreter's lock.
template <typename F, typename... Args>
int unlocked(F* entry, Args... args) {
  struct Lock {
    PyThreadState* const state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return entry(args...);
}

int int_of(Call& c, PyObject* o) {
  const long v = PyLong_AsLong(o);
  c.need(v >= -kInt && v <= kInt && !PyErr_Occurred());
  return static_cast<int>(v);
}

struct OrderArgs {
  int32_t *offsets, *slots, *position;
  int64_t M, topk, E, rows, block;
};
// An order's tensors, and the block that its number of rows says.
bool order_of(Call& c, PyObject* offsets, PyObject* slots, PyObject* position, OrderArgs* o) {
  const at::Tensor *a = c.tensor(offsets), *b = c.tensor(slots), *p = c.tensor(position);
  if (!a || !b || !p || !c.need(a->dim() == 1 && b->dim() == 1 && p->dim() == 2)) return false;
  o->E = a->size(0) - 1, o->rows = b->size(0), o->M = p->size(0), o->topk = p->size(1);
  const int64_t n = o->M * o->topk;
  if (!c.need(o->E >= 1 && n >= 1 && o->rows >= n && o->E <= kInt && o->M <= kInt && o->topk <= kInt)) return false;
  o->block = (o->rows - n) / std::min(o->E, n) + 1;
  if (!c.need(o->block <= kInt && moe_w4a16_dispatch_rows(static_cast<int>(o->M), static_cast<int>(o->topk), static_cast<int>(o->E),
                                                          static_cast<int>(o->block)) == o->rows))
    return false;
  o->offsets = c.dense<int32_t>(offsets, at::kInt, {o->E + 1});
  o->slots = c.dense<int32_t>(slots, at::kInt, {o->rows});
  o->position = c.dense<int32_t>(position, at::kInt, {o->M, o->topk});
  return c.ok;
}

// (device, stream, x, offsets, slots, position, out)
PyObject* gather(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return with(v, n, 7, [&](Call& c) {
    long long stride;
    OrderArgs o;
    const at::Tensor* x = c.rows(v[2], &stride);
    if (!x || !order_of(c, v[3], v[4], v[5], &o) || !c.need(Call::type_of(*x, true) >= 0 && x->size(0) == o.M && x->size(1) <= kInt)) return 0;
    void* out = c.dense<void>(v[6], x->scalar_type(), {o.rows, x->size(1)});
    if (!c.ok) return 0;
    return unlocked(moe_w4a16_dispatch_gather, x->data_ptr(), Call::type_of(*x, true), stride, o.offsets, o.slots, o.position, out,
                    static_cast<int>(o.M), static_cast<int>(x->size(1)), static_cast<int>(o.topk), static_cast<int>(o.E),
                    static_cast<int>(o.block), c.stream);
  });
}

// (device, stream, x, ids, E, first expert, block, offsets, slots, position, out)
PyObject* sort_gather(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return with(v, n, 11, [&](Call& c) {
    long long stride;
    const at::Tensor *x = c.rows(v[2], &stride), *ids = c.tensor(v[3]);
    const int E = int_of(c, v[4]), begin = int_of(c, v[5]), block = int_of(c, v[6]);
    if (!x || !ids || !c.need(Call::type_of(*x, true) >= 0 && ids->dim() == 2 && x->size(1) <= kInt && ids->size(0) <= kInt &&
                              ids->size(1) <= kInt && x->size(0) == ids->size(0)))
      return 0;
    const int M = static_cast<int>(ids->size(0)), topk = static_cast<int>(ids->size(1));
    const long long rows = moe_w4a16_dispatch_rows(M, topk, E, block);
    if (!c.need(rows >= 0)) return 0;
    const auto* at = c.dense<int32_t>(v[3], at::kInt, {M, topk});
    auto* offsets = c.dense<int32_t>(v[7], at::kInt, {E + 1});
    auto* slots = c.dense<int32_t>(v[8], at::kInt, {rows});
    auto* position = c.dense<int32_t>(v[9], at::kInt, {M, topk});
    void* out = c.dense<void>(v[10], x->scalar_type(), {rows, x->size(1)});
    if (!c.ok) return 0;
    return unlocked(moe_w4a16_dispatch_sort_gather, x->data_ptr(), Call::type_of(*x, true), stride, at, M, static_cast<int>(x->size(1)),
                    topk, begin, E, block, offsets, slots, position, out, c.stream);
  });
}

// (device, stream, y, weights or None, slots, position, add or None, out)
PyObject* combine(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return with(v, n, 8, [&](Call& c) {
    const at::Tensor *y = c.matrix(v[2]), *slots = c.tensor(v[4]), *position = c.tensor(v[5]), *out = c.matrix(v[7]);
    if (!y || !slots || !position || !out || !c.need(slots->dim() == 1 && position->dim() == 2 && y->size(0) == slots->size(0))) return 0;
    const int64_t M = position->size(0), topk = position->size(1), K = y->size(1), rows = y->size(0);
    if (!c.need(M <= kInt && topk <= kInt && K <= kInt && rows <= kInt && out->size(0) == M && out->size(1) == K)) return 0;
    const auto* at = c.dense<int32_t>(v[5], at::kInt, {M, topk});
    const auto* w = c.dense_or_none<float>(v[3], at::kFloat, {M, topk});
    const void* add = c.dense_or_none<void>(v[6], out->scalar_type(), {M, K});
    if (!c.ok) return 0;
    return unlocked(moe_w4a16_combine, y->data_ptr(), Call::type_of(*y), w, at, add, out->data_ptr(), Call::type_of(*out),
                    static_cast<int>(M), static_cast<int>(K), static_cast<int>(topk), static_cast<int>(rows), c.stream);
  });
}

// (device, stream, dout, y, weights, offsets, slots, position, dy, dweights)
PyObject* combine_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return with(v, n, 10, [&](Call& c) {
    OrderArgs o;
    const at::Tensor *g = c.matrix(v[2]), *y = c.matrix(v[3]);
    if (!g || !y || !order_of(c, v[5], v[6], v[7], &o)) return 0;
    const int64_t K = g->size(1);
    if (!c.need(g->size(0) == o.M && y->size(0) == o.rows && y->size(1) == K && K <= kInt)) return 0;
    const auto* w = c.dense<float>(v[4], at::kFloat, {o.M, o.topk});
    void* dy = c.dense<void>(v[8], y->scalar_type(), {o.rows, K});
    auto* dw = c.dense<float>(v[9], at::kFloat, {o.M, o.topk});
    if (!c.ok) return 0;
    return unlocked(moe_w4a16_combine_backward, g->data_ptr(), Call::type_of(*g), y->data_ptr(), Call::type_of(*y), w, o.offsets,
                    o.slots, o.position, dy, dw, static_cast<int>(o.M), static_cast<int>(K), static_cast<int>(o.topk),
                    static_cast<int>(o.E), static_cast<int>(o.block), c.stream);
  });
}

// (device, stream, dweights, logits, ids, scoring, renormalize, scale, out)
PyObject* route_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return with(v, n, 9, [&](Call& c) {
    long long stride;
    const at::Tensor *l = c.rows(v[3], &stride), *ids = c.tensor(v[4]);
    const int scoring = int_of(c, v[5]), renormalize = PyObject_IsTrue(v[6]);
    const double scale = PyFloat_AsDouble(v[7]);
    if (!l || !ids || !c.need(!PyErr_Occurred() && renormalize >= 0 && ids->dim() == 2 && Call::type_of(*l) >= 0 && l->size(0) <= kInt &&
                              l->size(1) <= kInt && ids->size(1) <= kInt))
      return 0;
    const int64_t M = l->size(0), E = l->size(1), topk = ids->size(1);
    const auto* at = c.dense<int32_t>(v[4], at::kInt, {M, topk});
    const auto* g = c.dense<float>(v[2], at::kFloat, {M, topk});
    void* out = c.dense<void>(v[8], l->scalar_type(), {M, E});
    if (!c.ok) return 0;
    return unlocked(moe_w4a16_route_scored_backward, g, l->data_ptr(), Call::type_of(*l), stride, at, static_cast<int>(M),
                    static_cast<int>(E), static_cast<int>(topk), scoring, renormalize, static_cast<float>(scale), out, c.stream);
  });
}

// (device, stream, x, a, b, index, add or None, scale or None, out, most bytes of a workspace)
PyObject* lora(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return with(v, n, 10, [&](Call& c) {
    long long stride;
    const at::Tensor *x = c.rows(v[2], &stride), *a = c.tensor(v[3]), *b = c.tensor(v[4]), *out = c.matrix(v[8]);
    if (!x || !a || !b || !out || !c.need(x->scalar_type() == at::kBFloat16 && a->dim() == 3 && b->dim() == 3)) return 0;
    const int64_t M = x->size(0), K = x->size(1), L = a->size(0), r = a->size(1), N = b->size(1);
    if (!c.need(M <= kInt && K <= kInt && L <= kInt && r <= kInt && N <= kInt && out->size(0) == M && out->size(1) == N)) return 0;
    const auto* pa = c.dense<uint16_t>(v[3], at::kBFloat16, {L, r, K});
    const auto* pb = c.dense<uint16_t>(v[4], at::kBFloat16, {L, N, r});
    const auto* index = c.dense<int32_t>(v[5], at::kInt, {M});
    const at::Tensor* add = v[6] == Py_None ? nullptr : c.matrix(v[6]);
    const auto* scale = c.dense_or_none<float>(v[7], at::kFloat, {L});
    const size_t most = PyLong_AsSize_t(v[9]);
    if (!c.need(!add || (add->size(0) == M && add->size(1) == N)) || PyErr_Occurred()) return 0;
    const int m = static_cast<int>(M), k = static_cast<int>(K), nn = static_cast<int>(N), rr = static_cast<int>(r), l = static_cast<int>(L);
    if (!c.need(moe_w4a16_lora_workspace_size(m, k, nn, rr, l) <= most)) return 0;
    return unlocked(moe_w4a16_lora, static_cast<const uint16_t*>(x->data_ptr()), stride, pa, pb, scale, index,
                    add ? add->data_ptr() : nullptr, add ? Call::type_of(*add) : MOE_W4A16_F32, out->data_ptr(), Call::type_of(*out), m,
                    k, nn, rr, l, nullptr, size_t{0}, c.stream);
  });
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"gather", fast<gather>(), METH_FASTCALL, nullptr},
                         {"sort_gather", fast<sort_gather>(), METH_FASTCALL, nullptr},
                         {"combine", fast<combine>(), METH_FASTCALL, nullptr},
                         {"combine_backward", fast<combine_backward>(), METH_FASTCALL, nullptr},
                         {"route_backward", fast<route_backward>(), METH_FASTCALL, nullptr},
                         {"lora", fast<lora>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "moe_w4a16_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_moe_w4a16_calls() { return PyModule_Create(&module); }
