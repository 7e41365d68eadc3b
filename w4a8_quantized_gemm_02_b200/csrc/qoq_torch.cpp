// The calls of one decode step from torch tensors to the C ABI: the paged cache and
// the adapters.
//
// These kernels run a few microseconds, less than a call through ctypes takes: its
// checks, tensor by tensor, and the marshalling of 23 arguments came to 12 us of
// host time, the launches to 2 to 3 us each.  Here the checks read the tensors'
// fields.  A call whose arguments are all as the kernels take them, on the current
// device and its current stream, is made from here.  Any other returns None, and the
// Python function makes it the long way: that is where errors are put into words.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <limits.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "qoq.h"

namespace {

using at::Tensor;

// A plain tensor, null for anything else (None and subclasses among them).
const Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool fits(int64_t v) { return v >= 0 && v <= INT_MAX; }

// The device of a call: the current one.
struct Where {
  int device = -1;
  bool set(const Tensor* t) {
    if (!t || !t->is_cuda()) return false;
    device = t->get_device();
    return device == c10::cuda::current_device();
  }
  bool on(const Tensor* t, at::ScalarType type) const {
    return t && t->is_cuda() && t->scalar_type() == type && t->get_device() == device;
  }
  // a contiguous tensor of that type and shape
  bool is(const Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    return on(t, type) && t->sizes() == at::IntArrayRef(shape) && t->is_contiguous();
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

// Rows of `width` contiguous elements of a tensor of 2 or 3 dimensions: elements
// between rows, or -1.
int64_t row_step(const Tensor& t, int64_t width) {
  const int64_t n = t.dim();
  if (n != 2 && n != 3) return -1;
  int64_t at = 1;
  for (int64_t d = n - 1; d > 0; --d) {
    if (t.size(d) != 1 && t.stride(d) != at) return -1;
    at *= t.size(d);
  }
  if (at != width) return -1;
  const int64_t ld = t.size(0) > 1 ? t.stride(0) : width;
  return ld >= width && ld % 8 == 0 ? ld : -1;
}

struct Batch {
  const Tensor *kc, *vc, *sc, *q_start, *seqlen, *table;
  int pages, Hkv, page, B, width;
  // cache, q_start, seqlen and block_table, in the arguments' order
  bool set(PyObject* const* args, const Where& w) {
    if (!PyTuple_CheckExact(args[0]) || PyTuple_GET_SIZE(args[0]) != 3) return false;
    kc = tensor(PyTuple_GET_ITEM(args[0], 0));
    vc = tensor(PyTuple_GET_ITEM(args[0], 1));
    sc = tensor(PyTuple_GET_ITEM(args[0], 2));
    q_start = tensor(args[1]);
    seqlen = tensor(args[2]);
    table = tensor(args[3]);
    if (!w.on(sc, at::kHalf) || sc->dim() != 4 || !w.on(table, at::kInt) || table->dim() != 2)
      return false;
    const int64_t p = sc->size(0), h = sc->size(1), n = sc->size(2), b = table->size(0);
    if (!fits(p) || !fits(h) || !fits(n) || n % 16 != 0 || !fits(b) || !fits(table->size(1)))
      return false;
    pages = static_cast<int>(p);
    Hkv = static_cast<int>(h);
    page = static_cast<int>(n);
    B = static_cast<int>(b);
    width = static_cast<int>(table->size(1));
    return w.is(sc, at::kHalf, {p, h, n, 4}) && w.is(kc, at::kByte, {p, h, n / 16, 1024}) &&
           w.is(vc, at::kByte, {p, h, n / 16, 1024}) && table->is_contiguous() &&
           w.is(seqlen, at::kInt, {b}) && w.is(q_start, at::kInt, {b + 1});
  }
};

// A workspace: the caller's, or `need` bytes.
bool workspace(PyObject* given, const Where& w, const Tensor& like, size_t need, Tensor& ws) {
  if (given != Py_None) {
    const Tensor* t = tensor(given);
    if (!w.on(t, at::kByte) || !t->is_contiguous()) return false;
    ws = *t;
    return true;
  }
  ws = at::empty({static_cast<int64_t>(need)}, like.options().dtype(at::kByte));
  return true;
}

// `given`, or a new tensor of that shape like `like`; null: not as the kernels take it.
bool output(PyObject* given, const Where& w, const Tensor& like,
            std::initializer_list<int64_t> shape, Tensor& out) {
  if (given == Py_None) {
    out = at::empty(at::IntArrayRef(shape), like.options());
    return true;
  }
  const Tensor* t = tensor(given);
  if (!w.is(t, at::kHalf, shape)) return false;
  out = *t;
  return true;
}

bool integer(PyObject* o, int& v) {
  if (!PyLong_CheckExact(o)) return false;
  int overflow = 0;
  const long x = PyLong_AsLongAndOverflow(o, &overflow);
  if (overflow || x < 0 || x > INT_MAX) return false;
  v = static_cast<int>(x);
  return true;
}

// The interpreter's lock is free while the launches are made.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

PyObject* give(PyObject* given, Tensor&& out) {
  return given == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(given);
}

// (qkv, cache, q_start, seqlen, block_table, Hq, inv_freq, interleaved, factor, q_out, values)
PyObject* append(PyObject* const* args) {
  const Tensor* qkv = tensor(args[0]);
  Where w;
  Batch b;
  int Hq = 0, inter = 0;
  if (!w.set(qkv) || qkv->scalar_type() != at::kHalf || !b.set(args + 1, w) ||
      !integer(args[5], Hq) || !integer(args[7], inter) || !PyFloat_CheckExact(args[8]))
    Py_RETURN_NONE;
  const int64_t T = qkv->dim() ? qkv->size(0) : -1;
  if (!fits(T)) Py_RETURN_NONE;
  const int64_t ld = row_step(*qkv, (static_cast<int64_t>(Hq) + 2 * b.Hkv) * 128);
  if (ld < 0) Py_RETURN_NONE;
  const double* freq = nullptr;
  int rot = 0;
  if (args[6] != Py_None) {
    const Tensor* f = tensor(args[6]);
    if (!w.on(f, at::kDouble) || f->dim() != 1 || !f->is_contiguous() || f->size(0) > 64)
      Py_RETURN_NONE;
    freq = static_cast<const double*>(f->data_ptr());
    rot = 2 * static_cast<int>(f->size(0));
  }
  void *kh = nullptr, *vh = nullptr;
  if (args[10] != Py_None) {
    if (!PyTuple_CheckExact(args[10]) || PyTuple_GET_SIZE(args[10]) != 2) Py_RETURN_NONE;
    const Tensor* k = tensor(PyTuple_GET_ITEM(args[10], 0));
    const Tensor* v = tensor(PyTuple_GET_ITEM(args[10], 1));
    if (!w.is(k, at::kHalf, {T, b.Hkv, 128}) || !w.is(v, at::kHalf, {T, b.Hkv, 128}))
      Py_RETURN_NONE;
    kh = k->data_ptr();
    vh = v->data_ptr();
  }
  Tensor q;
  if (!output(args[9], w, *qkv, {T, Hq, 128}, q)) Py_RETURN_NONE;
  int st = 0;
  {
    const Unlocked unlocked;
    st = qoq_kv4_paged_append(
        qkv->data_ptr(), static_cast<size_t>(ld), static_cast<int>(T), Hq, b.Hkv, 128,
        static_cast<const int*>(b.q_start->data_ptr()), static_cast<const int*>(b.seqlen->data_ptr()),
        b.B, static_cast<const int*>(b.table->data_ptr()), b.width, b.pages, b.page, freq, rot, inter,
        PyFloat_AS_DOUBLE(args[8]), q.data_ptr(), static_cast<uint8_t*>(b.kc->data_ptr()),
        static_cast<uint8_t*>(b.vc->data_ptr()), b.sc->data_ptr(), kh, vh, w.stream());
  }
  if (st) Py_RETURN_NONE;
  return give(args[9], std::move(q));
}

// (Q, cache, q_start, seqlen, block_table, max_q, scale, out, ws)
PyObject* attention(PyObject* const* args) {
  const Tensor* Q = tensor(args[0]);
  Where w;
  Batch b;
  if (!w.set(Q) || Q->scalar_type() != at::kHalf || Q->dim() != 3 || Q->size(2) != 128 ||
      !b.set(args + 1, w) || !PyFloat_CheckExact(args[6]))
    Py_RETURN_NONE;
  const int64_t T = Q->size(0), Hq = Q->size(1);
  if (!fits(T) || !fits(Hq)) Py_RETURN_NONE;
  const int64_t ld = row_step(*Q, Hq * 128);
  int max_q = T > 0 ? static_cast<int>(T) : 1;
  if (ld < 0 || (args[5] != Py_None && !integer(args[5], max_q))) Py_RETURN_NONE;
  const int t = static_cast<int>(T), h = static_cast<int>(Hq);
  Tensor out, ws;
  if (!output(args[7], w, *Q, {T, Hq, 128}, out)) Py_RETURN_NONE;
  const size_t need = args[8] != Py_None ? 0
      : qoq_kv4_paged_attention_workspace_bytes(t, h, b.Hkv, 128, b.B, b.width, b.page, max_q);
  if (!workspace(args[8], w, *Q, need, ws)) Py_RETURN_NONE;
  int st = 0;
  {
    const Unlocked unlocked;
    st = qoq_kv4_paged_attention(
        Q->data_ptr(), static_cast<size_t>(ld), t, h, b.Hkv, 128,
        static_cast<const uint8_t*>(b.kc->data_ptr()), static_cast<const uint8_t*>(b.vc->data_ptr()),
        b.sc->data_ptr(), static_cast<const int*>(b.q_start->data_ptr()),
        static_cast<const int*>(b.seqlen->data_ptr()), b.B,
        static_cast<const int*>(b.table->data_ptr()), b.width, b.pages, b.page, max_q,
        static_cast<float>(PyFloat_AS_DOUBLE(args[6])), out.data_ptr(), ws.data_ptr(),
        static_cast<size_t>(ws.numel()), w.stream());
  }
  if (st) Py_RETURN_NONE;
  return give(args[7], std::move(out));
}

// (Y, X, A, B, ids, scaling, out, ws)
PyObject* lora(PyObject* const* args) {
  const Tensor *Y = tensor(args[0]), *X = tensor(args[1]), *A = tensor(args[2]);
  const Tensor *Bm = tensor(args[3]), *ids = tensor(args[4]), *scaling = tensor(args[5]);
  Where w;
  if (!w.set(X) || X->dim() != 2 || !w.on(Bm, at::kHalf) || Bm->dim() != 3) Py_RETURN_NONE;
  const int64_t T = X->size(0), K = X->size(1), n = Bm->size(0), N = Bm->size(1), R = Bm->size(2);
  if (!fits(T) || !fits(K) || !fits(n) || !fits(N) || !fits(R) ||
      !w.is(X, at::kHalf, {T, K}) || !w.is(Y, at::kHalf, {T, N}) || !w.is(A, at::kHalf, {n, R, K}) ||
      !w.is(Bm, at::kHalf, {n, N, R}) || !w.is(ids, at::kInt, {T}) ||
      !w.is(scaling, at::kFloat, {n}))
    Py_RETURN_NONE;
  const int t = static_cast<int>(T), k = static_cast<int>(K), nn = static_cast<int>(N);
  const int r = static_cast<int>(R), a = static_cast<int>(n);
  Tensor out, ws;
  if (!output(args[6], w, *Y, {T, N}, out)) Py_RETURN_NONE;
  const size_t need = args[7] != Py_None ? 0 : qoq_lora_workspace_bytes(t, k, nn, r, a);
  if (!workspace(args[7], w, *X, need, ws)) Py_RETURN_NONE;
  int st = 0;
  {
    const Unlocked unlocked;
    st = qoq_lora_add(Y->data_ptr(), X->data_ptr(), t, k, nn, A->data_ptr(), Bm->data_ptr(), r, a,
                      static_cast<const int*>(ids->data_ptr()),
                      static_cast<const float*>(scaling->data_ptr()), out.data_ptr(), ws.data_ptr(),
                      static_cast<size_t>(ws.numel()), w.stream());
  }
  if (st) Py_RETURN_NONE;
  return give(args[6], std::move(out));
}

// No C++ exception (an allocation that fails, a tensor without storage) leaves here.
template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return kCall(args);
  } catch (const std::exception&) {
    Py_RETURN_NONE;
  }
}

#define ENTRY(name, call, args) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<call, args>)), \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    ENTRY("paged_append", append, 11),
    ENTRY("paged_attention", attention, 9),
    ENTRY("lora_add", lora, 8),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
