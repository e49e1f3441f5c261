// wq_calls.cpp -- the KV cache calls of wq.py, from torch tensors to the C ABI: checks, outputs, the call.
//
// A call of few tokens costs the host more than the GPU: through ctypes, with its outputs allocated from Python, an attention
// call took 13 us of the host's time against 7 of the GPU's, here 5 (a call that is given its outputs 2.5).  wq.py hands over the
// cache (address of its wq_kv_cache, and what is checked against it), the device and the stream; a failed check raises
// AssertionError, a status other than WQ_OK comes back as an int, which wq.py raises.  Built beside libwq.so, whose functions it
// gets by their addresses.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ops/empty.h>
#include <cmath>
#include <initializer_list>

#include "../../include/wq.h"

namespace {

struct Lib {
  decltype(&wq_attend) attend;
  decltype(&wq_attend_ex) attend_ex;
  decltype(&wq_attend_workspace_bytes) workspace;
  decltype(&wq_attend_ex_workspace_bytes) ex_workspace;
  decltype(&wq_kv_append) append;
  decltype(&wq_kv_append_slots) append_slots;
  decltype(&wq_kv_read) read;
  decltype(&wq_kv_reserve) reserve;
  decltype(&wq_kv_release) release;
  decltype(&wq_kv_keep) keep;
  decltype(&wq_tree_mask_ex) tree_mask;
} lib;

// The leading arguments of every call: (cache address, heads, dim, batch, device, stream).
struct Where {
  const wq_kv_cache* cache;
  int64_t heads, dim, batch, device;
  void* stream;
};
constexpr int kLead = 6;

// Other threads of the interpreter run while memory is allocated or a launch waits for room in its queue.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

struct Refused {
  const char* what;
};
void want(bool ok, const char* what) {
  if (!ok) throw Refused{what};
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
const at::Tensor& tensor(PyObject* o) {
  want(THPVariable_Check(o), "a tensor is expected");
  return THPVariable_Unpack(o);
}
Where where(PyObject* const* a) {
  return Where{reinterpret_cast<const wq_kv_cache*>(PyLong_AsVoidPtr(a[0])), integer(a[1]), integer(a[2]), integer(a[3]), integer(a[4]),
               PyLong_AsVoidPtr(a[5])};
}
void placed(const Where& w, const at::Tensor& t, at::ScalarType type) {
  want(t.is_cuda() && t.get_device() == w.device, "a tensor is not on the cache's device");
  want(t.scalar_type() == type, "a tensor has another type than is taken");
}
// [batch, token, head, dim] view, dim contiguous; other strides as they are.
wq_heads heads_of(const Where& w, const at::Tensor& t, at::ScalarType type) {
  placed(w, t, type);
  want(t.stride(3) == 1, "the elements of a head are not contiguous");
  return wq_heads{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}
// A contiguous tensor of n values, or NULL.
template <class T>
T* values(const Where& w, PyObject* o, int64_t n, at::ScalarType type) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  placed(w, t, type);
  want(t.is_contiguous() && t.numel() == n, "a tensor of lengths, numbers or slots has another size or layout than is taken");
  return static_cast<T*>(t.data_ptr());
}
int32_t* ints(const Where& w, PyObject* o, int64_t n) { return values<int32_t>(w, o, n, at::kInt); }

at::TensorOptions on(const Where& w, at::ScalarType type) {
  return at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(w.device));
}
at::Tensor empty(at::IntArrayRef sizes, const Where& w, at::ScalarType type) {
  const Unlocked unlocked;
  return at::empty(sizes, on(w, type));
}
// An allocation costs as much as the launch, so outputs that are made together and are small lie in one: contiguous tensors over
// parts of it, each from a multiple of 16 bytes on.  It lives as long as one of them does, so what is larger has an allocation of
// its own: a log-sum-exp or a few counts that are kept hold no output and no slot map alive.  (A reservation of 256 prompts, whose
// map is 13 MB, then takes 2 us more of the host's time, beside 16 of the GPU's.)
constexpr int64_t kSmall = 65536;     // bytes
class Together {
 public:
  // What will be made, in this order.
  Together(const Where& w, std::initializer_list<int64_t> bytes) : w_(w) {
    for (const int64_t n : bytes) room_ += n <= kSmall ? rounded(n) : 0;
  }
  at::Tensor make(at::ScalarType type, at::IntArrayRef sizes) {
    const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
    const int64_t bytes = c10::multiply_integers(sizes) * static_cast<int64_t>(meta.itemsize());
    if (bytes > kSmall) return empty(sizes, w_, type);
    if (!whole_.defined()) whole_ = empty({room_}, w_, at::kByte);
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole_.storage()), whole_.key_set(), meta);
    t.unsafeGetTensorImpl()->set_storage_offset(from_ / static_cast<int64_t>(meta.itemsize()));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    from_ += rounded(bytes);
    return t;
  }

 private:
  static int64_t rounded(int64_t n) { return (n + 15) / 16 * 16; }
  const Where& w_;
  int64_t room_ = 0, from_ = 0;
  at::Tensor whole_;
};
// A function of libwq.
template <class F, class... Args>
auto run(F* f, Args... args) {
  const Unlocked unlocked;
  return f(args...);
}

PyObject* done(int rc) {
  if (rc != WQ_OK) return PyLong_FromLong(rc);
  Py_RETURN_NONE;
}
PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b), *t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

// (q, lens, counts, causal, window, scale, max_len, out, out_f32, return_lse, workspace, sinks, mask, depth)
PyObject* attend(const Where& w, PyObject* const* a) {
  const at::Tensor& q = tensor(a[0]);
  want(q.dim() == 4, "q is [batch, tokens, q_heads, dim]");
  const int64_t batch = q.size(0), tokens = q.size(1), q_heads = q.size(2), dim = q.size(3);
  want(dim == w.dim && batch <= w.batch, "q's heads are not of the cache's size, or more sequences than it has");
  const at::ScalarType type = truth(a[8]) ? at::kFloat : at::kBFloat16;
  const bool tree = a[12] != Py_None;
  const int64_t sinks = integer(a[11]), window = integer(a[4]), max_len = integer(a[6]);
  const bool sel = tree || sinks != 0;
  const wq_heads qh = heads_of(w, q, at::kBFloat16);
  const int32_t *lens = ints(w, a[1], batch), *counts = ints(w, a[2], batch);
  wq_tree t{};
  if (tree) {
    const at::Tensor& mask = tensor(a[12]);
    placed(w, mask, at::kInt);
    want(mask.dim() == 3 && mask.is_contiguous() && mask.size(1) == tokens && mask.size(2) == (tokens + 31) / 32 &&
             (mask.size(0) == 1 || mask.size(0) == batch), "the mask is [batch or 1, tokens, ceil(tokens / 32)]");
    t.mask = static_cast<const uint32_t*>(mask.data_ptr());
    t.mask_batch = mask.size(0) == batch ? tokens * mask.size(2) : 0;
    if (a[13] != Py_None) {
      const at::Tensor& depth = tensor(a[13]);
      placed(w, depth, at::kInt);
      want(depth.dim() == 2 && depth.is_contiguous() && depth.size(1) == tokens && (depth.size(0) == 1 || depth.size(0) == batch),
           "the depths are [batch or 1, tokens]");
      t.depth = static_cast<const int32_t*>(depth.data_ptr());
      t.depth_batch = depth.size(0) == batch ? tokens : 0;
    }
  }
  float scale;
  if (a[5] == Py_None) {
    scale = static_cast<float>(std::pow(static_cast<double>(dim), -0.5));
  } else {
    const double v = PyFloat_AsDouble(a[5]);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    scale = static_cast<float>(v);
  }
  const bool wants_lse = truth(a[9]);
  at::Tensor out, lse;
  if (a[7] == Py_None && wants_lse) {
    Together both(w, {q.numel() * (type == at::kFloat ? 4 : 2), batch * tokens * q_heads * 4});
    out = both.make(type, q.sizes());
    lse = both.make(at::kFloat, {batch, tokens, q_heads});
  } else if (a[7] == Py_None) {
    out = empty(q.sizes(), w, type);
  } else {
    out = tensor(a[7]);
    want(out.sizes() == q.sizes(), "out has another shape than q");
  }
  const wq_heads oh = heads_of(w, out, type);
  at::Tensor workspace;
  if (wants_lse && !lse.defined()) lse = empty({batch, tokens, q_heads}, w, at::kFloat);
  if (a[10] == Py_None) {
    const size_t need = (sel ? lib.ex_workspace : lib.workspace)(w.cache, batch, tokens, q_heads, max_len);
    if (need) workspace = empty({static_cast<int64_t>(need)}, w, at::kByte);
  } else {
    workspace = tensor(a[10]);
    placed(w, workspace, at::kByte);
    want(workspace.is_contiguous(), "the workspace is not contiguous");
  }
  float* lse_at = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
  void* work = workspace.defined() ? workspace.data_ptr() : nullptr;
  const size_t bytes = workspace.defined() ? workspace.numel() : 0;
  const unsigned flags = (truth(a[3]) ? WQ_FLAG_CAUSAL : 0u) | (type == at::kFloat ? WQ_FLAG_OUT_F32 : 0u);
  const int rc = sel ? run(lib.attend_ex, w.cache, &qh, &oh, lse_at, batch, tokens, q_heads, lens, counts, max_len, scale, window, sinks,
                                     tree ? &t : nullptr, flags, work, bytes, w.stream)
                     : run(lib.attend, w.cache, &qh, &oh, lse_at, batch, tokens, q_heads, lens, counts, max_len, scale, window, flags, work,
                                  bytes, w.stream);
  if (rc != WQ_OK) return PyLong_FromLong(rc);
  if (lse.defined()) return pair(out, lse);
  return THPVariable_Wrap(out);
}

// (k, v, start, counts)
PyObject* append(const Where& w, PyObject* const* a) {
  const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
  want(k.dim() == 4 && v.sizes() == k.sizes() && k.size(2) == w.heads && k.size(3) == w.dim && k.size(0) <= w.batch,
       "k and v are [batch, tokens, heads, dim], of the cache's heads and at most its sequences");
  const wq_heads kh = heads_of(w, k, at::kBFloat16), vh = heads_of(w, v, at::kBFloat16);
  return done(run(lib.append, w.cache, &kh, &vh, k.size(0), k.size(1), ints(w, a[2], k.size(0)), ints(w, a[3], k.size(0)), w.stream));
}

// (k, v, slots)
PyObject* append_slots(const Where& w, PyObject* const* a) {
  const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
  want(k.dim() == 3 && v.sizes() == k.sizes() && k.size(1) == w.heads && k.size(2) == w.dim, "k and v are [tokens, heads, dim], of the cache's heads");
  placed(w, k, at::kBFloat16);
  placed(w, v, at::kBFloat16);
  want(k.stride(2) == 1 && v.stride(2) == 1, "the elements of a head are not contiguous");
  want(a[2] != Py_None, "slots are expected");
  const wq_heads kh{k.data_ptr(), 0, k.stride(0), k.stride(1)}, vh{v.data_ptr(), 0, v.stride(0), v.stride(1)};
  return done(run(lib.append_slots, w.cache, &kh, &vh, k.size(0), values<int64_t>(w, a[2], k.size(0), at::kLong), w.stream));
}

// (tokens, start, counts, out_f32, batch)
PyObject* read(const Where& w, PyObject* const* a) {
  const int64_t tokens = integer(a[0]), batch = integer(a[4]);
  want(batch <= w.batch, "more sequences than the cache has");
  const at::ScalarType type = truth(a[3]) ? at::kFloat : at::kBFloat16;
  const int32_t *start = ints(w, a[1], batch), *counts = ints(w, a[2], batch);
  const at::Tensor k = empty({batch, tokens, w.heads, w.dim}, w, type), v = empty({batch, tokens, w.heads, w.dim}, w, type);
  const wq_heads kh = heads_of(w, k, type), vh = heads_of(w, v, type);
  const int rc = run(lib.read, w.cache, &kh, &vh, batch, tokens, start, counts, type == at::kFloat ? WQ_FLAG_OUT_F32 : 0u, w.stream);
  return rc != WQ_OK ? PyLong_FromLong(rc) : pair(k, v);
}

struct Turn {
  int32_t *free, *top, *top_out;
  const int32_t* lens;
  int64_t size, batch;
};
// (free, top, lens, ..., top_out)
Turn turn(const Where& w, PyObject* free, PyObject* top, PyObject* lens, PyObject* top_out) {
  want(w.cache->table != nullptr, "the cache has no table");
  const int64_t batch = tensor(lens).numel(), size = tensor(free).numel();
  want(batch <= w.batch, "the table has not that many rows");
  Turn t{ints(w, free, size), ints(w, top, 1), ints(w, top_out, 1), ints(w, lens, batch), size, batch};
  want(t.top != nullptr, "top is expected");
  if (!t.top_out) t.top_out = t.top;
  return t;
}

// (free, top, lens, counts, tokens, top_out, out)
PyObject* reserve(const Where& w, PyObject* const* a) {
  const Turn t = turn(w, a[0], a[1], a[2], a[5]);
  const int64_t tokens = integer(a[4]);
  const int32_t* counts = ints(w, a[3], t.batch);
  PyObject* out = a[6];
  if (out == Py_None) {
    want(tokens >= 0, "tokens is negative");
    Together four(w, {8 * tokens, 4 * tokens, 4 * (t.batch + 1), 4 * t.batch});
    const at::Tensor made[4] = {four.make(at::kLong, {tokens}), four.make(at::kInt, {tokens}), four.make(at::kInt, {t.batch + 1}),
                                four.make(at::kInt, {t.batch})};
    out = PyTuple_New(4);
    if (!out) throw python_error();
    for (int i = 0; i < 4; ++i) {
      PyObject* x = THPVariable_Wrap(made[i]);
      if (!x) {
        Py_DECREF(out);
        throw python_error();
      }
      PyTuple_SET_ITEM(out, i, x);
    }
  } else {
    want(PyTuple_Check(out) && PyTuple_GET_SIZE(out) == 4, "out is (slots, positions, starts, granted)");
    Py_INCREF(out);
  }
  THPObjectPtr held(out);
  int64_t* slots = values<int64_t>(w, PyTuple_GET_ITEM(out, 0), tokens, at::kLong);
  int32_t *positions = ints(w, PyTuple_GET_ITEM(out, 1), tokens), *starts = ints(w, PyTuple_GET_ITEM(out, 2), t.batch + 1);
  int32_t* granted = ints(w, PyTuple_GET_ITEM(out, 3), t.batch);
  const int rc = run(lib.reserve, w.cache, t.free, t.size, t.top, t.top_out, t.batch, t.lens, counts, granted, tokens, slots, positions, starts,
                             w.stream);
  return rc != WQ_OK ? PyLong_FromLong(rc) : held.release();
}

// (free, top, lens, keep, top_out)
PyObject* release(const Where& w, PyObject* const* a) {
  const Turn t = turn(w, a[0], a[1], a[2], a[4]);
  return done(run(lib.release, w.cache, t.free, t.size, t.top, t.top_out, t.batch, t.lens, ints(w, a[3], t.batch), w.stream));
}

// (start, path, counts)
PyObject* keep(const Where& w, PyObject* const* a) {
  const at::Tensor& path = tensor(a[1]);
  want(path.dim() == 2 && path.size(0) <= w.batch, "path is [batch, n], of at most the cache's sequences");
  const int64_t batch = path.size(0);
  return done(run(lib.keep, w.cache, ints(w, a[0], batch), batch, ints(w, a[1], path.numel()), path.size(1), ints(w, a[2], batch), w.stream));
}

// (parents, counts, window, sinks, lens); no cache
PyObject* tree_mask_ex(const Where& w, PyObject* const* a) {
  const at::Tensor& parents = tensor(a[0]);
  want(parents.dim() == 2, "parents is [batch, tokens]");
  const int64_t batch = parents.size(0), tokens = parents.size(1), window = integer(a[2]), sinks = integer(a[3]);
  const int32_t *up = ints(w, a[0], parents.numel()), *counts = ints(w, a[1], batch), *lens = ints(w, a[4], batch);
  const int64_t words = (tokens + 31) / 32;
  Together both(w, {batch * tokens * words * 4, batch * tokens * 4});
  const at::Tensor mask = both.make(at::kInt, {batch, tokens, words}), depth = both.make(at::kInt, {batch, tokens});
  const int rc = run(lib.tree_mask, up, batch, tokens, counts, window, sinks, lens, static_cast<uint32_t*>(mask.data_ptr()),
                               static_cast<int32_t*>(depth.data_ptr()), w.stream);
  return rc != WQ_OK ? PyLong_FromLong(rc) : pair(mask, depth);
}
// (parents, counts, window)
PyObject* tree_mask(const Where& w, PyObject* const* a) {
  THPObjectPtr none(PyLong_FromLong(0));
  if (!none.get()) throw python_error();
  PyObject* const all[5] = {a[0], a[1], a[2], none.get(), Py_None};
  return tree_mask_ex(w, all);
}

template <PyObject* (*F)(const Where&, PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kLead + N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    const Where w = where(args);
    if (PyErr_Occurred()) return nullptr;
    return F(w, args + kLead);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_AssertionError, r.what);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// Addresses of libwq's functions, in the order of Lib.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n * sizeof(void*) != sizeof(Lib)) {
    PyErr_SetString(PyExc_TypeError, "wrong number of functions");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    void* p = PyLong_AsVoidPtr(args[i]);
    if (!p) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function is missing");
      return nullptr;
    }
    reinterpret_cast<void**>(&lib)[i] = p;
  }
  Py_RETURN_NONE;
}

template <PyObject* (*F)(const Where&, PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<F, N>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&bind)), METH_FASTCALL, nullptr},
    method<attend, 14>("attend"),
    method<append, 4>("append"),
    method<append_slots, 3>("append_slots"),
    method<read, 5>("read"),
    method<reserve, 7>("reserve"),
    method<release, 5>("release"),
    method<keep, 3>("keep"),
    method<tree_mask, 3>("tree_mask"),
    method<tree_mask_ex, 5>("tree_mask_ex"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_wq_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__wq_calls(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", WQ_CALLS_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
