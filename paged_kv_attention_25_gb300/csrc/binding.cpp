// Python side of the calls that read their metadata on the device (trees,
// selected blocks, pages): checks of the tensors, outputs and workspaces that
// are not given, the stream.  The GPU part of a small call is shorter than its
// checks in Python and ctypes would be (attention over selected blocks: 17.5 us of
// host time a call there, 4.3 here, 2 of them the launch).
//
// Tensors live on the pool's device.  Without a stream a call runs on that
// device's current one.  What is not given is allocated for that stream; the
// workspace of calls on a current stream is kept with the pool, one for each
// stream, as calls on one stream follow one another.  A call that is being
// captured, or that names a stream, gets a workspace of its own (a captured
// graph keeps it), and so does one on a stream that torch does not own: such a
// stream may be destroyed while its work runs, and another come back under its
// handle.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <new>
#include <optional>
#include <string>
#include <unordered_map>

#include "pkv.h"

namespace {

PyObject* g_error = nullptr;   // PkvError

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& msg) {
  PyErr_SetString(type, msg.c_str());
  throw Raised{};
}

void check(int rc) {
  if (rc == PKV_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", rc, pkv_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// A library call, without the interpreter's lock: it may wait for the pool's (another thread's plan of a batch).
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};
template <class... P, class... A>
void run(int (*call)(P...), A... args) {   // (the arguments are made, and refused, with the lock)
  int rc;
  {
    const Unlocked unlocked;
    rc = call(args...);
  }
  check(rc);
}

struct Pool {
  PyObject_HEAD
  pkv_pool* handle;
  int device;
  int64_t num_blocks, num_kv_heads, head_dim;
  std::unordered_map<cudaStream_t, at::Tensor>* buf;   // workspaces of the current streams
};

// One call's stream, and where its outputs are allocated.
class Call {
 public:
  Call(Pool* pool, PyObject* stream) : pool_(pool), given_(stream != Py_None) {
    if (given_) {
      PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
      if (!raw) throw Raised{};
      stream_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
      Py_DECREF(raw);
      if (PyErr_Occurred()) throw Raised{};
    } else {
      const c10::cuda::CUDAStream s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(pool->device));
      stream_ = s.stream();
      // (torch's own have small ids, others their handle for an id)
      foreign_ = stream_ && static_cast<uint64_t>(s.id()) == reinterpret_cast<uintptr_t>(stream_);
    }
  }
  void* stream() const { return stream_; }

  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    const at::Device device(at::kCUDA, static_cast<c10::DeviceIndex>(pool_->device));
    if (!given_) return at::detail::empty_cuda(shape, type, device, std::nullopt);
    const c10::cuda::CUDAStreamGuard guard(
        c10::cuda::getStreamFromExternal(stream_, static_cast<c10::DeviceIndex>(pool_->device)));
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
  }

  // `size` bytes: the caller's tensor (any size: the library checks it), the pool's, or a new one.
  // (Held by the call: another thread's may replace the pool's while this one runs.)
  at::Tensor workspace(PyObject* given, size_t size);

 private:
  Pool* pool_;
  bool given_, foreign_ = false;
  cudaStream_t stream_ = nullptr;
};

const at::Tensor& tensor(PyObject* o, const char* name, int64_t dims) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != dims) raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dims) + " dimensions");
  return t;
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "int32";
    case at::kChar: return "int8";
    case at::kByte: return "uint8";
    case at::kBFloat16: return "bfloat16";
    default: return "float32";
  }
}

// The address of a contiguous tensor of this type and shape on the pool's device.
template <class T = void>
T* address(const Pool* pool, PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  const bool is = THPVariable_Check(o);
  if (!is || !THPVariable_Unpack(o).is_cuda() || THPVariable_Unpack(o).scalar_type() != type ||
      !THPVariable_Unpack(o).is_contiguous())
    raise(PyExc_TypeError, std::string(name) + " must be a contiguous " + type_name(type) + " CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.get_device() != pool->device) raise(PyExc_ValueError, std::string(name) + " must be on the pool's device");
  if (t.sizes() != shape) {
    std::string s;
    for (const int64_t x : shape) s += (s.empty() ? "" : ", ") + std::to_string(x);
    raise(PyExc_ValueError, std::string(name) + " must have shape (" + s + ")");
  }
  return static_cast<T*>(t.data_ptr());
}

at::Tensor Call::workspace(PyObject* given, size_t size) {
  if (given != Py_None) {
    const at::Tensor& t = tensor(given, "workspace", 1);
    address(pool_, given, "workspace", at::kByte, t.sizes());
    return t;
  }
  const int64_t n = static_cast<int64_t>(size);
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  const bool kept = !given_ && !foreign_;
  if (kept) {
    const cudaError_t e = cudaStreamIsCapturing(stream_, &capturing);
    if (e != cudaSuccess) raise(PyExc_RuntimeError, std::string("cudaStreamIsCapturing: ") + cudaGetErrorString(e));
  }
  if (!kept || capturing != cudaStreamCaptureStatusNone) return make({n}, at::kByte);
  at::Tensor& t = (*pool_->buf)[stream_];
  if (!t.defined() || t.numel() < n) t = make({n}, at::kByte);
  return t;
}

int count(int64_t n) {   // a size for the library's int arguments
  if (n > INT_MAX) raise(PyExc_ValueError, "a size exceeds 2^31 - 1");
  return static_cast<int>(n);
}
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < INT_MIN || v > INT_MAX) raise(PyExc_ValueError, "an argument exceeds 32 bits");
  return static_cast<int>(v);
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

// Requests, table width, and the addresses of the tables and of cu.
struct Batch {
  int64_t reqs, width;
  const int32_t *tables, *cu;
  Batch(const Pool* pool, PyObject* block_tables, PyObject* cu_q_lens, const char* cu_name) {
    reqs = tensor(cu_q_lens, cu_name, 1).size(0) - 1;
    if (reqs < 0) raise(PyExc_ValueError, std::string(cu_name) + " must hold num_reqs + 1 entries");
    width = tensor(block_tables, "block_tables", 2).size(1);
    tables = address<int32_t>(pool, block_tables, "block_tables", at::kInt, {reqs, width});
    cu = address<int32_t>(pool, cu_q_lens, cu_name, at::kInt, {reqs + 1});
  }
};

struct Summary {
  int8_t *codes, *exps;
  Summary(const Pool* pool, PyObject* c, PyObject* e) {
    const int64_t nb = pool->num_blocks, hkv = pool->num_kv_heads;
    codes = address<int8_t>(pool, c, "summary.codes", at::kChar, {nb, hkv, 2, pool->head_dim});
    exps = address<int8_t>(pool, e, "summary.exps", at::kChar, {nb, hkv});
  }
};

// Queries, and O and LSE, made if they are not given.
struct Query {
  int64_t tokens, heads;
  const void* q;
  Query(const Pool* pool, PyObject* o) {
    const at::Tensor& t = tensor(o, "q", 3);
    tokens = t.size(0);
    heads = t.size(1);
    q = address(pool, o, "q", at::kBFloat16, {tokens, heads, pool->head_dim});
  }
};
struct Output {
  at::Tensor made_o, made_lse;
  PyObject *given_o, *given_lse;
  void* o;
  float* lse = nullptr;
  Output(const Pool* pool, const Call& call, const Query& q, PyObject* out, PyObject* lse_in, bool want_lse)
      : given_o(out), given_lse(lse_in) {
    const int64_t shape[3] = {q.tokens, q.heads, pool->head_dim};
    if (out == Py_None) {
      made_o = call.make(shape, at::kBFloat16);
      o = made_o.data_ptr();
    } else {
      o = address(pool, out, "out", at::kBFloat16, shape);
    }
    if (lse_in != Py_None) {
      lse = address<float>(pool, lse_in, "lse", at::kFloat, {q.tokens, q.heads});
    } else if (want_lse) {
      made_lse = call.make({q.tokens, q.heads}, at::kFloat);
      lse = static_cast<float*>(made_lse.data_ptr());
    }
  }
  PyObject* result() {
    PyObject* a = made_o.defined() ? THPVariable_Wrap(std::move(made_o)) : Py_NewRef(given_o);
    PyObject* b = made_lse.defined() ? THPVariable_Wrap(std::move(made_lse)) : Py_NewRef(given_lse);
    PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
  }
};

// An output tensor that is not a query's: given, or made.
struct Table {
  at::Tensor made;
  PyObject* given;
  void* data;
  int32_t* at;   // data as int32
  Table(const Pool* pool, const Call& call, PyObject* o, const char* name, at::IntArrayRef shape,
        at::ScalarType type = at::kInt)
      : given(o) {
    if (o == Py_None) {
      made = call.make(shape, type);
      data = made.data_ptr();
    } else {
      data = address(pool, o, name, type, shape);
    }
    at = static_cast<int32_t*>(data);
  }
  PyObject* result() { return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(given); }
};

using Args = PyObject* const*;

// parents, cu_q_lens, mask_words or None, max_nodes or None, out or None, stream or None
PyObject* tree_mask(Pool* p, Args a) {
  const int64_t T = tensor(a[0], "parents", 1).size(0);
  const int32_t* parents = address<int32_t>(p, a[0], "parents", at::kInt, {T});
  const int64_t R = tensor(a[1], "cu_q_lens", 1).size(0) - 1;
  const int32_t* cu = address<int32_t>(p, a[1], "cu_q_lens", at::kInt, {R + 1});
  const Call call(p, a[5]);
  int64_t words;
  if (a[4] != Py_None) {
    words = tensor(a[4], "out", 2).size(1);
  } else if (a[2] != Py_None) {
    words = integer(a[2]);
  } else {
    const int64_t nodes = a[3] != Py_None ? integer(a[3]) : 0;
    words = std::max<int64_t>(1, ((nodes ? nodes : T) + 31) / 32);
  }
  if (words < 0) raise(PyExc_ValueError, "mask_words must be >= 0");
  Table out(p, call, a[4], "out", {T, words});
  run(pkv_tree_mask, p->handle, parents, cu, count(R), count(T), reinterpret_cast<uint32_t*>(out.at), count(words),
      call.stream());
  return out.result();
}

// q, block_tables, ctx_lens, prefix_lens, cu_q_lens, tree_mask, scale, out, lse, workspace, stream, want_lse
PyObject* tree_attn(Pool* p, Args a) {
  const Batch b(p, a[1], a[4], "cu_q_lens");
  const Query q(p, a[0]);
  const int64_t words = tensor(a[5], "tree_mask", 2).size(1);
  const int32_t* ctx = address<int32_t>(p, a[2], "ctx_lens", at::kInt, {b.reqs});
  const int32_t* prefix = address<int32_t>(p, a[3], "prefix_lens", at::kInt, {b.reqs});
  const int32_t* mask = address<int32_t>(p, a[5], "tree_mask", at::kInt, {q.tokens, words});
  const float scale = number(a[6]);
  Call call(p, a[10]);
  Output out(p, call, q, a[7], a[8], a[11] == Py_True);
  size_t size = 0;
  check(pkv_tree_attn_workspace_size(p->handle, count(q.heads), count(b.width), count(b.reqs), count(q.tokens), &size));
  const at::Tensor ws = call.workspace(a[9], size);
  run(pkv_tree_attn, p->handle, q.q, count(q.heads), b.tables, count(b.width), ctx, prefix, b.cu, count(b.reqs),
      count(q.tokens), reinterpret_cast<const uint32_t*>(mask), count(words), scale, out.o, out.lse, ws.data_ptr(),
      static_cast<size_t>(ws.numel()), call.stream());
  return out.result();
}

// codes, exps, block_tables, cu_q_lens, positions, ctx_lens, stream
PyObject* summarize(Pool* p, Args a) {
  const Batch b(p, a[2], a[3], "cu_q_lens");
  const int64_t T = tensor(a[4], "positions", 1).size(0);
  const int32_t* pos = address<int32_t>(p, a[4], "positions", at::kInt, {T});
  const int32_t* ctx = address<int32_t>(p, a[5], "ctx_lens", at::kInt, {b.reqs});
  const Summary s(p, a[0], a[1]);
  const Call call(p, a[6]);
  run(pkv_summarize, p->handle, b.tables, count(b.width), count(b.reqs), b.cu, pos, ctx, count(T), s.codes, s.exps,
      call.stream());
  Py_RETURN_NONE;
}

// codes, exps, q, q_positions, block_tables, cu_q_lens, top_k, sinks, recent, out, workspace, stream
PyObject* select_blocks(Pool* p, Args a) {
  const Batch b(p, a[4], a[5], "cu_q_lens");
  const Query q(p, a[2]);
  const int32_t* pos = address<int32_t>(p, a[3], "q_positions", at::kInt, {q.tokens});
  const int top_k = integer(a[6]), sinks = integer(a[7]), recent = integer(a[8]);
  if (top_k < 1) raise(PyExc_ValueError, "top_k must be >= 1");
  const Summary s(p, a[0], a[1]);
  Call call(p, a[11]);
  Table out(p, call, a[9], "out", {q.tokens, p->num_kv_heads, top_k});
  size_t size = 0;
  check(pkv_select_blocks_workspace_size(p->handle, count(b.width), count(q.tokens), &size));
  const at::Tensor ws = call.workspace(a[10], size);
  run(pkv_select_blocks, p->handle, q.q, count(q.heads), pos, b.tables, count(b.width), b.cu, count(b.reqs),
      count(q.tokens), s.codes, s.exps, top_k, sinks, recent, out.at, ws.data_ptr(), static_cast<size_t>(ws.numel()),
      call.stream());
  return out.result();
}

// q, q_positions, block_tables, cu_q_lens, selected, scale, out, lse, workspace, stream, want_lse
PyObject* sparse_attn(Pool* p, Args a) {
  const Batch b(p, a[2], a[3], "cu_q_lens");
  const Query q(p, a[0]);
  const int32_t* pos = address<int32_t>(p, a[1], "q_positions", at::kInt, {q.tokens});
  const int64_t k = tensor(a[4], "selected", 3).size(2);
  const int32_t* sel = address<int32_t>(p, a[4], "selected", at::kInt, {q.tokens, p->num_kv_heads, k});
  const float scale = number(a[5]);
  Call call(p, a[9]);
  Output out(p, call, q, a[6], a[7], a[10] == Py_True);
  size_t size = 0;
  check(pkv_sparse_attn_workspace_size(p->handle, &size));
  const at::Tensor ws = call.workspace(a[8], size);
  run(pkv_sparse_attn, p->handle, q.q, count(q.heads), pos, b.tables, count(b.width), b.cu, count(b.reqs),
      count(q.tokens), sel, count(k), scale, out.o, out.lse, ws.data_ptr(), static_cast<size_t>(ws.numel()),
      call.stream());
  return out.result();
}

// tables, lens, caps, parents, new_caps, refs, out_tables, out_refs, codes, exps, workspace, stream
PyObject* fork(Pool* p, Args a) {
  const at::Tensor& t = tensor(a[0], "tables", 2);
  const int64_t R = t.size(0), width = t.size(1), N = tensor(a[3], "parents", 1).size(0);
  const int32_t* tables = address<int32_t>(p, a[0], "tables", at::kInt, {R, width});
  const int32_t* lens = address<int32_t>(p, a[1], "lens", at::kInt, {R});
  const int32_t* caps = address<int32_t>(p, a[2], "caps", at::kInt, {R});
  const int32_t* parents = address<int32_t>(p, a[3], "parents", at::kInt, {N});
  const int32_t* new_caps = address<int32_t>(p, a[4], "new_caps", at::kInt, {N});
  const int32_t* refs = address<int32_t>(p, a[5], "refs", at::kInt, {p->num_blocks});
  PyObject* refs_out = a[7] == Py_None ? a[5] : a[7];
  int32_t* out_refs = address<int32_t>(p, refs_out, "out_refs", at::kInt, {p->num_blocks});
  std::optional<Summary> s;
  if (a[8] != Py_None || a[9] != Py_None) s.emplace(p, a[8], a[9]);
  Call call(p, a[11]);
  Table out(p, call, a[6], "out_tables", {N, width});
  size_t size = 0;
  check(pkv_fork_workspace_size(p->handle, count(R), count(N), &size));
  const at::Tensor ws = call.workspace(a[10], size);
  run(pkv_fork, p->handle, tables, count(R), count(width), lens, caps, parents, new_caps, count(N), out.at, refs,
      out_refs, s ? s->codes : nullptr, s ? s->exps : nullptr, ws.data_ptr(), static_cast<size_t>(ws.numel()),
      call.stream());
  PyObject* made = out.result();
  if (!made) return nullptr;
  PyObject* r = PyTuple_Pack(2, made, refs_out);
  Py_DECREF(made);
  return r;
}

// src, dst, codes, exps, stream
PyObject* copy_blocks(Pool* p, Args a) {
  const int64_t n = tensor(a[0], "src", 1).size(0);
  const int32_t* src = address<int32_t>(p, a[0], "src", at::kInt, {n});
  const int32_t* dst = address<int32_t>(p, a[1], "dst", at::kInt, {n});
  std::optional<Summary> s;
  if (a[2] != Py_None || a[3] != Py_None) s.emplace(p, a[2], a[3]);
  const Call call(p, a[4]);
  run(pkv_copy_blocks, p->handle, src, dst, count(n), s ? s->codes : nullptr, s ? s->exps : nullptr, call.stream());
  Py_RETURN_NONE;
}

// block_tables, cu_keep, src_positions, dst_starts, stream
PyObject* compact(Pool* p, Args a) {
  const Batch b(p, a[0], a[1], "cu_keep");
  const int64_t n = tensor(a[2], "src_positions", 1).size(0);
  const int32_t* src = address<int32_t>(p, a[2], "src_positions", at::kInt, {n});
  const int32_t* dst = address<int32_t>(p, a[3], "dst_starts", at::kInt, {b.reqs});
  const Call call(p, a[4]);
  run(pkv_compact, p->handle, b.tables, count(b.width), count(b.reqs), b.cu, src, dst, count(n), call.stream());
  Py_RETURN_NONE;
}

#include "binding_score.h"

// codes, exps
PyObject* check_summary(Pool* p, Args a) {
  const Summary s(p, a[0], a[1]);
  (void)s;
  Py_RETURN_NONE;
}

// The pool has been destroyed: calls are refused from now on.
PyObject* close(Pool* p, Args) {
  p->handle = nullptr;
  p->buf->clear();
  Py_RETURN_NONE;
}

template <PyObject* (*F)(Pool*, Args), Py_ssize_t N>
PyObject* method(PyObject* self, Args args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", N, n);
    return nullptr;
  }
  try {
    return F(reinterpret_cast<Pool*>(self), args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(Pool*, Args), Py_ssize_t N>
PyMethodDef entry(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&method<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {entry<tree_mask, 6>("tree_mask"),         entry<tree_attn, 12>("tree_attn"),
                          entry<summarize, 7>("summarize"),         entry<select_blocks, 12>("select_blocks"),
                          entry<sparse_attn, 11>("sparse_attn"),    entry<fork, 12>("fork"),
                          entry<copy_blocks, 5>("copy_blocks"),     entry<compact, 5>("compact"),
                          entry<check_summary, 2>("check_summary"), entry<close, 0>("close"),
                          entry<append_int8, 7>("append_int8"),     entry<read_rows, 6>("read_rows"),
                          entry<score_attn, 16>("score_attn"),
                          {nullptr, nullptr, 0, nullptr}};

// Pool(handle, device, num_blocks, num_kv_heads, head_dim)
PyObject* pool_new(PyTypeObject* type, PyObject* args, PyObject*) {
  unsigned long long handle;
  int device;
  long long nb, hkv, d;
  if (!PyArg_ParseTuple(args, "KiLLL", &handle, &device, &nb, &hkv, &d)) return nullptr;
  Pool* p = reinterpret_cast<Pool*>(type->tp_alloc(type, 0));
  if (!p) return nullptr;
  p->handle = reinterpret_cast<pkv_pool*>(static_cast<uintptr_t>(handle));
  p->device = device;
  p->num_blocks = nb;
  p->num_kv_heads = hkv;
  p->head_dim = d;
  p->buf = new (std::nothrow) std::unordered_map<cudaStream_t, at::Tensor>();
  if (!p->buf) {
    Py_DECREF(p);
    return PyErr_NoMemory();
  }
  return reinterpret_cast<PyObject*>(p);
}

void pool_dealloc(PyObject* self) {
  delete reinterpret_cast<Pool*>(self)->buf;
  Py_TYPE(self)->tp_free(self);
}

PyTypeObject pool_type() {
  PyTypeObject t = {PyVarObject_HEAD_INIT(nullptr, 0)};
  t.tp_name = "pkv_binding.Pool";
  t.tp_basicsize = sizeof(Pool);
  t.tp_dealloc = pool_dealloc;
  t.tp_flags = Py_TPFLAGS_DEFAULT;
  t.tp_methods = kMethods;
  t.tp_new = pool_new;
  return t;
}
PyTypeObject g_pool_type = pool_type();

// The exception class of a refused call, PkvError(code, message).
PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XSETREF(g_error, Py_NewRef(cls));
  Py_RETURN_NONE;
}

PyMethodDef kModuleMethods[] = {{"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "pkv_binding", nullptr, -1, kModuleMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pkv_binding() {
  if (PyType_Ready(&g_pool_type) < 0) return nullptr;
  PyObject* m = PyModule_Create(&kModule);
  if (!m) return nullptr;
  if (PyModule_AddObjectRef(m, "Pool", reinterpret_cast<PyObject*>(&g_pool_type)) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
