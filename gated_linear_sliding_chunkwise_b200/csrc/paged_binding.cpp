// Python entry of the paged cache (module _paged_call, used by paged.py):
// looks the tensors over, allocates outputs and workspaces with torch, packs
// the C structs and calls liblizard.so.
//
// A serving step makes these calls for every layer and token, and the smallest
// of them run for 10 us on the GPU: a pass of one token, host included, took
// 18.7 us with the same checks in Python on ctypes and takes 13.3 with these, a
// row's turnover (two calls) 20.2 and 13.6.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "../../include/lizard.h"

namespace {

using at::Tensor;

// What a caller did wrong, as the Python exception that says it.
struct Refusal {
  PyObject *type;
  std::string what;
};
[[noreturn]] void refuse(const std::string &what) { throw Refusal{PyExc_ValueError, what}; }

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// A tensor argument; null for None where that is allowed.
const Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return &THPVariable_Unpack(o);
}
void dims(const Tensor &t, const char *name, int64_t n, const char *layout) {
  if (t.dim() != n) refuse(std::string(name) + ": " + layout + " expected, got " + text(t.sizes()));
}
// The library takes pointers on 16-byte boundaries; a slice may begin elsewhere.
void aligned(const Tensor &t, const char *name) {
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15)
    refuse(std::string(name) + " must begin on a 16-byte boundary (clone the slice)");
}
// A contiguous tensor of this shape and type on the cache's device.
void fits(const Tensor *t, const char *name, at::IntArrayRef shape, at::ScalarType type, at::Device device) {
  if (!t) return;
  if (t->scalar_type() != type || t->sizes() != shape)
    refuse(std::string(name) + ": " + c10::toString(type) + " of shape " + text(shape) + " expected, got " +
           c10::toString(t->scalar_type()) + " " + text(t->sizes()));
  if (t->device() != device) refuse(std::string(name) + " is on " + t->device().str() + ", the cache on " + device.str());
  if (!t->is_contiguous()) refuse(std::string(name) + " must be contiguous");
  aligned(*t, name);
}
void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
int32_t *ints(const Tensor *t) { return static_cast<int32_t *>(ptr(t)); }
int type_code(at::ScalarType t) {
  if (t == at::kBFloat16) return LIZARD_BF16;
  if (t == at::kFloat) return LIZARD_FP32;
  throw Refusal{PyExc_TypeError, std::string("activations must be bf16 or fp32, got ") + c10::toString(t)};
}
int32_t number(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v > INT32_MAX || v < INT32_MIN) refuse(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}

// The call's device and stream, both made current: the device's current stream
// unless a handle is given.  So what is allocated for the call comes from the
// memory of the stream that it runs on: a block of the current stream may
// still be in use there, and would go back there while the other stream works.
struct Place {
  c10::cuda::CUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard on;
  c10::cuda::CUDAStream stream;
  Place(at::Device device, PyObject *handle)
      : guard(device), stream(c10::cuda::getCurrentCUDAStream(device.index())) {
    if (handle == Py_None) return;
    const unsigned long long h = PyLong_AsUnsignedLongLong(handle);
    if (PyErr_Occurred()) throw python_error();
    stream = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(h), device.index());
    on.reset_stream(stream);
  }
  lizard_stream_t handle() const { return reinterpret_cast<lizard_stream_t>(stream.stream()); }
};
// The caller's workspace, or one from torch's allocator.
Tensor space(const Tensor *given, size_t bytes, at::Device device) {
  if (given) {
    if (given->device() != device || !given->is_contiguous())
      refuse("workspace must be contiguous and on " + device.str());
    aligned(*given, "workspace");
    return *given;
  }
  return at::empty({(int64_t)(bytes > 256 ? bytes : 256)}, at::TensorOptions().dtype(at::kByte).device(device));
}
void cuda_only(at::Device device) {
  if (!device.is_cuda()) refuse("the cache must be on a CUDA device");
}

// Without the interpreter's lock while it lives: an allocation may wait for the
// device, and a launch for room in the stream's queue, which a callback of
// another thread's may have to make.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs f; what it throws becomes the Python exception.
template <typename F> PyObject *guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refusal &r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject *give(const Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

// attn(q, k, v, k_pages, v_pages, table, lens, cu_q, row, out, workspace, max_q, layer, window, sinks,
//      softmax_scale, want_lse, impl, stream) -> (status, o, lse, workspace)
PyObject *attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 19) throw Refusal{PyExc_TypeError, "attn takes 19 arguments"};
    const Tensor *q = tensor(a[0], "q"), *k = tensor(a[1], "k", true), *v = tensor(a[2], "v", true),
                 *kp = tensor(a[3], "k_pages"), *vp = tensor(a[4], "v_pages"), *table = tensor(a[5], "table"),
                 *lens = tensor(a[6], "lens"), *cu = tensor(a[7], "cu_q"), *row = tensor(a[8], "row", true),
                 *out = tensor(a[9], "out", true), *given = tensor(a[10], "workspace", true);
    lizard_paged_args c{};
    const at::ScalarType type = kp->scalar_type();
    const at::Device device = kp->device();
    c.dtype = type_code(type);
    dims(*kp, "k_pages", 5, "[layers, num_pages, Hkv, page, d]");
    dims(*q, "q", 3, "[T, H, d]");
    dims(*table, "table", 2, "[rows, max_pages]");
    dims(*cu, "cu_q", 1, "[B + 1]");
    if (cu->size(0) < 1) refuse("cu_q: [B + 1] expected, got nothing");
    const int64_t T = q->size(0), H = q->size(1), B = cu->size(0) - 1, Hkv = kp->size(2), d = kp->size(4),
                  rows = table->size(0);
    for (int64_t x : {T, H, B, rows, table->size(1), kp->size(0), kp->size(1), Hkv, kp->size(3), d})
      if (x > INT32_MAX) refuse("a size does not fit 32 bits");
    if (!k != !v) refuse("k and v go together");
    if (!row && B > rows)
      refuse(std::to_string(B) + " sequences, but the table has " + std::to_string(rows) + " rows");
    fits(q, "q", {T, H, d}, type, device);
    fits(k, "k", {T, Hkv, d}, type, device);
    fits(v, "v", {T, Hkv, d}, type, device);
    fits(kp, "k_pages", kp->sizes(), type, device);
    fits(vp, "v_pages", kp->sizes(), type, device);
    fits(table, "table", table->sizes(), at::kInt, device);
    fits(lens, "lens", {rows}, at::kInt, device);
    fits(cu, "cu_q", {B + 1}, at::kInt, device);
    fits(row, "row", {B}, at::kInt, device);
    fits(out, "out", {T, H, d}, type, device);
    c.layers = kp->size(0); c.num_pages = kp->size(1); c.Hkv = Hkv; c.page = kp->size(3); c.d = d;
    c.rows = rows; c.max_pages = table->size(1);
    c.B = B; c.T = T; c.H = H;
    c.max_q = number(a[11], "max_q"); c.layer = number(a[12], "layer");
    c.window = number(a[13], "window"); c.sinks = number(a[14], "sinks");
    c.softmax_scale = (float)PyFloat_AsDouble(a[15]);
    if (PyErr_Occurred()) throw python_error();
    const int want_lse = PyObject_IsTrue(a[16]);
    if (want_lse < 0) throw python_error();
    c.impl = number(a[17], "impl");
    cuda_only(device);
    const Place place(device, a[18]);
    Tensor o, lse, ws;
    lizard_status st;
    {
      const Unlocked unlocked;
      o = out ? *out : at::empty({T, H, d}, q->options());
      if (want_lse) lse = at::empty({T, H}, q->options().dtype(at::kFloat));
      ws = space(given, lizard_paged_attn_workspace_size(&c), device);
      c.q = ptr(q); c.k = ptr(k); c.v = ptr(v); c.k_pages = ptr(kp); c.v_pages = ptr(vp);
      c.table = ints(table); c.lens = ints(lens); c.cu_q = ints(cu); c.row = ints(row);
      c.o = ptr(&o);
      c.lse = lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr;
      c.workspace = ws.data_ptr();
      c.workspace_bytes = ws.nbytes();
      st = lizard_paged_attn(&c, place.handle());
    }
    return Py_BuildValue("(iNNN)", (int)st, give(o), give(lse), give(ws));
  });
}

// bookkeep(op, refs, table, lens, row, src, grow, page, k_pages, v_pages, table_out, refs_out, workspace, stream)
//   -> (status, table_out, refs_out, workspace); op: 0 reserve, 1 free, 2 fork, 3 compact
PyObject *bookkeep(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 14) throw Refusal{PyExc_TypeError, "bookkeep takes 14 arguments"};
    const int op = number(a[0], "op");
    const bool list = op != 3, contents = op >= 2;
    const Tensor *refs = tensor(a[1], "refs"), *table = tensor(a[2], "table"), *lens = tensor(a[3], "lens", !list),
                 *row = tensor(a[4], "row", !list), *src = tensor(a[5], "src", op != 2),
                 *grow = tensor(a[6], "grow", op != 0), *kp = tensor(a[8], "k_pages", !contents),
                 *vp = tensor(a[9], "v_pages", !contents), *table_out = tensor(a[10], "table_out", true),
                 *refs_out = tensor(a[11], "refs_out", true), *given = tensor(a[12], "workspace", true);
    const at::Device device = refs->device();
    dims(*refs, "refs", 1, "[num_pages]");
    dims(*table, "table", 2, "[rows, max_pages]");
    if (row) dims(*row, "row", 1, "[n]");
    const int64_t P = refs->size(0), rows = table->size(0), count = row ? row->size(0) : 0;
    lizard_pages_args c{};
    c.page = contents ? 0 : number(a[7], "page");
    if (contents) {
      c.dtype = type_code(kp->scalar_type());
      dims(*kp, "k_pages", 5, "[layers, num_pages, Hkv, page, d]");
      if (kp->size(1) != P)
        refuse("refs counts " + std::to_string(P) + " pages, the pool has " + std::to_string(kp->size(1)));
      fits(kp, "k_pages", kp->sizes(), kp->scalar_type(), device);
      fits(vp, "v_pages", kp->sizes(), kp->scalar_type(), device);
      for (int64_t x : kp->sizes())
        if (x > INT32_MAX) refuse("a size does not fit 32 bits");
      c.layers = kp->size(0); c.Hkv = kp->size(2); c.page = kp->size(3); c.d = kp->size(4);
      c.k_pages = ptr(kp); c.v_pages = ptr(vp);
    }
    for (int64_t x : {P, rows, table->size(1), count})
      if (x > INT32_MAX) refuse("a size does not fit 32 bits");
    fits(refs, "refs", {P}, at::kInt, device);
    fits(table, "table", table->sizes(), at::kInt, device);
    fits(lens, "lens", {rows}, at::kInt, device);
    fits(row, "row", {count}, at::kInt, device);
    fits(src, "src", {count}, at::kInt, device);
    fits(grow, "grow", {count}, at::kInt, device);
    fits(table_out, "table_out", table->sizes(), at::kInt, device);
    fits(refs_out, "refs_out", {P}, at::kInt, device);
    cuda_only(device);
    const Place place(device, a[13]);
    Tensor to, ro, ws;
    lizard_status st;
    {
      const Unlocked unlocked;
      if (op == 3) {
        to = table_out ? *table_out : at::empty(table->sizes(), table->options());
        ro = refs_out ? *refs_out : at::empty({P}, refs->options());
        c.table_out = ints(&to);
        c.refs_out = ints(&ro);
      }
      c.num_pages = P; c.rows = rows; c.max_pages = table->size(1); c.n = count;
      ws = space(given, lizard_pages_workspace_size(&c), device);
      c.refs = ints(refs); c.table = ints(table); c.lens = ints(lens);
      c.row = ints(row); c.src = ints(src); c.grow = ints(grow);
      c.workspace = ws.data_ptr();
      c.workspace_bytes = ws.nbytes();
      const auto call = op == 0   ? lizard_pages_reserve
                        : op == 1 ? lizard_pages_free
                        : op == 2 ? lizard_pages_fork
                                  : lizard_pages_compact;
      st = call(&c, place.handle());
    }
    return Py_BuildValue("(iNNN)", (int)st, give(to), give(ro), give(ws));
  });
}

PyMethodDef methods[] = {
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn)), METH_FASTCALL, nullptr},
    {"bookkeep", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bookkeep)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_call(void) { return PyModule_Create(&module); }
