// Native half of the language operators' binding (vla_dual_expert_b200/language.py): tensor checks, outputs and
// workspaces from torch's allocator, and the call into the C ABI of dm0.h.  A call on a few tokens is bound by
// the host; in Python and ctypes it took 15 us for the boundary norms of 50 rows, here 6.
//
// Every function takes the context's address and device first and the stream last (None: torch's current one), and
// returns the outputs, or the C ABI's status as an int where that is not DM0_OK.  A malformed tensor raises
// TypeError (kind, device, layout) or ValueError (shape).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "dm0.h"

namespace {

using at::Tensor;
using c10::ScalarType;

struct TypeErr : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct ValueErr : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PyErr : std::exception {};   // a Python error is already set

constexpr ScalarType kF32 = ScalarType::Float, kBf16 = ScalarType::BFloat16;

std::string text(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + ")";
}
std::string text(std::initializer_list<ScalarType> kinds) {
  std::string s;
  for (ScalarType k : kinds) s += (s.empty() ? "" : " or ") + std::string(c10::toString(k));
  return s;
}
bool among(ScalarType k, std::initializer_list<ScalarType> kinds) {
  for (ScalarType x : kinds)
    if (x == k) return true;
  return false;
}

// One call: its context, device and stream.
struct Call {
  dm0_ctx* ctx;
  int device;
  PyObject* given;   // the stream argument
  cudaStream_t stream;
  bool foreign = false;   // not torch's current stream, whose pool the allocator takes blocks from

  Call(PyObject* const* args, PyObject* stream_arg) : given(stream_arg) {
    ctx = static_cast<dm0_ctx*>(PyLong_AsVoidPtr(args[0]));
    device = static_cast<int>(PyLong_AsLong(args[1]));
    if (PyErr_Occurred()) throw PyErr();
    stream = nullptr;
  }
  // after the tensors' checks: nothing before needs a GPU
  void open() {
    const cudaStream_t current = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    stream = given == Py_None ? current : static_cast<cudaStream_t>(PyLong_AsVoidPtr(given));
    if (PyErr_Occurred()) throw PyErr();
    foreign = stream != current;
  }
  // A tensor of the call's stream's own pool: the allocator hands out a block that was freed a moment ago, while
  // kernels on the block's stream still use it, so a block of another stream's pool would be written too early.
  Tensor take(at::IntArrayRef shape, ScalarType kind) const {
    return at::detail::empty_cuda(shape, kind, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                  std::nullopt);
  }
  // an output; the current stream is where the caller goes on, so the block is kept until that is past it too
  Tensor make(at::IntArrayRef shape, ScalarType kind) const {
    if (!foreign) return take(shape, kind);
    const c10::cuda::CUDAStream here = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device));
    const c10::cuda::CUDAStreamGuard there(target());
    Tensor t = take(shape, kind);
    if (t.numel()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), here);
    return t;
  }
  // a workspace, freed when the call returns: what takes its block next follows on the same stream
  Tensor scratch(size_t bytes) const {
    const int64_t n = static_cast<int64_t>(bytes < 16 ? 16 : bytes);
    if (!foreign) return take({n}, ScalarType::Byte);
    const c10::cuda::CUDAStreamGuard there(target());
    return take({n}, ScalarType::Byte);
  }
  c10::cuda::CUDAStream target() const {
    return c10::cuda::getStreamFromExternal(stream, static_cast<c10::DeviceIndex>(device));
  }

  void kind_ok(const Tensor& t, std::initializer_list<ScalarType> kinds, const char* name) const {
    if (!t.is_cuda() || t.get_device() != device || !among(t.scalar_type(), kinds))
      throw TypeErr(std::string(name) + " must be a tensor on cuda:" + std::to_string(device) + " of " + text(kinds));
  }
  static void shape_ok(const Tensor& t, at::IntArrayRef shape, const char* name) {
    if (t.sizes() != shape)
      throw ValueErr(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
  }
  // a contiguous tensor of `shape`
  void* dense(const Tensor& t, std::initializer_list<ScalarType> kinds, at::IntArrayRef shape, const char* name) const {
    shape_ok(t, shape, name);
    kind_ok(t, kinds, name);
    if (!t.is_contiguous()) throw TypeErr(std::string(name) + " must be contiguous");
    return t.data_ptr();
  }
  // rows that are contiguous themselves: [T][H] or [B][T][H]
  void* rows(const Tensor& t, at::IntArrayRef shape, const char* name, int64_t* batch, int64_t* row) const {
    shape_ok(t, shape, name);
    kind_ok(t, {kBf16, kF32}, name);
    const int64_t n = t.dim();
    if (t.stride(n - 1) != 1) throw ValueErr("the rows of " + std::string(name) + " must be contiguous");
    // the stride of a dimension of one says nothing
    *batch = n == 3 && shape[0] > 1 ? t.stride(0) : 0;
    *row = shape[n - 2] > 1 ? t.stride(n - 2) : shape[n - 1];
    return t.data_ptr();
  }
};

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw TypeErr(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
float number(PyObject* o) {
  const double d = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw PyErr();
  return static_cast<float>(d);
}
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (PyErr_Occurred()) throw PyErr();
  if (v < INT32_MIN || v > INT32_MAX) throw ValueErr("integer out of range");
  return static_cast<int>(v);
}
int fit(int64_t v) {   // a size as the C ABI takes it; larger ones are refused there as out of range
  return v > INT32_MAX ? INT32_MAX : static_cast<int>(v);
}
bool is_f32(const Tensor& t) { return t.scalar_type() == kF32; }

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* status(dm0_status st) { return PyLong_FromLong(st); }

// a function's body with C++ exceptions turned into Python ones
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const PyErr&) {
  } catch (const TypeErr& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const ValueErr& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* kind = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_Clear();
    PyErr_SetString(kind ? kind : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(kind);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
template <class F>
dm0_status without_gil(F&& call) {
  struct Released {
    PyThreadState* save = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(save); }
  } released;
  return call();
}

struct IdList {
  void* p;
  int wide, B, T;
  c10::SmallVector<int64_t, 4> shape;   // of the ids, then room for the hidden size
};
IdList id_list(const Call& c, const Tensor& ids) {
  if (ids.dim() != 1 && ids.dim() != 2) throw ValueErr("ids must be [T] or [B][T]");
  IdList l;
  l.shape.append(ids.sizes().begin(), ids.sizes().end());
  l.p = c.dense(ids, {ScalarType::Long, ScalarType::Int}, ids.sizes(), "ids");
  l.wide = ids.scalar_type() == ScalarType::Long;
  l.B = ids.dim() == 1 ? 1 : fit(ids.size(0));
  l.T = fit(ids.size(-1));
  return l;
}

// (ctx, device, table, ids, scale, out, stream)
PyObject* embed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c(a, a[6]);
    const Tensor& table = tensor(a[2], "table");
    IdList l = id_list(c, tensor(a[3], "ids"));
    if (table.dim() != 2) throw ValueErr("table must be [vocab][hidden]");
    const void* tp = c.dense(table, {kBf16}, table.sizes(), "table");
    const int64_t H = table.size(1);
    l.shape.push_back(H);
    const float scale = number(a[4]);
    const Tensor* given = maybe(a[5], "out");
    int64_t bs = 0, rs = 0;
    if (given) c.rows(*given, l.shape, "out", &bs, &rs);
    c.open();
    const Tensor out = given ? *given : c.make(l.shape, kBf16);
    void* op = c.rows(out, l.shape, "out", &bs, &rs);
    const dm0_status st = without_gil([&] {
      return dm0_embed(c.ctx, tp, l.p, l.wide, l.B, l.T, fit(table.size(0)), fit(H), scale, op, is_f32(out), bs, rs,
                       c.stream);
    });
    return st ? status(st) : wrap(out);
  });
}

// (ctx, device, ids, dout, vocab, scale, grad, accumulate, stream)
PyObject* embed_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Call c(a, a[8]);
    IdList l = id_list(c, tensor(a[2], "ids"));
    const Tensor& dout = tensor(a[3], "dout");
    if (dout.dim() < 1) throw ValueErr("dout must have rows");
    const int64_t H = dout.size(-1);
    l.shape.push_back(H);
    int64_t bs, rs;
    const void* dp = c.rows(dout, l.shape, "dout", &bs, &rs);
    const int vocab = integer(a[4]);
    const float scale = number(a[5]);
    const Tensor* given = maybe(a[6], "grad");
    const int add = PyObject_IsTrue(a[7]);
    if (add < 0) throw PyErr();
    if (add && !given) throw ValueErr("accumulate needs grad");
    if (vocab < 0) throw ValueErr("vocab must not be negative");
    if (given) c.dense(*given, {kF32}, {vocab, H}, "grad");
    c.open();
    const Tensor grad = given ? *given : c.make({vocab, H}, kF32);
    const size_t bytes = dm0_embed_grad_workspace(l.B, l.T, vocab, fit(H));
    const Tensor ws = c.scratch(bytes);
    const dm0_status st = without_gil([&] {
      return dm0_embed_grad(c.ctx, l.p, l.wide, l.B, l.T, vocab, fit(H), scale, dp, is_f32(dout), bs, rs,
                            grad.data_ptr<float>(), add, ws.data_ptr(), bytes, c.stream);
    });
    return st ? status(st) : wrap(grad);
  });
}

// a per-sample vector: [H], or [B][H] rows at *stride
const float* vector(const Call& c, const Tensor* v, int64_t B, int64_t H, const char* name, int* stride) {
  *stride = 0;
  if (!v) return nullptr;
  const bool one = v->dim() == 1 ? v->size(0) == H : v->dim() == 2 && B == 1 && v->size(0) == 1 && v->size(1) == H;
  if (!one && !(v->dim() == 2 && v->size(0) == B && v->size(1) == H))
    throw ValueErr(std::string(name) + " has shape " + text(v->sizes()) + ", expected " + text({H}) + " or " + text({B, H}));
  c.kind_ok(*v, {kF32}, name);
  if (H > 1 && v->stride(-1) != 1) throw TypeErr("the rows of " + std::string(name) + " must be contiguous");
  if (!one) {
    if (v->stride(0) < H) throw ValueErr("the rows of " + std::string(name) + " overlap");
    *stride = fit(v->stride(0));
  }
  return v->data_ptr<float>();
}

struct Norm {
  dm0_norm a;
  void *h, *y;
  c10::SmallVector<int64_t, 4> rows;   // the shape without the hidden size
};
Norm norm_of(const Call& c, const Tensor& h, const Tensor* y, const Tensor* post, const Tensor* gate, float scale,
             const Tensor* pre, const Tensor* ms, const Tensor* mt) {
  if (h.dim() != 2 && h.dim() != 3) throw ValueErr("the residual stream must be [T][hidden] or [B][T][hidden]");
  const int64_t B = h.dim() == 3 ? h.size(0) : 1, T = h.size(-2), H = h.size(-1);
  Norm r{};
  r.h = c.dense(h, {kBf16, kF32}, h.sizes(), "the residual stream");
  r.y = y ? c.dense(*y, {kBf16, kF32}, h.sizes(), "y") : nullptr;
  r.rows.append(h.sizes().begin(), h.sizes().end() - 1);
  dm0_norm& a = r.a;
  a.batch = fit(B), a.tokens = fit(T), a.hidden = fit(H);
  a.h_f32 = is_f32(h), a.y_f32 = y && is_f32(*y);
  a.scale = scale;
  a.post_gain = post ? static_cast<float*>(c.dense(*post, {kF32}, {H}, "post_gain")) : nullptr;
  a.pre_gain = pre ? static_cast<float*>(c.dense(*pre, {kF32}, {H}, "pre_gain")) : nullptr;
  int s1, s2;
  a.gate = vector(c, gate, B, H, "gate", &a.gate_stride);
  a.mod_scale = vector(c, ms, B, H, "mod_scale", &s1);
  a.mod_shift = vector(c, mt, B, H, "mod_shift", &s2);
  if (ms && mt && s1 != s2) throw ValueErr("mod_scale and mod_shift must be laid out alike");
  a.mod_stride = ms ? s1 : s2;
  return r;
}

// (ctx, device, h, y, post_gain, gate, scale, pre_gain, mod_scale, mod_shift, h_out, n_out, stream)
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    Call c(a, a[12]);
    const Tensor& h = tensor(a[2], "h");
    const Tensor *y = maybe(a[3], "y"), *post = maybe(a[4], "post_gain");
    const Norm r = norm_of(c, h, y, post, maybe(a[5], "gate"), number(a[6]), maybe(a[7], "pre_gain"),
                           maybe(a[8], "mod_scale"), maybe(a[9], "mod_shift"));
    const Tensor *hg = maybe(a[10], "h_out"), *ng = maybe(a[11], "n_out");
    if (hg) c.dense(*hg, {h.scalar_type()}, h.sizes(), "h_out");
    if (ng) c.dense(*ng, {kBf16}, h.sizes(), "n_out");
    c.open();
    const Tensor h_out = hg ? *hg : c.make(h.sizes(), h.scalar_type());
    const Tensor n_out = ng ? *ng : c.make(h.sizes(), kBf16);
    const Tensor r_pre = c.make(r.rows, kF32);
    Tensor r_post;
    if (post) r_post = c.make(r.rows, kF32);
    const dm0_status st = without_gil([&] {
      return dm0_residual_norm(c.ctx, &r.a, r.h, r.y, h_out.data_ptr(), n_out.data_ptr(),
                               post ? r_post.data_ptr<float>() : nullptr, r_pre.data_ptr<float>(), c.stream);
    });
    if (st) return status(st);
    PyObject* t = PyTuple_New(4);
    if (!t) throw PyErr();
    PyTuple_SET_ITEM(t, 0, wrap(h_out));
    PyTuple_SET_ITEM(t, 1, wrap(n_out));
    PyTuple_SET_ITEM(t, 2, post ? wrap(r_post) : Py_NewRef(Py_None));
    PyTuple_SET_ITEM(t, 3, wrap(r_pre));
    return t;
  });
}

void put(PyObject* dict, const char* key, const Tensor& t) {
  PyObject* o = wrap(t);
  const int bad = !o || PyDict_SetItemString(dict, key, o);
  Py_XDECREF(o);
  if (bad) {
    Py_DECREF(dict);
    throw PyErr();
  }
}

// (ctx, device, dn, dh_out, h_out, y, r_post, r_pre, post_gain, gate, scale, pre_gain, mod_scale, mod_shift, stream)
PyObject* residual_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    Call c(a, a[14]);
    const Tensor &dn = tensor(a[2], "dn"), &h = tensor(a[4], "h_out"), &r_pre = tensor(a[7], "r_pre");
    const Tensor *up = maybe(a[3], "dh_out"), *y = maybe(a[5], "y"), *r_post = maybe(a[6], "r_post");
    const Tensor *post = maybe(a[8], "post_gain"), *gate = maybe(a[9], "gate"), *pre = maybe(a[11], "pre_gain");
    const Tensor *ms = maybe(a[12], "mod_scale"), *mt = maybe(a[13], "mod_shift");
    const Norm r = norm_of(c, h, y, post, gate, number(a[10]), pre, ms, mt);
    const void* np = c.dense(dn, {kBf16, kF32}, h.sizes(), "dn");
    const void* pp = up ? c.dense(*up, {h.scalar_type()}, h.sizes(), "dh_out") : nullptr;
    const float* rp = static_cast<float*>(c.dense(r_pre, {kF32}, r.rows, "r_pre"));
    const float* rq = r_post ? static_cast<float*>(c.dense(*r_post, {kF32}, r.rows, "r_post")) : nullptr;
    c.open();
    const Tensor dh = c.make(h.sizes(), h.scalar_type());
    Tensor dy;
    if (y) dy = c.make(h.sizes(), y->scalar_type());
    dm0_norm_grads g{};
    Tensor out[5];
    const Tensor* vec[5] = {post, gate, pre, ms, mt};
    float** dst[5] = {&g.post_gain, &g.gate, &g.pre_gain, &g.mod_scale, &g.mod_shift};
    for (int k = 0; k < 5; ++k)
      if (vec[k]) {
        out[k] = c.make(vec[k]->sizes(), kF32);
        *dst[k] = out[k].data_ptr<float>();
      }
    const size_t bytes = dm0_residual_norm_grad_workspace(&r.a);
    const Tensor ws = c.scratch(bytes);
    const dm0_status st = without_gil([&] {
      return dm0_residual_norm_grad(c.ctx, &r.a, np, is_f32(dn), pp, r.h, r.y, rq, rp, dh.data_ptr(),
                                    y ? dy.data_ptr() : nullptr, &g, ws.data_ptr(), bytes, c.stream);
    });
    if (st) return status(st);
    PyObject* d = PyDict_New();
    if (!d) throw PyErr();
    put(d, "h", dh);
    if (y) put(d, "y", dy);
    static const char* const names[5] = {"post_gain", "gate", "pre_gain", "mod_scale", "mod_shift"};
    for (int k = 0; k < 5; ++k)
      if (vec[k]) put(d, names[k], out[k]);
    return d;
  });
}

struct Vocab {
  int64_t N, V, H;
  void *h, *w, *t;
  int wide;
};
Vocab vocab_of(const Call& c, const Tensor& hidden, const Tensor& weight, const Tensor& targets) {
  if (hidden.dim() != 2 || weight.dim() != 2 || weight.size(1) != hidden.size(1))
    throw ValueErr("hidden must be [tokens][H] and weight [vocab][H]");
  Vocab v{hidden.size(0), weight.size(0), hidden.size(1)};
  v.h = c.dense(hidden, {kBf16}, hidden.sizes(), "hidden");
  v.w = c.dense(weight, {kBf16}, weight.sizes(), "weight");
  v.t = c.dense(targets, {ScalarType::Long, ScalarType::Int}, {v.N}, "targets");
  v.wide = targets.scalar_type() == ScalarType::Long;
  return v;
}
PyObject* pair(PyObject* x, PyObject* y) {
  PyObject* t = x && y ? PyTuple_New(2) : nullptr;
  if (!t) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    throw PyErr();
  }
  PyTuple_SET_ITEM(t, 0, x);
  PyTuple_SET_ITEM(t, 1, y);
  return t;
}

// (ctx, device, hidden, weight, targets, stream)
PyObject* vocab_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    Call c(a, a[5]);
    const Vocab v = vocab_of(c, tensor(a[2], "hidden"), tensor(a[3], "weight"), tensor(a[4], "targets"));
    c.open();
    const Tensor loss = c.make({v.N}, kF32), lse = c.make({v.N}, kF32);
    const size_t bytes = dm0_vocab_loss_workspace(fit(v.N), fit(v.V), fit(v.H));
    const Tensor ws = c.scratch(bytes);
    const dm0_status st = without_gil([&] {
      return dm0_vocab_loss(c.ctx, v.h, v.w, v.t, v.wide, fit(v.N), fit(v.V), fit(v.H), loss.data_ptr<float>(),
                            lse.data_ptr<float>(), ws.data_ptr(), bytes, c.stream);
    });
    return st ? status(st) : pair(wrap(loss), wrap(lse));
  });
}

// (ctx, device, hidden, weight, targets, lse, dloss, dhidden, dweight, accumulate, stream); a gradient is None (made
// here), False (left out) or a tensor
PyObject* vocab_loss_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    Call c(a, a[10]);
    const Tensor &hidden = tensor(a[2], "hidden"), &weight = tensor(a[3], "weight");
    const Vocab v = vocab_of(c, hidden, weight, tensor(a[4], "targets"));
    const float* lse = static_cast<float*>(c.dense(tensor(a[5], "lse"), {kF32}, {v.N}, "lse"));
    const float* dloss = static_cast<float*>(c.dense(tensor(a[6], "dloss"), {kF32}, {v.N}, "dloss"));
    const int add = PyObject_IsTrue(a[9]);
    if (add < 0) throw PyErr();
    Tensor out[2];
    const Tensor* like[2] = {&hidden, &weight};
    for (int k = 0; k < 2; ++k) {
      PyObject* o = a[7 + k];
      if (o == Py_None || o == Py_False) continue;
      out[k] = tensor(o, k ? "dweight" : "dhidden");
      c.dense(out[k], {kBf16, kF32}, like[k]->sizes(), k ? "dweight" : "dhidden");
    }
    if (add && !out[1].defined()) throw ValueErr("accumulate needs dweight");
    c.open();
    for (int k = 0; k < 2; ++k)
      if (a[7 + k] == Py_None) out[k] = c.make(like[k]->sizes(), kBf16);
    const bool dh = out[0].defined(), dw = out[1].defined();
    const size_t bytes = dm0_vocab_loss_grad_workspace(fit(v.N), fit(v.V), fit(v.H));
    const Tensor ws = c.scratch(bytes);
    const dm0_status st = without_gil([&] {
      return dm0_vocab_loss_grad(c.ctx, v.h, v.w, v.t, v.wide, lse, dloss, fit(v.N), fit(v.V), fit(v.H),
                                 dh ? out[0].data_ptr() : nullptr, dh && is_f32(out[0]), dw ? out[1].data_ptr() : nullptr,
                                 dw && is_f32(out[1]), add, ws.data_ptr(), bytes, c.stream);
    });
    if (st) return status(st);
    return pair(dh ? wrap(out[0]) : Py_NewRef(Py_None), dw ? wrap(out[1]) : Py_NewRef(Py_None));
  });
}

#define DM0_FN(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DM0_FN(embed),      DM0_FN(embed_grad), DM0_FN(residual_norm), DM0_FN(residual_norm_grad),
                         DM0_FN(vocab_loss), DM0_FN(vocab_loss_grad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_language", "Native half of the language operators' binding.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__language(void) { return PyModule_Create(&module); }
