// Python entry points of the calls that take microseconds (routing, block norms,
// the adapter projection): argument checks and marshalling only, as in _lib.py,
// but compiled.  The checks of a dozen tensors cost the interpreter 3 to 10 us a
// call on the host, more than the kernels of a decode batch take.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <string>

#include "moe_gb300.h"

namespace {

struct Refused {};   // the Python error is set

PyObject* g_check = nullptr;   // _lib._check: raises MoeError for a status
PyObject* g_error = nullptr;   // _lib.MoeError

// Raises MoeError(MOE_ERR_INVALID, why).
[[noreturn]] void refuse(const std::string& why) {
  if (PyObject* e = PyObject_CallFunction(g_error, "is", (int)MOE_ERR_INVALID, why.c_str())) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument; null for None.
const at::Tensor* tensor(PyObject* o, const char* what) {
  if (!o || o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", what, Py_TYPE(o)->tp_name);
    throw Refused();
  }
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* what) {
  const at::Tensor* t = tensor(o, what);
  if (!t) {
    PyErr_Format(PyExc_ValueError, "%s is needed", what);
    throw Refused();
  }
  return *t;
}
const at::Tensor& matrix(PyObject* o, const char* what) {
  const at::Tensor& t = needed(o, what);
  if (t.dim() != 2) {
    PyErr_Format(PyExc_ValueError, "%s must have two dimensions, got %s", what, shape_text(t.sizes()).c_str());
    throw Refused();
  }
  return t;
}

int dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MOE_DT_F32;
    case at::kBFloat16: return MOE_DT_BF16;
    case at::kHalf: return MOE_DT_F16;
    case at::kShort: return MOE_DT_BF16;   // bf16 bits, as the expert calls take them
    default: break;
  }
  PyErr_Format(PyExc_ValueError, "unsupported tensor type %s", c10::toString(t.scalar_type()));
  throw Refused();
}
void same_type(const at::Tensor* t, at::ScalarType d, const char* what) {
  if (t && t->scalar_type() != d) {
    PyErr_Format(PyExc_ValueError, "%s must be of type %s, got %s", what, c10::toString(d),
                 c10::toString(t->scalar_type()));
    throw Refused();
  }
}

// The tensors of a call, in the order in which they pass their own checks.
struct Tensors {
  const at::Tensor* t[20];
  const char* what[20];
  int n = 0;
  void add(const at::Tensor* a, const char* name) {
    if (n < 20) t[n] = a, what[n++] = name;
  }
  // Every tensor is on the first one's GPU: the kernels would read a host address as their own.
  void on_one_gpu() const {
    for (int i = 0; i < n; ++i) {
      if (t[i]->is_cuda() && t[i]->device() == t[0]->device()) continue;
      refuse(std::string(what[i]) + (t[i]->is_cuda() ? " is on another GPU than " + std::string(what[0])
                                                     : " is not on a GPU (" + t[i]->device().str() + ")"));
    }
  }
};

struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};
// A [T, n] tensor whose rows may be strided (null: none).
Rows rows(Tensors& all, const at::Tensor* t, int64_t T, int64_t n, const char* what) {
  if (!t) return {};
  if (t->dim() != 2 || t->size(0) != T || t->size(1) != n) {
    PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld], got %s", what, (long long)T, (long long)n,
                 shape_text(t->sizes()).c_str());
    throw Refused();
  }
  int64_t sr = t->stride(0);
  if (t->stride(1) != 1 && n > 1) {
    PyErr_Format(PyExc_ValueError, "%s: the elements of a row must be adjacent (strides %s)", what,
                 shape_text(t->strides()).c_str());
    throw Refused();
  }
  if (T <= 1) {
    sr = n;   // one row: the distance to the next is not used, whatever tensor it was taken from
  } else if (sr < n) {
    PyErr_Format(PyExc_ValueError, "%s: rows overlap (strides %s)", what, shape_text(t->strides()).c_str());
    throw Refused();
  }
  all.add(t, what);
  return {t->data_ptr(), sr};
}
// A dense tensor of the given shape and type (null: none).
void* dense(Tensors& all, const at::Tensor* t, std::initializer_list<int64_t> shape, at::ScalarType d, const char* what) {
  if (!t) return nullptr;
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t->sizes() != want || t->scalar_type() != d) {
    PyErr_Format(PyExc_ValueError, "%s must be %s of %s, got %s of %s", what, shape_text(want).c_str(),
                 c10::toString(d), shape_text(t->sizes()).c_str(), c10::toString(t->scalar_type()));
    throw Refused();
  }
  if (!t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s of shape %s and strides %s is not contiguous", what,
                 shape_text(t->sizes()).c_str(), shape_text(t->strides()).c_str());
    throw Refused();
  }
  all.add(t, what);
  return t->data_ptr();
}
// A workspace's address and bytes.
void* space(Tensors& all, const at::Tensor* t, size_t& bytes) {
  if (!t->is_contiguous()) {
    PyErr_SetString(PyExc_ValueError, "workspace is not contiguous");
    throw Refused();
  }
  all.add(t, "workspace");
  bytes = t->nbytes();
  return t->data_ptr();
}
int to_int(int64_t v, const char* what) {
  if (v > 0x7fffffffLL) {
    PyErr_Format(PyExc_ValueError, "%s is too large (%lld)", what, (long long)v);
    throw Refused();
  }
  return (int)v;
}

cudaStream_t stream_of(PyObject* o) {
  if (!o || o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  PyObject* h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Refused();
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!p && PyErr_Occurred()) throw Refused();
  return (cudaStream_t)p;
}

// Where a call runs, once its arguments have passed their own checks: on its tensors' GPU.
struct Place {
  c10::cuda::OptionalCUDAGuard gpu;
  cudaStream_t stream;
  Place(const Tensors& all, PyObject* stream_arg) {
    all.on_one_gpu();
    gpu.set_device(all.t[0]->device());
    stream = stream_of(stream_arg);
  }
};

// Tensors that the caller did not bring: held, and handed out as results.
struct Results {
  static PyObject* of(PyObject* given, const at::Tensor& made) {
    if (given && given != Py_None) return Py_NewRef(given);
    if (made.defined()) return THPVariable_Wrap(made);
    return Py_NewRef(Py_None);
  }
};

// A tensor that the caller did not bring, from the memory of the stream that the call runs on: what is
// free there has no work of another stream before it.  A result is known to the current stream too,
// where the caller takes it on (once that waits for the call's) and lets go of it.
at::Tensor make(at::IntArrayRef shape, const at::TensorOptions& o, PyObject* stream_arg, bool result = true) {
  if (!stream_arg || stream_arg == Py_None || !o.device().is_cuda()) return at::empty(shape, o);
  const cudaStream_t s = stream_of(stream_arg);
  const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(o.device().index());
  if (s == now.stream()) return at::empty(shape, o);
  at::Tensor t;
  {
    const c10::cuda::CUDAStreamGuard there(c10::cuda::getStreamFromExternal(s, o.device().index()));
    t = at::empty(shape, o);
  }
  if (result && t.numel()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), now);
  return t;
}

void check(moe_status st) {
  if (st == MOE_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", (int)st);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "a library call failed");
  throw Refused();
}

// Calls f without the interpreter's lock, as ctypes does.
template <typename F>
moe_status unlocked(F f) {
  moe_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused&) {
  } catch (...) {   // torch's own errors keep their Python types (out of memory among them)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

const at::Tensor* either(PyObject* given, const char* what, at::Tensor& made, at::IntArrayRef shape,
                         const at::TensorOptions& o, PyObject* stream_arg) {
  if (const at::Tensor* t = tensor(given, what)) return t;
  made = make(shape, o, stream_arg);
  return &made;
}

const uint8_t* mask_ptr(Tensors& all, PyObject* o, int64_t T) {
  const at::Tensor* m = tensor(o, "token_mask");
  return (const uint8_t*)dense(all, m, {T}, m && m->scalar_type() == at::kBool ? at::kBool : at::kByte, "token_mask");
}

PyObject* route(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"logits", "k", "score", "bias", "n_group", "topk_group", "group_score", "renorm",
                                "scale", "token_mask", "topk_ids", "topk_w", "load", "stream", nullptr};
  PyObject *logits, *bias = nullptr, *mask = nullptr, *ids = nullptr, *w = nullptr, *load = nullptr, *st = nullptr;
  int k, score = MOE_SCORE_SOFTMAX, ng = 1, tg = 1, gs = MOE_GROUP_TOP2, renorm = 1;
  double scale = 1.0;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "Oi|iOiiipdOOOOO", (char**)names, &logits, &k, &score, &bias, &ng, &tg,
                                   &gs, &renorm, &scale, &mask, &ids, &w, &load, &st))
    return nullptr;
  return guarded([&] {
    Tensors all;
    const at::Tensor& lg = matrix(logits, "logits");
    const int T = to_int(lg.size(0), "T"), E = to_int(lg.size(1), "E"), d = dtype_code(lg);
    at::Tensor mi, mw;
    const int64_t made = k >= 0 && k <= E ? k : 0;   // any other k is refused by the library
    const at::Tensor* ti = either(ids, "topk_ids", mi, {T, made}, lg.options().dtype(at::kInt), st);
    const at::Tensor* tw = either(w, "topk_w", mw, {T, made}, lg.options().dtype(at::kFloat), st);
    const Rows r = rows(all, &lg, T, E, "logits");
    auto* pb = (const float*)dense(all, tensor(bias, "bias"), {E}, at::kFloat, "bias");
    auto* pm = mask_ptr(all, mask, T);
    auto* pi = (int32_t*)dense(all, ti, {T, mi.defined() ? made : k}, at::kInt, "topk_ids");
    auto* pw = (float*)dense(all, tw, {T, mw.defined() ? made : k}, at::kFloat, "topk_w");
    auto* pl = (int32_t*)dense(all, tensor(load, "load"), {E}, at::kInt, "load");
    const Place at(all, st);
    check(unlocked([&] {
      return moe_route(r.p, d, r.ld, T, E, k, score, pb, ng, tg, gs, renorm, (float)scale, pm, pi, pw, pl, at.stream);
    }));
    return Py_BuildValue("(NN)", Results::of(ids, mi), Results::of(w, mw));
  });
}

PyObject* route_backward(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"logits", "topk_ids", "d_w", "score", "renorm", "scale", "token_mask", "d_logits",
                                "stream", nullptr};
  PyObject *logits, *ids, *dw, *mask = nullptr, *dl = nullptr, *st = nullptr;
  int score = MOE_SCORE_SOFTMAX, renorm = 1;
  double scale = 1.0;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "OOO|ipdOOO", (char**)names, &logits, &ids, &dw, &score, &renorm, &scale,
                                   &mask, &dl, &st))
    return nullptr;
  return guarded([&] {
    Tensors all;
    const at::Tensor &lg = matrix(logits, "logits"), &ti = matrix(ids, "topk_ids");
    const int T = to_int(lg.size(0), "T"), E = to_int(lg.size(1), "E"), k = to_int(ti.size(1), "k"), d = dtype_code(lg);
    at::Tensor made;
    const at::Tensor* td = either(dl, "d_logits", made, {T, E}, lg.options(), st);
    same_type(td, lg.scalar_type(), "d_logits");
    const Rows r = rows(all, &lg, T, E, "logits"), rd = rows(all, td, T, E, "d_logits");
    auto* pm = mask_ptr(all, mask, T);
    auto* pi = (const int32_t*)dense(all, &ti, {T, k}, at::kInt, "topk_ids");
    auto* pd = (const float*)dense(all, &needed(dw, "d_w"), {T, k}, at::kFloat, "d_w");
    const Place at(all, st);
    check(unlocked([&] {
      return moe_route_backward(r.p, d, r.ld, T, E, k, score, renorm, (float)scale, pm, pi, pd, rd.p, rd.ld, at.stream);
    }));
    return Results::of(dl, made);
  });
}

// The weights of the norms: all of one type, which the first that is given sets.
struct NormWeights {
  int dtype = MOE_DT_F32, mode = MOE_GATE_NONE;
  const at::Tensor *tp, *tg, *tn;
  void *post, *gate, *next;
  NormWeights(Tensors& all, PyObject* p, PyObject* g, PyObject* n, int64_t T, int64_t H) {
    tp = tensor(p, "post_weight"), tg = tensor(g, "gate"), tn = tensor(n, "next_weight");
    const at::Tensor* first = tp ? tp : tg ? tg : tn;
    if (first) dtype = dtype_code(*first);
    const at::ScalarType d = first ? first->scalar_type() : at::kFloat;
    post = dense(all, tp, {H}, d, "post_weight");
    if (tg) mode = tg->dim() == 1 ? MOE_GATE_CHANNEL : MOE_GATE_TOKEN;   // [H]: each channel; [T, 1]: each token
    gate = mode == MOE_GATE_TOKEN ? dense(all, tg, {T, 1}, d, "gate (of the weights' one type)")
                                  : dense(all, tg, {H}, d, "gate (of the weights' one type)");
    next = dense(all, tn, {H}, d, "next_weight (of the weights' one type)");
  }
};

PyObject* block_norm(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"x", "y", "post_weight", "gate", "residual_scale", "next_weight", "eps", "x_out", "h",
                                "stream", nullptr};
  PyObject *x, *y = nullptr, *post = nullptr, *gate = nullptr, *next = nullptr, *xo = nullptr, *h = nullptr,
               *st = nullptr;
  double alpha = 1.0, eps = 1e-6;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "O|OOOdOdOOO", (char**)names, &x, &y, &post, &gate, &alpha, &next, &eps,
                                   &xo, &h, &st))
    return nullptr;
  return guarded([&] {
    Tensors all;
    const at::Tensor& tx = matrix(x, "x");
    const int T = to_int(tx.size(0), "T"), H = to_int(tx.size(1), "H");
    all.add(&tx, "x");   // first: the call runs on its GPU
    const NormWeights w(all, post, gate, next, T, H);
    const at::Tensor *ty = tensor(y, "y"), *th = tensor(h, "h"), *txo = tensor(xo, "x_out");
    const at::Tensor& like = ty ? *ty : th ? *th : tx;
    at::Tensor mxo, mh;
    if (!txo && ty) txo = &(mxo = make({T, H}, tx.options(), st));
    if (!th && w.tn) th = &(mh = make({T, H}, like.options(), st));
    same_type(txo, tx.scalar_type(), "x_out");
    same_type(th, like.scalar_type(), "h");
    const int dx = dtype_code(tx), dy = dtype_code(like);
    const Rows rx = rows(all, &tx, T, H, "x"), ry = rows(all, ty, T, H, "y"), ro = rows(all, txo, T, H, "x_out"),
               rh = rows(all, th, T, H, "h");
    const Place at(all, st);
    check(unlocked([&] {
      return moe_block_norm(T, H, dx, dy, w.dtype, rx.p, rx.ld, ry.p, ry.ld, w.post, w.gate, w.mode, (float)alpha,
                            w.next, (float)eps, ro.p, ro.ld, rh.p, rh.ld, at.stream);
    }));
    return Py_BuildValue("(NN)", Results::of(xo, mxo), Results::of(h, mh));
  });
}

PyObject* block_norm_backward(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"x", "y", "d_x_out", "d_h", "post_weight", "gate", "residual_scale", "next_weight",
                                "eps", "d_x", "d_y", "d_post_weight", "d_gate", "d_next_weight", "workspace", "stream",
                                nullptr};
  PyObject *x, *y, *du, *dh, *post = nullptr, *gate = nullptr, *next = nullptr, *dx = nullptr, *dy = nullptr,
                             *dp = nullptr, *dg = nullptr, *dn = nullptr, *ws = nullptr, *st = nullptr;
  double alpha = 1.0, eps = 1e-6;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "OOOO|OOdOdOOOOOOO", (char**)names, &x, &y, &du, &dh, &post, &gate, &alpha,
                                   &next, &eps, &dx, &dy, &dp, &dg, &dn, &ws, &st))
    return nullptr;
  return guarded([&] {
    Tensors all;
    const at::Tensor& tx = matrix(x, "x");
    const int T = to_int(tx.size(0), "T"), H = to_int(tx.size(1), "H");
    all.add(&tx, "x");   // first: the call runs on its GPU
    const NormWeights w(all, post, gate, next, T, H);
    const at::Tensor *ty = tensor(y, "y"), *tdu = tensor(du, "d_x_out"), *tdh = tensor(dh, "d_h");
    const at::Tensor& like = ty ? *ty : tdh ? *tdh : tx;
    const auto f32 = tx.options().dtype(at::kFloat);
    at::Tensor mdx, mdy, mdp, mdg, mdn, mws;
    const at::Tensor *tdx = either(dx, "d_x", mdx, {T, H}, tx.options(), st), *tdy = tensor(dy, "d_y");
    if (!tdy && ty) tdy = &(mdy = make({T, H}, ty->options(), st));
    same_type(tdu, tx.scalar_type(), "d_x_out");
    same_type(tdh, like.scalar_type(), "d_h");
    same_type(tdx, tx.scalar_type(), "d_x");
    same_type(tdy, like.scalar_type(), "d_y");
    const int xd = dtype_code(tx), yd = dtype_code(like);
    const Rows rx = rows(all, &tx, T, H, "x"), ry = rows(all, ty, T, H, "y"), ru = rows(all, tdu, T, H, "d_x_out"),
               rh = rows(all, tdh, T, H, "d_h"), rdx = rows(all, tdx, T, H, "d_x"), rdy = rows(all, tdy, T, H, "d_y");
    float *pp = nullptr, *pg = nullptr, *pn = nullptr;
    if (w.tp) pp = (float*)dense(all, either(dp, "d_post_weight", mdp, {H}, f32, st), {H}, at::kFloat, "d_post_weight");
    if (w.mode == MOE_GATE_CHANNEL) pg = (float*)dense(all, either(dg, "d_gate", mdg, {H}, f32, st), {H}, at::kFloat, "d_gate");
    if (w.mode == MOE_GATE_TOKEN)
      pg = (float*)dense(all, either(dg, "d_gate", mdg, {T, 1}, f32, st), {T, 1}, at::kFloat, "d_gate");
    if (w.tn) pn = (float*)dense(all, either(dn, "d_next_weight", mdn, {H}, f32, st), {H}, at::kFloat, "d_next_weight");
    const Place at(all, st);
    const at::Tensor* tws = tensor(ws, "workspace");
    if (!tws) tws = &(mws = make((int64_t)moe_block_norm_backward_workspace(T, H), tx.options().dtype(at::kByte), st, false));
    size_t nb;
    void* pws = space(all, tws, nb);
    all.on_one_gpu();
    check(unlocked([&] {
      return moe_block_norm_backward(T, H, xd, yd, w.dtype, rx.p, rx.ld, ry.p, ry.ld, ru.p, ru.ld, rh.p, rh.ld, w.post,
                                     w.gate, w.mode, (float)alpha, w.next, (float)eps, rdx.p, rdx.ld, rdy.p, rdy.ld, pp,
                                     pg, pn, pws, nb, at.stream);
    }));
    return Py_BuildValue("(NNNNN)", Results::of(dx, mdx), Results::of(dy, mdy), Results::of(w.tp ? dp : Py_None, mdp),
                         Results::of(w.tg ? dg : Py_None, mdg), Results::of(w.tn ? dn : Py_None, mdn));
  });
}

PyObject* adapter_linear(PyObject*, PyObject* args, PyObject* kw) {
  static const char* names[] = {"x", "weight", "lora_a", "lora_b", "adapter_ids", "lora_scale", "out", "out_dtype",
                                "workspace", "d_error", "stream", nullptr};
  PyObject *x, *wt, *la = nullptr, *lb = nullptr, *ids = nullptr, *ls = nullptr, *out = nullptr, *od = nullptr,
                    *ws = nullptr, *err = nullptr, *st = nullptr;
  if (!PyArg_ParseTupleAndKeywords(args, kw, "OO|OOOOOOOOO", (char**)names, &x, &wt, &la, &lb, &ids, &ls, &out, &od,
                                   &ws, &err, &st))
    return nullptr;
  return guarded([&] {
    Tensors all;
    const at::Tensor &tx = matrix(x, "x"), &tw = matrix(wt, "weight");
    const int T = to_int(tx.size(0), "T"), H = to_int(tx.size(1), "H"), N = to_int(tw.size(0), "N");
    const at::ScalarType d = tx.scalar_type();
    const Rows rx = rows(all, &tx, T, H, "x"), rw = rows(all, &tw, N, H, "weight");
    same_type(&tw, d, "weight (as x)");
    int n = 0, R = 0;
    void *pa = nullptr, *pb = nullptr, *pws = nullptr;
    const int32_t* pi = nullptr;
    const float* ps = nullptr;
    size_t nb = 0;
    at::Tensor mws, mout;
    if (const at::Tensor* ta = tensor(la, "lora_a")) {
      if (ta->dim() != 3) {
        PyErr_Format(PyExc_ValueError, "lora_a must be [n, R, %d], got %s", H, shape_text(ta->sizes()).c_str());
        throw Refused();
      }
      n = to_int(ta->size(0), "n"), R = to_int(ta->size(1), "R");
      pa = dense(all, ta, {n, R, H}, d, "lora_a");
      pb = dense(all, &needed(lb, "lora_b"), {n, N, R}, d, "lora_b");
      pi = (const int32_t*)dense(all, &needed(ids, "adapter_ids"), {T}, at::kInt, "adapter_ids");
      ps = (const float*)dense(all, tensor(ls, "lora_scale"), {n}, at::kFloat, "lora_scale");
    }
    const at::Tensor* to = tensor(out, "out");
    if (!to) {
      if (od && od != Py_None && !THPDtype_Check(od)) {
        PyErr_SetString(PyExc_TypeError, "out_dtype must be a torch.dtype");
        throw Refused();
      }
      const at::ScalarType t = od && od != Py_None ? reinterpret_cast<THPDtype*>(od)->scalar_type : d;
      to = &(mout = make({T, N}, tx.options().dtype(t), st));
    }
    const int xd = dtype_code(tx), ot = dtype_code(*to);
    const Rows ro = rows(all, to, T, N, "out");
    auto* pe = (int32_t*)dense(all, tensor(err, "d_error"), {1}, at::kInt, "d_error");
    const Place at(all, st);
    if (n) {
      const at::Tensor* tws = tensor(ws, "workspace");
      if (!tws)
        tws = &(mws = make((int64_t)moe_adapter_linear_workspace(T, H, N, n, R), tx.options().dtype(at::kByte), st, false));
      pws = space(all, tws, nb);
      all.on_one_gpu();
    }
    check(unlocked([&] {
      return moe_adapter_linear(T, H, N, xd, ot, rx.p, rx.ld, rw.p, rw.ld, n, R, pa, pb, pi, ps, ro.p, ro.ld, pws, nb,
                                pe, at.stream);
    }));
    return Results::of(out, mout);
  });
}

PyObject* set_check(PyObject*, PyObject* args) {
  PyObject *f, *e;
  if (!PyArg_ParseTuple(args, "OO", &f, &e)) return nullptr;
  Py_XSETREF(g_check, Py_NewRef(f));
  Py_XSETREF(g_error, Py_NewRef(e));
  Py_RETURN_NONE;
}

#define KW(f) (PyCFunction)(void (*)(void)) f, METH_VARARGS | METH_KEYWORDS
PyMethodDef methods[] = {
    {"moe_route", KW(route),
     "moe_route(logits, k, score=MOE_SCORE_SOFTMAX, bias=None, n_group=1, topk_group=1, group_score=MOE_GROUP_TOP2, "
     "renorm=True, scale=1.0, token_mask=None, topk_ids=None, topk_w=None, load=None, stream=None)\n\n"
     "(topk_ids, topk_w) of logits [T, E] (fp32, bf16 or f16; rows may be strided)."},
    {"moe_route_backward", KW(route_backward),
     "moe_route_backward(logits, topk_ids, d_w, score=MOE_SCORE_SOFTMAX, renorm=True, scale=1.0, token_mask=None, "
     "d_logits=None, stream=None)\n\n"
     "d_logits [T, E] (the logits' type) from d_w [T, k], the choice topk_ids held fixed."},
    {"moe_block_norm", KW(block_norm),
     "moe_block_norm(x, y=None, post_weight=None, gate=None, residual_scale=1.0, next_weight=None, eps=1e-6, "
     "x_out=None, h=None, stream=None)\n\n"
     "(x_out, h) = (residual_scale x + gate n(y) post_weight, n(x_out) next_weight).\n\n"
     "x [T, H] is the residual stream, y [T, H] a block's output (None: the norm before a first block alone, no\n"
     "x_out unless one is given); gate [H] (each channel) or [T, 1] (each token).  Without next_weight h is None."},
    {"moe_block_norm_backward", KW(block_norm_backward),
     "moe_block_norm_backward(x, y, d_x_out, d_h, post_weight=None, gate=None, residual_scale=1.0, next_weight=None, "
     "eps=1e-6, d_x=None, d_y=None, d_post_weight=None, d_gate=None, d_next_weight=None, workspace=None, "
     "stream=None)\n\n"
     "(d_x, d_y, d_post_weight, d_gate, d_next_weight) of moe_block_norm; the weights' gradients are fp32, and None\n"
     "where the weight is not given."},
    {"moe_adapter_linear", KW(adapter_linear),
     "moe_adapter_linear(x, weight, lora_a=None, lora_b=None, adapter_ids=None, lora_scale=None, out=None, "
     "out_dtype=None, workspace=None, d_error=None, stream=None)\n\n"
     "out [T, N] = x weight^T + lora_scale[a] (x lora_a[a]^T) lora_b[a]^T, a = adapter_ids[t] (< 0: none).\n\n"
     "x [T, H] and weight [N, H] (rows may be strided), lora_a [n, R, H], lora_b [n, N, R], all bf16 or all f16; out\n"
     "of x's type or fp32.  Without lora_a the projection alone."},
    {"set_check", set_check, METH_VARARGS, "The function that raises for a status other than MOE_OK, and what it raises."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Compiled entry points of short calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
