// ssm_marshal.cpp -- native marshalling behind layers.py: checks the tensors of a call, allocates its outputs and scratch
// with torch on their device, fills the C ABI's argument struct and calls the entry point on torch's current stream.
// Nothing is computed here. A call of these operators is often shorter on the GPU (2 to 10 us) than the same checks in
// Python are on the host; here they take about 1 us.
//
// Arguments are positional and complete; layers.py documents and defaults them.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ssm_scan.h"

namespace {

using at::ScalarType;
using Shape = at::IntArrayRef;

template <typename... A> [[noreturn]] void refuse(PyObject *type, const char *fmt, A... a) {
  PyErr_Format(type, fmt, a...);
  throw python_error();
}

const char *type_name(ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kBool: return "torch.bool";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}
std::string shape_text(Shape s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); i++) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const at::Tensor &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}
int32_t code(const char *name, ScalarType t) {
  if (t != at::kFloat && t != at::kBFloat16) refuse(PyExc_TypeError, "%s must be float32 or bfloat16", name);
  return t == at::kFloat ? SSM_F32 : SSM_BF16;
}

// The call's leading tensor: its device and type are the others'.
struct Lead {
  const at::Tensor &t;
  at::Device dev;
  ScalarType act;
  Lead(const char *name, PyObject *o) : t(tensor(name, o)), dev(t.device()), act(t.scalar_type()) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor (the library has no CPU path)", name);
    code(name, act);
  }
  void check(const char *name, const at::Tensor &u, ScalarType type, Shape shape) const {
    if (u.device() != dev)
      refuse(PyExc_ValueError, "%s must be a CUDA tensor on %s, got %s", name, dev.str().c_str(), u.device().str().c_str());
    if (u.scalar_type() != type)
      refuse(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(u.scalar_type()));
    if (u.sizes() != shape)
      refuse(PyExc_ValueError, "%s must be %s, got %s", name, shape_text(shape).c_str(), shape_text(u.sizes()).c_str());
  }
  // The address of a dense tensor of this type and shape.
  void *need(const char *name, PyObject *o, ScalarType type, Shape shape) const {
    const at::Tensor &u = tensor(name, o);
    check(name, u, type, shape);
    if (!u.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return u.data_ptr();
  }
  void *maybe(const char *name, PyObject *o, ScalarType type, Shape shape) const {
    return o == Py_None ? nullptr : need(name, o, type, shape);
  }
  float *f32(const char *name, PyObject *o, Shape shape) const { return static_cast<float *>(need(name, o, at::kFloat, shape)); }
  float *maybe_f32(const char *name, PyObject *o, Shape shape) const {
    return static_cast<float *>(maybe(name, o, at::kFloat, shape));
  }
  at::Tensor empty(Shape shape, ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  }
};

ScalarType out_type(const char *name, PyObject *o, ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.dtype", name);
  const ScalarType t = reinterpret_cast<THPDtype *>(o)->scalar_type;
  code(name, t);
  return t;
}
float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}
int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// A status as the exception that the other entry points raise.
[[noreturn]] void fail(const char *name, int status) {
  PyObject *m = PyImport_ImportModule("selective_state_space_34_b200._abi");
  if (m) {
    PyObject *r = PyObject_CallMethod(m, "check", "si", name, status);
    Py_XDECREF(r);
    Py_DECREF(m);
  }
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, status);
  throw python_error();
}

// Run an entry point on the current stream of a device, which need not be the current one; other threads may run meanwhile.
template <typename A> void run(const char *name, ssm_status (*fn)(const A *, void *), const A &a, at::Device dev) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != dev.index()) guard.set_device(dev);
  void *stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  PyThreadState *ts = PyEval_SaveThread();
  const ssm_status st = fn(&a, stream);
  PyEval_RestoreThread(ts);
  if (st != SSM_OK) fail(name, st);
}

// Scratch: the caller's workspace where that is large enough, else an allocation; from its first 256-byte boundary.
void *scratch(const Lead &lead, size_t need, PyObject *given, at::Tensor &held) {
  auto align = [](void *p) { return (reinterpret_cast<uintptr_t>(p) + 255) & ~uintptr_t(255); };
  if (given != Py_None) {
    const at::Tensor &w = tensor("workspace", given);
    if (w.device() != lead.dev || !w.is_contiguous())
      refuse(PyExc_ValueError, "workspace must be a contiguous CUDA tensor on %s", lead.dev.str().c_str());
    const uintptr_t at = align(w.data_ptr());
    if (at + need <= reinterpret_cast<uintptr_t>(w.data_ptr()) + w.nbytes()) return reinterpret_cast<void *>(at);
  }
  held = lead.empty({(int64_t)need + 256}, at::kByte);
  return reinterpret_cast<void *>(align(held.data_ptr()));
}

PyObject *wrap(const at::Tensor &t) {
  PyObject *o = THPVariable_Wrap(t);
  if (!o) throw python_error();
  return o;
}
// A dict under construction.
struct Dict {
  PyObject *d = PyDict_New();
  ~Dict() { Py_XDECREF(d); }
  void put(const char *key, const at::Tensor &t) {
    PyObject *o = wrap(t);
    const int bad = PyDict_SetItemString(d, key, o);
    Py_DECREF(o);
    if (bad) throw python_error();
  }
  PyObject *take() {
    PyObject *r = d;
    d = nullptr;
    return r;
  }
};
PyObject *given_or(PyObject *given, const at::Tensor &made) {
  if (given == Py_None) return wrap(made);
  Py_INCREF(given);
  return given;
}

// ---- gated linear recurrence -------------------------------------------------------------------

// x r i lam r_bias i_bias c h0 reset lengths
Lead lru_args(PyObject *const *v, ssm_lru_args &a) {
  Lead x("x", v[0]);
  const Shape s = x.t.sizes();
  if (s.size() != 3) refuse(PyExc_ValueError, "x must be (Bt, Dn, L)");
  const int64_t Bt = s[0], Dn = s[1], L = s[2];
  a.x = x.need("x", v[0], x.act, s);
  a.r = x.need("r", v[1], x.act, s);
  a.i = x.need("i", v[2], x.act, s);
  a.lam = x.f32("lam", v[3], {Dn});
  a.r_bias = x.maybe_f32("r_bias", v[4], {Dn});
  a.i_bias = x.maybe_f32("i_bias", v[5], {Dn});
  a.c = number(v[6]);
  a.h0 = x.maybe_f32("h0", v[7], {Bt, Dn});
  if (v[8] != Py_None) {
    const ScalarType t = tensor("reset", v[8]).scalar_type();
    if (t != at::kBool && t != at::kByte) refuse(PyExc_TypeError, "reset must be bool or uint8");
    a.reset = static_cast<const uint8_t *>(x.need("reset", v[8], t, {Bt, L}));
  }
  a.lengths = static_cast<const int32_t *>(x.maybe("lengths", v[9], at::kInt, {Bt}));
  a.Bt = Bt;
  a.Dn = Dn;
  a.L = L;
  a.in_dtype = code("x", x.act);
  return x;
}

// + out_dtype save_states return_state out
PyObject *lru_fwd(PyObject *const *v) {
  ssm_lru_args a = {};
  const Lead x = lru_args(v, a);
  const ScalarType od = out_type("out_dtype", v[10], x.act);
  const bool states = truth(v[11]), state = truth(v[12]);
  at::Tensor out, st, hl;
  if (v[13] == Py_None) {
    out = x.empty(x.t.sizes(), od);
    a.out = out.data_ptr();
  } else {
    a.out = x.need("out", v[13], od, x.t.sizes());
  }
  a.out_dtype = code("out_dtype", od);
  if (states) {
    st = x.empty({a.Bt, a.Dn, ssm_lru_num_states(a.L)}, at::kFloat);
    a.chunk_states = st.data_ptr<float>();
  }
  if (state) {
    hl = x.empty({a.Bt, a.Dn}, at::kFloat);
    a.h_last = hl.data_ptr<float>();
  }
  run("ssm_lru_fwd", ssm_lru_fwd, a, x.dev);
  if (!states && !state) return given_or(v[13], out);
  Dict d;
  PyObject *o = given_or(v[13], out);
  const int bad = PyDict_SetItemString(d.d, "out", o);
  Py_DECREF(o);
  if (bad) throw python_error();
  if (states) d.put("chunk_states", st);
  if (state) d.put("h_last", hl);
  return d.take();
}

// dout, the ten of lru_args, chunk_states dh_last grad_dtype workspace
PyObject *lru_bwd(PyObject *const *v) {
  ssm_lru_bwd_args q = {};
  ssm_lru_args &a = q.fwd;
  const Lead x = lru_args(v + 1, a);
  const Shape s = x.t.sizes();
  q.dout = x.need("dout", v[0], x.act, s);
  a.chunk_states = x.maybe_f32("chunk_states", v[11], {a.Bt, a.Dn, ssm_lru_num_states(a.L)});
  q.dh_last = x.maybe_f32("dh_last", v[12], {a.Bt, a.Dn});
  const ScalarType gd = out_type("grad_dtype", v[13], at::kFloat);
  q.grad_dtype = code("grad_dtype", gd);
  Dict d;
  auto make = [&](const char *name, Shape shape, ScalarType type) {
    const at::Tensor t = x.empty(shape, type);
    d.put(name, t);
    return t.data_ptr();
  };
  q.dx = make("dx", s, gd);
  q.dr = make("dr", s, gd);
  q.di = make("di", s, gd);
  q.dlam = static_cast<float *>(make("dlam", {a.Dn}, at::kFloat));
  if (a.r_bias || v[5] != Py_None) q.dr_bias = static_cast<float *>(make("dr_bias", {a.Dn}, at::kFloat));
  if (a.i_bias || v[6] != Py_None) q.di_bias = static_cast<float *>(make("di_bias", {a.Dn}, at::kFloat));
  if (v[8] != Py_None || v[12] != Py_None) q.dh0 = static_cast<float *>(make("dh0", {a.Bt, a.Dn}, at::kFloat));
  at::Tensor ws;
  if (const size_t need = ssm_lru_bwd_workspace_size(&q)) {
    q.workspace = scratch(x, need, v[14], ws);
    q.workspace_bytes = need;
  }
  run("ssm_lru_bwd", ssm_lru_bwd, q, x.dev);
  return d.take();
}

// x r i lam h r_bias i_bias c out_dtype out
PyObject *lru_step(PyObject *const *v) {
  const Lead x("x", v[0]);
  const Shape s = x.t.sizes();
  if (s.size() != 2) refuse(PyExc_ValueError, "x must be (Bt, Dn)");
  const int64_t Dn = s[1];
  ssm_lru_step_args a = {};
  a.x = x.need("x", v[0], x.act, s);
  a.r = x.need("r", v[1], x.act, s);
  a.i = x.need("i", v[2], x.act, s);
  a.lam = x.f32("lam", v[3], {Dn});
  a.h = x.f32("h", v[4], s);
  a.r_bias = x.maybe_f32("r_bias", v[5], {Dn});
  a.i_bias = x.maybe_f32("i_bias", v[6], {Dn});
  a.c = number(v[7]);
  const ScalarType od = out_type("out_dtype", v[8], x.act);
  at::Tensor out;
  if (v[9] == Py_None) {
    out = x.empty(s, od);
    a.out = out.data_ptr();
  } else {
    a.out = x.need("out", v[9], od, s);
  }
  a.Bt = s[0];
  a.Dn = Dn;
  a.in_dtype = code("x", x.act);
  a.out_dtype = code("out_dtype", od);
  run("ssm_lru_step", ssm_lru_step, a, x.dev);
  return given_or(v[9], out);
}

// ---- queries and keys --------------------------------------------------------------------------

// Batch, head and row stride of a (Bt, L, H, D) or, with time innermost, (Bt, H, D, L) tensor whose last axis is dense.
struct Heads {
  void *p;
  int64_t sb, sh, sr;
};
Heads heads(const Lead &lead, const char *name, PyObject *o, ScalarType type, Shape shape, bool time) {
  const at::Tensor &u = tensor(name, o);
  lead.check(name, u, type, shape);
  const Shape st = u.strides();
  if (st[3] != 1 && shape[3] > 1) refuse(PyExc_ValueError, "%s must be contiguous along its last axis", name);
  return {u.data_ptr(), st[0], time ? st[1] : st[2], time ? st[2] : st[1]};
}
#define SSM_PUT_HEADS(args, field, h) \
  do {                                \
    const Heads h_ = (h);             \
    (args).field = h_.p;              \
    (args).field##_sb = h_.sb;        \
    (args).field##_sh = h_.sh;        \
    (args).field##_sr = h_.sr;        \
  } while (0)

struct QkShapes {
  Lead q;
  bool time, keys;
  std::array<int64_t, 4> k;  // shape of k
};
// q k q_weight k_weight inv_freq positions pos0 norm eps interleaved rot_scale layout
QkShapes qk_args(PyObject *const *v, ssm_qk_args &a) {
  const Lead q("q", v[0]);
  a.layout = (int32_t)integer(v[11]);
  QkShapes r{q, a.layout == SSM_QK_TIME_LAST, v[1] != Py_None, {}};
  const Shape s = q.t.sizes();
  if (s.size() != 4) refuse(PyExc_ValueError, "q must be 4-dimensional, got %s", shape_text(s).c_str());
  const int head = r.time ? 1 : 2;
  a.Bt = s[0];
  a.L = r.time ? s[3] : s[1];
  a.D = r.time ? s[2] : s[3];
  a.Hq = s[head];
  SSM_PUT_HEADS(a, q, heads(q, "q", v[0], q.act, s, r.time));
  if (r.keys) {
    const at::Tensor &k = tensor("k", v[1]);
    if (k.dim() != 4) refuse(PyExc_ValueError, "k must be 4-dimensional, got %s", shape_text(k.sizes()).c_str());
    std::copy(s.begin(), s.end(), r.k.begin());
    r.k[head] = a.Hk = k.size(head);
    SSM_PUT_HEADS(a, k, heads(q, "k", v[1], q.act, r.k, r.time));
  } else if (v[3] != Py_None) {
    refuse(PyExc_ValueError, "k_weight without k");
  }
  a.q_weight = q.maybe_f32("q_weight", v[2], {a.D});
  a.k_weight = q.maybe_f32("k_weight", v[3], {a.D});
  a.norm = truth(v[7]);
  if (!a.norm && (v[2] != Py_None || v[3] != Py_None)) refuse(PyExc_ValueError, "weights need norm=True");
  if (v[4] != Py_None) {
    const at::Tensor &f = tensor("inv_freq", v[4]);
    const ScalarType t = f.scalar_type();
    if (t != at::kFloat && t != at::kDouble) refuse(PyExc_TypeError, "inv_freq must be float32 or float64");
    if (f.dim() != 1) refuse(PyExc_ValueError, "inv_freq must be (rot / 2,)");
    if (2 * f.size(0) > a.D)
      refuse(PyExc_ValueError, "inv_freq has %lld pairs, more than the %lld elements of a head hold", (long long)f.size(0),
             (long long)a.D);
    a.inv_freq = q.need("inv_freq", v[4], t, f.sizes());
    a.freq_f64 = t == at::kDouble;
    a.rot = 2 * f.size(0);
  }
  if (v[5] != Py_None) {
    const ScalarType t = tensor("positions", v[5]).scalar_type();
    if (t != at::kInt && t != at::kLong) refuse(PyExc_TypeError, "positions must be int32 or int64");
    a.positions = q.need("positions", v[5], t, {a.Bt, a.L});
    a.pos_i64 = t == at::kLong;
  }
  a.pos0 = integer(v[6]);
  a.eps = number(v[8]);
  a.interleaved = truth(v[9]);
  a.rot_scale = number(v[10]);
  a.in_dtype = code("q", q.act);
  return r;
}

PyObject *pair(PyObject *a, PyObject *b) {
  PyObject *t = PyTuple_Pack(2, a, b);
  Py_DECREF(a);
  Py_DECREF(b);
  if (!t) throw python_error();
  return t;
}
PyObject *held(PyObject *o) {
  Py_INCREF(o);
  return o;
}

// + out_dtype q_out k_out
PyObject *qk_fwd(PyObject *const *v) {
  ssm_qk_args a = {};
  const QkShapes r = qk_args(v, a);
  const ScalarType od = out_type("out_dtype", v[12], r.q.act);
  a.out_dtype = code("out_dtype", od);
  PyObject *qo = nullptr, *ko = nullptr;
  try {  // any of these may throw, an allocation without room too
    qo = v[13] == Py_None ? wrap(r.q.empty(r.q.t.sizes(), od)) : held(v[13]);
    ko = r.keys && v[14] == Py_None ? wrap(r.q.empty(r.k, od)) : held(r.keys ? v[14] : Py_None);
    SSM_PUT_HEADS(a, q_out, heads(r.q, "q_out", qo, od, r.q.t.sizes(), r.time));
    if (r.keys) SSM_PUT_HEADS(a, k_out, heads(r.q, "k_out", ko, od, r.k, r.time));
    run("ssm_qk_norm_rope_fwd", ssm_qk_norm_rope_fwd, a, r.q.dev);
  } catch (...) {
    Py_XDECREF(qo);
    Py_XDECREF(ko);
    throw;
  }
  return pair(qo, ko);
}

// dq_out dk_out, the twelve of qk_args, grad_dtype workspace
PyObject *qk_bwd(PyObject *const *v) {
  ssm_qk_bwd_args b = {};
  ssm_qk_args &a = b.fwd;
  if ((v[1] == Py_None) != (v[3] == Py_None)) refuse(PyExc_ValueError, "k and dk_out come together");
  const QkShapes r = qk_args(v + 2, a);
  const Lead dq("dq_out", v[0]);
  const ScalarType gd = out_type("grad_dtype", v[14], at::kFloat);
  b.dout_dtype = code("dq_out", dq.act);
  b.grad_dtype = code("grad_dtype", gd);
  Dict d;
  const Heads g = heads(r.q, "dq_out", v[0], dq.act, r.q.t.sizes(), r.time);
  b.dq_out = g.p;
  a.q_out_sb = g.sb;
  a.q_out_sh = g.sh;
  a.q_out_sr = g.sr;
  auto make = [&](const char *name, Shape shape, int64_t &sb, int64_t &sh, int64_t &sr) {
    const at::Tensor t = r.q.empty(shape, gd);
    d.put(name, t);
    const Shape st = t.strides();
    sb = st[0];
    sh = r.time ? st[1] : st[2];
    sr = r.time ? st[2] : st[1];
    return t.data_ptr();
  };
  b.dq = make("dq", r.q.t.sizes(), b.dq_sb, b.dq_sh, b.dq_sr);
  if (r.keys) {
    const Heads h = heads(r.q, "dk_out", v[1], dq.act, r.k, r.time);
    b.dk_out = h.p;
    a.k_out_sb = h.sb;
    a.k_out_sh = h.sh;
    a.k_out_sr = h.sr;
    b.dk = make("dk", r.k, b.dk_sb, b.dk_sh, b.dk_sr);
  }
  auto weight = [&](const char *name) {
    const at::Tensor t = r.q.empty({a.D}, at::kFloat);
    d.put(name, t);
    return t.data_ptr<float>();
  };
  if (v[4] != Py_None) b.dq_weight = weight("dq_weight");
  if (v[5] != Py_None) b.dk_weight = weight("dk_weight");
  at::Tensor ws;
  if (const size_t need = ssm_qk_norm_rope_bwd_workspace_size(&b)) {
    b.workspace = scratch(r.q, need, v[15], ws);
    b.workspace_bytes = need;
  }
  run("ssm_qk_norm_rope_bwd", ssm_qk_norm_rope_bwd, b, r.q.dev);
  return d.take();
}

// ---- state-space-dual step ---------------------------------------------------------------------

// x dt A_log B C h D dt_bias delta_softplus out_dtype discretization out
PyObject *ssd_step(PyObject *const *v) {
  const Lead x("x", v[0]);
  const Shape s = x.t.sizes();
  if (s.size() != 3) refuse(PyExc_ValueError, "x must be (Bt, H, P)");
  const at::Tensor &B = tensor("B", v[3]);
  if (B.dim() != 2) refuse(PyExc_ValueError, "B must be (Bt, N)");
  ssm_ssd_step_args a = {};
  a.Bt = s[0];
  a.H = s[1];
  a.P = s[2];
  a.N = B.size(1);
  a.x = x.need("x", v[0], x.act, s);
  a.dt = x.need("dt", v[1], x.act, {a.Bt, a.H});
  a.A_log = x.f32("A_log", v[2], {a.H});
  a.B = x.need("B", v[3], x.act, {a.Bt, a.N});
  a.C = x.need("C", v[4], x.act, {a.Bt, a.N});
  a.h = x.f32("h", v[5], {a.Bt, a.H, a.N, a.P});
  a.D = x.maybe_f32("D", v[6], {a.H});
  a.dt_bias = x.maybe_f32("dt_bias", v[7], {a.H});
  a.delta_softplus = truth(v[8]);
  const ScalarType od = out_type("out_dtype", v[9], x.act);
  a.discretization = (int32_t)integer(v[10]);
  at::Tensor out;
  if (v[11] == Py_None) {
    out = x.empty(s, od);
    a.out = out.data_ptr();
  } else {
    a.out = x.need("out", v[11], od, s);
  }
  a.in_dtype = code("x", x.act);
  a.out_dtype = code("out_dtype", od);
  run("ssm_ssd_step", ssm_ssd_step, a, x.dev);
  return given_or(v[11], out);
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) refuse(PyExc_TypeError, "%d arguments are wanted, got %zd", N, n);
  return F(v);
  END_HANDLE_TH_ERRORS
}
#define SSM_METHOD(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {SSM_METHOD(lru_fwd, 14), SSM_METHOD(lru_bwd, 15), SSM_METHOD(lru_step, 10), SSM_METHOD(qk_fwd, 15),
                         SSM_METHOD(qk_bwd, 16),  SSM_METHOD(ssd_step, 12), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", SSM_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
