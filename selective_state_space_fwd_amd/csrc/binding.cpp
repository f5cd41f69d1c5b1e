// The short way from Python into the entry points of block.py (conv, conv_step, scan_step,
// ssd_step, norm and the gradients) and of linattn.py (linattn, linattn_step, qk_norm and the
// gradients), which a decode loop or a training step makes once per layer and where marshalling
// through ctypes can take longer than the kernels. Each function here takes
// the arguments of its Python namesake in order, and either
//   * makes the call, when every argument is what the C ABI takes as it stands (a device tensor
//     of the right dtype and shape, on the current device, contiguous or strided where the ABI
//     takes strides), and returns its result, or
//   * returns None without having done anything; block.py or linattn.py then looks at the
//     arguments one by one, copies what needs copying, switches devices, or names what is wrong.
// So the checks here decide only which way a call goes, and those stay the one place that
// refuses arguments. The library's functions come in as addresses (bind).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "ssm_conv.h"
#include "ssm_linattn.h"
#include "ssm_norm.h"
#include "ssm_qk.h"
#include "ssm_step.h"

namespace {

decltype(&ssm_conv_fwd) g_conv_fwd;
decltype(&ssm_conv_step) g_conv_step;
decltype(&ssm_scan_step) g_scan_step;
decltype(&ssm_ssd_step) g_ssd_step;
decltype(&ssm_norm_fwd) g_norm_fwd;
decltype(&ssm_conv_bwd) g_conv_bwd;
decltype(&ssm_conv_bwd_workspace_bytes) g_conv_ws;
decltype(&ssm_norm_bwd) g_norm_bwd;
decltype(&ssm_norm_bwd_workspace_bytes) g_norm_ws;
decltype(&ssm_norm_fwd_workspace_bytes) g_norm_fwd_ws;
decltype(&ssm_linattn_fwd) g_linattn_fwd;
decltype(&ssm_linattn_fwd_workspace_bytes) g_linattn_fwd_ws;
decltype(&ssm_linattn_bwd) g_linattn_bwd;
decltype(&ssm_linattn_bwd_workspace_bytes) g_linattn_bwd_ws;
decltype(&ssm_linattn_step) g_linattn_step;
decltype(&ssm_qk_norm_fwd) g_qk_fwd;
decltype(&ssm_qk_norm_bwd) g_qk_bwd;
decltype(&ssm_qk_norm_bwd_workspace_bytes) g_qk_bwd_ws;
PyObject* g_error;  // SsmScanError

// An argument as a tensor: a plain torch.Tensor, or None (`t` undefined). `ok` turns false for
// anything else, a view whose memory holds the negative of its values among them.
struct Arg {
  const at::Tensor* t = nullptr;
  Arg(PyObject* o, bool* ok) {
    if (o == Py_None) return;
    if (THPVariable_CheckExact(o) && !THPVariable_Unpack(o).is_neg())
      t = &THPVariable_Unpack(o);
    else
      *ok = false;
  }
  explicit operator bool() const { return t != nullptr; }
  const at::Tensor* operator->() const { return t; }
  const void* data() const { return t ? t->const_data_ptr() : nullptr; }
  void* mut() const { return t ? t->data_ptr() : nullptr; }
};

// A call wrote t in place: autograd, if it holds t for a backward pass, has to see that.
void wrote(const Arg& t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

bool flag_of(PyObject* o, bool* ok) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    *ok = false;
  }
  return v > 0;
}

// t has this type and shape and is on device dev (and contiguous).
bool is(const Arg& t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  return t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->layout() == at::kStrided &&
         t->sizes() == at::IntArrayRef(shape.begin(), shape.size());
}
bool dense(const Arg& t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  return is(t, type, dev, shape) && t->is_contiguous();
}
bool dense_or_none(const Arg& t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  return !t || dense(t, type, dev, shape);
}
// Rows with the last axis contiguous.
bool rows(const Arg& t, at::ScalarType type, int dev, int64_t n, int64_t cols) {
  return is(t, type, dev, {n, cols}) && (cols <= 1 || t->stride(1) == 1);
}
// [batch, dim, seqlen] with the steps or the channels contiguous.
bool ordered(const Arg& t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  return is(t, type, dev, shape) &&
         (t->size(2) <= 1 || t->stride(2) == 1 || (t->size(1) > 1 && t->stride(1) == 1));
}

// The storage type's flag, or -1.
int io_of(const Arg& t) {
  return t->scalar_type() == at::kBFloat16 ? int(SSM_IO_BF16) : t->scalar_type() == at::kFloat ? int(SSM_IO_F32) : -1;
}

// The device of the call: t's, if it is the current one, else -1.
int device_of(const Arg& t) {
  return t && t->is_cuda() && t->get_device() == c10::hip::current_device() ? int(t->get_device()) : -1;
}

void* stream_of(int dev) { return c10::hip::getCurrentHIPStream(dev).stream(); }

// The interpreter's lock given up, and taken back however the scope ends.
struct Unlocked {
  PyThreadState* s = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(s); }
};

// The call f() without the interpreter's lock; false with the error set if it fails.
template <typename F>
bool made(F f) {
  int status;
  {
    const Unlocked u;
    status = f();
  }
  if (status == SSM_OK) return true;
  PyObject* e = PyObject_CallFunction(g_error, "i", status);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return false;
}

// The result: the caller's own tensor again, or the one made here.
PyObject* give(PyObject* own, const at::Tensor& t) {
  if (own == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(own);
  return own;
}

#define SSM_NEED(cond) \
  if (!(cond)) Py_RETURN_NONE

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kFunctions = 10;
  if (n != kFunctions + 1) {
    PyErr_SetString(PyExc_TypeError, "bind takes ten addresses and the error class");
    return nullptr;
  }
  void* f[kFunctions];
  for (int i = 0; i < kFunctions; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_conv_fwd = reinterpret_cast<decltype(g_conv_fwd)>(f[0]);
  g_conv_step = reinterpret_cast<decltype(g_conv_step)>(f[1]);
  g_scan_step = reinterpret_cast<decltype(g_scan_step)>(f[2]);
  g_ssd_step = reinterpret_cast<decltype(g_ssd_step)>(f[3]);
  g_norm_fwd = reinterpret_cast<decltype(g_norm_fwd)>(f[4]);
  g_conv_bwd = reinterpret_cast<decltype(g_conv_bwd)>(f[5]);
  g_conv_ws = reinterpret_cast<decltype(g_conv_ws)>(f[6]);
  g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(f[7]);
  g_norm_ws = reinterpret_cast<decltype(g_norm_ws)>(f[8]);
  g_norm_fwd_ws = reinterpret_cast<decltype(g_norm_fwd_ws)>(f[9]);
  Py_INCREF(a[kFunctions]);
  Py_XDECREF(g_error);
  g_error = a[kFunctions];
  Py_RETURN_NONE;
}

// An uninitialised tensor of t's shape and contiguous axis.
at::Tensor empty_in_order(const Arg& t) {
  const int64_t b = t->size(0), d = t->size(1), L = t->size(2);
  if (L <= 1 || t->stride(2) == 1) return at::empty({b, d, L}, t->options());
  return at::empty({b, L, d}, t->options()).transpose(1, 2);
}

// A workspace of `need` bytes: the caller's, or one made here (`made_ws`). Null if neither will do.
void* workspace_of(const Arg& ws, int64_t need, int dev, const at::Tensor& like, at::Tensor* made_ws, int64_t* bytes) {
  if (need < 0) return nullptr;
  if (ws) {
    if (ws->scalar_type() != at::kByte || !ws->is_cuda() || ws->get_device() != dev || !ws->is_contiguous() ||
        ws->numel() < need)
      return nullptr;
    *bytes = ws->numel();
    return ws.mut();
  }
  *bytes = need > 0 ? need : 1;
  *made_ws = at::empty({*bytes}, like.options().dtype(at::kByte));
  return made_ws->data_ptr();
}

// A new tuple of results; an undefined tensor is None.
PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New(Py_ssize_t(ts.size()));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None);
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// conv(x, weight, bias, silu, initial_state, lengths, out, final_state, return_final_state)
PyObject* conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 9;
  SSM_NEED(ok && g_conv_fwd);
  const Arg x(a[0], &ok), w(a[1], &ok), bias(a[2], &ok), init(a[4], &ok), lengths(a[5], &ok), out(a[6], &ok),
      fin(a[7], &ok);
  const bool silu = flag_of(a[3], &ok), want = flag_of(a[8], &ok);
  SSM_NEED(ok && x && w && x->dim() == 3 && w->dim() == 2);
  const int dev = device_of(x), io = io_of(x);
  const at::ScalarType type = x->scalar_type();
  const int64_t b = x->size(0), d = x->size(1), L = x->size(2), W = w->size(1);
  SSM_NEED(dev >= 0 && io >= 0 && W >= 2 && ordered(x, type, dev, {b, d, L}) &&
           dense(w, at::kFloat, dev, {d, W}) && dense_or_none(bias, at::kFloat, dev, {d}) &&
           dense_or_none(init, type, dev, {b, d, W - 1}) && dense_or_none(lengths, at::kInt, dev, {b}) &&
           dense_or_none(out, type, dev, {b, d, L}) && dense_or_none(fin, type, dev, {b, d, W - 1}));
  at::Tensor made_out, made_fin;
  if (!out) made_out = at::empty({b, d, L}, x->options());
  if (!fin && want) made_fin = at::empty({b, d, W - 1}, x->options());
  void* op = out ? out.mut() : made_out.data_ptr();
  void* fp = fin ? fin.mut() : want ? made_fin.data_ptr() : nullptr;
  const int64_t strides[3] = {x->stride(0), x->stride(1), x->stride(2)};
  if (!made([&] {
        return g_conv_fwd(x.data(), strides, static_cast<const float*>(w.data()),
                          static_cast<const float*>(bias.data()), init.data(),
                          static_cast<const int32_t*>(lengths.data()), uint32_t(io) | (silu ? SSM_CONV_SILU : 0),
                          op, fp, b, d, W, L, stream_of(dev));
      }))
    return nullptr;
  wrote(out);
  wrote(fin);
  PyObject* o = give(a[6], made_out);
  PyObject* f = fin || want ? give(a[7], made_fin) : (Py_INCREF(Py_None), Py_None);
  PyObject* both = PyTuple_Pack(2, o, f);
  Py_DECREF(o);
  Py_DECREF(f);
  return both;
  END_HANDLE_TH_ERRORS
}

// conv_step(x, state, weight, bias, silu, slots, out)
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 7;
  SSM_NEED(ok && g_conv_step);
  const Arg x(a[0], &ok), state(a[1], &ok), w(a[2], &ok), bias(a[3], &ok), slots(a[5], &ok), out(a[6], &ok);
  const bool silu = flag_of(a[4], &ok);
  SSM_NEED(ok && x && state && w && x->dim() == 2 && state->dim() == 3);
  const int dev = device_of(x), io = io_of(x);
  const at::ScalarType type = x->scalar_type();
  const int64_t b = x->size(0), d = x->size(1), ns = state->size(0), past = state->size(2);
  SSM_NEED(dev >= 0 && io >= 0 && rows(x, type, dev, b, d) && dense(state, type, dev, {ns, d, past}) &&
           dense(w, at::kFloat, dev, {d, past + 1}) && dense_or_none(bias, at::kFloat, dev, {d}) &&
           dense_or_none(slots, at::kInt, dev, {b}) && dense_or_none(out, type, dev, {b, d}));
  at::Tensor made_out;
  if (!out) made_out = at::empty({b, d}, x->options());
  void* op = out ? out.mut() : made_out.data_ptr();
  if (!made([&] {
        return g_conv_step(x.data(), x->stride(0), state.mut(), static_cast<const float*>(w.data()),
                           static_cast<const float*>(bias.data()), static_cast<const int32_t*>(slots.data()),
                           uint32_t(io) | (silu ? SSM_CONV_SILU : 0), op, b, ns, d, past + 1, stream_of(dev));
      }))
    return nullptr;
  wrote(state);
  wrote(out);
  return give(a[6], made_out);
  END_HANDLE_TH_ERRORS
}

// state_step(per_head, x, dt, A, B, C, state, D, z, dt_bias, softplus, slots, out)
PyObject* state_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 13;
  SSM_NEED(ok && g_scan_step);
  const bool per_head = flag_of(a[0], &ok), softplus = flag_of(a[10], &ok);
  const Arg x(a[1], &ok), dt(a[2], &ok), A(a[3], &ok), B(a[4], &ok), C(a[5], &ok), state(a[6], &ok), D(a[7], &ok),
      z(a[8], &ok), bias(a[9], &ok), slots(a[11], &ok), out(a[12], &ok);
  SSM_NEED(ok && x && dt && A && B && C && state && x->dim() == 2 && state->dim() == 3 &&
           A->dim() == (per_head ? 1 : 2));
  const int dev = device_of(x), io = io_of(x);
  const at::ScalarType type = x->scalar_type();
  const int64_t b = x->size(0), d = x->size(1), ns = state->size(0), N = state->size(2), heads = A->size(0);
  SSM_NEED(heads > 0 && d % heads == 0);
  SSM_NEED(dev >= 0 && io >= 0 && rows(x, type, dev, b, d) && rows(dt, type, dev, b, heads) &&
           rows(B, type, dev, b, N) && rows(C, type, dev, b, N) && dense(state, at::kFloat, dev, {ns, d, N}) &&
           (per_head ? dense(A, at::kFloat, dev, {heads}) : dense(A, at::kFloat, dev, {d, N})) &&
           dense_or_none(D, at::kFloat, dev, {d}) && (!z || rows(z, type, dev, b, d)) &&
           dense_or_none(bias, at::kFloat, dev, {heads}) && dense_or_none(slots, at::kInt, dev, {b}) &&
           dense_or_none(out, type, dev, {b, d}));
  at::Tensor made_out;
  if (!out) made_out = at::empty({b, d}, x->options());
  void* op = out ? out.mut() : made_out.data_ptr();
  const auto f32 = [](const Arg& t) { return static_cast<const float*>(t.data()); };
  const uint32_t flags = uint32_t(io) | (softplus ? SSM_DELTA_SOFTPLUS : 0);
  const int64_t zs = z ? z->stride(0) : 0;
  if (!made([&] {
        const auto* sl = static_cast<const int32_t*>(slots.data());
        float* st = static_cast<float*>(state.mut());
        return per_head ? g_ssd_step(x.data(), x->stride(0), dt.data(), dt->stride(0), f32(A), B.data(), B->stride(0),
                                     C.data(), C->stride(0), f32(D), z.data(), zs, f32(bias), sl, flags, st, op, b,
                                     ns, heads, d / heads, N, stream_of(dev))
                        : g_scan_step(x.data(), x->stride(0), dt.data(), dt->stride(0), f32(A), B.data(),
                                      B->stride(0), C.data(), C->stride(0), f32(D), z.data(), zs, f32(bias), sl,
                                      flags, st, op, b, ns, d, N, stream_of(dev));
      }))
    return nullptr;
  wrote(state);
  wrote(out);
  return give(a[12], made_out);
  END_HANDLE_TH_ERRORS
}

// norm(y, weight, z, eps, groups, norm_before_gate, token_major, out, save): (out, rstd or None)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 9;
  SSM_NEED(ok && g_norm_fwd && PyFloat_CheckExact(a[3]) && PyLong_CheckExact(a[4]));
  const Arg y(a[0], &ok), w(a[1], &ok), z(a[2], &ok), out(a[7], &ok);
  const bool first = flag_of(a[5], &ok), token = flag_of(a[6], &ok), save = flag_of(a[8], &ok);
  const double eps = PyFloat_AS_DOUBLE(a[3]);
  const long groups = PyLong_AsLong(a[4]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    ok = false;
  }
  SSM_NEED(ok && y && w && y->dim() == 3 && groups >= 1);
  const int dev = device_of(y), io = io_of(y);
  const at::ScalarType type = y->scalar_type();
  const int64_t b = y->size(0), d = y->size(1), L = y->size(2);
  SSM_NEED(dev >= 0 && io >= 0 && d % groups == 0 && ordered(y, type, dev, {b, d, L}) &&
           (!z || ordered(z, type, dev, {b, d, L})) && dense(w, at::kFloat, dev, {d}) &&
           (!out || (token ? dense(out, type, dev, {b, L, d}) : dense(out, type, dev, {b, d, L}))));
  at::Tensor made_out, rstd;
  if (!out) made_out = token ? at::empty({b, L, d}, y->options()) : at::empty({b, d, L}, y->options());
  if (save) rstd = at::empty({b, groups, L}, y->options().dtype(at::kFloat));
  // Not needed, and not made, for a decode step: channels contiguous throughout, and nothing that
  // the library could take for steps contiguous (one channel, or both at once).
  at::Tensor made_ws;
  int64_t bytes = 0;
  void* wp = nullptr;
  const auto channels = [&](const Arg& t) { return t->stride(1) == 1 && (L == 1 || t->stride(2) != 1); };
  if (d == 1 || !channels(y) || (z && !channels(z)) || !(token || L == 1) || d / groups > 4096) {
    wp = workspace_of(Arg(Py_None, &ok), g_norm_fwd_ws(b, d, groups, L, uint32_t(io)), dev, *y.t, &made_ws, &bytes);
    SSM_NEED(wp);
  }
  void* op = out ? out.mut() : made_out.data_ptr();
  const int64_t ys[3] = {y->stride(0), y->stride(1), y->stride(2)}, os[3] = {L * d, 1, d};
  int64_t zs[3] = {0, 0, 0};
  if (z)
    for (int i = 0; i < 3; ++i) zs[i] = z->stride(i);
  if (!made([&] {
        return g_norm_fwd(y.data(), ys, z.data(), z ? zs : nullptr, static_cast<const float*>(w.data()), float(eps),
                          uint32_t(io) | (first ? SSM_NORM_BEFORE_GATE : 0), op, token ? os : nullptr,
                          save ? static_cast<float*>(rstd.data_ptr()) : nullptr, wp, bytes, b, d, groups, L,
                          stream_of(dev));
      }))
    return nullptr;
  wrote(out);
  PyObject* o = give(a[7], made_out);
  PyObject* r = save ? THPVariable_Wrap(rstd) : (Py_INCREF(Py_None), Py_None);
  PyObject* both = PyTuple_Pack(2, o, r);
  Py_DECREF(o);
  Py_DECREF(r);
  return both;
  END_HANDLE_TH_ERRORS
}

// conv_backward(x, weight, dout, bias, silu, initial_state, lengths, dfinal, want_dinitial, workspace):
// (dx, dweight, dbias or None, dinitial or None)
PyObject* conv_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 10;
  SSM_NEED(ok && g_conv_bwd);
  const Arg x(a[0], &ok), w(a[1], &ok), g(a[2], &ok), bias(a[3], &ok), init(a[5], &ok), lengths(a[6], &ok),
      dfin(a[7], &ok), ws(a[9], &ok);
  const bool silu = flag_of(a[4], &ok), want = a[8] == Py_None ? bool(init) : flag_of(a[8], &ok);
  SSM_NEED(ok && x && w && g && x->dim() == 3 && w->dim() == 2);
  const int dev = device_of(x), io = io_of(x);
  const at::ScalarType type = x->scalar_type();
  const int64_t b = x->size(0), d = x->size(1), L = x->size(2), W = w->size(1);
  SSM_NEED(dev >= 0 && io >= 0 && W >= 2 && ordered(x, type, dev, {b, d, L}) &&
           dense(w, at::kFloat, dev, {d, W}) && dense(g, type, dev, {b, d, L}) &&
           dense_or_none(bias, at::kFloat, dev, {d}) && dense_or_none(init, type, dev, {b, d, W - 1}) &&
           dense_or_none(lengths, at::kInt, dev, {b}) && dense_or_none(dfin, type, dev, {b, d, W - 1}));
  const uint32_t flags = uint32_t(io) | (silu ? SSM_CONV_SILU : 0);
  at::Tensor made_ws;
  int64_t bytes = 0;
  void* wp = workspace_of(ws, g_conv_ws(b, d, W, L, flags), dev, *x.t, &made_ws, &bytes);
  SSM_NEED(wp);
  const at::Tensor dx = empty_in_order(x), dw = at::empty({d, W}, w->options());
  const at::Tensor db = bias ? at::empty({d}, w->options()) : at::Tensor();
  const at::Tensor di = want ? at::empty({b, d, W - 1}, x->options()) : at::Tensor();
  const int64_t xs[3] = {x->stride(0), x->stride(1), x->stride(2)}, ds[3] = {dx.stride(0), dx.stride(1), dx.stride(2)};
  if (!made([&] {
        return g_conv_bwd(x.data(), xs, static_cast<const float*>(w.data()), static_cast<const float*>(bias.data()),
                          init.data(), static_cast<const int32_t*>(lengths.data()), flags, g.data(), dfin.data(),
                          dx.data_ptr(), ds, static_cast<float*>(dw.data_ptr()),
                          bias ? static_cast<float*>(db.data_ptr()) : nullptr, want ? di.data_ptr() : nullptr, wp,
                          bytes, b, d, W, L, stream_of(dev));
      }))
    return nullptr;
  return tuple_of({dx, dw, db, di});
  END_HANDLE_TH_ERRORS
}

// norm_backward(y, weight, rstd, dout, z, groups, norm_before_gate, token_major, workspace):
// (dy, dz or None, dweight)
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 9;
  SSM_NEED(ok && g_norm_bwd && PyLong_CheckExact(a[5]));
  const Arg y(a[0], &ok), w(a[1], &ok), rstd(a[2], &ok), g(a[3], &ok), z(a[4], &ok), ws(a[8], &ok);
  const bool first = flag_of(a[6], &ok), token = flag_of(a[7], &ok);
  const long groups = PyLong_AsLong(a[5]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    ok = false;
  }
  SSM_NEED(ok && y && w && rstd && g && y->dim() == 3 && groups >= 1);
  const int dev = device_of(y), io = io_of(y);
  const at::ScalarType type = y->scalar_type();
  const int64_t b = y->size(0), d = y->size(1), L = y->size(2);
  SSM_NEED(dev >= 0 && io >= 0 && d % groups == 0 && ordered(y, type, dev, {b, d, L}) &&
           (!z || ordered(z, type, dev, {b, d, L})) && dense(w, at::kFloat, dev, {d}) &&
           dense(rstd, at::kFloat, dev, {b, groups, L}) &&
           (token ? dense(g, type, dev, {b, L, d}) : dense(g, type, dev, {b, d, L})));
  const uint32_t flags = uint32_t(io) | (first ? SSM_NORM_BEFORE_GATE : 0);
  at::Tensor made_ws;
  int64_t bytes = 0;
  void* wp = workspace_of(ws, g_norm_ws(b, d, groups, L, flags), dev, *y.t, &made_ws, &bytes);
  SSM_NEED(wp);
  const at::Tensor dy = empty_in_order(y), dz = z ? empty_in_order(z) : at::Tensor();
  const at::Tensor dw = at::empty({d}, w->options());
  const int64_t ys[3] = {y->stride(0), y->stride(1), y->stride(2)}, gs[3] = {L * d, 1, d};
  const int64_t dys[3] = {dy.stride(0), dy.stride(1), dy.stride(2)};
  int64_t zs[3] = {0, 0, 0}, dzs[3] = {0, 0, 0};
  if (z)
    for (int i = 0; i < 3; ++i) {
      zs[i] = z->stride(i);
      dzs[i] = dz.stride(i);
    }
  if (!made([&] {
        return g_norm_bwd(y.data(), ys, z.data(), z ? zs : nullptr, static_cast<const float*>(w.data()),
                          static_cast<const float*>(rstd.data()), g.data(), token ? gs : nullptr, flags,
                          dy.data_ptr(), dys, z ? dz.data_ptr() : nullptr, z ? dzs : nullptr,
                          static_cast<float*>(dw.data_ptr()), wp, bytes, b, d, groups, L, stream_of(dev));
      }))
    return nullptr;
  return tuple_of({dy, dz, dw});
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- linear attention

// The addresses of linattn.py's entry points, after bind.
PyObject* bind_linattn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kFunctions = 8;
  if (n != kFunctions) {
    PyErr_SetString(PyExc_TypeError, "bind_linattn takes eight addresses");
    return nullptr;
  }
  void* f[kFunctions];
  for (int i = 0; i < kFunctions; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_linattn_fwd = reinterpret_cast<decltype(g_linattn_fwd)>(f[0]);
  g_linattn_fwd_ws = reinterpret_cast<decltype(g_linattn_fwd_ws)>(f[1]);
  g_linattn_bwd = reinterpret_cast<decltype(g_linattn_bwd)>(f[2]);
  g_linattn_bwd_ws = reinterpret_cast<decltype(g_linattn_bwd_ws)>(f[3]);
  g_linattn_step = reinterpret_cast<decltype(g_linattn_step)>(f[4]);
  g_qk_fwd = reinterpret_cast<decltype(g_qk_fwd)>(f[5]);
  g_qk_bwd = reinterpret_cast<decltype(g_qk_bwd)>(f[6]);
  g_qk_bwd_ws = reinterpret_cast<decltype(g_qk_bwd_ws)>(f[7]);
  Py_RETURN_NONE;
}

// Heads of values, the last axis contiguous.
bool heads_of(const Arg& t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  return is(t, type, dev, shape) && (t->size(-1) <= 1 || t->stride(-1) == 1);
}

// The strides of all axes but the last.
struct Lead {
  int64_t s[3] = {0, 0, 0};
  explicit Lead(const Arg& t) {
    if (t)
      for (int64_t i = 0; i + 1 < t->dim() && i < 3; ++i) s[i] = t->stride(i);
  }
};

// Log decays: one for each head, or for each row (and step) and head. Its strides.
bool decays_of(const Arg& g, int dev, std::initializer_list<int64_t> shape, int64_t* strides) {
  if (!g) return true;
  const size_t lead = shape.size() - 1;
  const int64_t heads = *(shape.end() - 1);
  if (g->dim() == 1) {
    for (size_t i = 0; i < lead; ++i) strides[i] = 0;
    strides[lead] = g->stride(0);
    return is(g, at::kFloat, dev, {heads});
  }
  if (!is(g, at::kFloat, dev, shape)) return false;
  for (size_t i = 0; i <= lead; ++i) strides[i] = g->stride(int64_t(i));
  return true;
}

// A float, or None for `otherwise`.
float float_of(PyObject* o, double otherwise, bool* ok) {
  if (o == Py_None) return float(otherwise);
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    *ok = false;
  }
  return float(v);
}

const float* f32_of(const Arg& t) { return static_cast<const float*>(t.data()); }
const int32_t* i32_of(const Arg& t) { return static_cast<const int32_t*>(t.data()); }

// linattn(q, k, v, g, scale, initial_state, lengths, out, final_state, return_final_state, workspace)
PyObject* linattn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 11;
  SSM_NEED(ok && g_linattn_fwd);
  const Arg q(a[0], &ok), k(a[1], &ok), v(a[2], &ok), g(a[3], &ok), init(a[5], &ok), lengths(a[6], &ok),
      out(a[7], &ok), fin(a[8], &ok), ws(a[10], &ok);
  const bool want = flag_of(a[9], &ok);
  SSM_NEED(ok && q && k && v && q->dim() == 4 && v->dim() == 4);
  const int dev = device_of(q), io = io_of(q);
  const at::ScalarType type = q->scalar_type();
  const int64_t b = q->size(0), L = q->size(1), hk = q->size(2), dk = q->size(3), h = v->size(2), dv = v->size(3);
  const float scale = float_of(a[4], 1.0 / std::sqrt(double(dk)), &ok);
  int64_t gs[3];
  SSM_NEED(ok && dev >= 0 && io >= 0 && hk > 0 && h > 0 && h % hk == 0 && heads_of(q, type, dev, {b, L, hk, dk}) &&
           heads_of(k, type, dev, {b, L, hk, dk}) && heads_of(v, type, dev, {b, L, h, dv}) &&
           decays_of(g, dev, {b, L, h}, gs) && dense_or_none(init, at::kFloat, dev, {b, h, dv, dk}) &&
           dense_or_none(lengths, at::kInt, dev, {b}) && dense_or_none(out, type, dev, {b, L, h, dv}) &&
           dense_or_none(fin, at::kFloat, dev, {b, h, dv, dk}));
  at::Tensor made_ws, made_out, made_fin;
  int64_t bytes = 0;
  const int64_t need = g_linattn_fwd_ws(b, L, h, dk, dv, uint32_t(io));
  void* wp = nullptr;
  if (need != 0 || ws) {
    wp = workspace_of(ws, need, dev, *q.t, &made_ws, &bytes);
    SSM_NEED(wp);
  }
  if (!out) made_out = at::empty({b, L, h, dv}, v->options());
  if (!fin && want) made_fin = at::empty({b, h, dv, dk}, v->options().dtype(at::kFloat));
  void* op = out ? out.mut() : made_out.data_ptr();
  void* fp = fin ? fin.mut() : want ? made_fin.data_ptr() : nullptr;
  const Lead qs(q), ks(k), vs(v);
  if (!made([&] {
        return g_linattn_fwd(q.data(), qs.s, k.data(), ks.s, v.data(), vs.s, f32_of(g), g ? gs : nullptr,
                             f32_of(init), i32_of(lengths), scale, uint32_t(io), op, static_cast<float*>(fp), wp,
                             bytes, b, L, hk, h, dk, dv, stream_of(dev));
      }))
    return nullptr;
  wrote(out);
  wrote(fin);
  PyObject* o = give(a[7], made_out);
  PyObject* f = fin || want ? give(a[8], made_fin) : (Py_INCREF(Py_None), Py_None);
  PyObject* both = PyTuple_Pack(2, o, f);
  Py_DECREF(o);
  Py_DECREF(f);
  return both;
  END_HANDLE_TH_ERRORS
}

// linattn_backward(q, k, v, dout, g, scale, initial_state, lengths, dfinal, want_dg, want_dinitial,
// workspace): (dq, dk, dv, dg or None, dinitial or None)
PyObject* linattn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 12;
  SSM_NEED(ok && g_linattn_bwd);
  const Arg q(a[0], &ok), k(a[1], &ok), v(a[2], &ok), dout(a[3], &ok), g(a[4], &ok), init(a[6], &ok),
      lengths(a[7], &ok), dfin(a[8], &ok), ws(a[11], &ok);
  const bool want_dg = a[9] == Py_None ? bool(g) : flag_of(a[9], &ok);
  const bool want_di = a[10] == Py_None ? bool(init) : flag_of(a[10], &ok);
  SSM_NEED(ok && q && k && v && dout && q->dim() == 4 && v->dim() == 4 && (g || !want_dg));
  const int dev = device_of(q), io = io_of(q);
  const at::ScalarType type = q->scalar_type();
  const int64_t b = q->size(0), L = q->size(1), hk = q->size(2), dk = q->size(3), h = v->size(2), dv = v->size(3);
  const float scale = float_of(a[5], 1.0 / std::sqrt(double(dk)), &ok);
  int64_t gs[3];
  SSM_NEED(ok && dev >= 0 && io >= 0 && hk > 0 && h > 0 && h % hk == 0 && heads_of(q, type, dev, {b, L, hk, dk}) &&
           heads_of(k, type, dev, {b, L, hk, dk}) && heads_of(v, type, dev, {b, L, h, dv}) &&
           heads_of(dout, type, dev, {b, L, h, dv}) && decays_of(g, dev, {b, L, h}, gs) &&
           dense_or_none(init, at::kFloat, dev, {b, h, dv, dk}) && dense_or_none(lengths, at::kInt, dev, {b}) &&
           dense_or_none(dfin, at::kFloat, dev, {b, h, dv, dk}));
  const uint32_t flags = uint32_t(io) | (want_dg && g->dim() == 1 ? SSM_LINATTN_HEAD_DG : 0);
  at::Tensor made_ws;
  int64_t bytes = 0;
  void* wp = workspace_of(ws, g_linattn_bwd_ws(b, L, h, dk, dv, flags), dev, *q.t, &made_ws, &bytes);
  SSM_NEED(wp);
  const at::Tensor dq = at::empty({b, L, hk, dk}, q->options()), dkt = at::empty({b, L, hk, dk}, q->options()),
                   dvt = at::empty({b, L, h, dv}, q->options());
  const auto f32 = q->options().dtype(at::kFloat);
  const at::Tensor dg = want_dg ? at::empty(g->sizes(), f32) : at::Tensor();
  const at::Tensor di = want_di ? at::empty({b, h, dv, dk}, f32) : at::Tensor();
  const Lead qs(q), ks(k), vs(v), os(dout);
  if (!made([&] {
        return g_linattn_bwd(q.data(), qs.s, k.data(), ks.s, v.data(), vs.s, dout.data(), os.s, f32_of(g),
                             g ? gs : nullptr, f32_of(init), i32_of(lengths), f32_of(dfin), scale, flags,
                             dq.data_ptr(), dkt.data_ptr(), dvt.data_ptr(),
                             want_dg ? static_cast<float*>(dg.data_ptr()) : nullptr,
                             want_di ? static_cast<float*>(di.data_ptr()) : nullptr, wp, bytes, b, L, hk, h, dk, dv,
                             stream_of(dev));
      }))
    return nullptr;
  return tuple_of({dq, dkt, dvt, dg, di});
  END_HANDLE_TH_ERRORS
}

// linattn_step(q, k, v, state, g, scale, slots, out)
PyObject* linattn_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 8;
  SSM_NEED(ok && g_linattn_step);
  const Arg q(a[0], &ok), k(a[1], &ok), v(a[2], &ok), state(a[3], &ok), g(a[4], &ok), slots(a[6], &ok),
      out(a[7], &ok);
  SSM_NEED(ok && q && k && v && state && q->dim() == 3 && v->dim() == 3 && state->dim() == 4);
  const int dev = device_of(q), io = io_of(q);
  const at::ScalarType type = q->scalar_type();
  const int64_t b = q->size(0), hk = q->size(1), dk = q->size(2), h = v->size(1), dv = v->size(2), ns = state->size(0);
  const float scale = float_of(a[5], 1.0 / std::sqrt(double(dk)), &ok);
  int64_t gs[2];
  SSM_NEED(ok && dev >= 0 && io >= 0 && hk > 0 && h > 0 && h % hk == 0 && heads_of(q, type, dev, {b, hk, dk}) &&
           heads_of(k, type, dev, {b, hk, dk}) && heads_of(v, type, dev, {b, h, dv}) &&
           decays_of(g, dev, {b, h}, gs) && dense(state, at::kFloat, dev, {ns, h, dv, dk}) &&
           dense_or_none(slots, at::kInt, dev, {b}) && dense_or_none(out, type, dev, {b, h, dv}));
  at::Tensor made_out;
  if (!out) made_out = at::empty({b, h, dv}, v->options());
  void* op = out ? out.mut() : made_out.data_ptr();
  const Lead qs(q), ks(k), vs(v);
  if (!made([&] {
        return g_linattn_step(q.data(), qs.s, k.data(), ks.s, v.data(), vs.s, f32_of(g), g ? gs : nullptr,
                              i32_of(slots), scale, uint32_t(io), static_cast<float*>(state.mut()), op, b, ns, hk, h,
                              dk, dv, stream_of(dev));
      }))
    return nullptr;
  wrote(state);
  wrote(out);
  return give(a[7], made_out);
  END_HANDLE_TH_ERRORS
}

// What qk_norm and its gradient check alike.
struct QkCall {
  const Arg q, k, qw, kw, cos, sin, pos;
  float eps = 0;
  int dev = -1, io = -1;
  int64_t b = 0, L = 0, hq = 0, hk = 0, d = 0, rot = 0, rows = 0;
  uint32_t flags = 0;
  bool good = false;
  // o: q_weight, k_weight, cos, sin, positions, eps, interleaved
  QkCall(PyObject* q_, PyObject* k_, PyObject* const* o, bool* ok)
      : q(q_, ok), k(k_, ok), qw(o[0], ok), kw(o[1], ok), cos(o[2], ok), sin(o[3], ok), pos(o[4], ok) {
    eps = float_of(o[5], 1e-6, ok);
    const bool interleaved = flag_of(o[6], ok);
    if (!*ok || !q || !k || q->dim() != 4 || k->dim() != 4 || bool(cos) != bool(sin)) return;
    dev = device_of(q), io = io_of(q);
    b = q->size(0), L = q->size(1), hq = q->size(2), d = q->size(3), hk = k->size(2);
    const at::ScalarType type = q->scalar_type();
    if (dev < 0 || io < 0) return;
    if (cos) {
      if (cos->dim() != 2 || 2 * cos->size(1) > d) return;
      rows = cos->size(0), rot = 2 * cos->size(1);
      if (!dense(cos, at::kFloat, dev, {rows, rot / 2}) || !dense(sin, at::kFloat, dev, {rows, rot / 2}) ||
          (!pos && rows < L))
        return;
    }
    flags = uint32_t(io) | (interleaved ? SSM_QK_INTERLEAVED : 0);
    good = heads_of(q, type, dev, {b, L, hq, d}) && heads_of(k, type, dev, {b, L, hk, d}) &&
           dense_or_none(qw, at::kFloat, dev, {d}) && dense_or_none(kw, at::kFloat, dev, {d}) &&
           dense_or_none(pos, at::kInt, dev, {b, L});
  }
};

// qk_norm(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, q_out, k_out)
PyObject* qk_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 11;
  SSM_NEED(ok && g_qk_fwd);
  const QkCall c(a[0], a[1], a + 2, &ok);
  const Arg qo(a[9], &ok), ko(a[10], &ok);
  SSM_NEED(ok && c.good);
  const at::ScalarType type = c.q->scalar_type();
  SSM_NEED(dense_or_none(qo, type, c.dev, {c.b, c.L, c.hq, c.d}) && dense_or_none(ko, type, c.dev, {c.b, c.L, c.hk, c.d}));
  at::Tensor made_q, made_k;
  if (!qo) made_q = at::empty({c.b, c.L, c.hq, c.d}, c.q->options());
  if (!ko) made_k = at::empty({c.b, c.L, c.hk, c.d}, c.q->options());
  void* qp = qo ? qo.mut() : made_q.data_ptr();
  void* kp = ko ? ko.mut() : made_k.data_ptr();
  const Lead qs(c.q), ks(c.k);
  if (!made([&] {
        return g_qk_fwd(c.q.data(), qs.s, c.k.data(), ks.s, f32_of(c.qw), f32_of(c.kw), f32_of(c.cos), f32_of(c.sin),
                        i32_of(c.pos), c.eps, c.flags, qp, kp, c.b, c.L, c.hq, c.hk, c.d, c.rot, c.rows,
                        stream_of(c.dev));
      }))
    return nullptr;
  wrote(qo);
  wrote(ko);
  PyObject* x = give(a[9], made_q);
  PyObject* y = give(a[10], made_k);
  PyObject* both = PyTuple_Pack(2, x, y);
  Py_DECREF(x);
  Py_DECREF(y);
  return both;
  END_HANDLE_TH_ERRORS
}

// qk_norm_backward(q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, positions, eps, interleaved,
// workspace): (dq, dk, dq_weight or None, dk_weight or None)
PyObject* qk_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 12;
  SSM_NEED(ok && g_qk_bwd);
  const QkCall c(a[0], a[1], a + 4, &ok);
  const Arg gq(a[2], &ok), gk(a[3], &ok), ws(a[11], &ok);
  SSM_NEED(ok && c.good && gq && gk);
  const at::ScalarType type = c.q->scalar_type();
  SSM_NEED(heads_of(gq, type, c.dev, {c.b, c.L, c.hq, c.d}) && heads_of(gk, type, c.dev, {c.b, c.L, c.hk, c.d}));
  at::Tensor made_ws;
  int64_t bytes = 0;
  void* wp = workspace_of(ws, g_qk_bwd_ws(c.b, c.L, c.hq, c.hk, c.d, c.rot, c.flags), c.dev, *c.q.t, &made_ws, &bytes);
  SSM_NEED(wp);
  const at::Tensor dq = at::empty({c.b, c.L, c.hq, c.d}, c.q->options()),
                   dk = at::empty({c.b, c.L, c.hk, c.d}, c.q->options());
  const auto f32 = c.q->options().dtype(at::kFloat);
  const at::Tensor dqw = c.qw ? at::empty({c.d}, f32) : at::Tensor(), dkw = c.kw ? at::empty({c.d}, f32) : at::Tensor();
  const Lead qs(c.q), ks(c.k), gqs(gq), gks(gk);
  if (!made([&] {
        return g_qk_bwd(c.q.data(), qs.s, c.k.data(), ks.s, gq.data(), gqs.s, gk.data(), gks.s, f32_of(c.qw),
                        f32_of(c.kw), f32_of(c.cos), f32_of(c.sin), i32_of(c.pos), c.eps, c.flags, dq.data_ptr(),
                        dk.data_ptr(), c.qw ? static_cast<float*>(dqw.data_ptr()) : nullptr,
                        c.kw ? static_cast<float*>(dkw.data_ptr()) : nullptr, wp, bytes, c.b, c.L, c.hq, c.hk, c.d,
                        c.rot, c.rows, stream_of(c.dev));
      }))
    return nullptr;
  return tuple_of({dq, dk, dqw, dkw});
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef g_methods[] = {{"bind", fast<bind>(), METH_FASTCALL, nullptr},
                           {"conv", fast<conv>(), METH_FASTCALL, nullptr},
                           {"conv_step", fast<conv_step>(), METH_FASTCALL, nullptr},
                           {"state_step", fast<state_step>(), METH_FASTCALL, nullptr},
                           {"norm", fast<norm>(), METH_FASTCALL, nullptr},
                           {"conv_backward", fast<conv_backward>(), METH_FASTCALL, nullptr},
                           {"norm_backward", fast<norm_backward>(), METH_FASTCALL, nullptr},
                           {"bind_linattn", fast<bind_linattn>(), METH_FASTCALL, nullptr},
                           {"linattn", fast<linattn>(), METH_FASTCALL, nullptr},
                           {"linattn_backward", fast<linattn_backward>(), METH_FASTCALL, nullptr},
                           {"linattn_step", fast<linattn_step>(), METH_FASTCALL, nullptr},
                           {"qk_norm", fast<qk_norm>(), METH_FASTCALL, nullptr},
                           {"qk_norm_backward", fast<qk_norm_backward>(), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
