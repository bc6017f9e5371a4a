// bind.cpp -- CPython binding of the block operators for torch tensors (block.py): argument checks,
// outputs and workspaces from PyTorch's allocator, and the C calls of include/moe.h, whose addresses
// the package hands over (bind), so that this module and ctypes use one loaded library.
//
// In Python, checks and ctypes structures of one call cost 13 to 24 us, several times what the kernels
// of a decoding step take; here a call costs a few.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "moe.h"

namespace {

using at::Tensor;

struct {
  decltype(&::moe_norm_in) norm_in;
  decltype(&::moe_norm_out) norm_out;
  decltype(&::moe_norm_workspace) norm_workspace;
  decltype(&::moe_norm_in_backward) norm_in_backward;
  decltype(&::moe_norm_out_backward) norm_out_backward;
  decltype(&::moe_adapters_apply) adapters_apply;
  decltype(&::moe_adapters_last_error) adapters_last_error;
  decltype(&::moe_ffn_workspace) ffn_workspace;
  decltype(&::moe_ffn_forward) ffn_forward;
  decltype(&::moe_ffn_backward) ffn_backward;
} lib;
PyObject *moe_error = nullptr;

struct Refused {
  std::string what;
};
struct Raised {};  // a Python error is set

[[noreturn]] void refuse(const char *name, const std::string &what) { throw Refused{std::string(name) + ": " + what}; }

void check(moe_status s, const char *what, const char *detail = nullptr) {
  if (s == MOE_OK) return;
  const std::string text = detail ? std::string(what) + ": " + detail : what;
  PyObject *e = PyObject_CallFunction(moe_error, "is", static_cast<int>(s), text.c_str());
  if (e) {
    PyErr_SetObject(moe_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

int code(const Tensor &t) {
  const auto s = t.scalar_type();
  return s == at::kFloat ? MOE_F32 : s == at::kBFloat16 ? MOE_BF16 : -1;
}
at::ScalarType type_of(int c) { return c == MOE_BF16 ? at::kBFloat16 : at::kFloat; }

std::string str(const Tensor &t) {
  std::string s = c10::toString(t.scalar_type());
  s += " (";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  s += ") with strides (";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.stride(i));
  return s + ") on " + t.device().str();
}

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(name, "is not a tensor");
  const Tensor &t = THPVariable_Unpack(o);
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse(name, "requires grad, but the call leaves nothing for autograd: make it under torch.no_grad() and take the "
                 "gradients from the _backward functions");
  return t;
}
bool given(PyObject *o) { return o != Py_None; }

// A 2-D float32 or bfloat16 CUDA tensor (rows, cols, type: -1 any) with contiguous rows; its row stride.
int64_t matrix(const Tensor &t, const char *name, c10::Device dev, int64_t rows, int64_t cols, int type = -1,
               bool dense = false) {
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (cols >= 0 && t.size(1) != cols) || t.numel() == 0)
    refuse(name, str(t) + ": wrong shape, expected [" + (rows < 0 ? "n" : std::to_string(rows)) + ", " +
                     (cols < 0 ? "d" : std::to_string(cols)) + "], not empty");
  if (t.device() != dev || !dev.is_cuda()) refuse(name, str(t) + ": expected a CUDA tensor on " + dev.str());
  const int c = code(t);
  if (c < 0 || (type >= 0 && c != type))
    refuse(name, str(t) + ": expected " + (type == MOE_F32 ? "float32" : type == MOE_BF16 ? "bfloat16" : "float32 or bfloat16"));
  const int64_t d = t.size(1), ld = t.size(0) > 1 ? t.stride(0) : d;
  if ((t.stride(1) != 1 && d > 1) || ld < d || (dense && ld != d))
    refuse(name, str(t) + (dense ? ": must be contiguous" : ": rows must be contiguous"));
  if (t.size(0) > INT32_MAX || d > INT32_MAX) refuse(name, str(t) + ": too large");
  return ld;
}

void vector(const Tensor &t, const char *name, c10::Device dev, int64_t n, at::ScalarType type) {
  if (t.dim() != 1 || t.size(0) != n || t.device() != dev || t.scalar_type() != type || (t.stride(0) != 1 && n > 1))
    refuse(name, str(t) + ": expected " + c10::toString(type) + " [" + std::to_string(n) + "], contiguous, on " + dev.str());
}
void weights(const Tensor &t, const char *name, c10::Device dev, int64_t n) {
  vector(t, name, dev, n, code(t) == MOE_BF16 ? at::kBFloat16 : at::kFloat);
}

// The bytes a tensor spans: rows of `width` bytes, `pitch` apart (0: one row).
struct Span {
  uintptr_t lo, hi, width, pitch;
  explicit Span(const Tensor &t) {
    const int64_t size = t.element_size(), rows = t.dim() == 2 ? t.size(0) : 1;
    lo = reinterpret_cast<uintptr_t>(t.data_ptr());
    width = t.size(-1) * size;
    pitch = rows > 1 ? t.stride(0) * size : 0;
    hi = lo + (rows - 1) * pitch + width;
  }
  // Rows between the other one's, as of two column ranges of one matrix.
  bool beside(const Span &b) const {
    if (!pitch || pitch != b.pitch) return false;
    const uintptr_t at = b.lo >= lo ? (b.lo - lo) % pitch : (pitch - (lo - b.lo) % pitch) % pitch;
    return at >= width && at + b.width <= pitch;
  }
};
// An output shares no memory with an input, unless `may` and it is that input: same start, strides, type.
void apart(const Tensor &out, const char *name, const Tensor &in, bool may = false) {
  const Span a(out), b(in);
  if (a.lo >= b.hi || b.lo >= a.hi || a.beside(b)) return;
  if (may && a.lo == b.lo && out.strides() == in.strides() && out.scalar_type() == in.scalar_type()) return;
  refuse(name, "overlaps another tensor of the call");
}

Tensor fresh(int64_t n, int64_t d, int type, c10::Device dev) {
  return at::empty({n, d}, at::TensorOptions().dtype(type_of(type)).device(dev));
}
Tensor bytes(uint64_t n, c10::Device dev) {
  return at::empty({static_cast<int64_t>(n < 16 ? 16 : n)}, at::TensorOptions().dtype(at::kByte).device(dev));
}

struct Args {
  PyObject *const *v;
  Py_ssize_t n, i = 0;
  PyObject *next() {
    if (i >= n) refuse("call", "too few arguments");
    return v[i++];
  }
  float number() {
    const double d = PyFloat_AsDouble(next());
    if (d == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(d);
  }
  int64_t whole() {
    const int64_t d = PyLong_AsLongLong(next());
    if (d == -1 && PyErr_Occurred()) throw Raised{};
    return d;
  }
};

PyObject *wrap(const Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <size_t N>
PyObject *tuple(const Tensor (&t)[N]) {
  PyObject *r = PyTuple_New(N);
  if (!r) throw Raised{};
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(r, i, wrap(t[i]));
  return r;
}

void *stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
void cuda_only(const Tensor &t, const char *name) {
  if (!t.is_cuda()) refuse(name, str(t) + ": expected a CUDA tensor");
}

// norm_in(x, weight, eps, unit_offset, out, out_type)
PyObject *norm_in(Args a) {
  const Tensor &x = tensor(a.next(), "x"), &w = tensor(a.next(), "weight");
  const float eps = a.number();
  const int off = a.whole();
  PyObject *po = a.next();
  int type = a.whole();
  cuda_only(x, "x");
  const auto dev = x.device();
  const int64_t ld = matrix(x, "x", dev, -1, -1), n = x.size(0), d = x.size(1);
  weights(w, "weight", dev, d);
  c10::cuda::CUDAGuard guard(dev);
  Tensor out;
  int64_t old = d;
  if (given(po)) {
    out = tensor(po, "out");
    old = matrix(out, "out", dev, n, d, type);
    apart(out, "out", x, true);
    apart(out, "out", w);
  } else {
    out = fresh(n, d, type < 0 ? code(x) : type, dev);
  }
  check(lib.norm_in(x.data_ptr(), code(x), ld, w.data_ptr(), code(w), eps, off, out.data_ptr(), code(out), old, n, d,
                    stream_of(dev)),
        "moe_norm_in");
  return wrap(out);
}

struct Gate {
  int kind = MOE_GATE_NONE, type = 0;
  const void *p = nullptr;
  int64_t ld = 0;
  Gate(PyObject *o, c10::Device dev, int64_t n, int64_t d) {
    if (!given(o)) return;
    const Tensor &g = tensor(o, "gate");
    if (g.dim() == 1) {
      weights(g, "gate", dev, d);
      kind = MOE_GATE_CHANNEL;
    } else {
      const bool token = g.dim() == 2 && g.size(1) == 1;
      ld = matrix(g, "gate", dev, n, token ? 1 : d);
      kind = token ? MOE_GATE_TOKEN : MOE_GATE_FULL;
    }
    type = code(g);
    p = g.data_ptr();
  }
};

// norm_out(o, residual, weight, eps, unit_offset, gate, gate_act, scale, next_weight, next_eps, next_type, out,
//          out_type, next_out)
PyObject *norm_out(Args a) {
  const Tensor &o = tensor(a.next(), "o"), &res = tensor(a.next(), "residual");
  PyObject *pw = a.next();
  moe_norm_out_args p{};
  p.struct_size = sizeof p;
  p.eps = a.number();
  p.unit_offset = a.whole();
  PyObject *pg = a.next();
  p.gate_act = a.whole();
  p.scale = a.number();
  PyObject *pn = a.next();
  p.next_eps = a.number();
  const int h_type = a.whole();
  PyObject *po = a.next();
  const int out_type = a.whole();
  PyObject *ph = a.next();
  cuda_only(o, "o");
  const auto dev = o.device();
  p.o_stride = matrix(o, "o", dev, -1, -1);
  const int64_t n = o.size(0), d = o.size(1);
  p.n_tokens = n, p.d_model = d;
  p.o = o.data_ptr(), p.o_dtype = code(o);
  p.res_stride = matrix(res, "residual", dev, n, d);
  p.residual = res.data_ptr(), p.res_dtype = code(res);
  const Tensor *w = nullptr, *wn = nullptr;
  if (given(pw)) {
    w = &tensor(pw, "weight");
    weights(*w, "weight", dev, d);
    p.weight = w->data_ptr(), p.w_dtype = code(*w);
  }
  if (given(pn)) {
    wn = &tensor(pn, "next_weight");
    weights(*wn, "next_weight", dev, d);
    if (w && code(*w) != code(*wn)) refuse("next_weight", "has another type than weight");
    p.next_weight = wn->data_ptr(), p.w_dtype = code(*wn);
  }
  const Gate g(pg, dev, n, d);
  p.gate = g.p, p.gate_kind = g.kind, p.gate_dtype = g.type, p.gate_stride = g.ld;
  c10::cuda::CUDAGuard guard(dev);
  auto clear = [&](const Tensor &t, const char *name, bool may_res) {
    apart(t, name, o, true);
    apart(t, name, res, may_res);
    if (w) apart(t, name, *w);
    if (wn) apart(t, name, *wn);
    if (g.p) apart(t, name, THPVariable_Unpack(pg));
  };
  Tensor out, h;
  p.res_out_stride = p.h_stride = d;
  if (given(po)) {
    out = tensor(po, "out");
    p.res_out_stride = matrix(out, "out", dev, n, d, out_type);
    clear(out, "out", true);
  } else {
    out = fresh(n, d, out_type < 0 ? code(res) : out_type, dev);
  }
  p.res_out = out.data_ptr(), p.res_out_dtype = code(out);
  if (wn) {
    if (given(ph)) {
      h = tensor(ph, "next_out");
      p.h_stride = matrix(h, "next_out", dev, n, d, h_type);
      clear(h, "next_out", false);
      apart(h, "next_out", out);
    } else {
      h = fresh(n, d, h_type < 0 ? code(o) : h_type, dev);
    }
    p.h = h.data_ptr(), p.h_dtype = code(h);
  } else if (given(ph)) {
    refuse("next_out", "given without next_weight");
  }
  check(lib.norm_out(&p, stream_of(dev)), "moe_norm_out");
  if (!wn) return wrap(out);
  const Tensor r[2] = {out, h};
  return tuple(r);
}

// norm_in_backward(x, weight, dh, eps, unit_offset, d_residual)
PyObject *norm_in_backward(Args a) {
  const Tensor &x = tensor(a.next(), "x"), &w = tensor(a.next(), "weight"), &dh = tensor(a.next(), "dh");
  moe_norm_in_bwd_args p{};
  p.struct_size = sizeof p;
  p.eps = a.number();
  p.unit_offset = a.whole();
  PyObject *pr = a.next();
  cuda_only(x, "x");
  const auto dev = x.device();
  p.x_stride = matrix(x, "x", dev, -1, -1);
  const int64_t n = x.size(0), d = x.size(1);
  weights(w, "weight", dev, d);
  p.dh_stride = matrix(dh, "dh", dev, n, d);
  int type = code(x);
  if (given(pr)) {
    const Tensor &r = tensor(pr, "d_residual");
    p.dres_stride = matrix(r, "d_residual", dev, n, d);
    p.dres = r.data_ptr();
    type = p.dres_dtype = code(r);
  }
  c10::cuda::CUDAGuard guard(dev);
  const Tensor r[2] = {fresh(n, d, type, dev), at::empty_like(w)};
  const Tensor ws = bytes(lib.norm_workspace(n, d), dev);
  p.n_tokens = n, p.d_model = d;
  p.x = x.data_ptr(), p.x_dtype = code(x), p.weight = w.data_ptr(), p.w_dtype = code(w);
  p.dh = dh.data_ptr(), p.dh_dtype = code(dh);
  p.dx = r[0].data_ptr(), p.dx_dtype = type, p.dx_stride = d, p.dweight = r[1].data_ptr();
  p.workspace = ws.data_ptr(), p.workspace_bytes = ws.numel();
  check(lib.norm_in_backward(&p, stream_of(dev)), "moe_norm_in_backward");
  return tuple(r);
}

// norm_out_backward(o, d_res, weight, eps, unit_offset, gate, gate_act, scale)
PyObject *norm_out_backward(Args a) {
  const Tensor &o = tensor(a.next(), "o"), &dr = tensor(a.next(), "d_res");
  PyObject *pw = a.next();
  moe_norm_out_bwd_args p{};
  p.struct_size = sizeof p;
  p.eps = a.number();
  p.unit_offset = a.whole();
  PyObject *pg = a.next();
  p.gate_act = a.whole();
  p.scale = a.number();
  cuda_only(o, "o");
  const auto dev = o.device();
  p.o_stride = matrix(o, "o", dev, -1, -1);
  const int64_t n = o.size(0), d = o.size(1);
  p.dres_stride = matrix(dr, "d_res", dev, n, d);
  const Gate g(pg, dev, n, d);
  c10::cuda::CUDAGuard guard(dev);
  Tensor r[3];
  r[0] = fresh(n, d, code(o), dev);
  if (given(pw)) {
    const Tensor &w = tensor(pw, "weight");
    weights(w, "weight", dev, d);
    r[1] = at::empty_like(w);
    p.weight = w.data_ptr(), p.w_dtype = code(w), p.dweight = r[1].data_ptr();
  }
  if (g.p) {
    const Tensor &gt = THPVariable_Unpack(pg);
    r[2] = at::empty(gt.sizes(), gt.options());
    p.dgate = r[2].data_ptr(), p.dgate_stride = gt.size(-1);
  }
  const Tensor ws = bytes(lib.norm_workspace(n, d), dev);
  p.n_tokens = n, p.d_model = d;
  p.o = o.data_ptr(), p.o_dtype = code(o), p.dres = dr.data_ptr(), p.dres_dtype = code(dr);
  p.gate = g.p, p.gate_kind = g.kind, p.gate_dtype = g.type, p.gate_stride = g.ld;
  p.d_o = r[0].data_ptr(), p.do_stride = d;
  p.workspace = ws.data_ptr(), p.workspace_bytes = ws.numel();
  check(lib.norm_out_backward(&p, stream_of(dev)), "moe_norm_out_backward");
  return tuple(r);
}

// adapters_apply(handle, device index, d_in, d_out, x, base, ids, out)
PyObject *adapters_apply(Args a) {
  moe_adapters *h = reinterpret_cast<moe_adapters *>(a.whole());
  const c10::Device dev(c10::kCUDA, static_cast<c10::DeviceIndex>(a.whole()));
  const int64_t d_in = a.whole(), d_out = a.whole();
  const Tensor &x = tensor(a.next(), "x"), &base = tensor(a.next(), "base"), &ids = tensor(a.next(), "ids");
  PyObject *po = a.next();
  const int64_t x_ld = matrix(x, "x", dev, -1, d_in), n = x.size(0);
  const int64_t b_ld = matrix(base, "base", dev, n, d_out);
  vector(ids, "ids", dev, n, at::kInt);
  Tensor out;
  int64_t o_ld = d_out;
  if (given(po)) {
    out = tensor(po, "out");
    o_ld = matrix(out, "out", dev, n, d_out, code(base));
    apart(out, "out", x);
    apart(out, "out", ids);
    apart(out, "out", base, true);
  } else {
    out = fresh(n, d_out, code(base), dev);
  }
  const moe_status s = lib.adapters_apply(h, x.data_ptr(), code(x), x_ld, base.data_ptr(), b_ld, out.data_ptr(), o_ld,
                                          code(out), ids.data_ptr<int32_t>(), n, stream_of(dev));
  if (s != MOE_OK) check(s, "moe_adapters_apply", lib.adapters_last_error(h));
  return wrap(out);
}

struct FfnWeights {
  int64_t n, d, f, x_ld;
  const Tensor &wg, &wu, &wd;
  FfnWeights(const Tensor &x, const Tensor &g, const Tensor &u, const Tensor &w) : wg(g), wu(u), wd(w) {
    cuda_only(x, "x");
    const auto dev = x.device();
    x_ld = matrix(x, "x", dev, -1, -1, MOE_BF16);
    n = x.size(0), d = x.size(1);
    matrix(wg, "w_gate", dev, -1, d, MOE_BF16, true);
    f = wg.size(0);
    matrix(wu, "w_up", dev, f, d, MOE_BF16, true);
    matrix(wd, "w_down", dev, d, f, MOE_BF16, true);
  }
};

// ffn_forward(x, w_gate, w_up, w_down, add, out, out_type, save)
PyObject *ffn_forward(Args a) {
  const Tensor &x = tensor(a.next(), "x"), &wg = tensor(a.next(), "w_gate"), &wu = tensor(a.next(), "w_up"),
               &wd = tensor(a.next(), "w_down");
  PyObject *pa = a.next(), *po = a.next();
  const int type = a.whole();
  const bool save = a.whole();
  const FfnWeights w(x, wg, wu, wd);
  const auto dev = x.device();
  moe_ffn_args p{};
  p.struct_size = sizeof p;
  p.n_tokens = w.n, p.d_model = w.d, p.d_ff = w.f;
  p.x = x.data_ptr(), p.x_stride = w.x_ld;
  p.w_gate = wg.data_ptr(), p.w_up = wu.data_ptr(), p.w_down = wd.data_ptr();
  if (given(pa)) {
    const Tensor &add = tensor(pa, "add");
    p.add_stride = matrix(add, "add", dev, w.n, w.d);
    p.add = add.data_ptr(), p.add_dtype = code(add);
  }
  c10::cuda::CUDAGuard guard(dev);
  Tensor out, g, u;
  p.y_stride = w.d;
  if (given(po)) {
    out = tensor(po, "out");
    p.y_stride = matrix(out, "out", dev, w.n, w.d, type);
    for (const Tensor *t : {&x, &wg, &wu, &wd}) apart(out, "out", *t);
    if (p.add) apart(out, "out", THPVariable_Unpack(pa), true);
  } else {
    out = fresh(w.n, w.d, type < 0 ? MOE_BF16 : type, dev);
  }
  p.y = out.data_ptr(), p.y_dtype = code(out);
  if (save) {
    g = fresh(w.n, w.f, MOE_F32, dev), u = fresh(w.n, w.f, MOE_F32, dev);
    p.save_gate = g.data_ptr(), p.save_up = u.data_ptr();
  }
  p.workspace_bytes = lib.ffn_workspace(w.n, w.d, w.f, 0);
  const Tensor ws = bytes(p.workspace_bytes, dev);
  p.workspace = ws.data_ptr();
  check(lib.ffn_forward(&p, stream_of(dev)), "moe_ffn_forward");
  if (!save) return wrap(out);
  const Tensor r[3] = {out, g, u};
  return tuple(r);
}

// ffn_backward(dy, x, w_gate, w_up, w_down, saved gate, saved up, need_dx, need_dw)
PyObject *ffn_backward(Args a) {
  const Tensor &dy = tensor(a.next(), "dy"), &x = tensor(a.next(), "x"), &wg = tensor(a.next(), "w_gate"),
               &wu = tensor(a.next(), "w_up"), &wd = tensor(a.next(), "w_down"), &g = tensor(a.next(), "saved gate"),
               &u = tensor(a.next(), "saved up");
  const bool need_dx = a.whole(), need_dw = a.whole();
  const FfnWeights w(x, wg, wu, wd);
  const auto dev = x.device();
  moe_ffn_bwd_args p{};
  p.struct_size = sizeof p;
  p.n_tokens = w.n, p.d_model = w.d, p.d_ff = w.f;
  p.dy_stride = matrix(dy, "dy", dev, w.n, w.d, MOE_BF16);
  matrix(g, "saved gate", dev, w.n, w.f, MOE_F32, true);
  matrix(u, "saved up", dev, w.n, w.f, MOE_F32, true);
  if (!need_dx && !need_dw) refuse("need_dx, need_dw", "nothing to compute");
  p.dy = dy.data_ptr(), p.x = x.data_ptr(), p.x_stride = w.x_ld;
  p.w_gate = wg.data_ptr(), p.w_up = wu.data_ptr(), p.w_down = wd.data_ptr();
  p.save_gate = g.data_ptr(), p.save_up = u.data_ptr();
  c10::cuda::CUDAGuard guard(dev);
  Tensor r[4];
  if (need_dx) r[0] = fresh(w.n, w.d, MOE_BF16, dev), p.dx = r[0].data_ptr();
  p.dx_stride = w.d;
  if (need_dw) {
    r[1] = fresh(w.f, w.d, MOE_BF16, dev), r[2] = fresh(w.f, w.d, MOE_BF16, dev), r[3] = fresh(w.d, w.f, MOE_BF16, dev);
    p.dw_gate = r[1].data_ptr(), p.dw_up = r[2].data_ptr(), p.dw_down = r[3].data_ptr();
  }
  p.workspace_bytes = lib.ffn_workspace(w.n, w.d, w.f, 1);
  const Tensor ws = bytes(p.workspace_bytes, dev);
  p.workspace = ws.data_ptr();
  check(lib.ffn_backward(&p, stream_of(dev)), "moe_ffn_backward");
  return tuple(r);
}

template <PyObject *(*F)(Args)>
PyObject *entry(PyObject *, PyObject *const *v, Py_ssize_t n) {
  try {
    return F(Args{v, n});
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Raised &) {
  } catch (const c10::OutOfMemoryError &e) {
    PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// bind(MoeError, {name: address})
PyObject *bind(PyObject *, PyObject *args) {
  PyObject *err, *names;
  if (!PyArg_ParseTuple(args, "OO!", &err, &PyDict_Type, &names)) return nullptr;
#define BIND(name)                                                                                      \
  {                                                                                                     \
    PyObject *v = PyDict_GetItemString(names, "moe_" #name);                                            \
    void *p = v ? PyLong_AsVoidPtr(v) : nullptr;                                                        \
    if (!p) {                                                                                           \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, "moe_" #name);                             \
      return nullptr;                                                                                   \
    }                                                                                                   \
    lib.name = reinterpret_cast<decltype(lib.name)>(p);                                                 \
  }
  BIND(norm_in) BIND(norm_out) BIND(norm_workspace) BIND(norm_in_backward) BIND(norm_out_backward)
  BIND(adapters_apply) BIND(adapters_last_error) BIND(ffn_workspace) BIND(ffn_forward) BIND(ffn_backward)
#undef BIND
  Py_INCREF(err);
  Py_XDECREF(moe_error);
  moe_error = err;
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         METHOD(norm_in), METHOD(norm_out), METHOD(norm_in_backward), METHOD(norm_out_backward),
                         METHOD(adapters_apply), METHOD(ffn_forward), METHOD(ffn_backward),
                         {nullptr, nullptr, 0, nullptr}};
// Read from the file before it is loaded: a binding of another torch or Python is not.
__attribute__((used)) const char built_for[] = "moe-block-ext-for:" MOE_EXT_TARGET;

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_ext() { return PyModule_Create(&module); }
