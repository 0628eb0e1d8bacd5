// Python binding of the serving operators (argument marshalling only): checks of the tensors,
// output allocation, the current stream, and one call of the C ABI (include/kda.h).
//
// It is native because the calls are short: a single-token step of a small batch runs a few
// microseconds on the GPU, and checking ten tensors and converting twenty arguments in Python took
// three times as long. The functions are positional; serving.py has the public signatures.
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <string>

#include "../../include/kda.h"

namespace {

using at::IntArrayRef;
using at::Tensor;

// A refused argument: the Python exception's type and text.
struct Refused {
  PyObject *type;
  std::string text;
};
[[noreturn]] void type_error(const std::string &text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string &text) { throw Refused{PyExc_ValueError, text}; }

std::string tuple_text(IntArrayRef x) {
  std::string s = "(";
  for (size_t i = 0; i < x.size(); ++i) s += (i ? ", " : "") + std::to_string(x[i]);
  return s + (x.size() == 1 ? ",)" : ")");
}
const char *dtype_text(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return c10::toString(t);
  }
}

bool given(PyObject *o) { return o != Py_None; }

const Tensor &as_tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}
const Tensor &as_tensor(PyObject *o, const char *name, int dims, const char *text) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != dims)
    value_error(std::string(name) + " must be a " + std::to_string(dims) + "-D torch.Tensor " + text);
  return THPVariable_Unpack(o);
}

// Device, dtype, shape and layout (contiguous, or contiguous in the last dimension) of one tensor.
void need_layout(const Tensor &t, const char *name, at::ScalarType dtype, const at::Device &dev, bool contiguous) {
  if (t.device() != dev) value_error(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
  if (t.scalar_type() != dtype)
    type_error(std::string(name) + " must be " + dtype_text(dtype) + ", got " + dtype_text(t.scalar_type()));
  if (contiguous) {
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  } else if (t.dim() > 0 && t.stride(-1) != 1 && t.size(-1) > 1) {
    value_error(std::string(name) + " must be contiguous in its last dimension");
  }
}
void need(const Tensor &t, const char *name, at::ScalarType dtype, IntArrayRef shape, const at::Device &dev,
          bool contiguous = false) {
  if (t.device() == dev && t.scalar_type() == dtype && t.sizes() != shape)
    value_error(std::string(name) + " must have shape " + tuple_text(shape) + ", got " + tuple_text(t.sizes()));
  need_layout(t, name, dtype, dev, contiguous);
}
void need_aligned(const Tensor &t, const char *name) {
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 != 0) value_error(std::string(name) + " must begin on a 16-byte boundary");
}
// A tensor that is read in boxes of 16-byte pieces: its base, and the strides of all dimensions but the last.
void need_boxes(const Tensor &t, const char *name) {
  for (int i = 0; i + 1 < t.dim(); ++i)
    if (t.size(i) > 1 && (t.stride(i) <= 0 || t.stride(i) % 8 != 0))
      value_error(std::string(name) + " must have strides that are positive multiples of 8, got " + tuple_text(t.strides()));
  need_aligned(t, name);
}
void need_gpu(const Tensor &t, const char *name) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor (there is no CPU path)");
}

Tensor output(PyObject *out, const char *name, IntArrayRef shape, at::ScalarType dtype, const at::Device &dev) {
  if (!given(out)) return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
  const Tensor &t = as_tensor(out, name);
  need(t, name, dtype, shape, dev, true);
  return t;
}

const void *ptr(const Tensor &t) { return t.data_ptr(); }
const float *fptr(const Tensor &t) { return static_cast<const float *>(t.data_ptr()); }

double number(PyObject *o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}

// Runs f(stream) with the tensors' device current.
template <typename F>
kda_status_t on_stream(const at::Device &dev, F &&f) {
  c10::cuda::OptionalCUDAGuard guard(dev);
  return f(reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
}

// Raises KDAError for a status other than KDA_OK.
void check(const char *fn, kda_status_t status) {
  if (status == KDA_OK) return;
  THPObjectPtr mod(PyImport_ImportModule("chunked_gated_delta_02_gb300._lib"));
  if (!mod) throw python_error();
  THPObjectPtr r(PyObject_CallMethod(mod.get(), "check", "si", fn, (int)status));
  throw python_error();
}

// State pools and states: dtype and layout as flags.
uint32_t state_flags(const Tensor &t, bool kv) {
  if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
    type_error("the state must be float32 or bfloat16");
  return (kv ? KDA_STATE_KV : 0u) | (t.scalar_type() == at::kBFloat16 ? KDA_STATE_BF16 : 0u);
}

struct Pool {
  void *state;
  const int32_t *indices;
  int64_t rows;
  uint32_t flags;
};
Pool pool(PyObject *state, PyObject *indices, bool kv, int64_t N, int64_t H, int64_t K, int64_t V, const at::Device &dev) {
  const Tensor &t = as_tensor(state, "state", 4, "[rows,H,V,K] or [rows,H,K,V]");
  Pool p;
  p.flags = state_flags(t, kv);
  p.rows = t.size(0);
  p.state = t.data_ptr();
  p.indices = nullptr;
  const int64_t shape[4] = {p.rows, H, kv ? K : V, kv ? V : K};
  need(t, "state", t.scalar_type(), shape, dev, true);
  need_aligned(t, "state");
  if (given(indices)) {
    const Tensor &i = as_tensor(indices, "state_indices");
    const int64_t n[1] = {N};
    need(i, "state_indices", at::kInt, n, dev, true);
    p.indices = static_cast<const int32_t *>(i.data_ptr());
  } else if (p.rows < N) {
    value_error("state must hold " + std::to_string(N) + " rows, or state_indices say which it uses; got " +
                std::to_string(p.rows));
  }
  return p;
}

int checked_int(int64_t x) {
  if (x > 2147483647) value_error("a dimension is longer than 2^31 - 1");
  return (int)x;
}

// Copies the strides of a tensor's first n dimensions.
void strides_of(const Tensor &t, int64_t *dst, int n) {
  for (int i = 0; i < n; ++i) dst[i] = t.stride(i);
}

// (flags, strides) of a log decay: [H], or one per token, [*lead, H].
uint32_t decay_of(const Tensor &t, IntArrayRef lead, int64_t H, const at::Device &dev, int64_t *strides) {
  if (t.dim() == 1) {
    const int64_t shape[1] = {H};
    need(t, "log_decay", at::kFloat, shape, dev);
    for (size_t i = 0; i <= lead.size(); ++i) strides[i] = 0;
    return 0;
  }
  c10::SmallVector<int64_t, 4> shape(lead.begin(), lead.end());
  shape.push_back(H);
  if (t.device() == dev && t.scalar_type() == at::kFloat && t.sizes() != IntArrayRef(shape))
    value_error("log_decay must have shape " + tuple_text(shape) + ", got " + tuple_text(t.sizes()));
  if (t.device() != dev || t.scalar_type() != at::kFloat) need_layout(t, "log_decay", at::kFloat, dev, false);
  strides_of(t, strides, (int)lead.size() + 1);   // any strides: it is read element by element
  return KDA_LA_TOKEN_DECAY;
}

struct Heads { int64_t Hk, H, K, V; };
Heads heads(const Tensor &q, const Tensor &k, const Tensor &v, int lead) {
  const at::Device dev = q.device();
  Heads r{q.size(lead), v.size(lead), q.size(lead + 1), v.size(lead + 1)};
  need_layout(q, "q", at::kBFloat16, dev, false);
  need(k, "k", at::kBFloat16, q.sizes(), dev);
  c10::SmallVector<int64_t, 4> shape(q.sizes().begin(), q.sizes().end());
  shape[lead] = r.H;
  shape[lead + 1] = r.V;
  need(v, "v", at::kBFloat16, shape, dev);
  if (r.Hk < 1 || r.H % r.Hk != 0)
    value_error("the " + std::to_string(r.H) + " heads of v must be a multiple of the " + std::to_string(r.Hk) +
                " heads of q and k");
  return r;
}

// ---- step(q, k, v, g, beta, A_log, state, dt_bias, lower_bound, scale, state_indices, out, kv)
PyObject *step(PyObject *const *a) {
  const Tensor &q = as_tensor(a[0], "q", 3, "[N,H,K]"), &v = as_tensor(a[2], "v", 3, "[N,H,V]");
  const Tensor &k = as_tensor(a[1], "k"), &g = as_tensor(a[3], "g"), &beta = as_tensor(a[4], "beta");
  const Tensor &A_log = as_tensor(a[5], "A_log");
  const at::Device dev = q.device();
  const int64_t N = q.size(0), H = q.size(1), K = q.size(2), V = v.size(2);
  const int64_t vs[3] = {N, H, V}, nh[2] = {N, H}, hs[1] = {H};
  need_layout(q, "q", at::kBFloat16, dev, false);
  need(k, "k", at::kBFloat16, q.sizes(), dev);
  need(v, "v", at::kBFloat16, vs, dev);
  const Pool p = pool(a[6], a[10], a[12] == Py_True, N, H, K, V, dev);
  uint32_t flags = p.flags;
  kda_step_strides_t st;
  if (g.dim() == 2) {
    flags |= KDA_GATE_PER_HEAD;
    need(g, "g", at::kBFloat16, nh, dev);
  } else {
    need(g, "g", at::kBFloat16, q.sizes(), dev);
  }
  const bool f32 = beta.scalar_type() == at::kFloat;
  if (f32) flags |= KDA_BETA_F32;
  need(beta, "beta", f32 ? at::kFloat : at::kBFloat16, nh, dev);
  need(A_log, "A_log", at::kFloat, hs, dev);
  const float *dt = nullptr;
  if (given(a[7])) {
    const Tensor &t = as_tensor(a[7], "dt_bias");
    need_layout(t, "dt_bias", at::kFloat, dev, true);
    const int64_t want = (flags & KDA_GATE_PER_HEAD) ? H : H * K;
    if (t.numel() != want) value_error("dt_bias must hold " + std::to_string(want) + " values");
    dt = fptr(t);
  }
  const float lb = (float)number(a[8]), scale = (float)number(a[9]);
  Tensor o = output(a[11], "out", vs, at::kBFloat16, dev);
  need_gpu(q, "q");
  strides_of(q, st.q, 2);
  strides_of(k, st.k, 2);
  strides_of(v, st.v, 2);
  strides_of(g, st.g, 2);
  strides_of(beta, st.beta, 2);
  check("kda_step", on_stream(dev, [&](kda_stream_t s) {
    return kda_step(ptr(q), ptr(k), ptr(v), ptr(g), ptr(beta), fptr(A_log), dt, lb, scale, p.state, p.indices,
                    checked_int(N), checked_int(H), checked_int(K), checked_int(V), p.rows, &st, flags, o.data_ptr(), s);
  }));
  return THPVariable_Wrap(std::move(o));
}

// ---- la_step(q, k, v, log_decay, state, state_indices, scale, out, kv)
PyObject *la_step(PyObject *const *a) {
  const Tensor &q = as_tensor(a[0], "q", 3, "[N,Hk,K]"), &v = as_tensor(a[2], "v", 3, "[N,H,V]");
  const Tensor &k = as_tensor(a[1], "k"), &decay = as_tensor(a[3], "log_decay");
  const at::Device dev = q.device();
  const int64_t N = q.size(0);
  const Heads x = heads(q, k, v, 1);
  const Pool p = pool(a[4], a[5], a[8] == Py_True, N, x.H, x.K, x.V, dev);
  kda_step_strides_t st = {};
  const int64_t lead[1] = {N}, vs[3] = {N, x.H, x.V};
  const uint32_t flags = p.flags | decay_of(decay, lead, x.H, dev, st.g);
  const float scale = (float)number(a[6]);
  Tensor o = output(a[7], "out", vs, at::kBFloat16, dev);
  need_gpu(q, "q");
  strides_of(q, st.q, 2);
  strides_of(k, st.k, 2);
  strides_of(v, st.v, 2);
  check("kda_la_step", on_stream(dev, [&](kda_stream_t s) {
    return kda_la_step(ptr(q), ptr(k), ptr(v), fptr(decay), scale, p.state, p.indices, checked_int(N), checked_int(x.Hk),
                       checked_int(x.H), checked_int(x.K), checked_int(x.V), p.rows, &st, flags, o.data_ptr(), s);
  }));
  return THPVariable_Wrap(std::move(o));
}

// ---- la_fwd(q, k, v, log_decay, scale, initial_state, output_final_state, cu_seqlens, workspace, out,
//             final_state, kv, state is bf16 without an initial_state)
PyObject *la_fwd(PyObject *const *a) {
  const Tensor &q = as_tensor(a[0], "q", 4, "[B,T,Hk,K]"), &v = as_tensor(a[2], "v", 4, "[B,T,H,V]");
  const Tensor &k = as_tensor(a[1], "k"), &decay = as_tensor(a[3], "log_decay");
  const at::Device dev = q.device();
  const int64_t B = q.size(0), T = q.size(1);
  const Heads x = heads(q, k, v, 2);
  kda_la_strides_t st;
  const int64_t lead[2] = {B, T};
  uint32_t flags = decay_of(decay, lead, x.H, dev, st.log_decay);
  need_boxes(q, "q");
  need_boxes(k, "k");
  need_boxes(v, "v");
  int64_t N = B;
  const int32_t *cu = nullptr;
  if (given(a[7])) {
    const Tensor &t = as_tensor(a[7], "cu_seqlens");
    need_layout(t, "cu_seqlens", at::kInt, dev, true);
    if (t.dim() != 1 || t.numel() < 1) value_error("cu_seqlens must be a 1-D tensor of N + 1 offsets");
    if (B != 1) value_error("packed sequences (cu_seqlens) need B = 1");
    N = t.numel() - 1;
    cu = static_cast<const int32_t *>(t.data_ptr());
  }
  const bool kv = a[11] == Py_True;
  const int64_t ss[4] = {N, x.H, kv ? x.K : x.V, kv ? x.V : x.K}, os[4] = {B, T, x.H, x.V};
  at::ScalarType sdt = a[12] == Py_True ? at::kBFloat16 : at::kFloat;
  const void *init = nullptr;
  if (given(a[5])) {
    const Tensor &t = as_tensor(a[5], "initial_state");
    state_flags(t, kv);
    sdt = t.scalar_type();
    need(t, "initial_state", sdt, ss, dev, true);
    need_aligned(t, "initial_state");
    init = t.data_ptr();
  }
  flags |= (kv ? KDA_STATE_KV : 0u) | (sdt == at::kBFloat16 ? KDA_STATE_BF16 : 0u);
  const float scale = (float)number(a[4]);
  Tensor fs;
  if (a[6] == Py_True) fs = output(a[10], "final_state", ss, sdt, dev);
  Tensor o = output(a[9], "out", os, at::kBFloat16, dev);
  if (fs.defined()) need_aligned(fs, "final_state");
  need_aligned(o, "out");
  Tensor ws;
  if (given(a[8])) {
    ws = as_tensor(a[8], "workspace");
    need_layout(ws, "workspace", ws.scalar_type(), dev, true);
  }
  need_gpu(q, "q");
  const int b = checked_int(B), t = checked_int(T), hk = checked_int(x.Hk), h = checked_int(x.H), n = checked_int(N);
  size_t bytes = 0;
  const kda_status_t rc = on_stream(dev, [&](kda_stream_t s) {
    const size_t size = kda_la_workspace_size(b, t, h, (int)x.K, (int)x.V, n, cu != nullptr);
    if (ws.defined()) {
      bytes = (size_t)ws.numel() * ws.element_size();
      if (bytes < size) value_error("workspace too small: need " + std::to_string(size) + " bytes");
    } else if (size > 0) {
      ws = at::empty({(int64_t)size}, at::TensorOptions().dtype(at::kByte).device(dev));
      bytes = size;
    }
    strides_of(q, st.q, 3);
    strides_of(k, st.k, 3);
    strides_of(v, st.v, 3);
    return kda_la_fwd(ptr(q), ptr(k), ptr(v), fptr(decay), scale, init, fs.defined() ? fs.data_ptr() : nullptr, cu, b, t,
                      hk, h, checked_int(x.K), checked_int(x.V), n, &st, flags, o.data_ptr(),
                      ws.defined() ? ws.data_ptr() : nullptr, bytes, s);
  });
  check("kda_la_fwd", rc);
  THPObjectPtr po(THPVariable_Wrap(std::move(o)));
  if (!po) throw python_error();
  THPObjectPtr pf;
  if (fs.defined()) {
    pf = THPVariable_Wrap(std::move(fs));
    if (!pf) throw python_error();
  }
  return PyTuple_Pack(2, po.get(), pf ? pf.get() : Py_None);
}

// Rows of D values of a tensor [..., D]: how many (outer, inner) and their strides.
struct Rows { int64_t outer, inner, s0, s1; };
Rows rows_of(const Tensor &t, const char *name) {
  const int64_t D = t.size(-1);
  if (t.is_contiguous()) return {t.numel() / D, 1, D, D};
  if (t.dim() == 2) return {t.size(0), 1, t.stride(0), t.stride(0)};
  if (t.dim() == 3) return {t.size(0), t.size(1), t.stride(0), t.stride(1)};
  if (t.dim() == 4 && (t.size(0) == 1 || t.size(1) == 1 || t.stride(0) == t.size(1) * t.stride(1)))
    return {t.size(0) * t.size(1), t.size(2), t.size(1) == 1 ? t.stride(0) : t.stride(1), t.stride(2)};
  value_error(std::string(name) + " must be contiguous, or a strided tensor [rows,D], [rows,heads,D] or [B,T,heads,D] "
                                  "whose B and T are one dimension");
}

const Tensor &as_rows(PyObject *o) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() < 1 || THPVariable_Unpack(o).size(-1) < 1)
    value_error("x must be a torch.Tensor [..., D]");
  return THPVariable_Unpack(o);
}

const float *vector_of(PyObject *o, const char *name, int64_t D, const at::Device &dev) {
  if (!given(o)) return nullptr;
  const Tensor &t = as_tensor(o, name);
  const int64_t shape[1] = {D};
  need(t, name, at::kFloat, shape, dev);
  return fptr(t);
}

// ---- norm_gate(x, gate, weight, eps, silu, out)
PyObject *norm_gate(PyObject *const *a) {
  const Tensor &x = as_rows(a[0]), &gate = as_tensor(a[1], "gate");
  const at::Device dev = x.device();
  const int64_t D = x.size(-1);
  need_layout(x, "x", at::kBFloat16, dev, false);
  need(gate, "gate", at::kBFloat16, x.sizes(), dev);
  const float *w = vector_of(a[2], "weight", D, dev);
  const float eps = (float)number(a[3]);
  Rows rx = rows_of(x, "x"), rg = rows_of(gate, "gate");
  if (rx.inner != rg.inner) {   // one of them contiguous, with its rows not split yet: the other's split
    if (rx.inner == 1) rx = {rg.outer, rg.inner, rg.inner * D, D};
    else rg = {rx.outer, rx.inner, rx.inner * D, D};
  }
  Tensor y = output(a[5], "out", x.sizes(), at::kBFloat16, dev);
  need_gpu(x, "x");
  const int64_t strides[4] = {rx.s0, rx.s1, rg.s0, rg.s1};
  check("kda_norm_gate", on_stream(dev, [&](kda_stream_t s) {
    return kda_norm_gate(ptr(x), ptr(gate), w, eps, rx.outer, rx.inner < 1 ? 1 : rx.inner, checked_int(D), strides,
                         a[4] == Py_True ? KDA_NORM_SILU : 0u, y.data_ptr(), s);
  }));
  return THPVariable_Wrap(std::move(y));
}

int64_t row_stride(const Tensor &t, const char *name) {
  if (t.is_contiguous()) return t.size(-1);
  if (t.dim() != 2) value_error(std::string(name) + " must be contiguous, or [rows,D] with a row stride");
  return t.stride(0);
}

// ---- add_norm(x, residual, weight, post_weight, gate, residual_scale, eps, out, residual_out)
PyObject *add_norm(PyObject *const *a) {
  const Tensor &x = as_rows(a[0]), &residual = as_tensor(a[1], "residual");
  const at::Device dev = x.device();
  const int64_t D = x.size(-1);
  need_layout(x, "x", at::kBFloat16, dev, false);
  const at::ScalarType rdt = residual.scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
  need(residual, "residual", rdt, x.sizes(), dev);
  const float *w = vector_of(a[2], "weight", D, dev), *post = vector_of(a[3], "post_weight", D, dev);
  const Tensor *gate = nullptr;
  if (given(a[4])) {
    gate = &as_tensor(a[4], "gate");
    need(*gate, "gate", at::kBFloat16, x.sizes(), dev);
  }
  const float *vec = nullptr;
  float scale = 1.f;
  if (THPVariable_Check(a[5])) vec = vector_of(a[5], "residual_scale", D, dev);
  else scale = (float)number(a[5]);
  const float eps = (float)number(a[6]);
  const int64_t strides[3] = {row_stride(x, "x"), row_stride(residual, "residual"), gate ? row_stride(*gate, "gate") : 0};
  Tensor y = output(a[7], "out", x.sizes(), at::kBFloat16, dev);
  Tensor h = output(a[8], "residual_out", x.sizes(), rdt, dev);
  need_gpu(x, "x");
  check("kda_add_norm", on_stream(dev, [&](kda_stream_t s) {
    return kda_add_norm(ptr(x), ptr(residual), gate ? ptr(*gate) : nullptr, post, w, vec, scale, eps, x.numel() / D,
                        checked_int(D), strides, rdt == at::kFloat ? KDA_NORM_RESIDUAL_F32 : 0u, y.data_ptr(),
                        h.data_ptr(), s);
  }));
  THPObjectPtr py(THPVariable_Wrap(std::move(y))), ph(THPVariable_Wrap(std::move(h)));
  if (!py || !ph) throw python_error();
  return PyTuple_Pack(2, py.get(), ph.get());
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *), int N>
constexpr PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<step, 13>("step"),           method<la_step, 9>("la_step"),   method<la_fwd, 13>("la_fwd"),
    method<norm_gate, 6>("norm_gate"), method<add_norm, 9>("add_norm"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module_def); }
