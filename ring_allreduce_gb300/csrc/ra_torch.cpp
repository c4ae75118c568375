// ra_torch.cpp -- the Python extension _ra_torch: torch tensors checked and
// marshalled into the argument blocks of the model operators (ra_norm_*,
// ra_vocab_*, ra_ffn_*, ra_ckpt_* of include/ra.h).  A decode step is a few microseconds on the
// GPU, so the way to the launch has to be short: about 1 us here for a call
// of a dozen tensors, 8 to 10 us in interpreted Python.
//
// The functions of libra_gb300.so are reached through their addresses, handed
// over once by bind() (which library is loaded is the ctypes binding's
// business).  A wrong type, shape, device or stride raises ValueError; what
// the library returns comes back as an integer.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <stdexcept>
#include <string>

#include "ra.h"

namespace {

struct Api {
  decltype(&ra_norm_forward) norm_forward;
  decltype(&ra_norm_backward) norm_backward;
  decltype(&ra_vocab_logprobs) logprobs;
  decltype(&ra_vocab_logprobs_backward) logprobs_backward;
  decltype(&ra_vocab_distill) distill;
  decltype(&ra_vocab_distill_backward) distill_backward;
  decltype(&ra_ffn_forward) ffn_forward;
  decltype(&ra_ffn_backward) ffn_backward;
  decltype(&ra_ckpt_store) ckpt_store;
  decltype(&ra_ckpt_load) ckpt_load;
} api;

constexpr int kRanks = 32;

using Type = at::ScalarType;

// The arguments of one call, in order; errors as C++ exceptions up to guarded().
struct Args {
  PyObject* const* at;
  PyObject* const* end;
  PyObject* next() {
    if (at == end) throw std::invalid_argument("too few arguments");
    return *at++;
  }
  long long number() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw std::invalid_argument("an integer is expected");
    return v;
  }
  // an address or a raw handle: None is 0
  void* pointer() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw std::invalid_argument("an address is expected");
    return p;
  }
};

Type type_of(long long code) {
  switch (code) {
    case RA_BF16: return at::kBFloat16;
    case RA_F16: return at::kHalf;
    default: return at::kFloat;
  }
}

std::string shape_text(const int64_t* shape, int dims) {
  std::string s = "(";
  for (int i = 0; i < dims; ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + ")";
}

[[noreturn]] void wrong(const char* name, const char* what) { throw std::invalid_argument(std::string(name) + ": " + what); }

[[noreturn]] void mismatch(const char* name, PyObject* o, Type type, const int64_t* shape, int dims, int device) {
  std::string text = std::string(name) + ": " + at::toString(type) + " " + shape_text(shape, dims) + " on cuda:" +
                     std::to_string(device) + ", its last axis contiguous, is expected, got ";
  if (!THPVariable_Check(o)) {
    text += Py_TYPE(o)->tp_name;
  } else {
    const at::Tensor& t = THPVariable_Unpack(o);
    text += std::string(at::toString(t.scalar_type())) + " " + shape_text(t.sizes().data(), (int)t.dim()) + " on " +
            t.device().str();
    if (t.layout() == at::kStrided) text += ", strides " + shape_text(t.strides().data(), (int)t.dim());
  }
  throw std::invalid_argument(text);
}

const at::Tensor* strided(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == at::kStrided ? &t : nullptr;
}

bool fits(const at::Tensor* t, Type type, const int64_t* shape, int dims, int device) {
  if (!t || t->scalar_type() != type || t->dim() != dims || t->get_device() != device) return false;
  for (int i = 0; i < dims; ++i)
    if (t->size(i) != shape[i]) return false;
  return true;
}

// Checks of one call's tensors.
struct Call {
  int device;

  // Address of a contiguous tensor.
  void* flat(const char* name, PyObject* o, Type type, std::initializer_list<int64_t> shape) const {
    const at::Tensor* t = strided(o);
    if (!fits(t, type, shape.begin(), (int)shape.size(), device) || !t->is_contiguous())
      mismatch(name, o, type, shape.begin(), (int)shape.size(), device);
    return t->data_ptr();
  }
  void* maybe(const char* name, PyObject* o, Type type, std::initializer_list<int64_t> shape) const {
    return o == Py_None ? nullptr : flat(name, o, type, shape);
  }

  // Address and row stride of a tensor [rows, width] whose rows are contiguous.
  void* rows(const char* name, PyObject* o, Type type, int64_t rows, int64_t width, size_t* stride) const {
    const int64_t shape[2] = {rows, width};
    const at::Tensor* t = strided(o);
    if (!fits(t, type, shape, 2, device) || (t->stride(1) != 1 && width > 1)) mismatch(name, o, type, shape, 2, device);
    *stride = rows > 1 ? (size_t)t->stride(0) : (size_t)width;
    return t->data_ptr();
  }

  // Rank buffers [rows, width]: a sequence of tensors or one with a leading
  // axis; their number, R, or also 1 where `one` allows it.
  int ranks(const char* name, PyObject* o, int R, bool one, Type type, int64_t n_rows, int64_t width, void** p,
            size_t* stride) const {
    if (THPVariable_Check(o)) {
      const at::Tensor* t = strided(o);
      const int64_t n = t && t->dim() == 3 ? t->size(0) : -1;
      const int64_t shape[3] = {n == R || (one && n == 1) ? n : R, n_rows, width};
      if (!fits(t, type, shape, 3, device) || (t->stride(2) != 1 && width > 1)) mismatch(name, o, type, shape, 3, device);
      *stride = n_rows > 1 ? (size_t)t->stride(1) : (size_t)width;
      char* base = static_cast<char*>(t->data_ptr());
      const int64_t step = t->stride(0) * (int64_t)t->element_size();
      for (int r = 0; r < n; ++r) p[r] = base + r * step;
      return (int)n;
    }
    PyObject* seq = PySequence_Fast(o, "a sequence of rank buffers is expected");
    if (!seq) throw std::invalid_argument(std::string(name) + ": a sequence of rank buffers is expected");
    try {
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
      if (n != R && !(one && n == 1))
        wrong(name, ((one ? "1 or " : "") + std::to_string(R) + " rank buffers are expected, got " + std::to_string(n)).c_str());
      for (Py_ssize_t r = 0; r < n; ++r) {
        size_t s;
        p[r] = rows(name, PySequence_Fast_GET_ITEM(seq, r), type, n_rows, width, &s);
        if (r == 0) *stride = s;
        if (s != *stride) wrong(name, "the rank buffers' rows have different strides");
      }
      Py_DECREF(seq);
      return (int)n;
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
  }

  // The logits' shards [rows, min(C, V - r C)]; those without columns are not looked at.
  void shards(const char* name, PyObject* o, int R, int64_t V, Type type, int64_t n_rows, void** p, size_t* strides) const {
    PyObject* seq = PySequence_Fast(o, "a sequence of shards is expected");
    if (!seq) throw std::invalid_argument(std::string(name) + ": a sequence of shards is expected");
    try {
      if (PySequence_Fast_GET_SIZE(seq) != R)
        wrong(name, (std::to_string(R) + " shards are expected, got " + std::to_string(PySequence_Fast_GET_SIZE(seq))).c_str());
      const int64_t C = (V + R - 1) / R;
      for (int r = 0; r < R; ++r) {
        const int64_t width = std::min(C, V - r * C);
        p[r] = nullptr;
        strides[r] = 0;
        if (width > 0) p[r] = rows(name, PySequence_Fast_GET_ITEM(seq, r), type, n_rows, width, &strides[r]);
      }
      Py_DECREF(seq);
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
  }
};

// Axis `i` of a tensor of `dims` axes.
int64_t axis(const char* name, PyObject* o, int dims, int i, const char* want) {
  const at::Tensor* t = strided(o);
  if (!t || t->dim() != dims) wrong(name, want);
  return t->size(i);
}

template <class F> PyObject* guarded(F&& f) {
  try {
    return PyLong_FromLong(f());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred() || PyErr_ExceptionMatches(PyExc_TypeError)) {
      PyErr_Clear();
      PyErr_SetString(PyExc_ValueError, e.what());
    }
    return nullptr;
  }
}

// (handle, device, R, dim, dtype, residual_dtype, param_dtype) lead every norm call
struct NormConfig {
  ra_norm_handle h;
  Call call;
  int R;
  int64_t dim;
  Type type, residual, param;
  explicit NormConfig(Args& a) {
    h = static_cast<ra_norm_handle>(a.pointer());
    call.device = (int)a.number();
    R = (int)a.number();
    dim = a.number();
    type = type_of(a.number());
    residual = type_of(a.number());
    param = type_of(a.number());
  }
  const void* gate(PyObject* o, size_t* rows) const {
    *rows = 0;
    if (o == Py_None) return nullptr;
    const int64_t n = axis("gate", o, 2, 0, "a tensor [groups, dim] is expected");
    *rows = (size_t)n;
    return call.flat("gate", o, param, {n, dim});
  }
};

PyObject* norm_forward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    const NormConfig c(a);
    const Call& k = c.call;
    ra_norm_forward_args g{};
    void *in[kRanks], *out[kRanks];
    PyObject* parts = a.next();
    PyObject* residual = a.next();
    const int64_t T = axis("residual", residual, 2, 0, "a tensor [rows, dim] is expected");
    g.rows = (size_t)T;
    k.ranks("parts", parts, c.R, false, c.type, T, c.dim, in, &g.in_stride);
    g.residual = k.rows("residual", residual, c.residual, T, c.dim, &g.residual_stride);
    g.weight = k.flat("weight", a.next(), c.param, {c.dim});
    g.outs = k.ranks("outs", a.next(), c.R, true, c.type, T, c.dim, out, &g.out_stride);
    g.residual_out = k.rows("residual_out", a.next(), c.residual, T, c.dim, &g.residual_out_stride);
    g.post_weight = k.maybe("post_weight", a.next(), c.param, {c.dim});
    g.gate = c.gate(a.next(), &g.gate_rows);
    PyObject* total = a.next();
    if (total != Py_None) g.total = k.rows("total", total, c.type, T, c.dim, &g.total_stride);
    g.rstd = static_cast<float*>(k.maybe("rstd", a.next(), at::kFloat, {2, T}));
    g.in = in;
    g.out = out;
    return api.norm_forward(c.h, &g, a.pointer());
  });
}

PyObject* norm_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    const NormConfig c(a);
    const Call& k = c.call;
    ra_norm_backward_args g{};
    void *in[kRanks], *out[kRanks];
    PyObject* grad_outs = a.next();
    PyObject* grad_residual_out = a.next();
    PyObject* residual_out = a.next();
    const int64_t T = axis("residual_out", residual_out, 2, 0, "a tensor [rows, dim] is expected");
    g.rows = (size_t)T;
    g.grads = k.ranks("grad_outs", grad_outs, c.R, true, c.type, T, c.dim, in, &g.grad_out_stride);
    if (grad_residual_out != Py_None)
      g.grad_residual_out =
          k.rows("grad_residual_out", grad_residual_out, c.residual, T, c.dim, &g.grad_residual_out_stride);
    g.residual_out = k.rows("residual_out", residual_out, c.residual, T, c.dim, &g.residual_out_stride);
    g.rstd = static_cast<float*>(k.flat("rstd", a.next(), at::kFloat, {2, T}));
    g.weight = k.flat("weight", a.next(), c.param, {c.dim});
    g.outs = k.ranks("grad_ins", a.next(), c.R, true, c.type, T, c.dim, out, &g.grad_in_stride);
    g.grad_residual = k.rows("grad_residual", a.next(), c.residual, T, c.dim, &g.grad_residual_stride);
    g.grad_weight = static_cast<float*>(k.maybe("grad_weight", a.next(), at::kFloat, {c.dim}));
    g.post_weight = k.maybe("post_weight", a.next(), c.param, {c.dim});
    g.gate = c.gate(a.next(), &g.gate_rows);
    PyObject* total = a.next();
    if (total != Py_None) g.total = k.rows("total", total, c.type, T, c.dim, &g.total_stride);
    g.grad_post_weight = static_cast<float*>(k.maybe("grad_post_weight", a.next(), at::kFloat, {c.dim}));
    g.grad_gate = static_cast<float*>(k.maybe("grad_gate", a.next(), at::kFloat, {(int64_t)g.gate_rows, c.dim}));
    g.grad_out = in;
    g.grad_in = out;
    return api.norm_backward(c.h, &g, a.pointer());
  });
}

// (handle, device, R, vocab, dtype) lead every head call
struct HeadConfig {
  ra_vocab_handle h;
  Call call;
  int R;
  int64_t V;
  long long code;
  Type type;
  void* x[kRanks];
  size_t strides[kRanks];
  explicit HeadConfig(Args& a) {
    h = static_cast<ra_vocab_handle>(a.pointer());
    call.device = (int)a.number();
    R = (int)a.number();
    V = a.number();
    code = a.number();
    type = type_of(code);
  }
  void shards(PyObject* o, int64_t T) { call.shards("shards", o, R, V, type, T, x, strides); }
  float* floats(const char* name, PyObject* o, int64_t T) const {
    return static_cast<float*>(call.flat(name, o, at::kFloat, {T}));
  }
};

PyObject* logprobs(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    HeadConfig c(a);
    ra_vocab_logprobs_args g{};
    PyObject* shards = a.next();
    PyObject* targets = a.next();
    const int64_t T = axis("targets", targets, 1, 0, "a tensor [rows] is expected");
    g.rows = (size_t)T;
    c.shards(shards, T);
    g.shards = c.x;
    g.strides = c.strides;
    g.targets = static_cast<int64_t*>(c.call.flat("targets", targets, at::kLong, {T}));
    g.logprob = c.floats("logprob", a.next(), T);
    g.lse = c.floats("lse", a.next(), T);
    PyObject* entropy = a.next();
    if (entropy != Py_None) g.entropy = c.floats("entropy", entropy, T);
    PyObject* ids = a.next();
    PyObject* top = a.next();
    if ((ids == Py_None) != (top == Py_None)) wrong("top_ids, top_logprobs", "they go together");
    if (ids != Py_None) {
      const int64_t K = axis("top_ids", ids, 2, 1, "a tensor [rows, K] is expected");
      g.top = (int)std::min<int64_t>(K, 1 << 20);
      g.top_ids = static_cast<int64_t*>(c.call.flat("top_ids", ids, at::kLong, {T, K}));
      g.top_logprobs = static_cast<float*>(c.call.flat("top_logprobs", top, at::kFloat, {T, K}));
    }
    return api.logprobs(c.h, &g, a.pointer());
  });
}

PyObject* logprobs_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    HeadConfig c(a);
    ra_vocab_logprobs_backward_args g{};
    PyObject* shards = a.next();
    PyObject* targets = a.next();
    const int64_t T = axis("targets", targets, 1, 0, "a tensor [rows] is expected");
    g.rows = (size_t)T;
    c.shards(shards, T);
    g.shards = c.x;
    g.strides = c.strides;
    g.targets = static_cast<int64_t*>(c.call.flat("targets", targets, at::kLong, {T}));
    g.lse = c.floats("lse", a.next(), T);
    g.grad_logprob = c.floats("grad_logprob", a.next(), T);
    void* grads[kRanks];
    size_t grad_strides[kRanks];
    c.call.shards("grads", a.next(), c.R, c.V, c.type, T, grads, grad_strides);
    g.grads = grads;
    g.grad_strides = grad_strides;
    PyObject* entropy = a.next();
    PyObject* grad_entropy = a.next();
    if (grad_entropy != Py_None) {
      g.grad_entropy = c.floats("grad_entropy", grad_entropy, T);
      g.entropy = c.floats("entropy", entropy, T);
    }
    return api.logprobs_backward(c.h, &g, a.pointer());
  });
}

// The teacher's tokens of a call; answers the rows.
template <class G> int64_t teacher(const HeadConfig& c, PyObject* ids, PyObject* logits, G* g) {
  const int64_t T = axis("teacher_ids", ids, 2, 0, "a tensor [rows, K] is expected");
  const int64_t K = THPVariable_Unpack(ids).size(1);
  g->rows = (size_t)T;
  g->teacher_k = (int)std::min<int64_t>(K, 1 << 20);
  g->teacher_ids = static_cast<int64_t*>(c.call.flat("teacher_ids", ids, at::kLong, {T, K}));
  const at::Tensor* t = strided(logits);
  const bool f32 = t && t->scalar_type() == at::kFloat;
  g->teacher_logits = c.call.flat("teacher_logits", logits, f32 ? at::kFloat : c.type, {T, K});
  g->teacher_dtype = f32 ? RA_F32 : (ra_dtype)c.code;
  return T;
}

PyObject* distill(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    HeadConfig c(a);
    ra_vocab_distill_args g{};
    PyObject* shards = a.next();
    PyObject* ids = a.next();
    const int64_t T = teacher(c, ids, a.next(), &g);
    c.shards(shards, T);
    g.shards = c.x;
    g.strides = c.strides;
    g.loss = c.floats("loss", a.next(), T);
    g.lse = c.floats("lse", a.next(), T);
    return api.distill(c.h, &g, a.pointer());
  });
}

PyObject* distill_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    HeadConfig c(a);
    ra_vocab_distill_backward_args g{};
    PyObject* shards = a.next();
    PyObject* ids = a.next();
    const int64_t T = teacher(c, ids, a.next(), &g);
    c.shards(shards, T);
    g.shards = c.x;
    g.strides = c.strides;
    g.lse = c.floats("lse", a.next(), T);
    g.grad_loss = c.floats("grad_loss", a.next(), T);
    void* grads[kRanks];
    size_t grad_strides[kRanks];
    c.call.shards("grads", a.next(), c.R, c.V, c.type, T, grads, grad_strides);
    g.grads = grads;
    g.grad_strides = grad_strides;
    return api.distill_backward(c.h, &g, a.pointer());
  });
}

// A list of R tensors, one a rank's shard of `inner` columns (chunk plan: C
// columns a rank); those of ranks without columns are not looked at.
struct Shards {
  void* at[kRanks];
  size_t strides[kRanks];
};

// (handle, device, R, dim, inner, dtype, grad_dtype) lead every feed-forward call
struct FfnConfig {
  ra_ffn_handle h;
  Call call;
  mutable PyObject* made[2 * kRanks];   // lists of what can be gone through once only
  mutable int made_count = 0;
  int R;
  int64_t dim, inner, C;
  Type type, grad;
  explicit FfnConfig(Args& a) {
    h = static_cast<ra_ffn_handle>(a.pointer());
    call.device = (int)a.number();
    R = (int)a.number();
    dim = a.number();
    inner = a.number();
    C = (inner + R - 1) / R;
    type = type_of(a.number());
    grad = type_of(a.number());
  }
  FfnConfig(const FfnConfig&) = delete;
  ~FfnConfig() {
    while (made_count) Py_DECREF(made[--made_count]);
  }
  PyObject* again(PyObject* o) const {
    if (o == Py_None || THPVariable_Check(o) || PyList_Check(o) || PyTuple_Check(o) || made_count == 2 * kRanks) return o;
    PyObject* list = PySequence_List(o);
    if (!list) PyErr_Clear();
    if (list) made[made_count++] = list;
    return list ? list : o;   // what is no sequence is refused where it is looked at
  }
  // f(r, width, tensor) for every rank that holds columns
  template <class F> void each(const char* name, PyObject* o, F&& f) const {
    PyObject* seq = PySequence_Fast(o, "a sequence of shards is expected");
    if (!seq) throw std::invalid_argument(std::string(name) + ": a sequence of shards is expected");
    try {
      if (PySequence_Fast_GET_SIZE(seq) != R)
        wrong(name, (std::to_string(R) + " shards are expected, got " + std::to_string(PySequence_Fast_GET_SIZE(seq))).c_str());
      for (int r = 0; r < R; ++r) {
        const int64_t width = std::min(C, inner - r * C);
        if (width > 0) f(r, width, PySequence_Fast_GET_ITEM(seq, r));
      }
      Py_DECREF(seq);
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
  }
  void columns(const char* name, PyObject* o, Type t, int64_t T, Shards* s) const {
    each(name, o, [&](int r, int64_t width, PyObject* x) { s->at[r] = call.rows(name, x, t, T, width, &s->strides[r]); });
  }
  void weights(const char* name, PyObject* o, Type t, Shards* s) const {
    each(name, o, [&](int r, int64_t width, PyObject* x) { s->at[r] = call.rows(name, x, t, width, dim, &s->strides[r]); });
  }
  void scales(const char* name, PyObject* o, int64_t T, float** at) const {
    each(name, o, [&](int r, int64_t width, PyObject* x) {
      at[r] = static_cast<float*>(call.flat(name, x, at::kFloat, {T, (width + 127) / 128}));
    });
  }
  // 8 where the shards hold 8-bit codes, 16 where they hold the block's type
  int bits(PyObject* o) const {
    int n = 16;
    each("gate", o, [&](int r, int64_t, PyObject* x) {
      const at::Tensor* t = strided(x);
      if (r == 0 && t && t->scalar_type() == at::kChar) n = 8;
    });
    return n;
  }
};

// Rows of the rank buffers that a call goes by.
int64_t ranks_rows(const char* name, PyObject* o) {
  if (THPVariable_Check(o)) return axis(name, o, 3, 1, "rank buffers [rows, dim] are expected");
  PyObject* seq = PySequence_Fast(o, "a sequence of rank buffers is expected");
  if (!seq) throw std::invalid_argument(std::string(name) + ": a sequence of rank buffers is expected");
  PyObject* first = PySequence_Fast_GET_SIZE(seq) ? PySequence_Fast_GET_ITEM(seq, 0) : nullptr;
  const at::Tensor* t = first ? strided(first) : nullptr;
  const int64_t n = t && t->dim() == 2 ? t->size(0) : -1;
  Py_DECREF(seq);
  if (n < 0) wrong(name, "rank buffers [rows, dim] are expected");
  return n;
}

struct Kept {
  int bits = 0;
  Shards gate, up;
  float *gate_scales[kRanks], *up_scales[kRanks];
  Kept(const FfnConfig& c, PyObject* g, PyObject* u, PyObject* gs, PyObject* us, int64_t T) {
    if ((g == Py_None) != (u == Py_None)) wrong("gate, up", "they go together");
    if (g == Py_None) {
      if (gs != Py_None || us != Py_None) wrong("gate_scales, up_scales", "scales without gate and up");
      return;
    }
    bits = c.bits(g);
    const Type t = bits == 8 ? at::kChar : c.type;
    c.columns("gate", g, t, T, &gate);
    c.columns("up", u, t, T, &up);
    if (bits == 8) {
      c.scales("gate_scales", gs, T, gate_scales);
      c.scales("up_scales", us, T, up_scales);
    } else if (gs != Py_None || us != Py_None) {
      wrong("gate_scales, up_scales", "they go with 8-bit codes");
    }
  }
};

PyObject* ffn_forward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    const FfnConfig c(a);
    ra_ffn_forward_args g{};
    void *x[kRanks], *out[kRanks];
    Shards w[3], hidden;
    PyObject* xs = c.again(a.next());
    const int64_t T = ranks_rows("xs", xs);
    g.rows = (size_t)T;
    g.xs = c.call.ranks("xs", xs, c.R, true, c.type, T, c.dim, x, &g.x_stride);
    c.weights("w_gate", c.again(a.next()), c.type, &w[0]);
    c.weights("w_up", c.again(a.next()), c.type, &w[1]);
    c.weights("w_down", c.again(a.next()), c.type, &w[2]);
    c.columns("hidden", c.again(a.next()), c.type, T, &hidden);
    c.call.ranks("parts", c.again(a.next()), c.R, false, c.type, T, c.dim, out, &g.out_stride);
    PyObject* kept[4];
    for (PyObject*& o : kept) o = c.again(a.next());
    Kept k(c, kept[0], kept[1], kept[2], kept[3], T);
    g.x = x;
    g.w_gate = w[0].at;
    g.w_gate_strides = w[0].strides;
    g.w_up = w[1].at;
    g.w_up_strides = w[1].strides;
    g.w_down = w[2].at;
    g.w_down_strides = w[2].strides;
    g.hidden = hidden.at;
    g.hidden_strides = hidden.strides;
    g.out = out;
    g.keep_bits = k.bits;
    g.gate = k.gate.at;
    g.gate_strides = k.gate.strides;
    g.up = k.up.at;
    g.up_strides = k.up.strides;
    g.gate_scales = k.gate_scales;
    g.up_scales = k.up_scales;
    return api.ffn_forward(c.h, &g, a.pointer());
  });
}

PyObject* ffn_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    const FfnConfig c(a);
    ra_ffn_backward_args g{};
    void *dy[kRanks], *x[kRanks], *dx[kRanks];
    Shards w[3], hidden, pre[2], gw[3];
    PyObject* grad_parts = c.again(a.next());
    PyObject* xs = c.again(a.next());
    PyObject* weights[3];
    for (PyObject*& o : weights) o = c.again(a.next());
    PyObject* kept[2];
    for (PyObject*& o : kept) o = c.again(a.next());
    PyObject* hid = c.again(a.next());
    PyObject* pres[2];
    for (PyObject*& o : pres) o = c.again(a.next());
    PyObject* grad_xs = c.again(a.next());
    PyObject* grads[3];
    for (PyObject*& o : grads) o = c.again(a.next());
    PyObject* gate_scales = c.again(a.next());
    PyObject* up_scales = c.again(a.next());
    const int64_t T = ranks_rows("grad_parts", grad_parts);
    g.rows = (size_t)T;
    g.grads = c.call.ranks("grad_parts", grad_parts, c.R, true, c.type, T, c.dim, dy, &g.grad_out_stride);
    g.grad_out = dy;
    if (kept[0] == Py_None) wrong("gate", "what forward kept is expected");
    Kept k(c, kept[0], kept[1], gate_scales, up_scales, T);
    g.keep_bits = k.bits;
    g.gate = k.gate.at;
    g.gate_strides = k.gate.strides;
    g.up = k.up.at;
    g.up_strides = k.up.strides;
    g.gate_scales = k.gate_scales;
    g.up_scales = k.up_scales;
    c.weights("w_down", weights[2], c.type, &w[2]);
    g.w_down = w[2].at;
    g.w_down_strides = w[2].strides;
    if (hid != Py_None) {
      c.columns("hidden", hid, c.type, T, &hidden);
      g.hidden = hidden.at;
      g.hidden_strides = hidden.strides;
    }
    c.columns("grad_gate", pres[0], c.type, T, &pre[0]);
    c.columns("grad_up", pres[1], c.type, T, &pre[1]);
    g.grad_gate = pre[0].at;
    g.grad_gate_strides = pre[0].strides;
    g.grad_up = pre[1].at;
    g.grad_up_strides = pre[1].strides;
    if (grad_xs != Py_None) {
      c.weights("w_gate", weights[0], c.type, &w[0]);
      c.weights("w_up", weights[1], c.type, &w[1]);
      g.w_gate = w[0].at;
      g.w_gate_strides = w[0].strides;
      g.w_up = w[1].at;
      g.w_up_strides = w[1].strides;
      c.call.ranks("grad_xs", grad_xs, c.R, false, c.type, T, c.dim, dx, &g.grad_x_stride);
      g.grad_x = dx;
    }
    if (grads[0] != Py_None || grads[1] != Py_None) {
      g.xs = c.call.ranks("xs", xs, c.R, true, c.type, T, c.dim, x, &g.x_stride);
      g.x = x;
    }
    const char* names[3] = {"grad_w_gate", "grad_w_up", "grad_w_down"};
    for (int i = 0; i < 3; ++i)
      if (grads[i] != Py_None) c.weights(names[i], grads[i], c.grad, &gw[i]);
    if (grads[0] != Py_None) {
      g.grad_w_gate = gw[0].at;
      g.grad_w_gate_strides = gw[0].strides;
    }
    if (grads[1] != Py_None) {
      g.grad_w_up = gw[1].at;
      g.grad_w_up_strides = gw[1].strides;
    }
    if (grads[2] != Py_None) {
      g.grad_w_down = gw[2].at;
      g.grad_w_down_strides = gw[2].strides;
    }
    return api.ffn_backward(c.h, &g, a.pointer());
  });
}

// (handle, device, dim, dtype, normed_dtype, param_dtype) lead the calls for kept rows
struct CkptConfig {
  ra_ckpt_handle h;
  Call call;
  int64_t dim;
  Type type, normed, param;
  explicit CkptConfig(Args& a) {
    h = static_cast<ra_ckpt_handle>(a.pointer());
    call.device = (int)a.number();
    dim = a.number();
    type = type_of(a.number());
    normed = type_of(a.number());
    param = type_of(a.number());
  }
  float* scales(PyObject* o, int64_t T) const {
    return static_cast<float*>(call.flat("scales", o, at::kFloat, {T, (dim + 127) / 128}));
  }
};

PyObject* ckpt_store(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    const CkptConfig c(a);
    ra_ckpt_store_args g{};
    PyObject* values = a.next();
    const int64_t T = axis("values", values, 2, 0, "a tensor [rows, dim] is expected");
    g.rows = (size_t)T;
    g.values = c.call.rows("values", values, c.type, T, c.dim, &g.stride);
    g.codes = static_cast<signed char*>(c.call.rows("codes", a.next(), at::kChar, T, c.dim, &g.codes_stride));
    g.scales = c.scales(a.next(), T);
    return api.ckpt_store(c.h, &g, a.pointer());
  });
}

PyObject* ckpt_load(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    const CkptConfig c(a);
    ra_ckpt_load_args g{};
    PyObject* codes = a.next();
    const int64_t T = axis("codes", codes, 2, 0, "a tensor [rows, dim] is expected");
    g.rows = (size_t)T;
    g.codes = static_cast<signed char*>(c.call.rows("codes", codes, at::kChar, T, c.dim, &g.codes_stride));
    g.scales = c.scales(a.next(), T);
    PyObject* values = a.next();
    if (values != Py_None) g.values = c.call.rows("values", values, c.type, T, c.dim, &g.stride);
    PyObject* rstd = a.next();
    PyObject* weight = a.next();
    PyObject* normed = a.next();
    if (normed != Py_None) {
      g.rstd = static_cast<float*>(c.call.flat("rstd", rstd, at::kFloat, {T}));
      g.weight = c.call.flat("weight", weight, c.param, {c.dim});
      g.normed = c.call.rows("normed", normed, c.normed, T, c.dim, &g.normed_stride);
    }
    return api.ckpt_load(c.h, &g, a.pointer());
  });
}

// bind(norm_forward, norm_backward, logprobs, logprobs_backward, distill,
// distill_backward, ffn_forward, ffn_backward, ckpt_store, ckpt_load): the
// library's functions, by address
PyObject* bind(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> int {
    Args a{argv, argv + argc};
    api.norm_forward = reinterpret_cast<decltype(api.norm_forward)>(a.pointer());
    api.norm_backward = reinterpret_cast<decltype(api.norm_backward)>(a.pointer());
    api.logprobs = reinterpret_cast<decltype(api.logprobs)>(a.pointer());
    api.logprobs_backward = reinterpret_cast<decltype(api.logprobs_backward)>(a.pointer());
    api.distill = reinterpret_cast<decltype(api.distill)>(a.pointer());
    api.distill_backward = reinterpret_cast<decltype(api.distill_backward)>(a.pointer());
    api.ffn_forward = reinterpret_cast<decltype(api.ffn_forward)>(a.pointer());
    api.ffn_backward = reinterpret_cast<decltype(api.ffn_backward)>(a.pointer());
    api.ckpt_store = reinterpret_cast<decltype(api.ckpt_store)>(a.pointer());
    api.ckpt_load = reinterpret_cast<decltype(api.ckpt_load)>(a.pointer());
    return 0;
  });
}

#define RA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RA_METHOD(bind), RA_METHOD(norm_forward), RA_METHOD(norm_backward), RA_METHOD(logprobs),
                         RA_METHOD(logprobs_backward), RA_METHOD(distill), RA_METHOD(distill_backward),
                         RA_METHOD(ffn_forward), RA_METHOD(ffn_backward), RA_METHOD(ckpt_store), RA_METHOD(ckpt_load),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ra_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ra_torch() { return PyModule_Create(&module); }
