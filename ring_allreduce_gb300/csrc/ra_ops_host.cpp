// ra_ops_host.cpp -- host side of the model operators of include/ra.h
// (ra_norm_*, ra_vocab_*): handles, argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>

#include "ra.h"
#include "ra_ops.h"

namespace ra {
ra_status record_error(ra_status s, const char* fmt, ...);   // ra_host.cpp
}

namespace {

// Device memory of a handle.  Graphs that captured a call which uses it share
// it with the handle (`shared`, once there are any), and may be replayed when
// the handle is gone.  The last of them to go hands it over to retire(), on a
// thread of the driver's that may call nothing of CUDA: it waits in a list until
// a later call frees it.
struct Workspace {
  void* p = nullptr;
  cudaUserObject_t shared = nullptr;
  Workspace* next = nullptr;
};

struct Retired {
  std::mutex lock;
  Workspace* first = nullptr;
};
Retired& retired() {
  static Retired* r = new Retired;   // never destroyed: the driver's thread may outlive static objects
  return *r;
}

void CUDART_CB retire(void* w) {
  Retired& r = retired();
  std::lock_guard<std::mutex> hold(r.lock);
  static_cast<Workspace*>(w)->next = r.first;
  r.first = static_cast<Workspace*>(w);
}

void free_retired() {
  Workspace* w;
  {
    Retired& r = retired();
    std::lock_guard<std::mutex> hold(r.lock);
    w = r.first;
    r.first = nullptr;
  }
  while (w) {
    Workspace* next = w->next;
    cudaFree(w->p);
    delete w;
    w = next;
  }
}

}  // namespace

struct ra_norm_ctx {
  int R, dim, device, sms;
  ra_dtype dtype, residual_dtype, param_dtype;
  float eps, scale;
  bool check_pointers = true;
  Workspace* work = nullptr;   // column partials of the weights' gradients, from the first backward call on
  ra::OptedIn opted;
};

struct ra_vocab_ctx {
  int R, V, C, shards, device, sms;
  ra_dtype dtype;
  float tau;
  bool check_pointers = true;
};

namespace {

using ra::kMaxRanks;
using ra::record_error;

constexpr int64_t kMaxRows = 0x7FFFFFFF;

ra_status cuda_error(cudaError_t e, const char* what) {
  cudaGetLastError();   // clear a non-sticky error so the next call starts clean
  return record_error(e == cudaErrorMemoryAllocation ? RA_ERR_OOM : RA_ERR_CUDA, "%s: %s (%s)", what,
                      cudaGetErrorName(e), cudaGetErrorString(e));
}

// No C++ exception leaves the C entry points.
template <class F> ra_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return RA_ERR_OOM;   // the only ones there are: an error text that could not be stored
  }
}

// The handle's device for the duration of a call.
struct OnDevice {
  int prev = -1;
  cudaError_t status;
  explicit OnDevice(int dev) {
    status = cudaGetDevice(&prev);
    if (status == cudaSuccess && prev != dev) {
      status = cudaSetDevice(dev);
    } else {
      prev = -1;   // nothing to put back
    }
  }
  ~OnDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

bool is_float(int d) { return d == RA_F32 || d == RA_BF16 || d == RA_F16; }
size_t bytes_of(int d) { return d == RA_F32 ? 4 : 2; }

// One buffer of a call: `rows` rows of `width` bytes, `stride` bytes apart.
struct Buffer {
  const char* name;
  int index;               // -1: the only one of its name
  uintptr_t lo;
  size_t width, stride, span;
  bool output;
  const void* twin;        // an output may stand in this buffer's place (same address and stride)
};

// The buffers of one call and what has to hold of them.
class Buffers {
 public:
  Buffers(int device, bool check_pointers, size_t rows)
      : device_(device), rows_(rows), check_pointers_(check_pointers) {}

  // A buffer of rows() rows (or `rows` of them) of `width` elements; `stride`
  // in elements, made the width where there is one row.  The checked stride comes back.
  ra_status add(const char* name, int index, const void* p, size_t elem, size_t width, size_t* stride, bool output,
                size_t rows, const void* twin = nullptr) {
    if (!p) return record_error(RA_ERR_INVALID, "%s is NULL", label(name, index));
    if ((uintptr_t)p % elem)
      return record_error(RA_ERR_INVALID, "%s=%p is not aligned to its elements", label(name, index), p);
    if (rows <= 1) *stride = width;
    if (*stride < width)
      return record_error(RA_ERR_INVALID, "%s: stride %zu below the row's %zu elements", label(name, index), *stride,
                          width);
    if (*stride > ((size_t)1 << 46) / rows)
      return record_error(RA_ERR_INVALID, "%s: stride %zu too large", label(name, index), *stride);
    if (count_ == kMost) return record_error(RA_ERR_INVALID, "too many buffers");
    Buffer& b = b_[count_++];
    b.name = name;
    b.index = index;
    b.lo = (uintptr_t)p;
    b.width = width * elem;
    b.stride = *stride * elem;
    b.span = (rows - 1) * b.stride + b.width;
    b.output = output;
    b.twin = twin;
    return RA_OK;
  }
  ra_status add(const char* name, int index, const void* p, size_t elem, size_t width, size_t* stride, bool output,
                const void* twin = nullptr) {
    return add(name, index, p, elem, width, stride, output, rows_, twin);
  }
  // `count` elements in a row
  ra_status flat(const char* name, const void* p, size_t elem, size_t count, bool output) {
    size_t stride = count;
    return add(name, -1, p, elem, count, &stride, output, 1);
  }

  ra_status check() {
    for (int i = 0; i < count_; ++i) {
      if (b_[i].output)
        for (int k = 0; k < count_; ++k)
          if (k != i && !(b_[k].output && k < i) && overlap(b_[i], b_[k])) {
            char other[32];
            std::strncpy(other, label(b_[k].name, b_[k].index), sizeof(other) - 1);
            other[sizeof(other) - 1] = 0;
            return record_error(RA_ERR_INVALID, "output %s overlaps %s", label(b_[i].name, b_[i].index), other);
          }
      if (!check_pointers_) continue;
      cudaPointerAttributes at;
      const void* p = (const void*)b_[i].lo;
      const cudaError_t e = cudaPointerGetAttributes(&at, p);
      if (e != cudaSuccess) {
        cudaGetLastError();
        return record_error(RA_ERR_INVALID, "%s=%p: not a CUDA pointer (%s)", label(b_[i].name, b_[i].index), p,
                            cudaGetErrorName(e));
      }
      if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
        return record_error(RA_ERR_INVALID, "%s=%p: not device memory", label(b_[i].name, b_[i].index), p);
      if (at.type == cudaMemoryTypeDevice && at.device != device_)
        return record_error(RA_ERR_INVALID, "%s=%p: memory of device %d, handle is on device %d",
                            label(b_[i].name, b_[i].index), p, at.device, device_);
    }
    register_debug();
    return RA_OK;
  }

  // Every row of every buffer so far starts on a 16-byte boundary, and rows
  // of `row_bytes` hold whole 16-byte vectors.
  bool aligned(size_t row_bytes) const {
    uintptr_t bits = row_bytes;
    for (int i = 0; i < count_; ++i) bits |= b_[i].lo | (b_[i].span > b_[i].width ? b_[i].stride : 0);
    return bits % 16 == 0;
  }

 private:
  static constexpr int kMost = 2 * kMaxRanks + 16;

  const char* label(const char* name, int index) {
    if (index < 0) return name;
    std::snprintf(text_, sizeof(text_), "%s[%d]", name, index);
    return text_;
  }

  static bool overlap(const Buffer& a, const Buffer& b) {
    if (a.lo >= b.lo + b.span || b.lo >= a.lo + a.span) return false;
    if (a.output && a.twin && (uintptr_t)a.twin == b.lo && a.lo == b.lo && a.stride == b.stride) return false;
    if (a.stride == b.stride && a.stride >= a.width + b.width) {
      // column slices of one matrix: b's columns begin d bytes after a's
      const size_t s = a.stride;
      const size_t d = b.lo >= a.lo ? (b.lo - a.lo) % s : (s - (a.lo - b.lo) % s) % s;
      if (d >= a.width && d + b.width <= s) return false;
    }
    return true;
  }

  void register_debug() {
#ifdef RA_DEBUG_BOUNDS
    ra::DebugTable& t = ra::debug_table();
    t.count = 0;
    t.report = ra::debug_report();
    for (int i = 0; i < count_ && t.count < ra::kDebugRanges; ++i, ++t.count) {
      t.r[t.count].lo = b_[i].lo;
      t.r[t.count].hi = b_[i].lo + b_[i].span;
    }
#endif
  }

  Buffer b_[kMost];
  int count_ = 0;
  int device_;
  size_t rows_;
  bool check_pointers_;
  char text_[32];
};

#define RA_TRY(call)                       \
  do {                                     \
    const ra_status try_status = (call);   \
    if (try_status != RA_OK) return try_status; \
  } while (0)

ra_status device_of(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
  if (e != cudaSuccess) return cuda_error(e, "cudaDeviceGetAttribute");
  return RA_OK;
}

ra_status check_rows(size_t rows) {
  if (rows > (size_t)kMaxRows) return record_error(RA_ERR_INVALID, "rows=%zu too large", rows);
  return RA_OK;
}

ra_status check_gate(const void* gate, size_t gate_rows, size_t rows) {
  if (!gate) return RA_OK;
  if (gate_rows < 1 || gate_rows > rows || rows % gate_rows)
    return record_error(RA_ERR_INVALID, "gate_rows=%zu does not divide rows=%zu", gate_rows, rows);
  return RA_OK;
}

ra_status check_ranks(const char* name, int count, int R) {
  if (count != 1 && count != R) return record_error(RA_ERR_INVALID, "%s=%d: 1 or R=%d expected", name, count, R);
  return RA_OK;
}

}  // namespace

// ---------------------------------------------------------------- block end

static ra_status norm_create(int R, int dim, ra_dtype dtype, ra_dtype rdtype, ra_dtype pdtype, float eps, float scale,
                             ra_norm_handle* out) {
  if (!out) return record_error(RA_ERR_INVALID, "NULL handle pointer");
  if (R < 1 || R > kMaxRanks) return record_error(RA_ERR_INVALID, "R=%d outside [1, %d]", R, kMaxRanks);
  if (dim < 1) return record_error(RA_ERR_INVALID, "dim=%d", dim);
  if (dim > ra::kNormMaxDim)
    return record_error(RA_ERR_UNSUPPORTED, "dim=%d above %d", dim, ra::kNormMaxDim);
  if (!is_float(dtype)) return record_error(RA_ERR_UNSUPPORTED, "dtype %d: f32, bf16 or f16 expected", (int)dtype);
  if (rdtype != RA_F32 && rdtype != dtype)
    return record_error(RA_ERR_UNSUPPORTED, "residual dtype %d: f32 or the block's type expected", (int)rdtype);
  if (pdtype != RA_F32 && pdtype != dtype)
    return record_error(RA_ERR_UNSUPPORTED, "parameter dtype %d: f32 or the block's type expected", (int)pdtype);
  if (!(eps >= 0.0f) || std::isinf(eps)) return record_error(RA_ERR_INVALID, "eps=%g", (double)eps);
  if (!std::isfinite(scale)) return record_error(RA_ERR_INVALID, "scale=%g", (double)scale);
  int dev = -1, sms = 0;
  RA_TRY(device_of(&dev, &sms));
  ra_norm_ctx* h = new (std::nothrow) ra_norm_ctx();
  if (!h) return record_error(RA_ERR_OOM, "host allocation failed");
  h->R = R;
  h->dim = dim;
  h->device = dev;
  h->sms = sms;
  h->dtype = dtype;
  h->residual_dtype = rdtype;
  h->param_dtype = pdtype;
  h->eps = eps;
  h->scale = scale;
  *out = h;
  return RA_OK;
}

static ra_status norm_forward(ra_norm_handle h, const ra_norm_forward_args* g, cudaStream_t st) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (!g) return record_error(RA_ERR_INVALID, "NULL arguments");
  if (g->rows == 0) return RA_OK;
  RA_TRY(check_rows(g->rows));
  RA_TRY(check_gate(g->gate, g->gate_rows, g->rows));
  RA_TRY(check_ranks("outs", g->outs, h->R));
  if (!g->in || !g->out) return record_error(RA_ERR_INVALID, "NULL pointer array");
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  const size_t b = bytes_of(h->dtype), rb = bytes_of(h->residual_dtype), pb = bytes_of(h->param_dtype);
  const size_t dim = (size_t)h->dim;
  size_t in_stride = g->in_stride, out_stride = g->out_stride, res_stride = g->residual_stride,
         res_out_stride = g->residual_out_stride, total_stride = g->total_stride, gate_stride = dim;
  ra::NormForward a{};
  Buffers buf(h->device, h->check_pointers, g->rows);
  for (int r = 0; r < h->R; ++r) {
    RA_TRY(buf.add("in", r, g->in[r], b, dim, &in_stride, false));
    a.in[r] = g->in[r];
  }
  RA_TRY(buf.add("residual", -1, g->residual, rb, dim, &res_stride, false));
  RA_TRY(buf.flat("weight", g->weight, pb, dim, false));
  if (g->post_weight) RA_TRY(buf.flat("post_weight", g->post_weight, pb, dim, false));
  if (g->gate) RA_TRY(buf.add("gate", -1, g->gate, pb, dim, &gate_stride, false, g->gate_rows));
  for (int q = 0; q < g->outs; ++q) {
    RA_TRY(buf.add("out", q, g->out[q], b, dim, &out_stride, true, g->in[q]));
    a.out[q] = g->out[q];
  }
  RA_TRY(buf.add("residual_out", -1, g->residual_out, rb, dim, &res_out_stride, true, g->residual));
  if (g->total) RA_TRY(buf.add("total", -1, g->total, b, dim, &total_stride, true));
  const bool aligned = buf.aligned(dim * b);
  if (g->rstd) RA_TRY(buf.flat("rstd", g->rstd, 4, 2 * g->rows, true));
  RA_TRY(buf.check());
  a.residual = g->residual;
  a.residual_out = g->residual_out;
  a.total = g->total;
  a.weight = g->weight;
  a.post_weight = g->post_weight;
  a.gate = g->gate;
  a.rstd = g->rstd;
  a.rows = (int64_t)g->rows;
  a.in_stride = (int64_t)in_stride;
  a.out_stride = (int64_t)out_stride;
  a.residual_stride = (int64_t)res_stride;
  a.residual_out_stride = (int64_t)res_out_stride;
  a.total_stride = (int64_t)total_stride;
  a.rows_per_gate = g->gate ? (int64_t)(g->rows / g->gate_rows) : (int64_t)g->rows;
  a.R = h->R;
  a.outs = g->outs;
  a.dim = h->dim;
  a.param_f32 = h->param_dtype == RA_F32;
  a.eps = h->eps;
  a.scale = h->scale;
  const cudaError_t e = ra::launch_norm_forward(h->dtype, h->residual_dtype, aligned, a, h->sms, h->opted, st);
  return e == cudaSuccess ? RA_OK : cuda_error(e, "norm forward launch");
}

// The sums over no rows: zeros, in every gate row there is.
static ra_status norm_backward_no_rows(ra_norm_handle h, const ra_norm_backward_args* g, cudaStream_t st) {
  const size_t dim = (size_t)h->dim;
  if (g->grad_gate) RA_TRY(check_rows(g->gate_rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  const struct { const char* name; float* p; size_t count; } sums[3] = {
      {"grad_weight", g->grad_weight, dim},
      {"grad_post_weight", g->grad_post_weight, dim},
      {"grad_gate", g->gate_rows ? g->grad_gate : nullptr, g->gate_rows * dim}};
  Buffers buf(h->device, h->check_pointers, 1);
  for (const auto& s : sums)
    if (s.p) RA_TRY(buf.flat(s.name, s.p, 4, s.count, true));
  RA_TRY(buf.check());
  for (const auto& s : sums) {
    const cudaError_t e = s.p ? cudaMemsetAsync(s.p, 0, s.count * sizeof(float), st) : cudaSuccess;
    if (e != cudaSuccess) return cuda_error(e, s.name);
  }
  return RA_OK;
}

static ra_status norm_backward(ra_norm_handle h, const ra_norm_backward_args* g, cudaStream_t st) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (!g) return record_error(RA_ERR_INVALID, "NULL arguments");
  const size_t dim = (size_t)h->dim;
  if (g->grad_post_weight && !g->post_weight)
    return record_error(RA_ERR_INVALID, "grad_post_weight without post_weight");
  if (g->grad_gate && !g->gate) return record_error(RA_ERR_INVALID, "grad_gate without gate");
  if (g->rows == 0) return norm_backward_no_rows(h, g, st);
  RA_TRY(check_rows(g->rows));
  RA_TRY(check_gate(g->gate, g->gate_rows, g->rows));
  RA_TRY(check_ranks("grads", g->grads, h->R));
  RA_TRY(check_ranks("outs", g->outs, h->R));
  if (!g->grad_out || !g->grad_in) return record_error(RA_ERR_INVALID, "NULL pointer array");
  const bool need_total = g->post_weight || g->grad_gate;
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  const size_t b = bytes_of(h->dtype), rb = bytes_of(h->residual_dtype), pb = bytes_of(h->param_dtype);
  size_t go_stride = g->grad_out_stride, gi_stride = g->grad_in_stride, gro_stride = g->grad_residual_out_stride,
         ro_stride = g->residual_out_stride, total_stride = g->total_stride, gr_stride = g->grad_residual_stride,
         gate_stride = dim, gg_stride = dim;
  ra::NormBackward a{};
  Buffers buf(h->device, h->check_pointers, g->rows);
  for (int r = 0; r < g->grads; ++r) {
    RA_TRY(buf.add("grad_out", r, g->grad_out[r], b, dim, &go_stride, false));
    a.grad_out[r] = g->grad_out[r];
  }
  if (g->grad_residual_out)
    RA_TRY(buf.add("grad_residual_out", -1, g->grad_residual_out, rb, dim, &gro_stride, false));
  RA_TRY(buf.add("residual_out", -1, g->residual_out, rb, dim, &ro_stride, false));
  if (need_total) RA_TRY(buf.add("total", -1, g->total, b, dim, &total_stride, false));
  RA_TRY(buf.flat("weight", g->weight, pb, dim, false));
  if (g->post_weight) RA_TRY(buf.flat("post_weight", g->post_weight, pb, dim, false));
  if (g->gate) RA_TRY(buf.add("gate", -1, g->gate, pb, dim, &gate_stride, false, g->gate_rows));
  for (int q = 0; q < g->outs; ++q) {
    RA_TRY(buf.add("grad_in", q, g->grad_in[q], b, dim, &gi_stride, true,
                   q < g->grads ? g->grad_out[q] : nullptr));
    a.grad_in[q] = g->grad_in[q];
  }
  RA_TRY(buf.add("grad_residual", -1, g->grad_residual, rb, dim, &gr_stride, true, g->grad_residual_out));
  if (g->grad_gate) RA_TRY(buf.add("grad_gate", -1, g->grad_gate, 4, dim, &gg_stride, true, g->gate_rows));
  const bool aligned = buf.aligned(dim * b);
  if (g->grad_weight) RA_TRY(buf.flat("grad_weight", g->grad_weight, 4, dim, true));
  if (g->grad_post_weight) RA_TRY(buf.flat("grad_post_weight", g->grad_post_weight, 4, dim, true));
  RA_TRY(buf.flat("rstd", g->rstd, 4, 2 * g->rows, false));
  const size_t work_bytes = ra::norm_workspace_floats(h->dim, h->sms) * sizeof(float);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  cudaGraph_t graph = nullptr;
  cudaError_t e = cudaStreamGetCaptureInfo(st, &cap, nullptr, &graph, nullptr, nullptr, nullptr);
  if (e != cudaSuccess) return cuda_error(e, "cudaStreamGetCaptureInfo");
  if (!h->work) {
    if (cap != cudaStreamCaptureStatusNone)
      return record_error(RA_ERR_UNSUPPORTED, "the first backward call allocates: make it before the capture");
    free_retired();
    Workspace* w = new (std::nothrow) Workspace();
    if (!w) return record_error(RA_ERR_OOM, "host allocation failed");
    e = cudaMalloc(&w->p, work_bytes);
    if (e != cudaSuccess) {
      delete w;
      return cuda_error(e, "column partials allocation");
    }
    h->work = w;
  }
  RA_TRY(buf.flat("workspace", h->work->p, 4, work_bytes / 4, true));
  RA_TRY(buf.check());
  if (cap == cudaStreamCaptureStatusActive) {
    cudaUserObject_t& shared = h->work->shared;
    e = shared ? cudaSuccess : cudaUserObjectCreate(&shared, h->work, retire, 1, cudaUserObjectNoDestructorSync);
    if (e == cudaSuccess) e = cudaGraphRetainUserObject(graph, shared, 1, 0);
    if (e != cudaSuccess) return cuda_error(e, "the graph's share in the workspace");
  }
  a.grad_residual_out = g->grad_residual_out;
  a.residual_out = g->residual_out;
  a.total = need_total ? g->total : nullptr;
  a.rstd = g->rstd;
  a.weight = g->weight;
  a.post_weight = g->post_weight;
  a.gate = g->gate;
  a.grad_residual = g->grad_residual;
  a.grad_weight = g->grad_weight;
  a.grad_post_weight = g->grad_post_weight;
  a.grad_gate = g->grad_gate;
  a.work = static_cast<float*>(h->work->p);
  a.rows = (int64_t)g->rows;
  a.grad_out_stride = (int64_t)go_stride;
  a.grad_in_stride = (int64_t)gi_stride;
  a.grad_residual_out_stride = (int64_t)gro_stride;
  a.residual_out_stride = (int64_t)ro_stride;
  a.total_stride = (int64_t)total_stride;
  a.grad_residual_stride = (int64_t)gr_stride;
  a.groups = g->gate ? (int64_t)g->gate_rows : 1;
  a.rows_per_gate = (int64_t)g->rows / a.groups;
  a.grads = g->grads;
  a.outs = g->outs;
  a.dim = h->dim;
  a.param_f32 = h->param_dtype == RA_F32;
  a.scale = h->scale;
  e = ra::launch_norm_backward(h->dtype, h->residual_dtype, aligned, a, h->sms, h->opted, st);
  return e == cudaSuccess ? RA_OK : cuda_error(e, "norm backward launch");
}

// --------------------------------------------------------- vocabulary's head

static ra_status vocab_create(int R, size_t V, ra_dtype dtype, float temperature, ra_vocab_handle* out) {
  if (!out) return record_error(RA_ERR_INVALID, "NULL handle pointer");
  if (R < 1 || R > kMaxRanks) return record_error(RA_ERR_INVALID, "R=%d outside [1, %d]", R, kMaxRanks);
  if (V < 1 || V > ((size_t)1 << 30)) return record_error(RA_ERR_INVALID, "V=%zu outside [1, 2^30]", V);
  if (!is_float(dtype)) return record_error(RA_ERR_UNSUPPORTED, "dtype %d: f32, bf16 or f16 expected", (int)dtype);
  // the kernels' factor is log2(e) / temperature, log2(e) below 1.5
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(1.5f / temperature))
    return record_error(RA_ERR_INVALID, "temperature=%g", (double)temperature);
  int dev = -1, sms = 0;
  RA_TRY(device_of(&dev, &sms));
  ra_vocab_ctx* h = new (std::nothrow) ra_vocab_ctx();
  if (!h) return record_error(RA_ERR_OOM, "host allocation failed");
  h->R = R;
  h->V = (int)V;
  h->C = (int)((V + (size_t)R - 1) / (size_t)R);
  h->shards = (h->V + h->C - 1) / h->C;
  h->device = dev;
  h->sms = sms;
  h->dtype = dtype;
  h->tau = temperature;
  *out = h;
  return RA_OK;
}

// The logits' shards of a call (or their gradients', as outputs).
static ra_status add_shards(const ra_vocab_ctx* h, Buffers& buf, const char* name, const void* const* p,
                            const size_t* strides, int64_t* checked, bool output, const void* const* twins) {
  if (!p || !strides) return record_error(RA_ERR_INVALID, "NULL pointer array");
  for (int r = 0; r < h->shards; ++r) {
    const int lo = r * h->C, len = h->V - lo < h->C ? h->V - lo : h->C;
    size_t stride = strides[r];
    RA_TRY(buf.add(name, r, p[r], bytes_of(h->dtype), (size_t)len, &stride, output, twins ? twins[r] : nullptr));
    checked[r] = (int64_t)stride;
  }
  return RA_OK;
}

static void set_rows(const ra_vocab_ctx* h, size_t rows, const void* const* shards, ra::VocabRows* x) {
  for (int r = 0; r < h->shards; ++r) x->shard[r] = shards[r];
  const size_t elem = bytes_of(h->dtype), bytes = (size_t)h->C * elem;
  uintptr_t bits = 0;
  for (int r = 0; r < h->shards; ++r) bits |= (uintptr_t)shards[r] | (rows > 1 ? (uintptr_t)x->stride[r] * elem : 0);
  // rows may start up to `lag` bytes into a 128-byte line
  const size_t lag = bits % 128 == 0 ? 0 : bits % 64 == 0 ? 64 : bits % 32 == 0 ? 96 : bits % 16 == 0 ? 112 : 126;
  x->slots = (int)((bytes + lag + 15) / 16);
  x->rows = (int64_t)rows;
  x->shards = h->shards;
  x->V = h->V;
  x->C = h->C;
  x->tau = h->tau;
  x->inv_tau = 1.0f / h->tau;
  x->scale = ra::kLog2e * x->inv_tau;
  const double unit = 1.0 / ((double)h->tau * (double)x->scale);
  x->unit = (float)unit;
  x->unit_rest = (float)(unit - (double)x->unit);
}

// The powers of two that what a probability is multiplied with may reach:
// `factor`, and a log p of up to 2^7.  (2^lift has to be in binary32's range.)
static void set_lift(float factor, ra::VocabBackward* a) {
  const float most = 120.0f, lift = 7.0f + (factor > 1.0f ? std::ceil(std::log2(factor)) : 0.0f);
  a->lift = lift < most ? lift : most;
  a->by_lift = std::ldexp(1.0f, -(int)a->lift);
}

static ra_status vocab_logprobs(ra_vocab_handle h, const ra_vocab_logprobs_args* g, cudaStream_t st) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (!g) return record_error(RA_ERR_INVALID, "NULL arguments");
  if (g->top < 0 || g->top > ra::kTopMax || g->top > h->V)
    return record_error(RA_ERR_INVALID, "top=%d outside [0, min(%d, V=%d)]", g->top, ra::kTopMax, h->V);
  if (g->rows == 0) return RA_OK;
  RA_TRY(check_rows(g->rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  ra::VocabForward a{};
  Buffers buf(h->device, h->check_pointers, g->rows);
  RA_TRY(add_shards(h, buf, "shards", g->shards, g->strides, a.x.stride, false, nullptr));
  RA_TRY(buf.flat("targets", g->targets, 8, g->rows, false));
  RA_TRY(buf.flat("logprob", g->logprob, 4, g->rows, true));
  RA_TRY(buf.flat("lse", g->lse, 4, g->rows, true));
  if (g->entropy) RA_TRY(buf.flat("entropy", g->entropy, 4, g->rows, true));
  if (g->top) {
    RA_TRY(buf.flat("top_ids", g->top_ids, 8, g->rows * (size_t)g->top, true));
    RA_TRY(buf.flat("top_logprobs", g->top_logprobs, 4, g->rows * (size_t)g->top, true));
  }
  RA_TRY(buf.check());
  set_rows(h, g->rows, g->shards, &a.x);
  a.targets = g->targets;
  a.logprob = g->logprob;
  a.lse = g->lse;
  a.entropy = g->entropy;
  a.top = g->top;
  a.top_ids = g->top_ids;
  a.top_logprobs = g->top_logprobs;
  const cudaError_t e = ra::launch_vocab_forward(h->dtype, a, h->sms, st);
  return e == cudaSuccess ? RA_OK : cuda_error(e, "log probabilities launch");
}

static ra_status vocab_logprobs_backward(ra_vocab_handle h, const ra_vocab_logprobs_backward_args* g,
                                         cudaStream_t st) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (!g) return record_error(RA_ERR_INVALID, "NULL arguments");
  if (g->rows == 0) return RA_OK;
  RA_TRY(check_rows(g->rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  ra::VocabBackward a{};
  Buffers buf(h->device, h->check_pointers, g->rows);
  RA_TRY(add_shards(h, buf, "shards", g->shards, g->strides, a.x.stride, false, nullptr));
  RA_TRY(buf.flat("targets", g->targets, 8, g->rows, false));
  RA_TRY(buf.flat("lse", g->lse, 4, g->rows, false));
  RA_TRY(buf.flat("grad_logprob", g->grad_logprob, 4, g->rows, false));
  if (g->grad_entropy) {
    RA_TRY(buf.flat("grad_entropy", g->grad_entropy, 4, g->rows, false));
    RA_TRY(buf.flat("entropy", g->entropy, 4, g->rows, false));
  }
  RA_TRY(add_shards(h, buf, "grads", (const void* const*)g->grads, g->grad_strides, a.grad_stride, true, g->shards));
  RA_TRY(buf.check());
  set_rows(h, g->rows, g->shards, &a.x);
  for (int r = 0; r < h->shards; ++r) a.grad[r] = g->grads[r];
  a.lse = g->lse;
  a.targets = g->targets;
  a.entropy = g->entropy;
  a.grad_entropy = g->grad_entropy;
  a.g = g->grad_logprob;
  set_lift(a.x.inv_tau, &a);
  const cudaError_t e = ra::launch_vocab_backward(h->dtype, a, h->sms, st);
  return e == cudaSuccess ? RA_OK : cuda_error(e, "log probabilities' gradient launch");
}

static ra_status add_teacher(const ra_vocab_ctx* h, Buffers& buf, size_t rows, int K, const int64_t* ids,
                             const void* logits, ra_dtype dtype) {
  if (K < 1 || K > ra::kTeacherMax)
    return record_error(RA_ERR_INVALID, "teacher_k=%d outside [1, %d]", K, ra::kTeacherMax);
  if (dtype != RA_F32 && dtype != h->dtype)
    return record_error(RA_ERR_UNSUPPORTED, "teacher dtype %d: f32 or the logits' type expected", (int)dtype);
  RA_TRY(buf.flat("teacher_ids", ids, 8, rows * (size_t)K, false));
  return buf.flat("teacher_logits", logits, bytes_of(dtype), rows * (size_t)K, false);
}

static ra_status vocab_distill(ra_vocab_handle h, const ra_vocab_distill_args* g, cudaStream_t st) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (!g) return record_error(RA_ERR_INVALID, "NULL arguments");
  if (g->rows == 0) return RA_OK;
  RA_TRY(check_rows(g->rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  ra::VocabForward a{};
  Buffers buf(h->device, h->check_pointers, g->rows);
  RA_TRY(add_shards(h, buf, "shards", g->shards, g->strides, a.x.stride, false, nullptr));
  RA_TRY(add_teacher(h, buf, g->rows, g->teacher_k, g->teacher_ids, g->teacher_logits, g->teacher_dtype));
  RA_TRY(buf.flat("loss", g->loss, 4, g->rows, true));
  RA_TRY(buf.flat("lse", g->lse, 4, g->rows, true));
  RA_TRY(buf.check());
  set_rows(h, g->rows, g->shards, &a.x);
  a.lse = g->lse;
  a.ids = g->teacher_ids;
  a.teacher = g->teacher_logits;
  a.loss = g->loss;
  a.K = g->teacher_k;
  a.teacher_f32 = g->teacher_dtype == RA_F32;
  const cudaError_t e = ra::launch_vocab_forward(h->dtype, a, h->sms, st);
  return e == cudaSuccess ? RA_OK : cuda_error(e, "distillation launch");
}

static ra_status vocab_distill_backward(ra_vocab_handle h, const ra_vocab_distill_backward_args* g, cudaStream_t st) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (!g) return record_error(RA_ERR_INVALID, "NULL arguments");
  if (g->rows == 0) return RA_OK;
  RA_TRY(check_rows(g->rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  ra::VocabBackward a{};
  Buffers buf(h->device, h->check_pointers, g->rows);
  RA_TRY(add_shards(h, buf, "shards", g->shards, g->strides, a.x.stride, false, nullptr));
  RA_TRY(add_teacher(h, buf, g->rows, g->teacher_k, g->teacher_ids, g->teacher_logits, g->teacher_dtype));
  RA_TRY(buf.flat("lse", g->lse, 4, g->rows, false));
  RA_TRY(buf.flat("grad_loss", g->grad_loss, 4, g->rows, false));
  RA_TRY(add_shards(h, buf, "grads", (const void* const*)g->grads, g->grad_strides, a.grad_stride, true, g->shards));
  RA_TRY(buf.check());
  set_rows(h, g->rows, g->shards, &a.x);
  for (int r = 0; r < h->shards; ++r) a.grad[r] = g->grads[r];
  a.lse = g->lse;
  a.g = g->grad_loss;
  set_lift(h->tau, &a);
  a.ids = g->teacher_ids;
  a.teacher = g->teacher_logits;
  a.K = g->teacher_k;
  a.teacher_f32 = g->teacher_dtype == RA_F32;
  const cudaError_t e = ra::launch_vocab_backward(h->dtype, a, h->sms, st);
  return e == cudaSuccess ? RA_OK : cuda_error(e, "distillation's gradient launch");
}

template <class H> static ra_status set_option(H h, int key, long long value) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (key != RA_OPT_CHECK_POINTERS) return record_error(RA_ERR_INVALID, "option %d: only RA_OPT_CHECK_POINTERS", key);
  if (value != 0 && value != 1) return record_error(RA_ERR_INVALID, "value %lld: 0 or 1", value);
  h->check_pointers = value != 0;
  return RA_OK;
}

extern "C" {

ra_status ra_norm_create(int R, int dim, ra_dtype dtype, ra_dtype residual_dtype, ra_dtype param_dtype, float eps,
                         float scale, ra_norm_handle* out) {
  return guarded([&] { return norm_create(R, dim, dtype, residual_dtype, param_dtype, eps, scale, out); });
}

ra_status ra_norm_destroy(ra_norm_handle h) {
  return guarded([&]() -> ra_status {
    if (!h) return RA_OK;
    ra_status s = RA_OK;
    {
      OnDevice on(h->device);
      const cudaError_t e = h->work ? cudaDeviceSynchronize() : cudaSuccess;
      if (h->work && h->work->shared) {
        cudaUserObjectRelease(h->work->shared, 1);   // graphs may have it still
      } else if (h->work) {
        cudaFree(h->work->p);
        delete h->work;
        free_retired();
      }
      if (e != cudaSuccess) s = cuda_error(e, "synchronise before destroy");
    }
    delete h;
    return s;
  });
}

ra_status ra_norm_set_option(ra_norm_handle h, int key, long long value) {
  return guarded([&] { return set_option(h, key, value); });
}

ra_status ra_vocab_set_option(ra_vocab_handle h, int key, long long value) {
  return guarded([&] { return set_option(h, key, value); });
}

ra_status ra_norm_forward(ra_norm_handle h, const ra_norm_forward_args* args, void* stream) {
  return guarded([&] { return norm_forward(h, args, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_norm_backward(ra_norm_handle h, const ra_norm_backward_args* args, void* stream) {
  return guarded([&] { return norm_backward(h, args, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_vocab_create(int R, size_t V, ra_dtype dtype, float temperature, ra_vocab_handle* out) {
  return guarded([&] { return vocab_create(R, V, dtype, temperature, out); });
}

ra_status ra_vocab_destroy(ra_vocab_handle h) {
  delete h;
  return RA_OK;
}

ra_status ra_vocab_logprobs(ra_vocab_handle h, const ra_vocab_logprobs_args* args, void* stream) {
  return guarded([&] { return vocab_logprobs(h, args, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_vocab_logprobs_backward(ra_vocab_handle h, const ra_vocab_logprobs_backward_args* args, void* stream) {
  return guarded([&] { return vocab_logprobs_backward(h, args, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_vocab_distill(ra_vocab_handle h, const ra_vocab_distill_args* args, void* stream) {
  return guarded([&] { return vocab_distill(h, args, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_vocab_distill_backward(ra_vocab_handle h, const ra_vocab_distill_backward_args* args, void* stream) {
  return guarded([&] { return vocab_distill_backward(h, args, static_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
