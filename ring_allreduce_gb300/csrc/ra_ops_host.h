// ra_ops_host.h -- what the host sides of the model operators share: errors,
// the device of a call, and the checks of its buffers.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>

#include "ra.h"
#include "ra_internal.h"

namespace ra {
ra_status record_error(ra_status s, const char* fmt, ...);   // ra_host.cpp

namespace {

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

// The buffers of one call, `Most` of them at most, and what has to hold of them.
template <int Most> class BuffersOf {
 public:
  BuffersOf(int device, bool check_pointers, size_t rows)
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
    if (count_ == Most) return record_error(RA_ERR_INVALID, "too many buffers");
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

  // Memory of the library's own that the call's kernels write (bounds checks of debug builds).
  void also(const void* p, size_t bytes) {
    own_ = (uintptr_t)p;
    own_bytes_ = bytes;
  }

  ra_status check() {
    const bool apart = spans_apart();
    for (int i = 0; i < count_; ++i) {
      if (b_[i].output && !apart)
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

  // No output's span of memory meets another buffer's: then no pair has to be
  // looked at (with 32 ranks a call has some 450 buffers).
  bool spans_apart() const {
    int order[Most];
    for (int i = 0; i < count_; ++i) order[i] = i;
    std::sort(order, order + count_, [&](int i, int k) { return b_[i].lo < b_[k].lo; });
    uintptr_t any = 0, written = 0;   // ends of what came before: of all buffers, of the outputs
    for (int n = 0; n < count_; ++n) {
      const Buffer& b = b_[order[n]];
      if (b.lo < (b.output ? any : written)) return false;
      any = std::max(any, b.lo + b.span);
      if (b.output) written = std::max(written, b.lo + b.span);
    }
    return true;
  }

  void register_debug() {
#ifdef RA_DEBUG_BOUNDS
    ra::DebugTable& t = ra::debug_table();
    t.count = 0;
    t.report = ra::debug_report();
    if (own_bytes_) t.r[t.count++] = {own_, own_ + own_bytes_};
    const int room = ra::kDebugRanges - t.count;
    for (int i = 0; i < count_; ++i) {
      ra::DebugRange& d = t.r[t.count < ra::kDebugRanges ? t.count++ : ra::kDebugRanges - 1];
      const bool more = i >= room;   // what the table has no room for shares its last range
      d.lo = more ? std::min<uint64_t>(d.lo, b_[i].lo) : b_[i].lo;
      d.hi = more ? std::max<uint64_t>(d.hi, b_[i].lo + b_[i].span) : b_[i].lo + b_[i].span;
    }
#endif
  }

  Buffer b_[Most];
  int count_ = 0;
  int device_;
  size_t rows_;
  bool check_pointers_;
  uintptr_t own_ = 0;
  size_t own_bytes_ = 0;
  char text_[32];
};

using Buffers = BuffersOf<2 * kMaxRanks + 16>;

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

ra_status check_ranks(const char* name, int count, int R) {
  if (count != 1 && count != R) return record_error(RA_ERR_INVALID, "%s=%d: 1 or R=%d expected", name, count, R);
  return RA_OK;
}

// Operators without other options: set_option for RA_OPT_CHECK_POINTERS alone.
template <class H> ra_status set_option(H h, int key, long long value) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (key != RA_OPT_CHECK_POINTERS) return record_error(RA_ERR_INVALID, "option %d: only RA_OPT_CHECK_POINTERS", key);
  if (value != 0 && value != 1) return record_error(RA_ERR_INVALID, "value %lld: 0 or 1", value);
  h->check_pointers = value != 0;
  return RA_OK;
}

}  // namespace
}  // namespace ra
