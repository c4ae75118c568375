// ra_vocab.cu -- the vocabulary-parallel head: a row of V logits held as R
// column shards (shard r: columns [r C, min((r+1) C, V)), C = ceil(V / R)).
//
//   x = L / tau;  lse = log sum_j e^{x_j};  log p_j = x_j - lse
//   log probabilities  log p_target, entropy H = -sum_j p_j log p_j, and the
//                      top K logits (ties to the lower column)
//     gradient         dL_j = (1/tau) (g ([j = target] - p_j) - gH p_j (log p_j + H))
//   distillation       q = softmax(t / tau) over the teacher's K tokens,
//                      loss = tau^2 sum_k q_k (log q_k - log p_{id_k})
//     gradient         dL_j = g tau (p_j - sum_{k: id_k = j} q_k)
//
// The forward pass reads the row once: every thread keeps its own running
// maximum m, sum s = sum e^{x-m} and u = sum (x-m) e^{x-m}, which are joined
// over the block; H = log s - u / s is then a sum of two terms that are never
// negative, with no cancellation.  All statistics are binary32.
//
// The top K come out of the same pass without a comparison per element
// against a list: each thread also keeps the largest logit it saw and where.
// The K-th largest of those maxima bounds the row's K-th largest logit from
// below, and only the K threads whose maximum reaches it can hold one of the
// top K: their columns, K / threads of the row, are read again.
//
// A row's 16-byte slots are numbered through all shards; a slot that a
// shard's first or last columns share with other memory is read element by
// element, so rows may start on any element.
#include "ra_ops.cuh"

namespace ra {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFarBelow = -200.0f;   // exponents are held above this: 2^-200 is 0 in binary32,
                                       // and 0 times the exponent then stays 0 (not 0 * inf)

constexpr float kNothingLeft = -1e30f;

template <class D> struct NegInf;
template <> struct NegInf<DF32> { static constexpr uint32_t bits = 0xFF800000u; };
template <> struct NegInf<DBF16> { static constexpr uint32_t bits = 0xFF80u; };
template <> struct NegInf<DF16> { static constexpr uint32_t bits = 0xFC00u; };

// A logit as a whole number of the same order: -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);   // 0xFFFFFFFF: a NaN
}
__device__ __forceinline__ uint64_t top_key(float x, uint32_t column) {
  return ((uint64_t)ordered(x) << 32) | (uint32_t)~column;
}

// One row's shards, in shared memory: first byte, columns and the element
// offset of the first byte within its 16-byte slot.
struct RowShards {
  uintptr_t first[kMaxRanks];
  int len[kMaxRanks];
};

template <class D>
__device__ __forceinline__ void load_row(const VocabRows& x, int64_t row, RowShards& s) {
  for (int r = threadIdx.x; r < x.shards; r += blockDim.x) {
    s.first[r] = reinterpret_cast<uintptr_t>(x.shard[r]) + (uintptr_t)(row * x.stride[r]) * sizeof(typename D::T);
    s.len[r] = min(x.C, x.V - r * x.C);
  }
}

// Slots per shard: the most that C columns can touch.
template <class D> __host__ __device__ __forceinline__ int slots_per_shard(int C) {
  return (int)(((int64_t)C * (int64_t)sizeof(typename D::T) + 15) / 16) + 1;
}

// Where slot g of a row lies: shard r, slot j of it; [lo, hi) are the slot's
// elements that belong to the shard, e0 the shard's column of its element 0.
template <class D> struct Slot {
  const uint4* at;
  int r, lo, hi, e0;
  __device__ __forceinline__ Slot(const RowShards& s, int rr, int j) : r(rr) {
    const uintptr_t a = s.first[rr];
    at = reinterpret_cast<const uint4*>(a & ~uintptr_t(15)) + j;
    e0 = j * D::kVec - (int)((a & 15u) / sizeof(typename D::T));
    lo = max(0, -e0);
    hi = min(D::kVec, s.len[rr] - e0);
  }
  __device__ __forceinline__ bool empty() const { return hi <= lo; }
  __device__ __forceinline__ bool whole() const { return lo == 0 && hi == D::kVec; }
  // the slot's logits; -inf where it has none
  __device__ __forceinline__ uint4 load() const {
    if (whole()) return ld_stream(at);
    uint32_t w[4];
    const typename D::T* p = reinterpret_cast<const typename D::T*>(at);
    constexpr uint32_t none = NegInf<D>::bits;
    if constexpr (sizeof(typename D::T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = i >= lo && i < hi ? __float_as_uint(ld_stream_scalar(p + i)) : none;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = 2 * i >= lo && 2 * i < hi ? ld_stream_scalar(p + 2 * i) : none;
        const uint32_t b = 2 * i + 1 >= lo && 2 * i + 1 < hi ? ld_stream_scalar(p + 2 * i + 1) : none;
        w[i] = a | b << 16;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The logit of column c (0 <= c < V).
template <class D>
__device__ __forceinline__ float logit_at(const VocabRows& x, int64_t row, int c) {
  const int r = c / x.C;
  const typename D::T* p = static_cast<const typename D::T*>(x.shard[r]) + row * x.stride[r] + (c - r * x.C);
  return widen<D>(ld_stream_scalar(p));
}

__device__ __forceinline__ float exponent(float x, float m, float scale) {
  return fmaxf((x - m) * scale, kFarBelow);
}

// Running statistics of a row relative to m (the largest logit so far, or the
// lowest finite number): s = sum 2^t, u = sum t 2^t, t = (x - m) log2(e) / tau.
struct Stats {
  float m, s, u;
  __device__ __forceinline__ void shift(float to, float scale) {
    const float t = exponent(m, to, scale);
    const float f = exp2_fast(t);
    u = __fmaf_rn(t, s, u) * f;
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Stats o, float scale) {
    const float to = max_nan(m, o.m);
    shift(to, scale);
    o.shift(to, scale);
    s += o.s;
    u += o.u;
  }
};

__device__ __forceinline__ Stats warp_stats(Stats v, float scale) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    Stats o;
    o.m = __shfl_xor_sync(0xFFFFFFFFu, v.m, d);
    o.s = __shfl_xor_sync(0xFFFFFFFFu, v.s, d);
    o.u = __shfl_xor_sync(0xFFFFFFFFu, v.u, d);
    v.join(o, scale);
  }
  return v;
}

// ---------------------------------------------- lists of a warp's 32 largest
// A warp holds 32 keys, falling from lane 0; 0 is no key.

// A bitonic sequence of 32 keys into falling order.
__device__ __forceinline__ uint64_t warp_fall(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, k, d);
    const bool up = lane & d;
    k = up ? (k < o ? k : o) : (k > o ? k : o);
  }
  return k;
}

// Any 32 keys into falling order.
__device__ __forceinline__ uint64_t warp_sort(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, k, d);
      const bool falling = (lane & size) == 0 || size == 32;
      const bool low = (lane & d) == 0;
      k = (falling == low) ? (k > o ? k : o) : (k < o ? k : o);
    }
  }
  return k;
}

// The 32 largest of two falling lists.
__device__ __forceinline__ uint64_t warp_merge(uint64_t a, uint64_t b) {
  const uint64_t back = __shfl_sync(0xFFFFFFFFu, b, 31 - (threadIdx.x & 31));
  return warp_fall(a > back ? a : back);
}

// The block's 32 largest of every warp's list, in warp 0.
__device__ __forceinline__ uint64_t block_merge(uint64_t k, uint64_t (*lists)[32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
  lists[w][lane] = k;
  __syncthreads();
  for (int step = 1; step < warps; step <<= 1) {
    if ((w & (2 * step - 1)) == 0 && w + step < warps) {
      k = warp_merge(k, lists[w + step][lane]);
      lists[w][lane] = k;
    }
    __syncthreads();
  }
  return k;
}

__device__ __forceinline__ uint64_t warp_insert(uint64_t mine, uint64_t key) {
  const int lane = threadIdx.x & 31;
  const int pos = __popc(__ballot_sync(0xFFFFFFFFu, mine > key));
  const uint64_t above = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
  return lane < pos ? mine : lane == pos ? key : above;
}

// ------------------------------------------------------------------ teacher

// The teacher's distribution over its tokens, in every thread of the block
// that runs this: q[k], log q[k] (0 where the token is absent), and whether
// the row has any.  ids[k] is -1 where the token is absent: a negative id or
// one that is no column, or a teacher logit of -inf.
struct Teacher {
  int id[kTeacherMax];
  float q[kTeacherMax];
  float logq[kTeacherMax];
};

template <class D>
__device__ __forceinline__ bool load_teacher(Teacher& t, const int64_t* ids, const void* teacher, int K, bool f32,
                                             int64_t row, int V, float inv_tau, float* red) {
  // one warp: K is at most 256, eight a lane
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    float m = -INFINITY;
    for (int k = lane; k < K; k += 32) {
      const int64_t id = ld_g(ids + row * K + k);
      float x = f32 ? ld_g(static_cast<const float*>(teacher) + row * K + k)
                    : widen<D>(ld_g(static_cast<const typename D::T*>(teacher) + row * K + k));
      const bool absent = id < 0 || id >= V || x == -INFINITY;
      t.id[k] = absent ? -1 : (int)id;
      t.logq[k] = x;
      if (!absent) m = max_nan(m, x);
    }
    m = warp_max_nan(m);
    float s = 0.0f;
    for (int k = lane; k < K; k += 32) {
      const float d = (t.logq[k] - m) * inv_tau;
      const float e = t.id[k] < 0 ? 0.0f : expf(d);
      t.q[k] = e;
      t.logq[k] = d;
      s += e;
    }
    s = warp_sum(s);
    const float log_s = logf(s);
    for (int k = lane; k < K; k += 32) {
      const bool some = t.id[k] >= 0;
      t.q[k] = some ? t.q[k] / s : 0.0f;
      t.logq[k] = some ? t.logq[k] - log_s : 0.0f;
    }
    if (lane == 0) red[0] = m;
  }
  __syncthreads();
  return red[0] != -INFINITY;   // NaN: the row has a teacher, and its values are NaN
}

// ------------------------------------------------------------------ forward

constexpr int kUnroll = 4;   // slots in flight per thread

struct ForwardShared {
  RowShards rows;
  Stats warp[32];
  uint64_t lists[32][32];
  float red[2];
};

template <class D, bool DISTILL>
__global__ void __launch_bounds__(512) vocab_forward_kernel(const __grid_constant__ VocabForward a) {
  constexpr int V = D::kVec;
  __shared__ ForwardShared sh;
  const int64_t row = blockIdx.x;
  const int n = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float scale = kLog2e * a.x.inv_tau;
  const int per = slots_per_shard<D>(a.x.C), slots = per * a.x.shards;
  load_row<D>(a.x, row, sh.rows);
  __syncthreads();

  Stats st{-FLT_MAX, 0.0f, 0.0f};
  float best = -INFINITY;   // the thread's largest logit and its slot (-1: it saw none)
  int best_at = -1;
  int r = tid / per, j = tid - r * per;
  for (int g = tid; g < slots; g += n * kUnroll) {
    uint4 raw[kUnroll];
    bool some[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      constexpr uint32_t none = sizeof(typename D::T) == 4 ? NegInf<D>::bits : NegInf<D>::bits * 0x10001u;
      raw[i] = make_uint4(none, none, none, none);
      some[i] = false;
      if (g + i * n < slots) {
        const Slot<D> s(sh.rows, r, j);
        some[i] = !s.empty();
        if (some[i]) raw[i] = s.load();
      }
      j += n;
      while (j >= per) {
        j -= per;
        ++r;
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (!some[i]) continue;
      float x[V];
      unpack<D>(raw[i], x);
      float vm = x[0];
#pragma unroll
      for (int e = 1; e < V; ++e) vm = max_nan(vm, x[e]);
      // of equals the first slot keeps the place; the first NaN takes it for good
      if (vm > best || best_at < 0 || (vm != vm && best == best)) {
        best = vm;
        best_at = g + i * n;
      }
      if (!(vm <= st.m)) st.shift(max_nan(st.m, vm), scale);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float t = exponent(x[e], st.m, scale);
        const float p = exp2_fast(t);
        st.s += p;
        if (!DISTILL) st.u = __fmaf_rn(t, p, st.u);
      }
    }
  }

  // the block's statistics, the same in every thread
  st = warp_stats(st, scale);
  if (lane == 0) sh.warp[warp] = st;
  __syncthreads();
  st = lane < (n >> 5) ? sh.warp[lane] : Stats{-FLT_MAX, 0.0f, 0.0f};
  st = warp_stats(st, scale);
  const bool empty = st.s == 0.0f && st.m == -FLT_MAX;   // nothing but -inf
  const bool broken = !(st.m < INFINITY);                // +inf or NaN: the row's values are NaN
  const float log_s = broken ? NAN : logf(st.s);         // empty: -inf
  const float lse = broken ? NAN : empty ? -INFINITY : __fmaf_rn(st.m, a.x.inv_tau, log_s);
  auto log_prob = [&](float x) { return empty ? -INFINITY : (x - st.m) * a.x.inv_tau - log_s; };
  if (tid == 0) st_g(a.lse + row, lse);

  if constexpr (DISTILL) {
    Teacher& t = *reinterpret_cast<Teacher*>(&sh.lists);
    const bool taught = load_teacher<D>(t, a.ids, a.teacher, a.K, a.teacher_f32, row, a.x.V, a.x.inv_tau, sh.red);
    if (warp == 0) {
      float loss = 0.0f;
      for (int k = lane; k < a.K; k += 32) {
        if (t.q[k] != 0.0f) {   // NaN included
          const float lp = log_prob(logit_at<D>(a.x, row, t.id[k]));
          loss += t.q[k] * (t.logq[k] - lp);
        }
      }
      loss = warp_sum(loss);
      if (lane == 0) st_g(a.loss + row, taught ? loss * a.x.tau * a.x.tau : 0.0f);
    }
  } else {
    if (tid == 0) {
      const int64_t target = ld_g(a.targets + row);
      // no target: 0; a target that is no column: NaN
      st_g(a.logprob + row, target < 0 ? 0.0f : target >= a.x.V ? NAN : log_prob(logit_at<D>(a.x, row, (int)target)));
      if (a.entropy) st_g(a.entropy + row, empty ? 0.0f : log_s - kLn2 * (st.u / st.s));
    }
    if (a.top > 0) {
      // the K-th largest of the threads' maxima, by (logit, slot)
      uint64_t k = best_at < 0 ? 0 : top_key(best, (uint32_t)best_at);
      k = block_merge(warp_sort(k), sh.lists);
      if (warp == 0) sh.lists[0][lane] = k;
      __syncthreads();
      const uint64_t mine = sh.lists[0][lane];
      const uint64_t bound = __shfl_sync(0xFFFFFFFFu, mine, a.top - 1);
      __syncthreads();
      // the threads that reach it: each warp reads its share of their slots again
      uint64_t list = 0;
      for (int q = warp; q < a.top; q += n >> 5) {
        const uint64_t key = __shfl_sync(0xFFFFFFFFu, mine, q);
        if (key == 0) continue;   // fewer threads than K saw a logit
        const int owner = (int)(~(uint32_t)key) % n;
        for (int g0 = owner; g0 < slots; g0 += 32 * n) {
          const int64_t g = g0 + (int64_t)lane * n;
          bool have = g < slots;
          uint4 raw = make_uint4(0, 0, 0, 0);
          int lo = 0, hi = 0, column = 0;
          if (have) {
            const int rr = (int)g / per;
            const Slot<D> s(sh.rows, rr, (int)g - rr * per);
            lo = s.lo;
            hi = s.hi;
            column = rr * a.x.C + s.e0;
            if (!s.empty()) raw = s.load();
          }
          float x[V];
          unpack<D>(raw, x);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const bool may = e >= lo && e < hi && top_key(x[e], (uint32_t)g) >= bound;
            uint32_t hits = __ballot_sync(0xFFFFFFFFu, may);
            const uint64_t full = top_key(x[e], (uint32_t)(column + e));
            while (hits) {
              const int from = __ffs(hits) - 1;
              hits &= hits - 1;
              list = warp_insert(list, __shfl_sync(0xFFFFFFFFu, full, from));
            }
          }
        }
      }
      list = block_merge(list, sh.lists);
      if (warp == 0 && lane < a.top) {
        st_g(a.top_ids + row * a.top + lane, (int64_t)(uint32_t)~(uint32_t)list);
        st_g(a.top_logprobs + row * a.top + lane, log_prob(from_ordered((uint32_t)(list >> 32))));
      }
    }
  }
}

// ----------------------------------------------------------------- backward

struct BackwardShared {
  RowShards rows;
  uintptr_t grad[kMaxRanks];
  Teacher teacher;
  float fix[kTeacherMax];
  float red[2];
};

template <class D, bool DISTILL>
__global__ void __launch_bounds__(512) vocab_backward_kernel(const __grid_constant__ VocabBackward a, int parts) {
  constexpr int V = D::kVec;
  using T = typename D::T;
  __shared__ BackwardShared sh;
  const int64_t row = blockIdx.x / parts;
  const int part = (int)(blockIdx.x - row * parts);
  const int n = blockDim.x, tid = threadIdx.x;
  const int per = slots_per_shard<D>(a.x.C), slots = per * a.x.shards;
  const int share = (slots + parts - 1) / parts;
  const int begin = part * share, end = min(slots, begin + share);
  const float inv_tau = a.x.inv_tau;
  load_row<D>(a.x, row, sh.rows);
  for (int r = tid; r < a.x.shards; r += n)
    sh.grad[r] = reinterpret_cast<uintptr_t>(a.grad[r]) + (uintptr_t)(row * a.grad_stride[r]) * sizeof(T);
  __syncthreads();

  // dL_j = p_j (A + B log p_j), plus what the target or the teacher adds
  float A, B = 0.0f, add = 0.0f;
  const float row_lse = ld_g(a.lse + row);
  // nothing left by the mask: -inf everywhere, or logits so low (the type's
  // lowest value) that lse cannot hold the logarithm of their sum beside them
  const bool empty = row_lse < kNothingLeft;
  bool zero = empty;
  const float lse = empty ? 0.0f : row_lse;
  int fixes = 0;
  if constexpr (DISTILL) {
    const bool taught =
        load_teacher<D>(sh.teacher, a.ids, a.teacher, a.K, a.teacher_f32, row, a.x.V, inv_tau, sh.red);
    zero = zero || !taught;
    A = zero ? 0.0f : ld_g(a.g + row) * a.x.tau;
    fixes = zero ? 0 : a.K;
  } else {
    const int64_t target = ld_g(a.targets + row);
    const float g = target < 0 ? 0.0f : target >= a.x.V ? NAN : ld_g(a.g + row);
    const float gh = a.grad_entropy ? ld_g(a.grad_entropy + row) : 0.0f;
    const float H = a.grad_entropy ? ld_g(a.entropy + row) : 0.0f;
    A = -(g + gh * H) * inv_tau;
    B = -gh * inv_tau;
    add = g * inv_tau;
    fixes = !zero && target >= 0 && target < a.x.V ? 1 : 0;
    if (tid == 0) sh.teacher.id[0] = (int)target;
    __syncthreads();
  }
  if (zero) A = B = 0.0f;
  auto gradient = [&](float x) {
    const float lp = __fmaf_rn(x, inv_tau, -lse);
    const float p = sizeof(T) == 4 ? expf(lp) : exp2_fast(lp * kLog2e);
    if (DISTILL || B == 0.0f) return A * p;
    return p * __fmaf_rn(B, fmaxf(lp, kFarBelow), A);
  };
  // the columns with more than that, read before any of them is written (the
  // gradient may stand in the logits' place); of equal tokens the first one
  // holds the sum
  for (int k = tid; k < fixes; k += n) {
    const int c = sh.teacher.id[k];
    float v = 0.0f;
    bool mine = false;
    if (c >= 0) {
      const int r = c / a.x.C;
      const int slot = r * per + (int)((sh.rows.first[r] & 15u) / sizeof(T) + (c - r * a.x.C)) / V;
      mine = slot >= begin && slot < end;
    }
    if (mine) {
      if (DISTILL) {
        for (int i = 0; i < a.K; ++i) {
          if (sh.teacher.id[i] == c) {
            add -= A * sh.teacher.q[i];
            if (i < k) mine = false;
          }
        }
      }
      if (mine) v = gradient(logit_at<D>(a.x, row, c)) + add;
      if (DISTILL) add = 0.0f;
    }
    sh.fix[k] = v;
    sh.teacher.logq[k] = mine ? 1.0f : 0.0f;   // no further use of logq here
  }
  __syncthreads();

  int g = begin + tid, r = g / per, j = g - r * per;
  for (; g < end; g += n * kUnroll) {
    uint4 raw[kUnroll];
    Slot<D> s[kUnroll] = {Slot<D>(sh.rows, 0, 0), Slot<D>(sh.rows, 0, 0), Slot<D>(sh.rows, 0, 0),
                          Slot<D>(sh.rows, 0, 0)};
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      s[i].hi = s[i].lo;
      if (g + i * n < end) {
        s[i] = Slot<D>(sh.rows, r, j);
        if (!s[i].empty()) raw[i] = s[i].load();
      }
      j += n;
      while (j >= per) {
        j -= per;
        ++r;
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (s[i].empty()) continue;
      float x[V];
      unpack<D>(raw[i], x);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = zero ? 0.0f : gradient(x[e]);
      T* to = reinterpret_cast<T*>(sh.grad[s[i].r]) + s[i].e0;
      if (s[i].whole() && (reinterpret_cast<uintptr_t>(to) & 15u) == 0) {
        st_stream(reinterpret_cast<uint4*>(to), pack<D>(x));
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e >= s[i].lo && e < s[i].hi) st_g(to + e, narrow<D>(x[e]));
      }
    }
  }
  if (fixes == 0) return;
  __syncthreads();
  for (int k = tid; k < fixes; k += n) {
    if (sh.teacher.logq[k] == 0.0f) continue;
    const int c = sh.teacher.id[k], q = c / a.x.C;
    st_g(reinterpret_cast<T*>(sh.grad[q]) + (c - q * a.x.C), narrow<D>(sh.fix[k]));
  }
}

template <class F> cudaError_t with_float(int dtype, F&& f) {
  switch (dtype) {
    case RA_F32: return f(DF32{});
    case RA_BF16: return f(DBF16{});
    case RA_F16: return f(DF16{});
    default: return cudaErrorInvalidValue;
  }
}

int threads_for(int slots) { return slots > 256 * kUnroll ? 512 : slots > 128 * kUnroll ? 256 : 128; }

}  // namespace

cudaError_t launch_vocab_forward(int dtype, const VocabForward& a, int, cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_float(dtype, [&](auto d) {
    using D = decltype(d);
    const int threads = threads_for(slots_per_shard<D>(a.x.C) * a.x.shards);
    if (a.ids)
      vocab_forward_kernel<D, true><<<(unsigned)a.x.rows, threads, 0, st>>>(a);
    else
      vocab_forward_kernel<D, false><<<(unsigned)a.x.rows, threads, 0, st>>>(a);
    return cudaGetLastError();
  });
}

cudaError_t launch_vocab_backward(int dtype, const VocabBackward& a, int sms, cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_float(dtype, [&](auto d) {
    using D = decltype(d);
    const int slots = slots_per_shard<D>(a.x.C) * a.x.shards;
    const int threads = threads_for(slots);
    // few rows: split each over CTAs until the SMs are covered, a batch of
    // slots each at least
    int64_t parts = ((int64_t)4 * sms + a.x.rows - 1) / a.x.rows;
    const int64_t most = (slots + threads * kUnroll - 1) / (threads * kUnroll);
    if (parts > most) parts = most;
    const unsigned grid = (unsigned)(a.x.rows * parts);
    if (a.ids)
      vocab_backward_kernel<D, true><<<grid, threads, 0, st>>>(a, (int)parts);
    else
      vocab_backward_kernel<D, false><<<grid, threads, 0, st>>>(a, (int)parts);
    return cudaGetLastError();
  });
}

}  // namespace ra
