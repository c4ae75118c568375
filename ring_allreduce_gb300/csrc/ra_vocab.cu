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
// The forward pass reads the row once.  With t = x log2(e) - ref, every thread
// keeps s = sum 2^t and u = sum t 2^t; ref is at most kLag below the largest x
// log2(e) that the thread saw, and s and u are moved when it is passed by more
// (rare after the first vectors), so 2^t never leaves its range.  Then lse =
// ref unit + ln2 log2 s, unit = 1 / (tau scale) of the rounded factor (ln2 but for
// that) in two parts so that lse is rounded once, and H = ln2 (log2 s - u / s).
// All statistics are binary32.
// ref is the rounded x log2(e) of a logit, t the exact one less ref, so t of
// that very logit is half a unit of ref's last place: |ref| is held to 2^24,
// where that is 1 at most.  (At 1e10 it would be 2^8, and 2^t infinite: a mask
// of such a value over a thread's first logits would take the row with it.)
// What lies below counts for nothing beside a logit above; a row that lies
// beyond it altogether has its largest logit taken off exactly (far_stats).
//
// The top K come out of the same pass without a comparison per element
// against a list: each thread also keeps the largest logit it saw, and its
// largest of every few chunks in shared memory.  The K-th largest of the
// threads' maxima bounds the row's K-th largest logit from below; a lane's
// part of a group of chunks is read again only where its largest reaches
// that, and the few logits that do are ranked against each other.
//
// A row's shards are cut into 16-byte slots, and these into chunks of 128, a
// lane's four 512 bytes apart; a warp takes every warps-th chunk.  A slot that
// a shard's first or last columns share with other memory is read element by
// element, so rows may start on any element.
//
// What bounds it: 16-bit logits arrive at 12 a clock and SM at the copy
// bandwidth, so that at three instructions a clock and scheduler quartet each
// may take eight: arithmetic on pairs, a maximum on packed halves, and no
// index arithmetic within a chunk.
#include "ra_ops.cuh"

#include <type_traits>

namespace ra {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFarBelow = -200.0f;   // 2^-200 is 0 in binary32: exponents that are multiplied with their power
                                       // are held above this, so that it stays 0 (not 0 * inf)
constexpr float kLag = 4.0f;
constexpr float kFar = 16777216.0f;    // 2^24: a row whose ref would be further from zero is a far one
constexpr float kNoRef = -kFar;        // ref before the first logit above it

constexpr float kNothingLeft = -1e30f;
constexpr float kSharp = 16384.0f;     // 2^14: binary32 holds an lse of that size to 2^-10, and with it every probability

template <class D> struct NegInf;
// -inf, and the type's lowest value, ordered()
template <> struct NegInf<DF32> { static constexpr uint32_t word = 0xFF800000u, one = 0xFF800000u, lowest = 0x00800000u; };
template <> struct NegInf<DBF16> { static constexpr uint32_t word = 0xFF80FF80u, one = 0xFF80u, lowest = 0x0080FFFFu; };
template <> struct NegInf<DF16> { static constexpr uint32_t word = 0xFC00FC00u, one = 0xFC00u, lowest = 0x38801FFFu; };
constexpr uint32_t kOrderedNegInf = 0x007FFFFFu;

// The largest of a slot's logits, NaN if there is one.
template <class D> __device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t word_max<DF32>(uint32_t a, uint32_t b) {
  return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
}
template <> __device__ __forceinline__ uint32_t word_max<DBF16>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <> __device__ __forceinline__ uint32_t word_max<DF16>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <class D> __device__ __forceinline__ uint32_t vector_max(uint4 v) {
  return word_max<D>(word_max<D>(v.x, v.y), word_max<D>(v.z, v.w));
}
template <class D> __device__ __forceinline__ float word_value(uint32_t w) {
  if constexpr (sizeof(typename D::T) == 4) {
    return __uint_as_float(w);
  } else {
    float x[2];
    unpack2<D>(w, x);
    return max_nan(x[0], x[1]);
  }
}

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

// One row's shards, in shared memory: the first byte, and the columns.
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

constexpr int kChunk = 128;                  // slots
constexpr uintptr_t kLine = 127;             // a shard's slots are counted from its first byte's 128-byte line on, so that
                                             // a warp's accesses are of whole lines
constexpr int kPerLane = kChunk / 32;

// Chunks per shard.
__host__ __device__ __forceinline__ int chunks_per_shard(const VocabRows& x) { return (x.slots + kChunk - 1) / kChunk; }

// Where slot j of a shard lies: [lo, hi) are the slot's elements that belong
// to the shard, e0 the shard's column of its element 0.
template <class D> struct Slot {
  const uint4* at;
  int lo, hi, e0;
  __device__ __forceinline__ Slot(uintptr_t first, int len, int j) {
    at = reinterpret_cast<const uint4*>(first & ~kLine) + j;
    e0 = j * D::kVec - (int)((first & kLine) / sizeof(typename D::T));
    lo = max(0, -e0);
    hi = min(D::kVec, len - e0);
  }
  __device__ __forceinline__ bool empty() const { return hi <= lo; }
  __device__ __forceinline__ bool whole() const { return lo == 0 && hi == D::kVec; }
  // the slot's logits; -inf where it has none
  __device__ __forceinline__ uint4 load() const {
    if (whole()) return ld_stream(at);
    uint32_t w[4];
    const typename D::T* p = reinterpret_cast<const typename D::T*>(at);
    constexpr uint32_t none = NegInf<D>::one;
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

// A warp's walk over the chunks q, q + step, ... below `end` of a row, chunk q
// being chunk k of shard r.  The same in every lane.
template <class D> struct Walk {
  const RowShards& s;
  int per, q, end, step;
  int r, k;
  uintptr_t first;
  int len;
  __device__ __forceinline__ Walk(const RowShards& rows, int chunks, int begin, int last, int by)
      : s(rows), per(chunks), q(begin), end(last), step(by) {
    r = q / per;
    k = q - r * per;
    open();
  }
  __device__ __forceinline__ void open() {
    if (q < end) {
      first = s.first[r];
      len = s.len[r];
    }
  }
  __device__ __forceinline__ bool more() const { return q < end; }
  __device__ __forceinline__ void next() {
    q += step;
    k += step;
    if (k >= per) {
      do {
        k -= per;
        ++r;
      } while (k >= per);
      open();
    }
  }
  // every slot is the shard's alone
  __device__ __forceinline__ bool whole() const {
    const int e0 = k * kChunk * D::kVec - (int)((first & kLine) / sizeof(typename D::T));
    return e0 >= 0 && e0 + kChunk * D::kVec <= len;
  }
  __device__ __forceinline__ int slot(int i) const { return k * kChunk + 32 * i + (int)(threadIdx.x & 31); }
  __device__ __forceinline__ Slot<D> at(int i) const { return Slot<D>(first, len, slot(i)); }
  // the lane's slots; whether any of them has a logit
  __device__ __forceinline__ bool load(uint4 (&raw)[kPerLane]) const {
    constexpr uint32_t none = NegInf<D>::word;
    if (whole()) {
      const uint4* p = reinterpret_cast<const uint4*>(first & ~kLine) + slot(0);
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) raw[i] = ld_stream(p + 32 * i);
      return true;
    }
    bool some = false;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      raw[i] = make_uint4(none, none, none, none);
      const Slot<D> t = at(i);
      if (t.empty()) continue;
      some = true;
      raw[i] = t.load();
    }
    return some;
  }
};

// The logit of column c (0 <= c < V).
template <class D>
__device__ __forceinline__ float logit_at(const VocabRows& x, int64_t row, int c) {
  const int r = c / x.C;
  const typename D::T* p = static_cast<const typename D::T*>(x.shard[r]) + row * x.stride[r] + (c - r * x.C);
  return widen<D>(ld_stream_scalar(p));
}

// Running statistics of a row: s = sum 2^t, u = sum t 2^t, t = x scale - ref.
struct Stats {
  float ref, s, u;
  __device__ __forceinline__ void move(float to) {
    const float t = fmaxf(ref - to, kFarBelow);
    const float f = exp2_fast(t);
    u = __fmaf_rn(t, s, u) * f;
    s *= f;
    ref = to;
  }
  __device__ __forceinline__ void join(Stats o) {
    const float to = fmaxf(ref, o.ref);
    move(to);
    o.move(to);
    s += o.s;
    u += o.u;
  }
};

// Joined over `lanes` neighbouring lanes (a power of two), the same in each of them.
__device__ __forceinline__ Stats warp_stats(Stats v, int lanes) {
#pragma unroll 1
  for (int d = lanes >> 1; d > 0; d >>= 1) {
    Stats o;
    o.ref = __shfl_xor_sync(0xFFFFFFFFu, v.ref, d);
    o.s = __shfl_xor_sync(0xFFFFFFFFu, v.s, d);
    o.u = __shfl_xor_sync(0xFFFFFFFFu, v.u, d);
    v.join(o);
  }
  return v;
}

// ------------------------------------------- the CTAs that share a row (few
// rows): one cluster, each CTA with a part of the chunks

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// `mine`'s place in the shared memory of CTA `rank`
__device__ __forceinline__ uint32_t in_cta(const void* mine, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(mine)), "r"(rank));
  return a;
}
// What another CTA is to read is stored into its shared memory before the
// barrier: read from here after it, a few rows would wait for the way there and
// back once more.
__device__ __forceinline__ void far_store(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void far_store(uint32_t a, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// ---------------------------------------------- lists of a warp's 32 largest
// A warp holds 32 keys, falling from lane 0; 0 is no key.

// (Called, not inlined: what runs once a row costs mostly its way into the
// instruction cache.)  A bitonic sequence of 32 keys into falling order.
__device__ __noinline__ uint64_t warp_fall(uint64_t k) {
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
__device__ __noinline__ uint64_t warp_sort(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll 1
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
__device__ __noinline__ uint64_t block_merge(uint64_t k, uint64_t (*lists)[32]) {
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

// A warp's 32 best logits so far (by value, then column), and the K-th of them.
struct Best {
  uint64_t list, last, bound;
  int top;
  // The lanes' slots, elements [lo, hi) of each: what comes before the bound
  // by (logit, chunk) and before the K-th.
  template <class D> __device__ __noinline__ void offer(uint4 raw, int lo, int hi, int chunk, int column) {
    float x[D::kVec];
    unpack<D>(raw, x);
    unsigned want = 0;
#pragma unroll
    for (int e = 0; e < D::kVec; ++e)
      if (e >= lo && e < hi && top_key(x[e], (uint32_t)chunk) > bound) want |= 1u << e;
    while (__any_sync(0xFFFFFFFFu, want != 0)) {   // a logit of each lane at a time
      const bool some = want != 0;
      const int e = some ? __ffs(want) - 1 : 0;
      want &= want - 1;   // of 0: 0
      float v = x[0];
#pragma unroll
      for (int k = 1; k < D::kVec; ++k) v = e == k ? x[k] : v;
      const uint64_t full = top_key(v, (uint32_t)(column + e));
      const bool may = some && full > last;
      unsigned hits = __ballot_sync(0xFFFFFFFFu, may);
      if (__popc(hits) > 8) {   // all of them at once
        list = warp_merge(list, warp_sort(may ? full : 0));
      } else {
        for (; hits; hits &= hits - 1) list = warp_insert(list, __shfl_sync(0xFFFFFFFFu, full, __ffs(hits) - 1));
      }
      last = __shfl_sync(0xFFFFFFFFu, list, top - 1);
    }
  }
};

// ------------------------------------------------------------------ teacher

// The teacher's tokens: columns (-1 where one is absent: an id that is no
// column, or a teacher logit of -inf), logits, and the student's logits there.
struct Teacher {
  alignas(16) int id[kTeacherMax];   // -1, too, up to the next multiple of four past the last
  float t[kTeacherMax];
  float x[kTeacherMax];
};

// Called by the whole block, before a barrier.
template <class D>
__device__ __forceinline__ void load_teacher(Teacher& to, const VocabRows& rows, const int64_t* ids,
                                             const void* teacher, int K, bool f32, int64_t row) {
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    const int64_t id = ld_g(ids + row * K + k);
    const float t = f32 ? ld_g(static_cast<const float*>(teacher) + row * K + k)
                        : widen<D>(ld_g(static_cast<const typename D::T*>(teacher) + row * K + k));
    const bool absent = id < 0 || id >= rows.V || t == -INFINITY;
    to.id[k] = absent ? -1 : (int)id;
    to.t[k] = t;
    to.x[k] = absent ? 0.0f : logit_at<D>(rows, row, (int)id);
  }
  if (threadIdx.x < (unsigned)(-K & 3)) to.id[K + threadIdx.x] = -1;
}

// The softmax's largest logit and sum over the tokens, in every lane of the
// warp that runs this (every warp that needs them does, so that no barrier
// follows); m is -inf where the row has none, NaN where a logit is.
struct Softmax {
  float m, s;
  __device__ __forceinline__ Softmax(const Teacher& t, int K, float inv_tau) {
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
    for (int k = lane; k < K; k += 32)
      if (t.id[k] >= 0) m = max_nan(m, t.t[k]);
    m = warp_max_nan(m);
    s = 0.0f;
    for (int k = lane; k < K; k += 32)
      if (t.id[k] >= 0) s += expf((t.t[k] - m) * inv_tau);
    s = warp_sum(s);
  }
  __device__ __forceinline__ bool taught() const { return m != -INFINITY; }
};

// A row's loss where the sum over its tokens left binary32's range: tokens at
// the type's lowest value, whose mean over tau is out of it though tau times
// that is not, or whose shares add up to a little more than 1.  The mean is no
// larger than the largest term.  Called by one warp, and not inlined: rare.
// (m, s: Softmax; base, ref, log2_s: tau log p = tau ln2 ((x - base) log2(e) / tau - ref - log2_s).)
__device__ __noinline__ float largest_loss(const Teacher& t, int K, float tau, float inv_tau, float m, float s,
                                           float base, float ref, float log2_s) {
  float loss = 0.0f, most = 0.0f;
  for (int k = threadIdx.x & 31; k < K; k += 32) {
    const float d = t.t[k] - m, p = t.id[k] < 0 ? 0.0f : expf(d * inv_tau) / s;
    if (p == 0.0f) continue;
    const float x = t.x[k] - base, e = __fmaf_rn(x, kLog2e * inv_tau, -ref);
    const float v = d - tau * logf(s) - (e == -INFINITY ? x : kLn2 * tau * (e - log2_s));
    loss += p * tau * v;   // the weight first: tau v may be out of the range, too
    most = fmaxf(most, v);
  }
  return fminf(warp_sum(loss), warp_max_nan(most) * tau);
}

// ------------------------------------------------------------------ forward

constexpr int kMaxThreads = 256;
constexpr int kMaxParts = 8;   // CTAs of a portable cluster
constexpr int kGroups = 12;    // a warp's chunks, in this many groups at most
constexpr int kCandidates = 256;   // at least 32 of each part of a row

struct RowShared {
  RowShards rows;
  Stats warp[kMaxThreads / 32];
  Stats block[kMaxParts];              // what the row's CTAs found, stored here by each of them
};
struct DistillShared : RowShared {
  Teacher teacher;
};
struct TopShared : RowShared {
  int target;                          // -1: none, -2: one that is no column
  float target_logit;
  int found;
  int lowest;                          // a logit of the type's lowest value was seen
  uint64_t lists[kMaxThreads / 32][32];
  uint64_t candidates[kCandidates];
};
// and for the top K, as many as there are warps: with static ones of eight
// warps' size an SM held fewer of the small CTAs that short rows take
struct alignas(16) WarpTop {
  uint32_t largest[kGroups][32];   // the lanes' largest logits of each group of chunks, ordered()
  uint32_t again[32];              // the groups and lanes to read again
};
extern __shared__ WarpTop g_warp_top[];
// behind them, where CTAs share a row: the K largest of each, stored into the first one's
using PartLists = uint64_t[kMaxParts][32];

// The block's statistics, the same in every thread (and of every CTA of the row).
__device__ __noinline__ Stats block_stats(Stats st, RowShared& sh, int part, int parts) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;   // a power of two
  st = warp_stats(st, 32);
  if (lane == 0) sh.warp[threadIdx.x >> 5] = st;
  __syncthreads();
  st = warp_stats(sh.warp[lane & (warps - 1)], warps);
  if (parts > 1) {   // a power of two, too
    if ((int)threadIdx.x < parts) {
      const uint32_t a = in_cta(&sh.block[part], threadIdx.x);
      far_store(a, st.ref);
      far_store(a + 4, st.s);
      far_store(a + 8, st.u);
    }
    __syncwarp();
    cluster_sync();
    st = warp_stats(sh.block[lane & (parts - 1)], parts);
  }
  return st;
}

// Far rows: no thread's ref has moved from kNoRef (-inf everywhere, or a mask's
// low value), or one lies above kFar.  Their largest logit m first, then t = (x - m) scale, which
// is 0 where x is m and exact wherever 2^t counts.  Rare, so it reads the row
// twice more; m comes back as `largest`.
template <class D>
__device__ __noinline__ Stats far_stats(const VocabForward& a, RowShared& sh, int per, int begin, int end, int part,
                                        int parts, float scale, float* largest) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float m = -INFINITY;
  uint4 raw[kPerLane];
  for (Walk<D> w(sh.rows, per, begin + (int)(threadIdx.x >> 5), end, warps); w.more(); w.next()) {
    w.load(raw);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) m = max_nan(m, word_value<D>(vector_max<D>(raw[i])));
  }
  m = warp_max_nan(m);
  __syncthreads();   // sh.warp is read no more
  if (lane == 0) sh.warp[threadIdx.x >> 5].s = m;
  __syncthreads();
  m = warp_max_nan(lane < warps ? sh.warp[lane].s : -INFINITY);
  if (parts > 1) {
    cluster_sync();   // sh.block is read no more
    if ((int)threadIdx.x < parts) far_store(in_cta(&sh.block[part], threadIdx.x) + 4, m);
    __syncwarp();
    cluster_sync();
    m = lane < parts ? sh.block[lane].s : -INFINITY;
    m = warp_max_nan(m);
    cluster_sync();
  }
  __syncthreads();
  *largest = m;
  Stats st{0.0f, m < INFINITY ? 0.0f : NAN, 0.0f};   // relative to m
  for (Walk<D> w(sh.rows, per, begin + (int)(threadIdx.x >> 5), end, warps); w.more() && m > -INFINITY; w.next()) {
    w.load(raw);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      float x[D::kVec];
      unpack<D>(raw[i], x);
#pragma unroll
      for (int e = 0; e < D::kVec; ++e) {
        const float t = fmaxf((x[e] - m) * scale, kFarBelow), p = exp2_fast(t);
        st.s += p;
        st.u = __fmaf_rn(t, p, st.u);
      }
    }
  }
  return block_stats(st, sh, part, parts);
}

// The lanes' slots, elements [lo, hi) of each: those that reach the bound
// become candidates, as far as there is room.
template <class D>
__device__ __noinline__ void collect(TopShared& sh, uint4 raw, int lo, int hi, int column, uint32_t bound) {
  const int lane = threadIdx.x & 31;
  float x[D::kVec];
  unpack<D>(raw, x);
  unsigned want = 0;
#pragma unroll
  for (int e = 0; e < D::kVec; ++e) {
    if (e < lo || e >= hi) continue;
    if (ordered(x[e]) >= bound) want |= 1u << e;
    if (ordered(x[e]) == NegInf<D>::lowest) sh.lowest = 1;
  }
  int before = __popc(want);   // and in the lanes below
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const int below = __shfl_up_sync(0xFFFFFFFFu, before, d);
    if (lane >= d) before += below;
  }
  const int all = __shfl_sync(0xFFFFFFFFu, before, 31);
  if (all == 0) return;
  int at = 0;
  if (lane == 0) at = atomicAdd(&sh.found, all);   // their order does not matter: they are ranked
  at = __shfl_sync(0xFFFFFFFFu, at, 0) + before - __popc(want);
  for (; want; want &= want - 1, ++at) {
    const int e = __ffs(want) - 1;
    float v = x[0];
#pragma unroll
    for (int k = 1; k < D::kVec; ++k) v = e == k ? x[k] : v;
    if (at < kCandidates) sh.candidates[at] = top_key(v, (uint32_t)(column + e));
  }
}

// The first column from chunk q on.
template <class D>
__device__ __forceinline__ int column_of(const RowShards& s, int q, int per, int chunks, int C, int V) {
  if (q >= chunks) return V;
  const int r = q / per;
  const int c = (q - r * per) * kChunk * D::kVec - (int)((s.first[r] & kLine) / sizeof(typename D::T));
  return r * C + min(max(c, 0), s.len[r]);
}

// lists[0]: the `top` largest of the candidates (0: none), falling; all keys
// but 0 differ.
__device__ __noinline__ void rank_candidates(TopShared& sh, int n, int top) {
  if (threadIdx.x < 32) sh.lists[0][threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const uint64_t key = sh.candidates[i];
    int rank = 0;
#pragma unroll 4
    for (int k = 0; k < n; ++k) rank += sh.candidates[k] > key;
    if (key != 0 && rank < top) sh.lists[0][rank] = key;
  }
  __syncthreads();
}

// The same where too many logits reach a bound of 16 bits (equal ones, mostly:
// a mask that leaves fewer than K).  The K-th largest of the threads' maxima
// by (logit, chunk): chunks are numbered in the columns' order, so whatever
// comes after that is beaten by K logits.  What comes before it is read again;
// what is equal to it lies in its chunk.
template <class D>
__device__ __noinline__ void top_of_many(TopShared& sh, uint32_t best, int best_at, int top, int C, int per,
                                         int begin, int end) {
  constexpr int V = D::kVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const uint64_t mine = best_at < 0 ? 0 : (uint64_t)best << 32 | (uint32_t)~best_at;
  __syncthreads();
  block_merge(warp_sort(mine), sh.lists);
  const uint64_t bound = sh.lists[0][top - 1];
  __syncthreads();
  Best best_of{0, 0, bound, top};
  if (__any_sync(0xFFFFFFFFu, mine > bound)) {   // else no logit of the warp comes before it
    const uint32_t least = (uint32_t)(bound >> 32);
    for (Walk<D> w(sh.rows, per, begin + warp, end, warps); w.more(); w.next()) {
      uint4 raw[kPerLane];
      w.load(raw);
#pragma unroll 1
      for (int i = 0; i < kPerLane; ++i) {
        const Slot<D> s = w.at(i);
        const uint4 v = i == 0 ? raw[0] : i == 1 ? raw[1] : i == 2 ? raw[2] : raw[3];
        const bool reach = ordered(word_value<D>(vector_max<D>(v))) >= least;
        if (__any_sync(0xFFFFFFFFu, reach)) best_of.offer<D>(v, s.lo, s.hi, w.q, w.r * C + s.e0);
      }
    }
  }
  // the first 32 of the logits equal to the bound in its chunk: one warp, in the columns' order
  const int tied = (int)~(uint32_t)bound;
  if (bound != 0 && (tied - begin) % warps == warp) {
    const int r = tied / per;
    int got = 0;
    for (int i = 0; i < kPerLane && got < 32; ++i) {
      const Slot<D> s(sh.rows.first[r], sh.rows.len[r], (tied - r * per) * kChunk + 32 * i + lane);
      float x[V];
      unpack<D>(s.empty() ? make_uint4(0, 0, 0, 0) : s.load(), x);
      unsigned equal = 0;
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e >= s.lo && e < s.hi && ordered(x[e]) == (uint32_t)(bound >> 32)) equal |= 1u << e;
      int before = __popc(equal);   // and in the lanes below
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const int below = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before += below;
      }
      int at = got + before - __popc(equal);
      for (; equal; equal &= equal - 1, ++at)
        if (at < 32)
          sh.lists[warp][at] =
              ((uint64_t)(uint32_t)(bound >> 32) << 32) | (uint32_t)~(uint32_t)(r * C + s.e0 + __ffs(equal) - 1);
      got += __shfl_sync(0xFFFFFFFFu, before, 31);
    }
    __syncwarp();
    best_of.list = warp_merge(best_of.list, lane < got ? sh.lists[warp][lane] : 0);
    __syncwarp();
  }
  block_merge(best_of.list, sh.lists);
}

// Measured, as parts of a copy's 6.8 TB/s for the logits' bytes: loss of 4096
// x 131072 bf16 in eight shards, 64 teacher tokens: 161 us, 0.99; log
// probabilities, entropy and five alternatives: 185 us, 0.86 (the entropy's
// multiply and the largest of every group of chunks: issue slots); one row
// with 20 alternatives: 8.9 us, 4 us of them the choice of the alternatives
// over a cluster of eight CTAs.  Short rows pay per row for the alternatives:
// 20000 x 8192 bf16 59 us without, 93 with five.  2048 x 131072 binary32:
// 154 us, 1.03, and 168, 0.94.
template <class D, bool DISTILL>
__global__ void __launch_bounds__(kMaxThreads, 4) vocab_forward_kernel(const __grid_constant__ VocabForward a,
                                                                       int parts) {
  constexpr int V = D::kVec;
  __shared__ typename std::conditional<DISTILL, DistillShared, TopShared>::type sh;
  after_predecessor();
  const int64_t row = blockIdx.x / parts;
  const int part = parts > 1 ? (int)cluster_rank() : 0;
  if (parts > 1) cluster_arrive();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const float scale = a.x.scale;
  const int per = chunks_per_shard(a.x), chunks = per * a.x.shards;
  const int share = (chunks + parts - 1) / parts;
  const int begin = part * share, end = min(chunks, begin + share);
  load_row<D>(a.x, row, sh.rows);
  if constexpr (!DISTILL)
    if (tid == 0) sh.found = sh.lowest = 0;
  __syncthreads();

  Stats st{kNoRef, 0.0f, 0.0f};
  float2 s2 = make_float2(0.0f, 0.0f), u2 = make_float2(0.0f, 0.0f);
  uint32_t best = 0;   // the thread's largest logit, ordered(), and the first chunk that has it (-1: it saw none)
  int best_at = -1;
  const int of_group = ((share + warps - 1) / warps + kGroups - 1) / kGroups;   // chunks
  int group = 0, in_group = 0;
  uint32_t group_best = 0;
  const float2 scale2 = make_float2(scale, scale);
  auto add = [&](const uint4(&raw)[kPerLane], int chunk, bool some) {
    uint32_t vm = vector_max<D>(raw[0]);
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) vm = word_max<D>(vm, vector_max<D>(raw[i]));
    const float largest = word_value<D>(vm);
    if (!DISTILL && a.top > 0) {
      const uint32_t o = some ? ordered(largest) : 0;
      best_at = o > best ? chunk : best_at;
      best = max(o, best);
      if (in_group == of_group) {
        ++group;
        in_group = 0;
        group_best = 0;
      }
      ++in_group;
      group_best = max(group_best, o);
      g_warp_top[warp].largest[group][lane] = group_best;
    }
    if (largest * scale > st.ref + kLag) {
      st.s = s2.x + s2.y;
      st.u = u2.x + u2.y;
      st.move(largest * scale);
      s2 = make_float2(st.s, 0.0f);
      u2 = make_float2(st.u, 0.0f);
    }
    const float2 ref2 = make_float2(-st.ref, -st.ref);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      float x[V];
      unpack<D>(raw[i], x);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 t = __ffma2_rn(make_float2(x[e], x[e + 1]), scale2, ref2);
        const float2 p = make_float2(exp2_fast(t.x), exp2_fast(t.y));
        s2 = __fadd2_rn(s2, p);
        if (!DISTILL) u2 = __ffma2_rn(make_float2(fmaxf(t.x, kFarBelow), fmaxf(t.y, kFarBelow)), p, u2);
      }
    }
  };
  {
    // one chunk ahead, in two sets of registers by turns
    uint4 one[kPerLane], two[kPerLane];
    Walk<D> w(sh.rows, per, begin + warp, end, warps);
    bool some_one = false, some_two = false;
    if (w.more()) some_one = w.load(one);
    // what is needed at the end, beside the row's first logits
    if (part == 0) {
      if constexpr (DISTILL) {
        load_teacher<D>(sh.teacher, a.x, a.ids, a.teacher, a.K, a.teacher_f32, row);
      } else if (tid == 0) {
        const int64_t target = ld_g(a.targets + row);
        sh.target = target < 0 ? -1 : target >= a.x.V ? -2 : 0;
        sh.target_logit = target < 0 || target >= a.x.V ? 0.0f : logit_at<D>(a.x, row, (int)target);
      }
    }
    while (w.more()) {
      int chunk = w.q;
      w.next();
      if (w.more()) some_two = w.load(two);
      add(one, chunk, some_one);
      if (!w.more()) break;
      chunk = w.q;
      w.next();
      if (w.more()) some_one = w.load(one);
      add(two, chunk, some_two);
    }
  }
  st.s = s2.x + s2.y;
  st.u = u2.x + u2.y;
  if (parts > 1) cluster_wait();   // every CTA of the row has begun
  st = block_stats(st, sh, part, parts);
  float row_max = 0.0f;   // of a far row
  const bool far = st.ref <= kNoRef || st.ref > kFar;   // ref is the largest of the threads' now
  if (far) st = far_stats<D>(a, sh, per, begin, end, part, parts, scale, &row_max);
  const bool empty = far && row_max == -INFINITY;   // nothing but -inf
  const float log2_s = log2f(st.s);                // NaN where the row has +inf or NaN
  const float lse = empty ? -INFINITY
                    : far ? __fmaf_rn(row_max, a.x.inv_tau, kLn2 * log2_s)
                          : __fmaf_rn(st.ref, a.x.unit, __fmaf_rn(st.ref, a.x.unit_rest, kLn2 * log2_s));
  // A row of one token has log2 s - t of a rounding's size, on either side of 0:
  // what cannot be below 0 is held there.  (NaN stays.)
  auto not_below = [](float v) { return v < 0.0f ? 0.0f : v; };
  // log p of a logit, or tau times that
  auto log_prob = [&](float x, bool by_tau = false) {
    if (empty) return -INFINITY;
    const float d = far ? x - row_max : x;
    const float t = __fmaf_rn(d, scale, far ? 0.0f : -st.ref);
    // a masked logit near the type's lowest value leaves binary32's range in t before it does so itself
    if (t == -INFINITY && log2_s == log2_s) return by_tau ? d : d * a.x.inv_tau;
    return by_tau ? kLn2 * a.x.tau * (t - log2_s) : kLn2 * -not_below(log2_s - t);
  };
  const bool first = part == 0;
  if (first && tid == 0) st_g(a.lse + row, lse);

  if constexpr (DISTILL) {
    if (first && warp == 0) {
      const Teacher& t = sh.teacher;
      const Softmax q(t, a.K, a.x.inv_tau);
      const float log_s = logf(q.s);
      float loss = 0.0f;
      for (int k = lane; k < a.K; k += 32) {
        if (t.id[k] < 0) continue;
        const float d = t.t[k] - q.m, p = expf(d * a.x.inv_tau) / q.s;
        // tau (log q - log p): within binary32's range wherever the logits are.  (NaN included)
        if (p != 0.0f) loss += p * ((d - a.x.tau * log_s) - log_prob(t.x[k], true));
      }
      loss = warp_sum(loss) * a.x.tau;
      if (loss == INFINITY && !empty)
        loss = largest_loss(t, a.K, a.x.tau, a.x.inv_tau, q.m, q.s, far ? row_max : 0.0f, far ? 0.0f : st.ref, log2_s);
      if (lane == 0) st_g(a.loss + row, q.taught() ? loss : 0.0f);
    }
  } else {
    if (first && tid == 0) {
      st_g(a.logprob + row, sh.target == -1 ? 0.0f : sh.target == -2 ? NAN : log_prob(sh.target_logit));
      if (a.entropy) st_g(a.entropy + row, empty ? 0.0f : kLn2 * not_below(log2_s - st.u / st.s));
    }
    if (a.top > 0) {
      // A bound that K threads' maxima reach: their K-th largest, cut to 16
      // bits, found bit by bit.  What reaches it is read again and ranked.
      uint32_t bound = 0;
#pragma unroll 1
      for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1)
        if (__syncthreads_count(best >= (bound | bit)) >= a.top) bound |= bit;
      // Fewer than K threads saw more than what a mask leaves (-inf, or the
      // type's lowest value): only that is read again.
      const bool masked = bound <= NegInf<D>::lowest;
      if (masked) bound = NegInf<D>::lowest + 1;
      uint32_t* again = g_warp_top[warp].again;   // group << 5 | lane
      const int groups = in_group ? group + 1 : 0;
      for (int g = 0; g < groups;) {
        int n = 0;
        for (; g < groups; ++g) {   // a group's lanes, and the next ones' while they fit
          const uint32_t largest = g_warp_top[warp].largest[g][lane];
          const unsigned hits = __ballot_sync(0xFFFFFFFFu, largest >= bound);
          if (largest == NegInf<D>::lowest) sh.lowest = 1;
          if (n + __popc(hits) > 32) break;
          if (hits >> lane & 1u) again[n + __popc(hits & ((1u << lane) - 1))] = (uint32_t)g << 5 | lane;
          n += __popc(hits);
        }
        __syncwarp();
        const int each = 4 * of_group;   // slots
        for (int i = lane; i - lane < n * each; i += 32) {
          const int k = i / each, u = i - k * each;
          uint4 raw = make_uint4(0, 0, 0, 0);
          int lo = 0, hi = 0, column = 0;
          if (k < n) {
            const int q = begin + warp + ((int)(again[k] >> 5) * of_group + (u >> 2)) * warps;
            if (q < end) {
              const int r = q / per;
              const Slot<D> s(sh.rows.first[r], sh.rows.len[r],
                              (q - r * per) * kChunk + 32 * (u & 3) + (int)(again[k] & 31u));
              lo = s.lo;
              hi = s.hi;
              column = r * a.x.C + s.e0;
              if (!s.empty()) raw = s.load();
            }
          }
          collect<D>(sh, raw, lo, hi, column, bound);
        }
        __syncwarp();
      }
      __syncthreads();
      bool many = sh.found > kCandidates;
      if (masked && sh.found < a.top) {
        // The rest of the K are masked ones, the lowest columns first.  Where
        // they are all -inf, the part's first K columns hold enough of them;
        // of the type's lowest value they may.
        const int had = sh.found;
        __syncthreads();
        if (warp == 0) {
          const int c = column_of<D>(sh.rows, begin, per, chunks, a.x.C, a.x.V) + lane;
          const bool in = lane < a.top && c < column_of<D>(sh.rows, end, per, chunks, a.x.C, a.x.V);
          const float x = in ? logit_at<D>(a.x, row, c) : 0.0f;
          const unsigned fill =
              __ballot_sync(0xFFFFFFFFu, in && ordered(x) == (sh.lowest ? NegInf<D>::lowest : kOrderedNegInf));
          if (fill >> lane & 1u) sh.candidates[had + __popc(fill & ((1u << lane) - 1))] = top_key(x, (uint32_t)c);
          if (lane == 0) sh.found = had + __popc(fill);
        }
        __syncthreads();
        many = sh.lowest && sh.found < a.top;
      }
      if (many)
        top_of_many<D>(sh, best, best_at, a.top, a.x.C, per, begin, end);
      else
        rank_candidates(sh, sh.found, a.top);
      // lists[0]: the K largest, falling
      if (parts > 1) {
        // the parts' lists, a warp each, joined in the first part
        PartLists& of = *reinterpret_cast<PartLists*>(g_warp_top + warps);
        if (first && warp >= parts) of[warp][lane] = 0;
        if (warp == 0) far_store(in_cta(&of[part][lane], 0), sh.lists[0][lane]);
        cluster_sync();
        if (first) {
          const uint64_t key = of[warp][lane];
          // a key's place is the sum of what every list has before it; all lists searched at once
          int before[kMaxParts] = {};
#pragma unroll
          for (int step = 16; step > 0; step >>= 1)
#pragma unroll
            for (int p = 0; p < kMaxParts; ++p) before[p] += of[p][before[p] + step - 1] > key ? step : 0;
          int rank = 0;
#pragma unroll
          for (int p = 0; p < kMaxParts; ++p) rank += before[p] + (of[p][before[p]] > key);
          __syncthreads();
          if (threadIdx.x < 32) sh.lists[0][lane] = 0;
          __syncthreads();
          if (key != 0 && rank < a.top) sh.lists[0][rank] = key;
          __syncthreads();
        }
      }
      if (first && warp == 0 && lane < a.top) {
        const uint64_t key = sh.lists[0][lane];
        st_g(a.top_ids + row * a.top + lane, (int64_t)(uint32_t)~(uint32_t)key);
        st_g(a.top_logprobs + row * a.top + lane, log_prob(from_ordered((uint32_t)(key >> 32))));
      }
    }
  }
}

// ----------------------------------------------------------------- backward

struct BackwardShared {
  RowShards rows;
  uintptr_t grad[kMaxRanks];
  Teacher teacher;
  // what the target or the teacher adds, and at which column (-1: nowhere); each thread's own tokens
  float add[kTeacherMax];
  int at[kTeacherMax];
  float by_warp[4];                    // of a far row
};

// A row whose lse is too far from zero to tell its probabilities apart (all of
// it masked with -1e9, say: lse is good to 32 there).  One CTA takes its
// largest logit m and log sum e^{(x - m) / tau} again, in two passes, and
// writes its gradient p (A + B log p) in a third, the tokens' parts on top.
// (Called, not inlined: rare, and other rows have no register to spare for it.)
template <class D>
__device__ __noinline__ void far_gradient(const VocabRows& x, BackwardShared& sh, int tokens, float A, float B) {
  using T = typename D::T;
  constexpr int V = D::kVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int per = chunks_per_shard(x), chunks = per * x.shards;
  const float inv_tau = x.inv_tau;
  uint4 raw[kPerLane];
  float m = -INFINITY;
  for (Walk<D> w(sh.rows, per, warp, chunks, warps); w.more(); w.next()) {
    w.load(raw);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) m = max_nan(m, word_value<D>(vector_max<D>(raw[i])));
  }
  m = warp_max_nan(m);
  if (lane == 0) sh.by_warp[warp] = m;
  __syncthreads();
  m = warp_max_nan(lane < warps ? sh.by_warp[lane] : -INFINITY);
  __syncthreads();
  float s = 0.0f;
  for (Walk<D> w(sh.rows, per, warp, chunks, warps); w.more(); w.next()) {
    w.load(raw);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      float v[V];
      unpack<D>(raw[i], v);
#pragma unroll
      for (int e = 0; e < V; ++e) s += expf((v[e] - m) * inv_tau);
    }
  }
  s = warp_sum(s);
  if (lane == 0) sh.by_warp[warp] = s;
  __syncthreads();
  const float log_s = logf(warp_sum(lane < warps ? sh.by_warp[lane] : 0.0f));
  auto gradient = [&](float v) {
    const float t = __fmaf_rn(v - m, inv_tau, -log_s);
    return expf(t) * __fmaf_rn(B, fmaxf(t, kFarBelow), A);
  };
  for (Walk<D> w(sh.rows, per, warp, chunks, warps); w.more(); w.next()) {
    w.load(raw);
    T* out = reinterpret_cast<T*>(sh.grad[w.r]);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const Slot<D> at = w.at(i);
      float v[V];
      unpack<D>(raw[i], v);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e >= at.lo && e < at.hi) st_g(out + at.e0 + e, narrow<D>(gradient(v[e])));
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < tokens; k += blockDim.x) {
    const int c = sh.at[k];
    if (c < 0) continue;
    const int r = c / x.C;
    st_g(reinterpret_cast<T*>(sh.grad[r]) + (c - r * x.C), narrow<D>(gradient(sh.teacher.x[k]) + sh.add[k]));
  }
}

// Every logit is read and its gradient written, element by element; what the
// target or the teacher adds is put on top after the CTA's columns are
// written.  Measured: log probabilities and entropy of 2048 x 65536 fp16: 85
// us, 0.93 of the copy bandwidth; distillation of 4096 x 100003 bf16 in eight
// shards, no row aligned: 269 us, 0.90; 2048 x 131072 binary32, with expf: 322
// and 326 us, 0.98 and 0.97.  Memory bounds them all.
template <class D, bool DISTILL>
__global__ void __launch_bounds__(128, 8) vocab_backward_kernel(const __grid_constant__ VocabBackward a, int parts) {
  constexpr int V = D::kVec;
  using T = typename D::T;
  __shared__ BackwardShared sh;
  after_predecessor();
  const int64_t row = blockIdx.x / parts;
  const int part = (int)(blockIdx.x - row * parts);
  const int n = blockDim.x, tid = threadIdx.x;
  const int per = chunks_per_shard(a.x), chunks = per * a.x.shards;
  const int share = (chunks + parts - 1) / parts;
  const int begin = part * share, end = min(chunks, begin + share);
  const float inv_tau = a.x.inv_tau;
  load_row<D>(a.x, row, sh.rows);
  for (int r = tid; r < a.x.shards; r += n)
    sh.grad[r] = reinterpret_cast<uintptr_t>(a.grad[r]) + (uintptr_t)(row * a.grad_stride[r]) * sizeof(T);
  __syncthreads();
  // the first chunk is on its way while the row's coefficients are made
  uint4 raw[kPerLane], ahead[kPerLane];
  Walk<D> w(sh.rows, per, begin + (tid >> 5), end, n >> 5);
  if (w.more()) w.load(raw);

  const float row_lse = ld_g(a.lse + row), row_g = ld_g(a.g + row);
  int64_t target = 0;
  float gh = 0.0f, H = 0.0f;
  if (!DISTILL) {
    target = ld_g(a.targets + row);
    if (a.grad_entropy) {
      gh = ld_g(a.grad_entropy + row);
      H = ld_g(a.entropy + row);
    }
  }
  // The columns where the target or the teacher adds something are read
  // before any column is written (the gradient may stand in the logits' place).
  if (DISTILL) {
    load_teacher<D>(sh.teacher, a.x, a.ids, a.teacher, a.K, a.teacher_f32, row);
  } else if (tid == 0) {
    const bool some = target >= 0 && target < a.x.V;
    sh.teacher.id[0] = some ? (int)target : -1;
    sh.teacher.x[0] = some ? logit_at<D>(a.x, row, (int)target) : 0.0f;
  }
  __syncthreads();
  // dL_j = p_j (A + B log p_j), plus that
  float A, B = 0.0f;
  // nothing left by the mask: -inf everywhere, or the type's lowest value
  bool zero = row_lse < kNothingLeft;
  if constexpr (DISTILL) {
    const Softmax q(sh.teacher, a.K, inv_tau);
    zero = zero || !q.taught();
    A = zero ? 0.0f : row_g * a.x.tau;
    for (int k = tid; k < a.K && !zero; k += n) {
      const int c = sh.teacher.id[k];
      sh.at[k] = -1;
      if (c < 0) continue;
      // Of equal tokens the first one adds for all.  They are rare, so they
      // are counted four at a time first (6783 x 12160 f16, 85 tokens: the
      // comparisons one by one were more work than the row).
      int equal = 0;
#pragma unroll 4
      for (int o = 0; o < a.K; o += 4) {
        const int4 v = *reinterpret_cast<const int4*>(sh.teacher.id + o);
        equal += (v.x == c) + (v.y == c) + (v.z == c) + (v.w == c);
      }
      bool earlier = false;
      float sum = 0.0f;
      if (equal == 1) {
        sum = expf((sh.teacher.t[k] - q.m) * inv_tau) / q.s;
      } else {
        for (int o = 0; o < a.K; ++o) {
          if (sh.teacher.id[o] != c) continue;
          earlier = earlier || o < k;
          sum += expf((sh.teacher.t[o] - q.m) * inv_tau) / q.s;
        }
      }
      if (earlier) continue;
      sh.add[k] = -A * sum;
      sh.at[k] = c;
    }
  } else {
    const float g = target < 0 ? 0.0f : target >= a.x.V ? NAN : row_g;
    A = -(g + gh * H) * inv_tau;
    B = -gh * inv_tau;
    if (tid == 0) {
      sh.add[0] = g * inv_tau;
      sh.at[0] = sh.teacher.id[0];
    }
  }
  if (zero) A = B = 0.0f;
  const float lse = zero ? 0.0f : row_lse;
  if (fabsf(lse) > kSharp) {
    // A far row is its first CTA's alone: the others' columns would have to be
    // read before they are written, where the gradient stands in the logits' place.
    if (part == 0) far_gradient<D>(a.x, sh, DISTILL ? a.K : 1, A, B);
    return;
  }
  // binary32 outputs show the exponent's rounding: expf there.  The others'
  // 2^t is 0 below 2^-126, where bf16 may still have the product with g / tau and
  // log p: it takes 2^(t + lift), and the factors 2^-lift.
  constexpr float kUnit = sizeof(T) == 4 ? 1.0f : kLog2e;
  const float lift = std::is_same<D, DBF16>::value ? a.lift : 0.0f;
  const float scale = inv_tau * kUnit, ref = __fmaf_rn(-lse, kUnit, lift);
  float slope = B / kUnit;
  if (std::is_same<D, DBF16>::value) {
    A = __fmaf_rn(-slope, lift, A) * a.by_lift;   // slope's t below is lift larger
    slope *= a.by_lift;
  }
  auto gradient = [&](float2 x) {
    const float2 t = __ffma2_rn(x, make_float2(scale, scale), make_float2(ref, ref));   // log p, in units of kUnit
    const float2 p = sizeof(T) == 4 ? make_float2(expf(t.x), expf(t.y)) : make_float2(exp2_fast(t.x), exp2_fast(t.y));
    float2 c = make_float2(A, A);
    if (!DISTILL && B != 0.0f)
      c = __ffma2_rn(make_float2(slope, slope), make_float2(fmaxf(t.x, kFarBelow), fmaxf(t.y, kFarBelow)), c);
    return __fmul2_rn(p, c);
  };
  auto write = [&](const uint4(&from)[kPerLane], int r, int j, uintptr_t first, int len, bool whole) {
    T* out = reinterpret_cast<T*>(sh.grad[r]) - (int)((first & kLine) / sizeof(T));   // element 0 of the shard's slot 0
    const bool vectors = whole && (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      float x[V];
      if (zero) {   // whatever the logits are
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = 0.0f;
      } else {
        unpack<D>(from[i], x);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 d = gradient(make_float2(x[e], x[e + 1]));
          x[e] = d.x;
          x[e + 1] = d.y;
        }
      }
      T* to = out + (int64_t)(j + 32 * i) * V;
      if (vectors) {
        st_stream(reinterpret_cast<uint4*>(to), pack<D>(x));
        continue;
      }
      const Slot<D> s(first, len, j + 32 * i);
      if (s.whole() && (reinterpret_cast<uintptr_t>(to) & 15u) == 0) {
        st_stream(reinterpret_cast<uint4*>(to), pack<D>(x));
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e >= s.lo && e < s.hi) st_g(to + e, narrow<D>(x[e]));
      }
    }
  };
  while (w.more()) {
    const bool whole = w.whole();
    const int r = w.r, j = w.slot(0), len = w.len;
    const uintptr_t first = w.first;
    w.next();
    if (w.more()) w.load(ahead);
    write(raw, r, j, first, len, whole);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) raw[i] = ahead[i];
  }
  __syncthreads();
  const int tokens = zero ? 0 : DISTILL ? a.K : 1;
  for (int k = tid; k < tokens; k += n) {
    const int c = sh.at[k];
    if (c < 0) continue;
    const int r = c / a.x.C, e = c - r * a.x.C;
    const int chunk = r * per + ((int)((sh.rows.first[r] & kLine) / sizeof(T)) + e) / (V * kChunk);
    if (chunk < begin || chunk >= end) continue;   // another CTA's part of the row
    st_g(reinterpret_cast<T*>(sh.grad[r]) + e,
         narrow<D>(gradient(make_float2(sh.teacher.x[k], 0.0f)).x + sh.add[k]));
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

}  // namespace

cudaError_t launch_vocab_forward(int dtype, const VocabForward& a, int sms, cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_float(dtype, [&](auto d) {
    using D = decltype(d);
    const int chunks = chunks_per_shard(a.x) * a.x.shards;
    // Many rows: CTAs of 128 threads at most, eight chunks a warp, so that
    // one's sums and lists overlap the others' reading (log probabilities with
    // five alternatives, and loss, in 128 and in 256 threads: 4096 x 131072
    // bf16 188 and 195 us, 162 and 164; 1200 rows 59 and 64, 51 and 53; 620 rows
    // 54 and 46, 33 and 37; of 50021 f32 34 and 36, 24 and 29).  Few rows: up to
    // 256 threads, a chunk a warp, and clusters that split a row
    // while less than five sixths of the SMs are covered, eight chunks a CTA
    // at least (61 x 50021 f32, 20 alternatives: 10.6 us in four parts, 12.0 in
    // two; 129 x 32003 f16: 11.8 in two, 10.6 in one).  Two threads an alternative
    // at least: the bound is one of the threads' maxima, and a low one lets
    // many logits through (20000 x 8192 bf16, 32 alternatives: 163 us with two
    // warps, 327 with one; with 20, 138 and 128).
    const bool many = a.x.rows >= 4 * (int64_t)sms;
    int threads = 32;
    while (threads < (many ? 128 : 256) && (threads / 32 * (many ? 8 : 1) < chunks || threads < 2 * a.top)) threads *= 2;
    int parts = 1;
    if (!many)
      while (parts < kMaxParts && a.x.rows * parts * 6 <= 5 * (int64_t)sms && chunks >= 16 * parts) parts *= 2;
    const size_t smem = a.top > 0 ? threads / 32 * sizeof(WarpTop) + (parts > 1 ? sizeof(PartLists) : 0) : 0;   // 15 KB at most
    auto kernel = a.ids ? vocab_forward_kernel<D, true> : vocab_forward_kernel<D, false>;
    return launch_after(kernel, dim3((unsigned)(a.x.rows * parts)), dim3((unsigned)threads), smem, st, parts, a, parts);
  });
}

cudaError_t launch_vocab_backward(int dtype, const VocabBackward& a, int sms, cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_float(dtype, [&](auto d) {
    using D = decltype(d);
    const int chunks = chunks_per_shard(a.x) * a.x.shards;
    // Many rows: CTAs of 128 threads at most, four chunks a warp (loss gradient
    // of 20000 x 8192 bf16, eight chunks a row: 129 us in CTAs of two warps, 133
    // of four, 172 of one; of 5184 x 503 f32, two chunks: 26 us of one, 28 of four).
    // Few rows: split each until there are four CTAs of 128 threads to an SM, a
    // chunk a warp at least.  (Every part reads the teacher's tokens again:
    // loss and gradient of 129 x 32003 f16 take 11.7 us so, 13.9 with eight.)
    const bool many = a.x.rows >= 4 * (int64_t)sms;
    int threads = many ? 32 : 128;
    while (threads < 128 && threads / 32 * 4 < chunks) threads *= 2;
    const int warps = threads / 32;
    int64_t parts = ((int64_t)4 * sms + a.x.rows - 1) / a.x.rows;
    const int64_t most = (chunks + warps - 1) / warps;
    if (parts > most) parts = most;
    auto kernel = a.ids ? vocab_backward_kernel<D, true> : vocab_backward_kernel<D, false>;
    return launch_after(kernel, dim3((unsigned)(a.x.rows * parts)), dim3((unsigned)threads), 0, st, 1, a, (int)parts);
  });
}

}  // namespace ra
