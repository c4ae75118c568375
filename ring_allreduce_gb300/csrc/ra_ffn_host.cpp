// ra_ffn_host.cpp -- host side of the feed-forward block and of rows kept in 8
// bits (ra_ffn_*, ra_ckpt_* of include/ra.h): handles, argument checks, the
// tensor maps of a call's operands, and which kernel runs.
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "ra_ffn.h"
#include "ra_ffn_mma.h"
#include "ra_ops_host.h"

struct ra_ffn_ctx {
  int R, dim, inner, C, ranks, device, sms;   // ranks: those that hold columns
  ra_dtype dtype, grad_dtype;
  int act;
  bool check_pointers = true;
  ra::WaitRecord* record; // the device's, of waits that gave up
  uint64_t seen;          // how often something new stood there when this handle last asked
};

struct ra_ckpt_ctx {
  int dim, device, sms;
  ra_dtype dtype, normed_dtype, param_dtype;
  bool check_pointers = true;
};

namespace {

using namespace ra;

constexpr int kMaxDim = 1 << 20, kMaxInner = 1 << 24;
constexpr size_t kMaxFfnRows = (size_t)1 << 27;   // sums over more would come near the waits' limit

using FfnBuffers = BuffersOf<17 * kMaxRanks>;

// Sharded buffers of a call: rank r's [rows][width_r], or, as a weight, [width_r][dim].
struct Shards {
  const char* name;
  const void* const* at;
  const size_t* strides;
  size_t elem;
  bool weight, output;
  const void* const* twins = nullptr;
};

ra_status add_shards(const ra_ffn_ctx* h, FfnBuffers& buf, size_t rows, const Shards& s, void** at, int64_t* strides) {
  if (!s.at || !s.strides) return record_error(RA_ERR_INVALID, "%s: NULL pointer array", s.name);
  for (int r = 0; r < h->ranks; ++r) {
    const size_t width = (size_t)(r + 1 < h->ranks ? h->C : h->inner - r * h->C);
    size_t stride = s.strides[r];
    if (s.weight)
      RA_TRY(buf.add(s.name, r, s.at[r], s.elem, (size_t)h->dim, &stride, s.output, width));
    else
      RA_TRY(buf.add(s.name, r, s.at[r], s.elem, width, &stride, s.output, rows, s.twins ? s.twins[r] : nullptr));
    at[r] = const_cast<void*>(s.at[r]);
    strides[r] = (int64_t)stride;
  }
  return RA_OK;
}

// 1 or R buffers [rows][dim], taken as R.
ra_status add_ranks(const ra_ffn_ctx* h, FfnBuffers& buf, const char* name, const void* const* p, int count,
                    size_t stride, bool output, const void** at, int64_t* checked) {
  if (!p) return record_error(RA_ERR_INVALID, "%s: NULL pointer array", name);
  for (int r = 0; r < count; ++r)
    RA_TRY(buf.add(name, r, p[r], 2, (size_t)h->dim, &stride, output));
  for (int r = 0; r < h->R; ++r) at[r] = p[count == 1 ? 0 : r];
  *checked = (int64_t)stride;
  return RA_OK;
}

ra_status add_scales(const ra_ffn_ctx* h, FfnBuffers& buf, const char* name, const float* const* p, bool output,
                     float** at) {
  if (!p) return record_error(RA_ERR_INVALID, "%s: NULL pointer array", name);
  for (int r = 0; r < h->ranks; ++r) {
    const size_t width = (size_t)(r + 1 < h->ranks ? h->C : h->inner - r * h->C);
    size_t stride = (width + kGroup - 1) / kGroup;
    RA_TRY(buf.add(name, r, p[r], 4, stride, &stride, output));
    at[r] = const_cast<float*>(p[r]);
  }
  return RA_OK;
}

ra_status add_kept(const ra_ffn_ctx* h, FfnBuffers& buf, size_t rows, int bits, bool output, const void* const* gate,
                   const size_t* gate_strides, const void* const* up, const size_t* up_strides,
                   const float* const* gate_scales, const float* const* up_scales, FfnArgs* a) {
  const size_t elem = bits == 8 ? 1 : 2;
  RA_TRY(add_shards(h, buf, rows, {"gate", gate, gate_strides, elem, false, output}, a->kept[0], a->kept_stride[0]));
  RA_TRY(add_shards(h, buf, rows, {"up", up, up_strides, elem, false, output}, a->kept[1], a->kept_stride[1]));
  if (bits == 8) {
    RA_TRY(add_scales(h, buf, "gate_scales", gate_scales, output, a->scales[0]));
    RA_TRY(add_scales(h, buf, "up_scales", up_scales, output, a->scales[1]));
  }
  return RA_OK;
}

FfnArgs args_of(const ra_ffn_ctx* h, size_t rows) {
  FfnArgs a{};
  a.rows = (int64_t)rows;
  a.R = h->R;
  a.dim = h->dim;
  a.inner = h->inner;
  a.C = h->C;
  a.act = h->act;
  a.grad_f32 = h->grad_dtype == RA_F32;
  return a;
}

ra_status check_ffn(ra_ffn_handle h, const void* args) {
  if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
  if (!args) return record_error(RA_ERR_INVALID, "NULL arguments");
  return RA_OK;
}

ra_status check_ffn_rows(size_t rows) {
  if (rows > kMaxFfnRows) return record_error(RA_ERR_INVALID, "rows=%zu above 2^27", rows);
  return RA_OK;
}

// A matrix of a product, [rows][columns] of `elem` bytes; NULL: there is none.
struct Matrix {
  const void* p;
  int64_t rows, columns, stride;   // in elements
  int elem;
  uintptr_t bits() const { return (uintptr_t)p | (rows > 1 ? (uintptr_t)(stride * elem) : 0); }
};

using Encode = decltype(&cuTensorMapEncodeTiled);

Encode encoder() {
  static const Encode f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return Encode(nullptr);
    return reinterpret_cast<Encode>(p);
  }();
  return f;
}

// The map that copies boxes of `box_bytes` (64 or 128, swizzled over as many) of `box_rows` rows.
bool encode(CUtensorMap* map, ra_dtype dtype, const Matrix& o, int box_bytes, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)o.columns, (cuuint64_t)o.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(o.rows > 1 ? o.stride * o.elem : (o.columns * o.elem + 15) / 16 * 16)};
  const cuuint32_t box[2] = {(cuuint32_t)(box_bytes / o.elem), (cuuint32_t)box_rows}, steps[2] = {1, 1};
  const CUtensorMapDataType type = o.elem == 4        ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : o.elem == 1      ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == RA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encoder()(map, type, 2, const_cast<void*>(o.p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A stage's matrices for rank r, laid out as MmaArgs has them.
struct Matrices {
  Matrix in[5] = {};    // operands
  Matrix out[5] = {};   // rows written, and kept rows read
  int outs = 0;         // written
  Matrices(FfnStage stage, const FfnArgs& f, int r) {
    const int64_t width = f.width(r), T = f.rows, D = f.dim;
    const int ke = f.keep_bits / 8, ge = f.grad_f32 ? 4 : 2;
    const Matrix x{f.x[r], T, D, f.x_stride, 2}, dy{f.grad_out[r], T, D, f.grad_out_stride, 2},
        hidden{f.hidden[r], T, width, f.hidden_stride[r], 2}, product{f.out[r], T, D, f.out_stride, 2};
    Matrix w[3], pre[2], kept[2];
    for (int k = 0; k < 3; ++k) w[k] = {f.w[k][r], width, D, f.w_stride[k][r], 2};
    for (int k = 0; k < 2; ++k) pre[k] = {f.grad_pre[k][r], T, width, f.grad_pre_stride[k][r], 2};
    for (int k = 0; k < 2; ++k) kept[k] = {f.kept[k][r], T, width, f.kept_stride[k][r], ke};
    switch (stage) {
      case kFfnHidden:
        in[0] = x, in[1] = w[0], in[2] = w[1];
        out[0] = hidden, out[1] = kept[0], out[2] = kept[1];
        outs = 3;
        break;
      case kFfnOut:
        in[0] = hidden, in[2] = w[2];
        out[0] = product;
        outs = 1;
        break;
      case kFfnGradHidden:
        in[0] = dy, in[1] = w[2];
        out[0] = pre[0], out[1] = pre[1], out[2] = hidden, out[3] = kept[0], out[4] = kept[1];
        outs = 3;
        break;
      case kFfnGradX:
        in[0] = pre[0], in[1] = pre[1], in[2] = w[0], in[3] = w[1];
        out[0] = product;
        outs = 1;
        break;
      default:   // what is not wanted has no operands
        outs = 3;
        for (int k = 0; k < 3; ++k)
          if (f.grad_w[k][r]) {
            in[k] = k == 2 ? hidden : pre[k];
            in[k == 2 ? 4 : 3] = k == 2 ? dy : x;
            out[k] = {f.grad_w[k][r], width, D, f.grad_w_stride[k][r], ge};
          }
    }
  }
};

// Tokens of a tile whose sums may be split: the CTAs' shares of both projections' sums, as much as this,
// lie in a ring of kFewRing.
constexpr int kFewMostSplit = 96;
static_assert(2 * kFewMostSplit * 128 * 4 <= kFewRing && kFewMostSplit % 8 == 0, "a cluster's sums outgrow the ring");

// Which kernel a product runs on: pairs of CTAs with tiles of 256 x 256, or
// CTAs with 128 of the weights' rows against `nt` tokens, `split` to a tile's sums.
struct Plan {
  bool few;
  int nt, split;
};

#ifdef RA_DEBUG_BOUNDS
thread_local Plan debug_plan{false, 0, 0};   // split 0: none
#endif

// The plan with the shortest estimate, in microseconds.  The estimates' form is
// what bounds either kernel -- steps of 64 terms, one after another, in as
// many rounds as there are tiles for the SMs; the bytes of an SM's steps; a turn
// of the ring, whose copies take some 1.8 us; the weights' bytes -- and their
// constants were fitted to 44 shapes (1 to 1200 tokens, 64 to 8192 by 64 to
// 28000 columns, 1 to 8 ranks) times five products, every plan of each measured.
// On these the plan chosen takes 5 % longer than the fastest on average, and
// the large tiles alone would take 42 %.  (The projections of 37 tokens, 4096 x
// 16384 in 8 ranks: 54 us large, 46 few; of 777, 1544 x 5005 in 3: 26 and 48.)
Plan plan_of(const ra_ffn_ctx* h, FfnStage stage, int64_t tokens, int keep_bits) {
  if (stage == kFfnGradW) return {false, 0, 0};   // sums over the tokens: nothing to split
#ifdef RA_DEBUG_BOUNDS
  if (debug_plan.split)
    return {debug_plan.few, (int)std::min<int64_t>(debug_plan.nt, (tokens + 15) / 16 * 16), debug_plan.split};
#endif
  const bool dual = stage == kFfnHidden, back = stage == kFfnGradHidden;
  const int64_t N = dual || back ? h->C : h->dim, K = dual || back ? h->dim : h->C;
  const auto up = [](int64_t n, int64_t by) { return (n + by - 1) / by; };
  const double steps = (double)up(K, 64) * (stage == kFfnGradX ? 2 : 1);
  const double memory = 2.0 * h->inner * h->dim * (dual || stage == kFfnGradX ? 2 : 1) / 6.6e6;
  const double waves = (double)up(up(tokens, 256) * up(N, dual ? 128 : 256) * h->R, h->sms / 2);
  Plan best{false, 0, 0};
  double least = 4.4 + std::max(waves * steps * 0.277, memory) + 1.8 * (waves - 1) +
                 (back ? 7.1 : !dual ? 1.1 : keep_bits == 8 ? 4.5 : 1.7);
  const double token = back ? 0.15 : !dual ? 0.07 : keep_bits == 8 ? 0.21 : 0.025;   // a token's outputs
  for (const int most : {16, 32, 64, 96, 128}) {
    const int nt = (int)std::min<int64_t>(most, up(tokens, 16) * 16);
    for (int split = 1; split <= 8 && (split == 1 || nt <= kFewMostSplit); split *= 2) {
      const double ctas = (double)(up(N, 128) * up(tokens, nt) * h->R * split);
      const double rounds = std::ceil(ctas / (2 * h->sms)), on_sm = ctas > h->sms ? 2 : 1;
      const int stage_bytes = few_stage_bytes(stage, nt);
      const int ring = std::min((on_sm > 1 ? kFewRing : kFewRingAlone) / stage_bytes, kFewMostStages);
      const double step = std::max(stage_bytes / 1024.0 * on_sm * 0.0117, 1.76 / ring);
      const int live = (int)std::min<int64_t>(nt, tokens);
      const double estimate =
          1.25 + std::max(rounds * steps / split * step, memory) +
          rounds * (3.3 + (split > 1 ? 0.33 + 0.07 * live + 0.144 * split : 0.0) + 8.0 * up(up(live, split), 8) * token +
                    (dual && keep_bits == 8 ? 2.0 : 0.0));
      if (estimate < least) {
        least = estimate;
        best = {true, nt, split};
      }
    }
    if (nt < most) break;
  }
  return best;
}

// One product on the tensor cores, in as few launches as its ranks fit into.
template <class Args> ra_status run_planned(ra_ffn_handle h, FfnStage stage, const Plan& plan, const FfnArgs& f,
                                            cudaStream_t st) {
  constexpr bool kFew = !std::is_same<Args, MmaArgs>::value;
  Args a;
  a.tokens = f.rows;
  a.segments = stage == kFfnGradX ? 2 : 1;
  a.dim = f.dim;
  a.keep_bits = f.keep_bits;
  a.act = f.act;
  a.grad_f32 = f.grad_f32;
  a.record = h->record;
  a.nt = plan.nt;
  a.split = plan.split;
  a.early = stage == kFfnOut || stage == kFfnGradX;
  const FfnStage as = stage == kFfnGradX ? kFfnOut : stage;
  const bool wide = stage == kFfnHidden, grads = stage == kFfnGradW;
  const int64_t N = wide || stage == kFfnGradHidden ? h->C : h->dim;   // columns of the product
  if (kFew) {
    a.tiles_m = (int)((N + 127) / 128);
    a.tiles_n = (int)((f.rows + plan.nt - 1) / plan.nt);
  } else {
    a.tiles_m = (int)(((grads ? h->C : f.rows) + 255) / 256);
    a.tiles_n = (int)(wide ? (N + 127) / 128 : (N + 255) / 256);
  }
  // rows of operands that run along the terms come 128 at a time, rows across them one a term, 64 at a time
  // (for few tokens, theirs as many as a tile has)
  const auto in_rows = [&](int k) {
    const bool tokens = as == kFfnOut ? k < 2 : k == 0;
    return grads ? 64 : kFew && tokens ? plan.nt : as == kFfnOut && k >= 2 ? 64 : 128;
  };
  const int launches = (h->R + Args::kRanks - 1) / Args::kRanks, most = (h->R + launches - 1) / launches;
  for (int r0 = 0; r0 < h->R; r0 += most) {
    const int ranks = h->R - r0 < most ? h->R - r0 : most;
    for (int& level : a.level) level = 2;
    for (int i = 0; i < ranks; ++i) {
      const int r = r0 + i;
      const Matrices m(stage, f, r);
      bool ok = true;
      MmaRank<Args::kMaps>& to = a.rank[i];
      to.width = f.width(r);
      for (int k = 0; k < 2; ++k) to.scales[k] = f.scales[k][r];
      // a rank without columns has no terms: its operands are not looked at, wherever they lie
      for (int k = 0; k < (kFew ? 4 : 5); ++k)
        if (to.width && m.in[k].p && m.in[k].rows) ok = ok && encode(&to.map[k], h->dtype, m.in[k], 128, in_rows(k));
      for (int k = 0; k < 5; ++k) {
        const Matrix& o = m.out[k];
        to.rows[k] = static_cast<char*>(const_cast<void*>(o.p));
        to.stride[k] = o.stride * o.elem;
        if (!o.p) continue;
        const uintptr_t bits = o.bits();
        const int level = bits % 16 == 0 ? 2 : bits % 8 == 0 ? 1 : 0;
        if (level < a.level[k]) a.level[k] = level;
        if constexpr (!kFew)
          if (k < m.outs && level == 2 && o.rows && o.columns)
            ok = ok && encode(&to.map[first_rows(as) + k], h->dtype, o, 64, 32);
      }
      if (!ok) return record_error(RA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    }
    a.tiles = (int64_t)a.tiles_m * a.tiles_n * (grads ? 3 * ranks : ranks);
    a.ring = a.tiles * plan.split <= h->sms ? kFewRingAlone : kFewRing;
    const bool bf16 = h->dtype == RA_BF16;
    cudaError_t e;
    if constexpr (kFew) e = bf16 ? launch_ffn_few<RA_BF16>(as, a, st) : launch_ffn_few<RA_F16>(as, a, st);
    else e = bf16 ? launch_ffn_mma<RA_BF16>(as, a, h->sms, st) : launch_ffn_mma<RA_F16>(as, a, h->sms, st);
    if (e != cudaSuccess) return cuda_error(e, "feed-forward launch");
  }
  return RA_OK;
}

ra_status run(ra_ffn_handle h, FfnStage stage, const FfnArgs& f, cudaStream_t st) {
  uintptr_t operands = 0;
  for (int r = 0; r < h->ranks; ++r) {
    const Matrices m(stage, f, r);
    for (const Matrix& o : m.in)
      if (o.p) operands |= o.bits();
  }
  if (operands % 16) {
    const cudaError_t e = launch_ffn_simple(h->dtype, stage, f, h->sms, st);
    return e == cudaSuccess ? RA_OK : cuda_error(e, "feed-forward launch");
  }
  if (!encoder()) return record_error(RA_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  const Plan plan = plan_of(h, stage, f.rows, f.keep_bits);
  if (!plan.few) return run_planned<MmaArgs>(h, stage, plan, f, st);
  return h->R <= kFewRanks ? run_planned<FewArgs<kFewRanks>>(h, stage, plan, f, st)
                           : run_planned<FewArgs<kMaxRanks>>(h, stage, plan, f, st);
}

// What the handles of a device know of its record.  Whoever asks takes what is
// new there; every handle is told once.
struct Reports {
  std::mutex lock;
  uint32_t counted = 0;      // the record's count when it was last read
  uint64_t times = 0;        // how often that was a new one
  ra_device_error last = {};
  uint64_t seen_now() {
    std::lock_guard<std::mutex> hold(lock);
    return times;
  }
  cudaError_t read(WaitRecord* record, cudaStream_t st) {
    WaitRecord got;
    cudaError_t e = cudaMemcpyAsync(&got, record, sizeof(got), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess || got.count == counted) return e;
    counted = got.count;
    ++times;
    last = got.first;
    if (!last.code) last = {2, -1, -1, -1, -1, 0, 0, 0};   // another came between the last reading and its clearing
    e = cudaMemsetAsync(&record->first, 0, sizeof(record->first), st);
    return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
  }
};

Reports& reports_of(int device) {
  static Reports all[64];
  return all[device & 63];
}

ra_status ffn_create(int R, int dim, size_t inner, ra_dtype dtype, int act, ra_dtype grad_dtype, ra_ffn_handle* out) {
  if (!out) return record_error(RA_ERR_INVALID, "NULL handle pointer");
  if (R < 1 || R > kMaxRanks) return record_error(RA_ERR_INVALID, "R=%d outside [1, %d]", R, kMaxRanks);
  if (dim < 1 || dim > kMaxDim) return record_error(RA_ERR_INVALID, "dim=%d outside [1, %d]", dim, kMaxDim);
  if (inner < 1 || inner > (size_t)kMaxInner)
    return record_error(RA_ERR_INVALID, "inner=%zu outside [1, %d]", inner, kMaxInner);
  if (dtype != RA_BF16 && dtype != RA_F16)
    return record_error(RA_ERR_UNSUPPORTED, "dtype %d: bf16 or f16 expected", (int)dtype);
  if (grad_dtype != RA_F32 && grad_dtype != dtype)
    return record_error(RA_ERR_UNSUPPORTED, "gradient dtype %d: f32 or the block's type expected", (int)grad_dtype);
  if (act != RA_SILU && act != RA_GELU) return record_error(RA_ERR_INVALID, "activation %d", act);
  int dev = -1, sms = 0;
  RA_TRY(device_of(&dev, &sms));
  WaitRecord* record = nullptr;
  const cudaError_t e = ffn_wait_record(&record);
  if (e != cudaSuccess) return cuda_error(e, "error record");
  ra_ffn_ctx* h = new (std::nothrow) ra_ffn_ctx();
  if (!h) return record_error(RA_ERR_OOM, "host allocation failed");
  h->record = record;
  h->seen = reports_of(dev).seen_now();
  h->R = R;
  h->dim = dim;
  h->inner = (int)inner;
  h->C = (h->inner + R - 1) / R;
  h->ranks = (h->inner + h->C - 1) / h->C;
  h->device = dev;
  h->sms = sms;
  h->dtype = dtype;
  h->grad_dtype = grad_dtype;
  h->act = act;
  *out = h;
  return RA_OK;
}

ra_status ffn_forward(ra_ffn_handle h, const ra_ffn_forward_args* g, cudaStream_t st) {
  RA_TRY(check_ffn(h, g));
  if (g->keep_bits != 0 && g->keep_bits != 8 && g->keep_bits != 16)
    return record_error(RA_ERR_INVALID, "keep_bits=%d: 0, 8 or 16 expected", g->keep_bits);
  RA_TRY(check_ranks("xs", g->xs, h->R));
  if (g->rows == 0) return RA_OK;
  RA_TRY(check_ffn_rows(g->rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  FfnArgs a = args_of(h, g->rows);
  a.keep_bits = g->keep_bits;
  FfnBuffers buf(h->device, h->check_pointers, g->rows);
  buf.also(h->record, sizeof(*h->record));
  RA_TRY(add_ranks(h, buf, "x", g->x, g->xs, g->x_stride, false, a.x, &a.x_stride));
  const Shards weights[3] = {{"w_gate", g->w_gate, g->w_gate_strides, 2, true, false},
                             {"w_up", g->w_up, g->w_up_strides, 2, true, false},
                             {"w_down", g->w_down, g->w_down_strides, 2, true, false}};
  for (int k = 0; k < 3; ++k)
    RA_TRY(add_shards(h, buf, g->rows, weights[k], const_cast<void**>(a.w[k]), a.w_stride[k]));
  RA_TRY(add_shards(h, buf, g->rows, {"hidden", (const void* const*)g->hidden, g->hidden_strides, 2, false, true},
                    a.hidden, a.hidden_stride));
  RA_TRY(add_ranks(h, buf, "out", (const void* const*)g->out, h->R, g->out_stride, true,
                   const_cast<const void**>(a.out), &a.out_stride));
  if (g->keep_bits)
    RA_TRY(add_kept(h, buf, g->rows, g->keep_bits, true, (const void* const*)g->gate, g->gate_strides,
                    (const void* const*)g->up, g->up_strides, (const float* const*)g->gate_scales,
                    (const float* const*)g->up_scales, &a));
  RA_TRY(buf.check());
  RA_TRY(run(h, kFfnHidden, a, st));
  return run(h, kFfnOut, a, st);
}

ra_status ffn_backward(ra_ffn_handle h, const ra_ffn_backward_args* g, cudaStream_t st) {
  RA_TRY(check_ffn(h, g));
  if (g->keep_bits != 8 && g->keep_bits != 16)
    return record_error(RA_ERR_INVALID, "keep_bits=%d: 8 or 16 expected", g->keep_bits);
  if (g->grad_w_down && !g->hidden) return record_error(RA_ERR_INVALID, "grad_w_down without hidden");
  RA_TRY(check_ranks("grads", g->grads, h->R));
  const bool need_x = g->grad_w_gate || g->grad_w_up;
  if (need_x) RA_TRY(check_ranks("xs", g->xs, h->R));
  RA_TRY(check_ffn_rows(g->rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  FfnArgs a = args_of(h, g->rows);
  a.keep_bits = g->keep_bits;
  const size_t gb = bytes_of(h->grad_dtype);
  FfnBuffers buf(h->device, h->check_pointers, g->rows);
  buf.also(h->record, sizeof(*h->record));
  const Shards grads[3] = {{"grad_w_gate", (const void* const*)g->grad_w_gate, g->grad_w_gate_strides, gb, true, true},
                           {"grad_w_up", (const void* const*)g->grad_w_up, g->grad_w_up_strides, gb, true, true},
                           {"grad_w_down", (const void* const*)g->grad_w_down, g->grad_w_down_strides, gb, true, true}};
  for (int k = 0; k < 3; ++k)
    if (grads[k].at) RA_TRY(add_shards(h, buf, g->rows, grads[k], a.grad_w[k], a.grad_w_stride[k]));
  const bool any_w = g->grad_w_gate || g->grad_w_up || g->grad_w_down;
  if (g->rows) {
    RA_TRY(add_ranks(h, buf, "grad_out", g->grad_out, g->grads, g->grad_out_stride, false, a.grad_out,
                     &a.grad_out_stride));
    if (need_x) RA_TRY(add_ranks(h, buf, "x", g->x, g->xs, g->x_stride, false, a.x, &a.x_stride));
    const Shards weights[3] = {{"w_gate", g->w_gate, g->w_gate_strides, 2, true, false},
                               {"w_up", g->w_up, g->w_up_strides, 2, true, false},
                               {"w_down", g->w_down, g->w_down_strides, 2, true, false}};
    for (int k = 0; k < 3; ++k)
      if (k == 2 || g->grad_x)
        RA_TRY(add_shards(h, buf, g->rows, weights[k], const_cast<void**>(a.w[k]), a.w_stride[k]));
    RA_TRY(add_kept(h, buf, g->rows, g->keep_bits, false, g->gate, g->gate_strides, g->up, g->up_strides,
                    g->gate_scales, g->up_scales, &a));
    if (g->hidden)
      RA_TRY(add_shards(h, buf, g->rows, {"hidden", (const void* const*)g->hidden, g->hidden_strides, 2, false, true},
                        a.hidden, a.hidden_stride));
    const bool in_place = g->keep_bits == 16;
    RA_TRY(add_shards(h, buf, g->rows, {"grad_gate", (const void* const*)g->grad_gate, g->grad_gate_strides, 2, false,
                                        true, in_place ? g->gate : nullptr},
                      a.grad_pre[0], a.grad_pre_stride[0]));
    RA_TRY(add_shards(h, buf, g->rows, {"grad_up", (const void* const*)g->grad_up, g->grad_up_strides, 2, false, true,
                                        in_place ? g->up : nullptr},
                      a.grad_pre[1], a.grad_pre_stride[1]));
    if (g->grad_x)
      RA_TRY(add_ranks(h, buf, "grad_x", (const void* const*)g->grad_x, h->R, g->grad_x_stride, true,
                       const_cast<const void**>(a.out), &a.out_stride));
  }
  RA_TRY(buf.check());
  if (g->rows) {
    RA_TRY(run(h, kFfnGradHidden, a, st));
    if (g->grad_x) RA_TRY(run(h, kFfnGradX, a, st));
  }
  return any_w ? run(h, kFfnGradW, a, st) : RA_OK;
}

// ---------------------------------------------------------------- kept rows

ra_status ckpt_create(int dim, ra_dtype dtype, ra_dtype ndtype, ra_dtype pdtype, ra_ckpt_handle* out) {
  if (!out) return record_error(RA_ERR_INVALID, "NULL handle pointer");
  if (dim < 1 || dim > kMaxInner) return record_error(RA_ERR_INVALID, "dim=%d outside [1, %d]", dim, kMaxInner);
  if (!is_float(dtype)) return record_error(RA_ERR_UNSUPPORTED, "dtype %d: f32, bf16 or f16 expected", (int)dtype);
  if (!is_float(ndtype))
    return record_error(RA_ERR_UNSUPPORTED, "normalised dtype %d: f32, bf16 or f16 expected", (int)ndtype);
  if (pdtype != RA_F32 && pdtype != ndtype)
    return record_error(RA_ERR_UNSUPPORTED, "parameter dtype %d: f32 or the normalised rows' type expected",
                        (int)pdtype);
  int dev = -1, sms = 0;
  RA_TRY(device_of(&dev, &sms));
  ra_ckpt_ctx* h = new (std::nothrow) ra_ckpt_ctx();
  if (!h) return record_error(RA_ERR_OOM, "host allocation failed");
  h->dim = dim;
  h->device = dev;
  h->sms = sms;
  h->dtype = dtype;
  h->normed_dtype = ndtype;
  h->param_dtype = pdtype;
  *out = h;
  return RA_OK;
}

// Rows that start on 16-byte boundaries (codes: 8), whole groups of 8 columns.
bool rows_wide(const void* p, size_t stride_bytes, size_t rows, size_t to) {
  return ((uintptr_t)p | (rows > 1 ? stride_bytes : 0)) % to == 0;
}

ra_status ckpt_store(ra_ckpt_handle h, const ra_ckpt_store_args* g, cudaStream_t st) {
  RA_TRY(!h ? record_error(RA_ERR_INVALID, "NULL handle") : RA_OK);
  if (!g) return record_error(RA_ERR_INVALID, "NULL arguments");
  if (g->rows == 0) return RA_OK;
  RA_TRY(check_rows(g->rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  const size_t dim = (size_t)h->dim, b = bytes_of(h->dtype), groups = (dim + kGroup - 1) / kGroup;
  size_t stride = g->stride, codes_stride = g->codes_stride;
  Buffers buf(h->device, h->check_pointers, g->rows);
  RA_TRY(buf.add("values", -1, g->values, b, dim, &stride, false));
  RA_TRY(buf.add("codes", -1, g->codes, 1, dim, &codes_stride, true));
  RA_TRY(buf.flat("scales", g->scales, 4, g->rows * groups, true));
  RA_TRY(buf.check());
  CkptArgs a{};
  a.values = const_cast<void*>(g->values);
  a.codes = reinterpret_cast<int8_t*>(g->codes);
  a.scales = g->scales;
  a.rows = (int64_t)g->rows;
  a.stride = (int64_t)stride;
  a.codes_stride = (int64_t)codes_stride;
  a.dim = h->dim;
  a.set_groups();
  const bool wide = dim % 8 == 0 && rows_wide(g->values, stride * b, g->rows, 16) &&
                    rows_wide(g->codes, codes_stride, g->rows, 8);
  const cudaError_t e = launch_ckpt_store(h->dtype, wide, a, h->sms, st);
  return e == cudaSuccess ? RA_OK : cuda_error(e, "checkpoint store launch");
}

ra_status ckpt_load(ra_ckpt_handle h, const ra_ckpt_load_args* g, cudaStream_t st) {
  RA_TRY(!h ? record_error(RA_ERR_INVALID, "NULL handle") : RA_OK);
  if (!g) return record_error(RA_ERR_INVALID, "NULL arguments");
  if (g->rows == 0) return RA_OK;
  if (!g->values && !g->normed) return record_error(RA_ERR_INVALID, "neither values nor normed");
  RA_TRY(check_rows(g->rows));
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
  const size_t dim = (size_t)h->dim, b = bytes_of(h->dtype), nb = bytes_of(h->normed_dtype),
               pb = bytes_of(h->param_dtype), groups = (dim + kGroup - 1) / kGroup;
  size_t stride = g->stride, codes_stride = g->codes_stride, normed_stride = g->normed_stride;
  Buffers buf(h->device, h->check_pointers, g->rows);
  RA_TRY(buf.add("codes", -1, g->codes, 1, dim, &codes_stride, false));
  RA_TRY(buf.flat("scales", g->scales, 4, g->rows * groups, false));
  bool wide = dim % 8 == 0 && rows_wide(g->codes, codes_stride, g->rows, 8);
  CkptArgs a{};
  if (g->values) {
    RA_TRY(buf.add("values", -1, g->values, b, dim, &stride, true));
    wide = wide && rows_wide(g->values, stride * b, g->rows, 16);
  }
  if (g->normed) {
    RA_TRY(buf.flat("rstd", g->rstd, 4, g->rows, false));
    RA_TRY(buf.flat("weight", g->weight, pb, dim, false));
    RA_TRY(buf.add("normed", -1, g->normed, nb, dim, &normed_stride, true));
    wide = wide && rows_wide(g->normed, normed_stride * nb, g->rows, 16) && (uintptr_t)g->weight % 16 == 0;
    a.rstd = g->rstd;
    a.weight = g->weight;
  }
  RA_TRY(buf.check());
  a.values = g->values;
  a.codes = reinterpret_cast<int8_t*>(const_cast<signed char*>(g->codes));
  a.scales = const_cast<float*>(g->scales);
  a.normed = g->normed;
  a.rows = (int64_t)g->rows;
  a.stride = (int64_t)stride;
  a.codes_stride = (int64_t)codes_stride;
  a.normed_stride = (int64_t)normed_stride;
  a.dim = h->dim;
  a.set_groups();
  const cudaError_t e = launch_ckpt_load(h->dtype, h->normed_dtype, h->param_dtype, wide, a, h->sms, st);
  return e == cudaSuccess ? RA_OK : cuda_error(e, "checkpoint load launch");
}

}  // namespace

extern "C" {

ra_status ra_ffn_create(int R, int dim, size_t inner, ra_dtype dtype, ra_activation activation, ra_dtype grad_dtype,
                        ra_ffn_handle* out) {
  return guarded([&] { return ffn_create(R, dim, inner, dtype, (int)activation, grad_dtype, out); });
}

ra_status ra_ffn_destroy(ra_ffn_handle h) {
  delete h;
  return RA_OK;
}

ra_status ra_ffn_set_option(ra_ffn_handle h, int key, long long value) {
  return guarded([&] { return set_option(h, key, value); });
}

ra_status ra_ffn_get_device_status(ra_ffn_handle h, void* stream, ra_device_error* err) {
  return guarded([&]() -> ra_status {
    if (!h) return record_error(RA_ERR_INVALID, "NULL handle");
    OnDevice on(h->device);
    if (on.status != cudaSuccess) return cuda_error(on.status, "cudaSetDevice");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(st, &capture);
    if (e != cudaSuccess) return cuda_error(e, "cudaStreamIsCapturing");
    if (capture != cudaStreamCaptureStatusNone)   // to wait for it would end the capture
      return record_error(RA_ERR_UNSUPPORTED, "the status of a stream that is being captured");
    Reports& reports = reports_of(h->device);
    std::lock_guard<std::mutex> hold(reports.lock);
    e = reports.read(h->record, st);
    if (e != cudaSuccess) return cuda_error(e, "error record");
    const bool news = h->seen != reports.times;
    h->seen = reports.times;
    if (err) *err = news ? reports.last : ra_device_error{};
    if (news) return record_error(RA_ERR_TIMEOUT, "a device wait of a feed-forward product gave up");
    return RA_OK;
  });
}

ra_status ra_ffn_forward(ra_ffn_handle h, const ra_ffn_forward_args* args, void* stream) {
  return guarded([&] { return ffn_forward(h, args, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_ffn_backward(ra_ffn_handle h, const ra_ffn_backward_args* args, void* stream) {
  return guarded([&] { return ffn_backward(h, args, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_ckpt_create(int dim, ra_dtype dtype, ra_dtype normed_dtype, ra_dtype param_dtype, ra_ckpt_handle* out) {
  return guarded([&] { return ckpt_create(dim, dtype, normed_dtype, param_dtype, out); });
}

ra_status ra_ckpt_destroy(ra_ckpt_handle h) {
  delete h;
  return RA_OK;
}

ra_status ra_ckpt_set_option(ra_ckpt_handle h, int key, long long value) {
  return guarded([&] { return set_option(h, key, value); });
}

ra_status ra_ckpt_store(ra_ckpt_handle h, const ra_ckpt_store_args* args, void* stream) {
  return guarded([&] { return ckpt_store(h, args, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_ckpt_load(ra_ckpt_handle h, const ra_ckpt_load_args* args, void* stream) {
  return guarded([&] { return ckpt_load(h, args, static_cast<cudaStream_t>(stream)); });
}

#ifdef RA_DEBUG_BOUNDS
// Debug builds: the plan of this host thread's next calls, but for the weights' gradients, which have one;
// among those that the estimate can come to. split 0: the estimate's again.
ra_status ra_debug_ffn_plan(int few, int nt, int split) {
  const bool valid = split == 0 || (!few && split == 1) ||
                     (few && nt >= 16 && nt <= 128 && nt % 16 == 0 &&
                      (split == 1 || ((split == 2 || split == 4 || split == 8) && nt <= kFewMostSplit)));
  if (!valid) return RA_ERR_INVALID;
  debug_plan = {few != 0, nt, split};
  return RA_OK;
}

// What a wait that gives up in a call of this handle writes down.
ra_status ra_debug_ffn_give_up(ra_ffn_handle h, void* stream) {
  return guarded([&]() -> ra_status {
    FfnBuffers buf(h->device, false, 0);
    buf.also(h->record, sizeof(*h->record));
    RA_TRY(buf.check());
    const cudaError_t e = launch_ffn_give_up(h->record, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RA_OK : cuda_error(e, "give-up launch");
  });
}
#endif

}  // extern "C"
