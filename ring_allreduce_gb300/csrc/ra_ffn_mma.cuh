// ra_ffn_mma.cuh -- the feed-forward block's products on the tensor cores.
//
// One kernel for all of them: D = A B with 16-bit operands and binary32 sums,
// and an epilogue for each (FfnStage).  A pair of CTAs on two SMs takes a tile
// of 256 x 256: each holds 128 rows of A and 128 columns of B of every 64
// terms, so that a byte fetched into shared memory serves 256 products; the
// instruction (M 256, N 256, 16 terms) reads both CTAs' halves.  The gated
// projections share one tile: its first 128 columns are the gate's, in one
// CTA, the other 128 the up projection's, in the other, and every thread of
// the epilogue holds both of its row.
//
// Roles in a CTA of 320 threads, one CTA an SM, tiles taken by turns:
//   warp 8   one thread copies operand tiles by tensor map into a ring of
//            kStages stages (out of range: zeros), the pair's bytes counted on
//            the first CTA's barrier
//   warp 9   of the first CTA: one thread issues the products, and frees
//            stages and hands over sums by commits to both CTAs' barriers
//   warps 0-3, 4-7  epilogue of the tiles whose sums lie in the first and in
//            the second 256 columns of tensor memory: the products of the next tile
//            run while one is written out; thread = row
// Operands are taken as they lie: rows along the terms (projections, dh) or
// across them (everything else); nothing is transposed or laid out anew.
#pragma once

#include "ra_ffn.cuh"
#include "ra_ffn_mma.h"
#include "ra_tensor.cuh"

namespace ra {

namespace {

constexpr int kBlockM = 128, kBlockN = 128, kBlockK = 64;   // of one CTA's operands
constexpr int kStages = 6;
constexpr int kOperandBytes = kBlockM * kBlockK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kMmaThreads = 320;
constexpr int kTileN = 2 * kBlockN;
constexpr uint32_t kTmemColumns = 2 * kTileN;
constexpr int kMmaShared = kStages * kStageBytes + 1024;   // and up to 1024 to align

struct MmaShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t sums_full[2], sums_empty[2];
  uint32_t tmem;
  int gave_up;
};

// What a tile is: its job (rank, and which weight), its place and its terms.
struct Tile {
  int r, which;        // which: of the weights' gradients
  int m0, n0;          // first row and column of the pair's
  int m, n;            // rows and columns there are
  int steps, half;     // steps of kBlockK terms; those of the first segment
};

template <int Stage> __device__ __forceinline__ bool tile_at(const MmaArgs& a, int64_t t, Tile* p) {
  const int64_t per = (int64_t)a.tiles_m * a.tiles_n;
  const int job = (int)(t / per);
  const int u = (int)(t - job * per);
  p->r = Stage == kFfnGradW ? job / 3 : job;
  p->which = Stage == kFfnGradW ? job - 3 * p->r : 0;
  // eight rows of tiles at a time, down before across: the tiles in flight share operands in L2
  const int band = u / (8 * a.tiles_n), top = band * 8, high = min(8, a.tiles_m - top);
  const int v = u - band * 8 * a.tiles_n;
  p->m0 = (top + v % high) * 256;
  constexpr int cols = Stage == kFfnHidden ? kBlockN : kTileN;
  p->n0 = v / high * cols;
  const FfnArgs& f = a.f;
  const int width = f.width(p->r);
  if constexpr (Stage == kFfnHidden || Stage == kFfnGradHidden) {
    p->m = (int)f.rows;
    p->n = width;
    p->steps = (f.dim + kBlockK - 1) / kBlockK;
  } else if constexpr (Stage == kFfnOut) {
    p->m = (int)f.rows;
    p->n = f.dim;
    p->half = (width + kBlockK - 1) / kBlockK;
    p->steps = p->half * a.segments;
  } else {
    p->m = width;
    p->n = f.dim;
    p->steps = (int)((f.rows + kBlockK - 1) / kBlockK);
    if (!f.grad_w[p->which][p->r]) return false;
  }
  return p->m0 < p->m && p->n0 < p->n;
}

// 32 columns of a row from `v`, of which `left` exist.  vec: 16-byte stores fit.
template <class D>
__device__ __forceinline__ void put_chunk(typename D::T* to, const float* v, int left, bool vec) {
  constexpr int kVec = D::kVec;
#pragma unroll
  for (int q = 0; q < 32 / kVec; ++q) {
    if (vec && left >= (q + 1) * kVec) {
      uint4* p = reinterpret_cast<uint4*>(to + q * kVec);
      if (RA_ACCESS_OK(p, 16u, 2u)) *p = pack<D>(v + q * kVec);
    } else {
#pragma unroll
      for (int j = q * kVec; j < (q + 1) * kVec; ++j)
        if (j < left) st_g(to + j, narrow<D>(v[j]));
    }
  }
}

__device__ __forceinline__ void put_codes(int8_t* to, const float* v, float by, int left, bool vec) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (vec && left >= (q + 1) * 16) {
      uint4* p = reinterpret_cast<uint4*>(to + q * 16);
      const float* x = v + q * 16;
      if (RA_ACCESS_OK(p, 16u, 2u))
        *p = make_uint4(codes4(x, by), codes4(x + 4, by), codes4(x + 8, by), codes4(x + 12, by));
    } else {
#pragma unroll
      for (int j = q * 16; j < (q + 1) * 16; ++j)
        if (j < left) st_g(to + j, code_of(v[j], by));
    }
  }
}

__device__ __forceinline__ void get_codes(const int8_t* from, float scale, int left, bool vec, float* v) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t w[4] = {};
    if (vec && left >= (q + 1) * 16) {
      const uint4 x = ld_plain(reinterpret_cast<const uint4*>(from + q * 16));
      w[0] = x.x;
      w[1] = x.y;
      w[2] = x.z;
      w[3] = x.w;
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (q * 16 + j < left) w[j / 4] |= (uint32_t)(uint8_t)ld_g(from + q * 16 + j) << (8 * (j % 4));
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[q * 16 + j] = code_value(bias_codes(w[j / 4]), j % 4) * scale;
  }
}

template <class D>
__device__ __forceinline__ void get_chunk(const typename D::T* from, int left, bool vec, float* v) {
  constexpr int kVec = D::kVec;
#pragma unroll
  for (int q = 0; q < 32 / kVec; ++q) {
    if (vec && left >= (q + 1) * kVec) {
      unpack<D>(ld_plain(reinterpret_cast<const uint4*>(from + q * kVec)), v + q * kVec);
    } else {
#pragma unroll
      for (int j = q * kVec; j < (q + 1) * kVec; ++j) v[j] = j < left ? widen<D>(ld_g(from + j)) : 0.0f;
    }
  }
}

// A chunk of 32 sums of this thread's row.
__device__ __forceinline__ void get_sums(uint32_t tmem, float* v) {
  __syncwarp();   // lanes beyond the last row have left the chunk before early
  tmem_load32(tmem, reinterpret_cast<uint32_t*>(v));
}

// One row of a finished tile.  `tmem`: its sums in this warp's lanes.
template <class D, int Stage, int Act>
__device__ void write_row(const MmaArgs& a, const Tile& p, uint32_t tmem, int64_t row) {
  using T = typename D::T;
  const FfnArgs& f = a.f;
  const int r = p.r;
  const bool in = row < p.m;
  if constexpr (Stage == kFfnHidden) {
    const int groups = (p.n + kGroup - 1) / kGroup;
    float by[2] = {};
    if (f.keep_bits == 8) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float most = 0.0f;
#pragma unroll 1
        for (int c = 0; c < kBlockN; c += 32) {
          float v[32];
          get_sums(tmem + b * kBlockN + c, v);
          tmem_wait_loads();
#pragma unroll
          for (int j = 0; j < 32; ++j) most = max_nan(most, fabsf(v[j]));
        }
        float scale;
        group_scale(most, &scale, &by[b]);
        if (in) st_g(f.scales[b][r] + row * groups + p.n0 / kGroup, scale);
      }
    }
    // a row of a vector of heads' worth of columns: 32 at a time
#pragma unroll 1
    for (int c = 0; c < kBlockN; c += 32) {
      const int col = p.n0 + c, left = p.n - col;
      if (left <= 0) break;
      float g[32], u[32], h[32];
      get_sums(tmem + c, g);
      get_sums(tmem + kBlockN + c, u);
      tmem_wait_loads();
      if (!in) continue;
      if (f.keep_bits == 8) {
        put_codes((int8_t*)f.kept[0][r] + row * f.kept_stride[0][r] + col, g, by[0], left, a.vec & kVecKept);
        put_codes((int8_t*)f.kept[1][r] + row * f.kept_stride[1][r] + col, u, by[1], left, a.vec & kVecKept);
      } else if (f.keep_bits == 16) {
        put_chunk<D>((T*)f.kept[0][r] + row * f.kept_stride[0][r] + col, g, left, a.vec & kVecKept);
        put_chunk<D>((T*)f.kept[1][r] + row * f.kept_stride[1][r] + col, u, left, a.vec & kVecKept);
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float act, slope;
        activate<Act, false>(g[j], &act, &slope);
        h[j] = act * u[j];
      }
      put_chunk<D>((T*)f.hidden[r] + row * f.hidden_stride[r] + col, h, left, a.vec & kVecHidden);
    }
  } else if constexpr (Stage == kFfnGradHidden) {
    const int groups = (p.n + kGroup - 1) / kGroup;
#pragma unroll 1
    for (int c = 0; c < kTileN; c += 32) {
      const int col = p.n0 + c, left = p.n - col;
      if (left <= 0) break;
      float dh[32], g[32], u[32];
      get_sums(tmem + c, dh);
      if (in) {
        if (f.keep_bits == 8) {
          const int64_t at = row * groups + col / kGroup;
          get_codes((const int8_t*)f.kept[0][r] + row * f.kept_stride[0][r] + col, ld_g(f.scales[0][r] + at), left,
                    a.vec & kVecKept, g);
          get_codes((const int8_t*)f.kept[1][r] + row * f.kept_stride[1][r] + col, ld_g(f.scales[1][r] + at), left,
                    a.vec & kVecKept, u);
        } else {
          get_chunk<D>((const T*)f.kept[0][r] + row * f.kept_stride[0][r] + col, left, a.vec & kVecKept, g);
          get_chunk<D>((const T*)f.kept[1][r] + row * f.kept_stride[1][r] + col, left, a.vec & kVecKept, u);
        }
      }
      tmem_wait_loads();
      if (!in) continue;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float act, slope;
        activate<Act, true>(g[j], &act, &slope);
        g[j] = dh[j] * u[j] * slope;
        u[j] = act * u[j];
        dh[j] = dh[j] * act;
      }
      put_chunk<D>((T*)f.grad_pre[0][r] + row * f.grad_pre_stride[0][r] + col, g, left, a.vec & kVecPre);
      put_chunk<D>((T*)f.grad_pre[1][r] + row * f.grad_pre_stride[1][r] + col, dh, left, a.vec & kVecPre);
      if (f.hidden[r])
        put_chunk<D>((T*)f.hidden[r] + row * f.hidden_stride[r] + col, u, left, a.vec & kVecHidden);
    }
  } else {
#pragma unroll 1
    for (int c = 0; c < kTileN; c += 32) {
      const int col = p.n0 + c, left = p.n - col;
      if (left <= 0) break;
      float v[32];
      get_sums(tmem + c, v);
      tmem_wait_loads();
      if (p.steps == 0) {   // a sum of nothing: the columns hold what an earlier tile left
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
      }
      if (!in) continue;
      if constexpr (Stage == kFfnGradW) {
        const int64_t at = row * f.grad_w_stride[p.which][r] + col;
        if (f.grad_f32)
          put_chunk<DF32>((float*)f.grad_w[p.which][r] + at, v, left, a.vec & kVecGradW);
        else
          put_chunk<D>((T*)f.grad_w[p.which][r] + at, v, left, a.vec & kVecGradW);
      } else {
        put_chunk<D>((T*)f.out[r] + row * f.out_stride + col, v, left, a.vec & kVecOut);
      }
    }
  }
}

}  // namespace

template <class D, int Stage, int Act>
__global__ void __launch_bounds__(kMmaThreads, 1) ffn_mma_kernel(const __grid_constant__ MmaArgs a) {
  // operands whose rows run across the terms: 64 terms of 64 elements a box, two boxes
  constexpr bool kAMn = Stage == kFfnGradW, kBMn = Stage == kFfnOut || Stage == kFfnGradW;
  constexpr uint32_t kDesc = product_desc(std::is_same<D, DBF16>::value, kAMn, kBMn, 2 * kBlockM, kTileN);
  extern __shared__ uint8_t dynamic[];
  __shared__ MmaShared sh;
  const uint32_t ring = (smem_addr(dynamic) + 1023u) & ~1023u;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t cta = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.sums_full[b], 1);
      mbar_init(&sh.sums_empty[b], 8);   // four warps of each CTA
    }
    sh.gave_up = 0;
    fence_mbar_init();
  }
  after_predecessor();
  if (warp == 9) tmem_alloc<2>(&sh.tmem, kTmemColumns);
  tensor_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tensor_fence_after();
  const uint32_t tmem = sh.tmem;
  const Waits wait{&sh.gave_up, a.err, Stage};
  const int64_t tiles = a.tiles, step = gridDim.x / 2;
  Tile p;

  if (warp == 8) {
    if (lane == 0) {
      uint32_t s = 0, round = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x / 2; ok && t < tiles; t += step) {
        if (!tile_at<Stage>(a, t, &p)) continue;
        const int m = p.m0 + (int)cta * kBlockM;
        const int n = p.n0 + (Stage == kFfnHidden ? 0 : (int)cta * kBlockN);
        for (int k = 0; k < p.steps; ++k) {
          ok = wait(&sh.empty[s], (round & 1) ^ 1, 0);
          if (!ok) break;
          const CUtensorMap *ma, *mb;
          int at = k * kBlockK;
          if constexpr (Stage == kFfnHidden) {
            ma = &a.a[0][p.r];
            mb = &a.b[cta][p.r];
          } else if constexpr (Stage == kFfnOut) {
            const int seg = k >= p.half;
            ma = &a.a[seg][p.r];
            mb = &a.b[seg][p.r];
            at -= seg * p.half * kBlockK;
          } else if constexpr (Stage == kFfnGradHidden) {
            ma = &a.a[0][p.r];
            mb = &a.b[0][p.r];
          } else {
            ma = &a.a[p.which][p.r];
            mb = &a.b[p.which == 2][p.r];
          }
          if (cta == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * kStageBytes);
          const uint32_t bar = in_cta(smem_addr(&sh.full[s]), 0);
          const uint32_t to = ring + s * kStageBytes;
          if constexpr (kAMn) {
            load_box<2>(to, ma, m, at, bar);
            load_box<2>(to + kOperandBytes / 2, ma, m + 64, at, bar);
          } else {
            load_box<2>(to, ma, at, m, bar);
          }
          if constexpr (kBMn) {
            load_box<2>(to + kOperandBytes, mb, n, at, bar);
            load_box<2>(to + kOperandBytes + kOperandBytes / 2, mb, n + 64, at, bar);
          } else {
            load_box<2>(to + kOperandBytes, mb, at, n, bar);
          }
          if (++s == kStages) {
            s = 0;
            ++round;
          }
        }
      }
      // until the last stages are free again: nothing arrives here any more
      for (int k = 0; ok && k < kStages; ++k) {
        ok = wait(&sh.empty[s], (round & 1) ^ 1, 1);
        if (++s == kStages) {
          s = 0;
          ++round;
        }
      }
    }
  } else if (warp == 9) {
    if (cta == 0 && lane == 0) {
      uint32_t s = 0, round = 0, it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x / 2; ok && t < tiles; t += step) {
        if (!tile_at<Stage>(a, t, &p)) continue;
        const uint32_t b = it & 1, to = tmem + b * kTileN;
        ok = wait(&sh.sums_empty[b], ((it >> 1) & 1) ^ 1, 2);
        if (!ok) break;
        tensor_fence_after();
        for (int k = 0; k < p.steps; ++k) {
          ok = wait(&sh.full[s], round & 1, 3);
          if (!ok) break;
          tensor_fence_after();
          const uint32_t at = ring + s * kStageBytes;
          const uint64_t da = operand_desc(at, kAMn ? kOperandBytes / 2 : 16, 1024);
          const uint64_t db = operand_desc(at + kOperandBytes, kBMn ? kOperandBytes / 2 : 16, 1024);
          // 16 terms on: 32 bytes along a row, or 16 rows of 128 bytes
#pragma unroll
          for (int j = 0; j < kBlockK / 16; ++j)
            multiply<2>(to, da + (uint64_t)(j * (kAMn ? 2048 : 32) >> 4), db + (uint64_t)(j * (kBMn ? 2048 : 32) >> 4),
                        kDesc, k > 0 || j > 0);
          commit<2>(&sh.empty[s]);
          if (++s == kStages) {
            s = 0;
            ++round;
          }
        }
        commit<2>(&sh.sums_full[b]);
        ++it;
      }
    }
  } else {
    const uint32_t b = warp / 4;
    uint32_t it = 0;
    for (int64_t t = blockIdx.x / 2; t < tiles; t += step) {
      if (!tile_at<Stage>(a, t, &p)) continue;
      if ((it++ & 1) != b) continue;
      if (!wait(&sh.sums_full[b], ((it - 1) >> 1) & 1, 4)) break;
      tensor_fence_after();
      const int64_t row = p.m0 + (int)cta * kBlockM + (warp % 4) * 32 + lane;
      write_row<D, Stage, Act>(a, p, tmem + b * kTileN + ((uint32_t)(warp % 4) * 32u << 16), row);
      tensor_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(in_cta(smem_addr(&sh.sums_empty[b]), 0));
    }
  }
  __syncwarp();
  __syncthreads();
  if (sh.gave_up) let_land();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (warp == 9) tmem_free<2>(tmem, kTmemColumns);
}

}  // namespace ra
