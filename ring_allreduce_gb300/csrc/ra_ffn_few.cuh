// ra_ffn_few.cuh -- the feed-forward block's products for few tokens.
//
// The weights are then most of what moves, so they take the tensor cores' long
// side: a CTA holds 128 of their rows (or columns) against `nt` tokens, 16 to
// 128, as D = W x^T with the weights' rows down tensor memory's lanes; of the
// gated projections both, 2 x nt columns of sums.  Where that makes few CTAs,
// the terms of a sum are split over a cluster: every CTA hands its partial sums
// of a share of the tokens to the CTA that finishes that share, through
// distributed shared memory, and they are added in the CTAs' order.
//
// One CTA an SM with a ring of 208 KB, or, where there are more, two with 104
// KB each: 20 to 30 MB of weights are in flight.  (Never more than two, which
// with 256 columns each always find room in tensor memory: a CTA that waited
// for that, while its cluster waited for it, could wait for ever.)
// Roles in a CTA of 320 threads: warps 0-7 epilogue, thread = weight row, four
// warps every other eight tokens; warp 8 copies; warp 9 issues the products.  A product whose predecessor in
// the stream is the call's own, which writes no weights, fetches its first weights
// before that has ended.
//
// What bounds it is DRAM where the weights are large: one token of 4096 x 16384
// in 8 ranks takes 67 us for 403 MB, 0.88 of the copy bandwidth, 37 tokens 75
// us (large tiles: 103 and 82).  Where they are not, a chain of steps: the
// predecessor's end 1 us, the first copy 1.5, the terms, a cluster's exchange
// 2 to 3, the epilogue 1: 7 us for a product of 1024 x 2048 a rank.
#pragma once

#include "ra_ffn.cuh"
#include "ra_ffn_mma.h"
#include "ra_tensor.cuh"

namespace ra {

namespace {

constexpr int kFewEpilogue = 8, kFewThreads = 32 * kFewEpilogue + 64, kFewRows = 128, kFewK = 64;

struct FewShared {
  uint64_t full[kFewMostStages], empty[kFewMostStages];
  uint64_t done;
  uint32_t most[4][2][128];   // of a warp's rows and a token, gate and up: the largest magnitude's bits
  uint32_t tmem;
  int gave_up;
};

__device__ __forceinline__ void st_cluster(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

}  // namespace

template <class D, int Stage, int Act, int Ranks>
__global__ void __launch_bounds__(kFewThreads, 2) ffn_few_kernel(const __grid_constant__ FewArgs<Ranks> a) {
  using T = typename D::T;
  constexpr bool kAMn = Stage == kFfnOut;   // the weights' rows run along the terms
  constexpr int kSums = few_sums(Stage);
  extern __shared__ uint8_t dynamic[];
  __shared__ FewShared sh;
  const uint32_t ring = (smem_addr(dynamic) + 1023u) & ~1023u;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, nt = a.nt;
  const int split = a.split, part = split > 1 ? (int)cluster_rank() : 0;
  const int stage_bytes = few_stage_bytes(Stage, nt), stages = min(a.ring / stage_bytes, kFewMostStages);
  // this CTA's tile: tokens run fastest, so that the CTAs that share weights run together
  const int64_t tile = blockIdx.x / split;
  const int per = a.tiles_m * a.tiles_n;
  const int r = (int)(tile / per), u = (int)(tile - (int64_t)r * per);
  const int m0 = u / a.tiles_n * kFewRows, t0 = u % a.tiles_n * nt;
  const auto& k = a.rank[r];
  const int width = k.width;
  const int m = Stage == kFfnOut ? a.dim : width;   // weight rows there are
  const int half = ((Stage == kFfnOut ? width : a.dim) + kFewK - 1) / kFewK;
  const int all = half * (Stage == kFfnOut ? a.segments : 1);
  const int first = (int)((int64_t)all * part / split), steps = (int)((int64_t)all * (part + 1) / split) - first;
  const bool some = m0 < m;
  const int maps = Stage == kFfnHidden ? 7 : Stage == kFfnGradHidden ? 3 : a.segments == 2 ? 15 : 5;
  if (threadIdx.x < 4 && some && width > 0 && maps >> threadIdx.x & 1) prefetch_map(&k.map[threadIdx.x]);

  uint32_t columns = 32;
  while (columns < (uint32_t)(kSums * nt)) columns *= 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.done, 1);
    sh.gave_up = 0;
    fence_mbar_init();
  }
  if (warp == kFewEpilogue + 1) tmem_alloc<1>(&sh.tmem, columns);
  tensor_fence_before();
  __syncthreads();
  tensor_fence_after();
  const uint32_t tmem = sh.tmem;
  if (!a.early) after_predecessor();   // what came before ran on beside all this
  const Waits wait{&sh.gave_up, a.record, 8 + Stage};

  if (warp == kFewEpilogue) {
    if (lane == 0) {
      const auto fetch = [&](int n, bool weights, bool tokens) {
        const int s = n % stages, step = first + n, seg = step >= half;
        const int at = (step - seg * half) * kFewK;
        uint32_t to = ring + s * stage_bytes;
        const uint32_t bar = smem_addr(&sh.full[s]);
        const int wa = Stage == kFfnOut ? 2 + seg : 1;
        if (weights) {
          if constexpr (kAMn) {
            load_box<1>(to, &k.map[wa], m0, at, bar);
            load_box<1>(to + kFewABytes / 2, &k.map[wa], m0 + 64, at, bar);
          } else {
#pragma unroll
            for (int i = 0; i < kSums; ++i) load_box<1>(to + i * kFewABytes, &k.map[wa + i], at, m0, bar);
          }
        }
        if (tokens) load_box<1>(to + kSums * kFewABytes, &k.map[seg], at, t0, bar);
      };
      int n = 0;
      if (a.early) {
        const int now = some ? min(stages, steps) : 0;
        for (; n < now; ++n) {
          mbar_arrive_expect_tx(&sh.full[n], stage_bytes);
          fetch(n, true, false);
        }
        after_predecessor();
        for (int i = 0; i < now; ++i) fetch(i, false, true);
      }
      for (; some && n < steps; ++n) {
        const int s = n % stages;
        if (!wait(&sh.empty[s], (n / stages & 1) ^ 1, 0)) break;
        mbar_arrive_expect_tx(&sh.full[s], stage_bytes);
        fetch(n, true, true);
      }
    } else if (a.early) {
      after_predecessor();
    }
  } else if (warp == kFewEpilogue + 1) {
    if (a.early) after_predecessor();
    if (lane == 0 && some) {
      const uint32_t desc = product_desc(std::is_same<D, DBF16>::value, kAMn, false, kFewRows, nt);
      bool ok = true;
      for (int n = 0; n < steps; ++n) {
        const int s = n % stages;
        ok = wait(&sh.full[s], n / stages & 1, 1);
        if (!ok) break;
        tensor_fence_after();
        const uint32_t at = ring + s * stage_bytes;
        const uint64_t db = operand_desc(at + kSums * kFewABytes, 16, 1024);
#pragma unroll
        for (int i = 0; i < kSums; ++i) {
          const uint64_t da = operand_desc(at + i * kFewABytes, kAMn ? kFewABytes / 2 : 16, 1024);
#pragma unroll
          for (int j = 0; j < kFewK / 16; ++j)
            multiply<1>(tmem + i * nt, da + (uint64_t)(j * (kAMn ? 2048 : 32) >> 4), db + (uint64_t)(j * 32 >> 4), desc,
                        n > 0 || j > 0);
        }
        commit<1>(&sh.empty[s]);
      }
      commit<1>(&sh.done);
    }
  } else {
    if (a.early) after_predecessor();
  }
  // every warp: the sums are whole (or a wait gave up, and what follows is of no use but ends)
  __syncwarp();
  if (some) wait.warp(&sh.done, 0, 2);
  tensor_fence_after();
  const uint32_t mine = tmem + ((uint32_t)(warp % 4) * 32u << 16);
  const int row = (warp % 4) * 32 + lane;
  const int turn = warp / 4 * 8;   // the first token that this warp takes, eight of every sixteen
  const int live = (int)min((int64_t)nt, a.tokens - t0);   // tokens of the tile that exist
  const int share = (live + split - 1) / split;            // those that a CTA of the cluster finishes
  // partial sums, [part][accumulator][token of the share][row], in the ring that the products have read
  const uint32_t slot = (uint32_t)(kSums * share * kFewRows) * 4u;
  if (split > 1) {
    cluster_arrive();
    cluster_wait();
    if (warp < kFewEpilogue && some) {
#pragma unroll 1
      for (int i = 0; i < kSums; ++i)
#pragma unroll 1
        for (int c = turn; c < live; c += 16) {
          uint32_t v[8];
          __syncwarp();
          tmem_load8(mine + i * nt + c, v);
          tmem_wait_loads();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int to = (c + j) / share;
            if (c + j < live)
              st_cluster(in_cta(ring + part * slot + (uint32_t)(((i * share + c + j - to * share) * kFewRows + row) * 4), (uint32_t)to),
                         steps ? __uint_as_float(v[j]) : 0.0f);
          }
        }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  // the tokens that this CTA finishes, eight at a time
  const int lo = min(part * share, live), hi = min(lo + share, live);
  const bool in = m0 + row < m;
  const float* const partial = reinterpret_cast<const float*>(dynamic + (ring - smem_addr(dynamic))) + row;
  const auto sums = [&](int i, int c, float* v) {
    if (split > 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll 1
      for (int q = 0; q < split; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < hi) v[j] = __fadd_rn(v[j], partial[q * (slot / 4) + (i * share + c + j - lo) * kFewRows]);
    } else {
      __syncwarp();
      tmem_load8(mine + i * nt + c, reinterpret_cast<uint32_t*>(v));
      tmem_wait_loads();
      if (!steps) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      }
    }
  };
  if (warp < kFewEpilogue && some) {
    if (Stage == kFfnHidden && a.keep_bits == 8) {
#pragma unroll 1
      for (int i = 0; i < kSums; ++i)
#pragma unroll 1
        for (int c = lo + turn; c < hi; c += 16) {
          float v[8];
          sums(i, c, v);
          uint32_t best = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            if (lane == j) best = most;
          }
          if (lane < 8 && c + lane < hi) sh.most[warp % 4][i][c + lane] = best;
        }
      asm volatile("bar.sync %0, 128;" ::"r"(1 + warp / 4) : "memory");   // the warps of the same tokens
    }
    const int64_t groups = (m + kGroup - 1) / kGroup, group = m0 / kGroup;
#pragma unroll 1
    for (int c = lo + turn; c < hi; c += 16) {
      float v[8], w[8];
      sums(0, c, v);
      if constexpr (kSums > 1) sums(1, c, w);
      const int count = min(8, hi - c);
      const auto at = [&](int i, int j, int elem) {
        return k.rows[i] + (t0 + (int64_t)(c + j)) * k.stride[i] + (int64_t)(m0 + row) * elem;
      };
      if constexpr (Stage == kFfnHidden) {
        if (a.keep_bits == 8) {
#pragma unroll 1
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (j >= count) continue;
              uint32_t most = 0;
#pragma unroll
              for (int q = 0; q < 4; ++q) most = max(most, sh.most[q][i][c + j]);
              float scale, by;
              group_scale(__uint_as_float(most), &scale, &by);
              if (row == 0) st_g(k.scales[i] + (t0 + c + j) * groups + group, scale);
              if (in) st_g(reinterpret_cast<int8_t*>(at(1 + i, j, 1)), code_of(i ? w[j] : v[j], by));
            }
        } else if (a.keep_bits == 16) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j >= count || !in) continue;
            st_g(reinterpret_cast<T*>(at(1, j, 2)), narrow<D>(v[j]));
            st_g(reinterpret_cast<T*>(at(2, j, 2)), narrow<D>(w[j]));
          }
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float2 act, slope;
          activate<Act, false>(make_float2(v[j], v[j + 1]), &act, &slope);
          if (j < count && in) st_g(reinterpret_cast<T*>(at(0, j, 2)), narrow<D>(act.x * w[j]));
          if (j + 1 < count && in) st_g(reinterpret_cast<T*>(at(0, j + 1, 2)), narrow<D>(act.y * w[j + 1]));
        }
      } else if constexpr (Stage == kFfnGradHidden) {
        float g[8], up[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g[j] = up[j] = 0.0f;
          if (j >= count || !in) continue;
          if (a.keep_bits == 8) {
            const int64_t n = (t0 + c + j) * groups + group;
            g[j] = (float)ld_g(reinterpret_cast<const int8_t*>(at(3, j, 1))) * ld_g(k.scales[0] + n);
            up[j] = (float)ld_g(reinterpret_cast<const int8_t*>(at(4, j, 1))) * ld_g(k.scales[1] + n);
          } else {
            g[j] = widen<D>(ld_g(reinterpret_cast<const T*>(at(3, j, 2))));
            up[j] = widen<D>(ld_g(reinterpret_cast<const T*>(at(4, j, 2))));
          }
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float2 act, slope;
          activate<Act, true>(make_float2(g[j], g[j + 1]), &act, &slope);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (j + i >= count || !in) continue;
            const float d = v[j + i], s = i ? slope.y : slope.x, f = i ? act.y : act.x;
            st_g(reinterpret_cast<T*>(at(0, j + i, 2)), narrow<D>(d * up[j + i] * s));
            st_g(reinterpret_cast<T*>(at(1, j + i, 2)), narrow<D>(d * f));
            if (k.rows[2]) st_g(reinterpret_cast<T*>(at(2, j + i, 2)), narrow<D>(f * up[j + i]));
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < count && in) st_g(reinterpret_cast<T*>(at(0, j, 2)), narrow<D>(v[j]));
      }
    }
  }
  tensor_fence_before();
  __syncwarp();
  __syncthreads();
  if (sh.gave_up) let_land();
  __syncwarp();
  if (warp == kFewEpilogue + 1) tmem_free<1>(tmem, columns);
}

}  // namespace ra
