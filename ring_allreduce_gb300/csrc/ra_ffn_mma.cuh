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
//            stages (out of range: zeros), the pair's bytes counted on
//            the first CTA's barrier
//   warp 9   of the first CTA: one thread issues the products, and frees
//            stages and hands over sums by commits to both CTAs' barriers
//   warps 0-7  epilogue: thread = row, the second four warps the second half
//            of the columns.  Tensor memory holds two tiles' sums, so the products
//            of the next tile run while one is written out
// Operands are taken as they lie: rows along the terms (projections, dh) or
// across them (everything else); nothing is transposed or laid out anew.
//
// The products keep the shared memory's path busy (a tile's 64 terms: 32 KB
// written and as much read an SM in 512 cycles), and whatever the epilogue sends
// through it costs them its time.  A store to global memory by lanes that each
// hold a row takes a cycle of it a row and 16 bytes; so the epilogue lays its
// outputs down in shared memory, 64 bytes of 32 rows at a time, and has them
// stored by tensor map, which also cuts them off at the last row and column
// (the projections of 8192 tokens, 4096 x 16384: 1108 -> 1079 us; their
// gradients' kernel, 4096 x 8192 from 2048 columns: 120 -> 112).
//
// Measured one by one, bf16: the projections of 8192 tokens, 4096 x 16384 in
// four ranks, at 2.04 PFLOP/s, the product back at 2.03; both together, over
// and over, 1.91 ms, 1.73 PFLOP/s, where the power limit holds a plain library
// product of that size to the same.  What bounds them beside the tensor cores is the way from L2: 64
// bytes a cycle and SM, 15 TB/s together.  The weights' gradients reach 1.8 to
// 1.9 PFLOP/s (their rows lie across the terms), the gradients of a and b 1.2
// to 1.6: of them the epilogue, which reads two kept tensors and writes three,
// takes 10 us a tile from codes and 13.7 from 16-bit values (SiLU; GELU 13 and
// 14.5), as long as the products of some 2400 columns and more.
#pragma once

#include "ra_ffn.cuh"
#include "ra_ffn_mma.h"
#include "ra_tensor.cuh"

namespace ra {

namespace {

constexpr int kBlockM = 128, kBlockN = 128, kBlockK = 64;   // of one CTA's operands
constexpr int kOperandBytes = kBlockM * kBlockK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kMmaThreads = 320;
constexpr int kTileN = 2 * kBlockN;
constexpr uint32_t kTmemColumns = 2 * kTileN;
constexpr int kUnitBytes = 32 * 64;   // 64 bytes of a warp's 32 rows

// dh's epilogue writes three outputs: more room for them, one stage less.
__host__ __device__ constexpr int stages(int stage) { return stage == kFfnGradHidden ? 5 : 6; }
__host__ __device__ constexpr int units(int stage) { return stage == kFfnGradHidden ? 4 : 2; }
__host__ __device__ constexpr int mma_shared(int stage) {
  return stages(stage) * kStageBytes + 8 * units(stage) * kUnitBytes + 1024;   // and up to 1024 to align
}

struct MmaShared {
  uint64_t full[6], empty[6];
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
  p->n0 = v / high * (Stage == kFfnHidden ? kBlockN : kTileN);
  const int width = a.rank[p->r].width;
  if constexpr (Stage == kFfnHidden || Stage == kFfnGradHidden) {
    p->m = (int)a.tokens;
    p->n = width;
    p->steps = (a.dim + kBlockK - 1) / kBlockK;
  } else if constexpr (Stage == kFfnOut) {
    p->m = (int)a.tokens;
    p->n = a.dim;
    p->half = (width + kBlockK - 1) / kBlockK;
    p->steps = p->half * a.segments;
  } else {
    p->m = width;
    p->n = a.dim;
    p->steps = (int)((a.tokens + kBlockK - 1) / kBlockK);
    if (!a.rank[p->r].rows[p->which]) return false;
  }
  return p->m0 < p->m && p->n0 < p->n;
}

// The maps of a tile's operands, as bits.
template <int Stage> __device__ __forceinline__ int operand_maps(const MmaArgs& a, const Tile& p) {
  if (Stage == kFfnGradW) return 1 << p.which | (p.which == 2 ? 16 : 8);
  return Stage == kFfnHidden ? 7 : Stage == kFfnGradHidden ? 3 : a.segments == 2 ? 15 : 5;
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The epilogue of a tile in one of eight warps.
template <int Stage> struct Epilogue {
  static constexpr int kUnits = units(Stage);
  const MmaArgs& a;
  uint32_t staging;        // kUnits units of this warp's, 512-byte aligned
  uint32_t next;           // the unit that is written next
  int half, lane;
  // of the tile
  uint32_t tmem;           // the warp's lanes of its sums
  int r;
  int64_t row0;            // the first lane's row
  int rows;                // how many of the lanes' exist
  uint32_t sums_empty;     // where the sums are handed back

  __device__ __forceinline__ int64_t row() const { return row0 + lane; }
  __device__ __forceinline__ bool in() const { return lane < rows; }
  // 32 columns of this thread's row
  __device__ __forceinline__ void sums(int column, float* v) const {
    __syncwarp();
    tmem_load32(tmem + column, reinterpret_cast<uint32_t*>(v));
  }
  // Every lane's loads from tensor memory have returned.
  __device__ __forceinline__ void release() const {
    tensor_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster_relaxed(sums_empty);
  }
  // Bytes [16 q, 16 q + 16) of this lane's row of a unit, swizzled as its copy by tensor map expects.
  __device__ __forceinline__ uint32_t piece(uint32_t unit, int q) const {
    return staging + unit * kUnitBytes + (uint32_t)lane * 64u + (((uint32_t)q ^ ((uint32_t)lane >> 1 & 3u)) << 4);
  }
  // The next unit, free to be written: all but the last kUnits - 1 copies have read theirs.
  __device__ __forceinline__ uint32_t take() {
    const uint32_t u = next;
    next = next + 1 == kUnits ? 0 : next + 1;
    if (lane == 0) bulk_wait_read<kUnits - 1>();
    __syncwarp();
    return u;
  }
  __device__ __forceinline__ void fill(uint32_t unit, const uint32_t* w) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) st_shared16(piece(unit, q), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  }
  // A filled unit to the columns from `column` on of rows `k`, elements of `elem` bytes, `left` columns to come.
  __device__ __forceinline__ void store(uint32_t unit, int k, int column, int left, int elem) const {
    const MmaRank<MmaArgs::kMaps>& t = a.rank[r];
    // (a copy is cut off to 16 bytes, not to the element)
    if (a.level[k] == 2 && (left * elem >= 64 || left * elem % 16 == 0)) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (left > 0 && rows > 0)
          asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                           &t.map[first_rows(Stage) + k]),
                       "r"(column), "r"((int)row0), "r"(staging + unit * kUnitBytes)
                       : "memory");
        bulk_commit();
      }
    } else {   // rows off the 16-byte grid, or that end on none: element by element, side by side
      __syncwarp();
      const int columns = max(min(left, 64 / elem), 1), n = left > 0 ? columns * rows : 0;
      const int down = 32 / columns, across = 32 - down * columns;   // 32 elements on
      int y = lane / columns, x = lane - y * columns;
#pragma unroll 2
      for (int i = lane; i < n; i += 32) {
        char* const to = t.rows[k] + (row0 + y) * t.stride[k] + (int64_t)(column + x) * elem;
        const uint32_t b = (uint32_t)(x * elem);
        const uint32_t from = staging + unit * kUnitBytes + (uint32_t)y * 64u + ((b >> 4 ^ ((uint32_t)y >> 1 & 3u)) << 4) + (b & 15u);
        uint32_t v;
        if (elem == 4) {
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(from) : "memory");
          st_g(reinterpret_cast<uint32_t*>(to), v);
        } else if (elem == 2) {
          asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(from) : "memory");
          st_g(reinterpret_cast<uint16_t*>(to), (uint16_t)v);
        } else {
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(from) : "memory");
          st_g(reinterpret_cast<uint8_t*>(to), (uint8_t)v);
        }
        x += across;
        y += down;
        if (x >= columns) {
          x -= columns;
          ++y;
        }
      }
      if (lane == 0) bulk_commit();   // of nothing: take() counts one a unit
      __syncwarp();
    }
  }
  // 32 values of a row, rounded to the block's type
  template <class D> __device__ __forceinline__ void put(int k, int column, const float* v, int left) {
    const uint32_t u = take();
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack2<D>(v[2 * j], v[2 * j + 1]);
    fill(u, w);
    store(u, k, column, left, 2);
  }
};

// 64 gated columns of a row.  Kept in 8 bits, the 128 columns that share a scale
// belong to two warps; each looks all of them through for the largest magnitude.
template <class D, int Act>
__device__ __forceinline__ void write_hidden(const MmaArgs& a, const Tile& p, Epilogue<kFfnHidden>& e) {
  const int r = p.r, first = p.n0 + e.half * 64, gate = e.half * 64, up = kBlockN + gate;
  if (a.keep_bits == 8) {
    float m[2] = {}, by[2], scale[2];
#pragma unroll 1
    for (int c = 0; c < kBlockN; c += 32) {
      float g[32], u[32];
      e.sums(c, g);
      e.sums(kBlockN + c, u);
      tmem_wait_loads();
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        m[0] = max_nan(m[0], fabsf(g[j]));
        m[1] = max_nan(m[1], fabsf(u[j]));
      }
    }
    group_scale(m[0], &scale[0], &by[0]);
    group_scale(m[1], &scale[1], &by[1]);
    if (e.in())
      st_g(a.rank[r].scales[e.half] + e.row() * ((p.n + kGroup - 1) / kGroup) + p.n0 / kGroup, e.half ? scale[1] : scale[0]);
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
      const uint32_t unit = e.take();
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        float v[32];
        e.sums((b ? up : gate) + c, v);
        tmem_wait_loads();
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = codes4(v + 4 * j, b ? by[1] : by[0]);
        st_shared16(e.piece(unit, c / 16), w[0], w[1], w[2], w[3]);
        st_shared16(e.piece(unit, c / 16 + 1), w[4], w[5], w[6], w[7]);
      }
      e.store(unit, 1 + b, first, p.n - first, 1);
    }
  }
#pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    const int col = first + c, left = p.n - col;
    float g[32], u[32];
    e.sums(gate + c, g);
    e.sums(up + c, u);
    tmem_wait_loads();
    if (c == 32) e.release();
    if (a.keep_bits == 16) {
      e.put<D>(1, col, g, left);
      e.put<D>(2, col, u, left);
    }
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      float2 act, slope;
      activate<Act, false>(make_float2(g[j], g[j + 1]), &act, &slope);
      const float2 h = __fmul2_rn(act, make_float2(u[j], u[j + 1]));
      g[j] = h.x;
      g[j + 1] = h.y;
    }
    e.put<D>(0, col, g, left);
  }
}

// 16 * kLanes bytes of a warp's 32 kept rows, gate or up: fetched with kLanes
// lanes to a row, so that a request takes a line of memory or half of one, and
// handed to the rows' lanes through shared memory.  (A row a lane, 32 bytes at
// a time, is four requests for a line; they took a third of the epilogue.)
template <int kLanes> struct KeptRows {
  static constexpr int kDown = 32 / kLanes;   // rows in a request
  uint4 q[kLanes];   // of rows lane / kLanes, lane / kLanes + kDown, ...: 16 bytes
  // From byte `first` of the rows on, of which `left` bytes are to come.
  __device__ __forceinline__ void fetch(const MmaArgs& a, const Epilogue<kFfnGradHidden>& e, int k, int64_t first, int left) {
    const int64_t stride = a.rank[e.r].stride[k];
    const int mine = left - e.lane % kLanes * 16, level = a.level[k];
    const char* const from = a.rank[e.r].rows[k] + e.row0 * stride + first + e.lane % kLanes * 16;
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
      const int y = e.lane / kLanes + kDown * i;
      const char* const at = from + y * stride;
      uint32_t w[4] = {};
      if (y < e.rows && mine > 0) {
        if (level == 2 && mine >= 16) {
          if (RA_ACCESS_OK(at, 16u, 1u)) {
            const uint4 x = *reinterpret_cast<const uint4*>(at);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            if (level && mine >= 4 * j + 8) {
              const uint2 x = ld_g(reinterpret_cast<const uint2*>(at) + j / 2);
              w[j] = x.x, w[j + 1] = x.y;
            } else {
#pragma unroll 1
              for (int n = 0; n < 8 && 4 * j + n < mine; ++n) {
                const uint32_t x = (uint32_t)ld_g(reinterpret_cast<const uint8_t*>(at) + 4 * j + n) << (8 * (n % 4));
                if (n < 4) w[j] |= x;
                else w[j + 1] |= x;
              }
            }
          }
        }
      }
      q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // Piece x of row y of what lies at `staging`: eight lanes' pieces on different banks, either way.
  static __device__ __forceinline__ uint32_t place(uint32_t staging, int y, int x) {
    return staging + (uint32_t)y * (16u * kLanes) + ((uint32_t)(x ^ (y / (8 / kLanes) % kLanes)) << 4);
  }
  __device__ __forceinline__ void put(uint32_t staging, int lane) const {
#pragma unroll
    for (int i = 0; i < kLanes; ++i)
      st_shared16(place(staging, lane / kLanes + kDown * i, lane % kLanes), q[i].x, q[i].y, q[i].z, q[i].w);
  }
  // This lane's row, as it lies.
  __device__ __forceinline__ void get(uint32_t staging, int lane) {
#pragma unroll
    for (int i = 0; i < kLanes; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w)
                   : "r"(place(staging, lane, i))
                   : "memory");
  }
};

__device__ __forceinline__ uint32_t word_of(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// 16 columns of a row: the gradients of a and b, and hidden, from dh and what was kept.
template <class D, int Act, class P>
__device__ __forceinline__ void gradients(const float* dh, const P& pair, uint32_t (*w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 g = pair(0, j), u = pair(1, j), d = make_float2(dh[2 * j], dh[2 * j + 1]);
    float2 act, slope;
    activate<Act, true>(g, &act, &slope);
    const float2 da = __fmul2_rn(__fmul2_rn(d, u), slope), db = __fmul2_rn(d, act), h = __fmul2_rn(act, u);
    w[0][j] = pack2<D>(da.x, da.y);
    w[1][j] = pack2<D>(db.x, db.y);
    w[2][j] = pack2<D>(h.x, h.y);
  }
}

// 128 columns of a row of dh, from which the gradients of a and b are made, 32
// at a time.  Kept codes are fetched while the products still run; 16-bit
// values, for which there are not the registers, a chunk ahead.
template <class D, int Act, bool Coded, class W>
__device__ __forceinline__ bool write_grad_hidden(const MmaArgs& a, const Tile& p, Epilogue<kFfnGradHidden>& e,
                                                  const W& wait, uint64_t* full, uint32_t parity) {
  const int r = p.r, first = p.n0 + e.half * kBlockN;
  constexpr int kLanes = Coded ? 8 : 4;
  float scale[2] = {};
  KeptRows<kLanes> kept[2];
  const auto fetch = [&](int col) {
#pragma unroll
    for (int b = 0; b < 2; ++b) kept[b].fetch(a, e, 3 + b, (int64_t)col * (Coded ? 1 : 2), (p.n - col) * (Coded ? 1 : 2));
  };
  fetch(first);
  if (Coded && e.in() && first < p.n) {
    const int64_t at = e.row() * ((p.n + kGroup - 1) / kGroup) + first / kGroup;
    scale[0] = ld_g(a.rank[r].scales[0] + at);
    scale[1] = ld_g(a.rank[r].scales[1] + at);
  }
  if (!wait.warp(full, parity, 4)) return false;
  tensor_fence_after();
  if constexpr (Coded) {
    if (e.lane == 0) bulk_wait_read<0>();   // all units are free
    __syncwarp();
    kept[0].put(e.staging, e.lane);
    kept[1].put(e.staging + 2 * kUnitBytes, e.lane);
    __syncwarp();
    kept[0].get(e.staging, e.lane);
    kept[1].get(e.staging + 2 * kUnitBytes, e.lane);
    __syncwarp();
  }
  // Codes are taken from the registers they were fetched into, which asks for
  // four copies of the body; with one, those that are left move to the front.
  // SiLU's body is short enough for four; the others outgrow the instruction
  // cache.  Two ranks of 8192 columns, 4096 tokens by 512 and by 2048, one
  // copy and four: SiLU 85 and 116 us, 76 and 117; GELU 93 and 117, 103 and 124;
  // 16-bit values with SiLU 99 and 126, 124 and 146.
  constexpr int kCopies = Coded && Act == RA_SILU ? 4 : 1;
#pragma unroll 1
  for (int c0 = 0; c0 < 4; c0 += kCopies) {
#pragma unroll
    for (int c1 = 0; c1 < kCopies; ++c1) {
      const int c = c0 + c1, col = first + 32 * c, left = p.n - col;
      float dh[32];
      e.sums(e.half * kBlockN + 32 * c, dh);
      KeptRows<kLanes> now[2] = {kept[0], kept[1]};
      if constexpr (!Coded) {
        if (left > 0) {
          // through the next unit, one after the other: the last copies' three are still being read
          if (e.lane == 0) bulk_wait_read<e.kUnits - 1>();
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            __syncwarp();
            kept[b].put(e.staging + e.next * kUnitBytes, e.lane);
            __syncwarp();
            now[b].get(e.staging + e.next * kUnitBytes, e.lane);
          }
          __syncwarp();
          if (c < 3 && left > 32) fetch(col + 32);
        }
      }
      tmem_wait_loads();
      if (c == 3) e.release();
      if (left <= 0) continue;
      uint32_t unit[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) unit[k] = (e.next + k) % e.kUnits;
      e.next = (e.next + (a.rank[r].rows[2] ? 3 : 2)) % e.kUnits;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[3][8];
        gradients<D, Act>(dh + 16 * h, [&](int b, int j) {
          if constexpr (Coded) {
            const uint32_t word = word_of(now[b].q[2 * c1 + h], j / 2);
            return __fmul2_rn(code_pair(bias_codes(word), 2 * (j % 2)), both(scale[b]));
          } else {
            float2 v;
            unpack2<D>(word_of(now[b].q[2 * h + j / 4], j % 4), reinterpret_cast<float*>(&v));
            return v;
          }
        }, w);
        if (h == 0) {   // three units at once: what was stored before the last copy has been read
          if (e.lane == 0) bulk_wait_read<e.kUnits - 3>();
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          if (k == 2 && !a.rank[r].rows[2]) continue;
          st_shared16(e.piece(unit[k], 2 * h), w[k][0], w[k][1], w[k][2], w[k][3]);
          st_shared16(e.piece(unit[k], 2 * h + 1), w[k][4], w[k][5], w[k][6], w[k][7]);
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < 2 || a.rank[r].rows[2]) e.store(unit[k], k, col, left, 2);
    }
    if constexpr (Coded && kCopies < 4) {
#pragma unroll
      for (int i = 0; i < 8 - 2 * kCopies; ++i)
        kept[0].q[i] = kept[0].q[i + 2 * kCopies], kept[1].q[i] = kept[1].q[i + 2 * kCopies];
    }
  }
  return true;
}

// 128 columns of a row, rounded.
template <class D, int Stage>
__device__ __forceinline__ void write_plain(const MmaArgs& a, const Tile& p, Epilogue<Stage>& e) {
  const int first = p.n0 + e.half * kBlockN;
#pragma unroll 1
  for (int c = 0; c < kBlockN; c += 32) {
    const int col = first + c, left = p.n - col;
    float v[32];
    e.sums(e.half * kBlockN + c, v);
    tmem_wait_loads();
    if (c == kBlockN - 32) e.release();
    if (p.steps == 0) {   // a sum of nothing: the columns hold what an earlier tile left
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.0f;
    }
    if (Stage == kFfnGradW && a.grad_f32) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t unit = e.take();
        e.fill(unit, reinterpret_cast<const uint32_t*>(v + 16 * q));
        e.store(unit, p.which, col + 16 * q, left - 16 * q, 4);
      }
    } else {
      e.template put<D>(p.which, col, v, left);
    }
  }
}

}  // namespace

template <class D, int Stage, int Act>
__global__ void __launch_bounds__(kMmaThreads, 1) ffn_mma_kernel(const __grid_constant__ MmaArgs a) {
  // operands whose rows run across the terms: 64 terms of 64 elements a box, two boxes
  constexpr bool kAMn = Stage == kFfnGradW, kBMn = Stage == kFfnOut || Stage == kFfnGradW;
  constexpr uint32_t kDesc = product_desc(std::is_same<D, DBF16>::value, kAMn, kBMn, 2 * kBlockM, kTileN);
  constexpr int kStages = stages(Stage);
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
      mbar_init(&sh.sums_empty[b], 16);   // eight warps of each CTA
    }
    sh.gave_up = 0;
    fence_mbar_init();
  }
  // (one CTA an SM, by its shared memory: the columns are free, and nothing is waited for)
  if (warp == 9) tmem_alloc<2>(&sh.tmem, kTmemColumns);
  Tile p;
  if (warp == 8 && lane < 8 && blockIdx.x / 2 < a.tiles && tile_at<Stage>(a, blockIdx.x / 2, &p) && p.steps > 0 &&
      operand_maps<Stage>(a, p) >> lane & 1)
    prefetch_map(&a.rank[p.r].map[lane]);
  tensor_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tensor_fence_after();
  const uint32_t tmem = sh.tmem;
  after_predecessor();   // what came before ran on beside all this
  const Waits wait{&sh.gave_up, a.record, Stage};
  const int64_t tiles = a.tiles, step = gridDim.x / 2;

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
          int ia = 0, ib = 1, at = k * kBlockK;
          if constexpr (Stage == kFfnHidden) {
            ib = 1 + (int)cta;
          } else if constexpr (Stage == kFfnOut) {
            ia = k >= p.half;
            ib = 2 + ia;
            at -= ia * p.half * kBlockK;
          } else if constexpr (Stage == kFfnGradW) {
            ia = p.which;
            ib = p.which == 2 ? 4 : 3;
          }
          const CUtensorMap *const ma = &a.rank[p.r].map[ia], *const mb = &a.rank[p.r].map[ib];
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
    Epilogue<Stage> e{a, ring + kStages * kStageBytes + (uint32_t)warp * (units(Stage) * kUnitBytes), 0, warp / 4, lane};
    uint32_t it = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x / 2; ok && t < tiles; t += step) {
      if (!tile_at<Stage>(a, t, &p)) continue;
      const uint32_t b = it & 1, parity = (it >> 1) & 1;
      e.tmem = tmem + b * kTileN + ((uint32_t)(warp % 4) * 32u << 16);
      e.r = p.r;
      e.row0 = p.m0 + (int)cta * kBlockM + (warp % 4) * 32;
      e.rows = (int)max((int64_t)0, min((int64_t)32, p.m - e.row0));
      e.sums_empty = in_cta(smem_addr(&sh.sums_empty[b]), 0);
      if constexpr (Stage == kFfnGradHidden) {
        ok = a.keep_bits == 8 ? write_grad_hidden<D, Act, true>(a, p, e, wait, &sh.sums_full[b], parity)
                              : write_grad_hidden<D, Act, false>(a, p, e, wait, &sh.sums_full[b], parity);
      } else {
        ok = wait.warp(&sh.sums_full[b], parity, 4);
        if (!ok) break;
        tensor_fence_after();
        if constexpr (Stage == kFfnHidden)
          write_hidden<D, Act>(a, p, e);
        else
          write_plain<D, Stage>(a, p, e);
      }
      ++it;
    }
    if (lane == 0) bulk_wait_all();   // what is stored by tensor map has been
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
