// Dense products on CTA pairs (tcgen05 cta_group::2): how a grid of tiles is
// cut and dealt to persistent pairs, and what an epilogue needs to bring an
// accumulator to memory.  Shared by the vocabulary head and the dense linear
// layer.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>

#include "tc.cuh"
#include "tmap.cuh"

namespace dmoe {
namespace tile {

using namespace dmoe::tc;

constexpr int BM = 128;   // rows of a CTA's half of a pair tile
constexpr int BN = 256;   // columns of a sub-tile
constexpr int BK = 64;    // K slice per stage (one 128-byte swizzle row)
constexpr int UMMA_K = 16;
constexpr uint32_t A_BYTES = BM * BK * 2;        // this CTA's A rows
constexpr uint32_t B_BYTES = (BN / 2) * BK * 2;  // this CTA's half of a sub-tile's B
constexpr uint32_t ATOM = 64 * BK * 2;           // MN-major operands: 64 MN x 64 K boxes
constexpr uint32_t SLAB32 = 32 * 32 * 2;         // an epilogue warp's 32 rows x 32 columns on their way out
constexpr size_t kSmemMax = 232448;
constexpr uint64_t kDrainNs = 1000 * 1000;
constexpr int kUnits = 76;  // CTA pairs of a GB300, for the rules that cut products

// Exact unsigned division by a number fixed on the host (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994,
// figure 4.1): a multiplication instead of some forty instructions, which a
// single issuing thread would wait for at every tile.
struct FastDiv {
  uint32_t d, m;
  int s;  // ceil(log2 d)
  void set(uint32_t v) {
    d = v;
    for (s = 0; (1ull << s) < v; ++s) {
    }
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - v)) / v + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    const uint32_t t = __umulhi(m, n);
    return s == 0 ? n : (t + ((n - t) >> 1)) >> (s - 1);
  }
};

// A grid of M x N tiles over K, cut into `parts` ranges of K slices, in groups
// of `raster` pair rows.
struct Grid {
  int cols;       // N
  int tile;       // columns of a tile: 512 (two sub-tiles), 256, for the logits also 128 or 64
  int64_t time;   // of its longest item, for the host: see item_time()
  int mt, nt;     // pair-tile rows, tile columns
  int raster;     // pair-tile rows per raster group
  int slices;     // K slices of 64
  int parts;
  int per_part;   // K slices of a part (the last one's may be fewer)
  int items;      // mt * nt * parts
  FastDiv tiles;  // mt * nt
  FastDiv group;  // tiles of a full raster group
  FastDiv high;   // raster
  FastDiv rest;   // pair rows of the last, smaller group
};

__device__ __forceinline__ uint4 pack8x(const float* f) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return u;
}

__device__ __forceinline__ void unpack8x(const uint4& u, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __bfloat1622float2(h[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// Waits for the loads of tmem_ld32; ties the registers to the wait, so that
// no use moves above it.
__device__ __forceinline__ void tmem_wait(float (&r)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
        "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
        "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]),
        "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
        "+f"(r[30]), "+f"(r[31])::"memory");
}

// M = 256 MMA of the CTA pair, descriptors as (low, high) words; `add`: 0
// overwrites the accumulator.
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi,
                                         uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(add)
      : "memory");
}

__device__ __forceinline__ void st_shared(uint32_t a, const uint4& q) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}

__device__ __forceinline__ uint4 ld_shared(uint32_t a) {
  uint4 q;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "r"(a)
               : "memory");
  return q;
}

// 32 rows x 32 columns held one row per lane go to global memory as coalesced
// 16-byte stores through the warp's 2 KB slab: every lane puts its row's
// 16-byte piece j at piece j ^ ((r >> 1) & 3) of row r (free of bank
// conflicts), then each store instruction writes 8 rows x 64 bytes.  Only
// rows below `rows` and 8-column pieces below `cols` exist (both counted from
// this corner).
__device__ __forceinline__ void write_rows32(uint32_t slab, int lane, const float* v, uint16_t* out, int64_t ld,
                                             int rows, int cols) {
  const int sw = (lane >> 1) & 3;
  const int j = lane & 3, r0 = lane >> 2;
  out += r0 * ld + 8 * j;
#pragma unroll
  for (int q = 0; q < 4; ++q) st_shared(slab + lane * 64 + ((q ^ sw) << 4), pack8x(v + 8 * q));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + r0;
    const uint4 u = ld_shared(slab + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
    if (r < rows && 8 * j < cols) *reinterpret_cast<uint4*>(out + 8 * i * ld) = u;
  }
  __syncwarp();
}

// A plain load, of memory that the kernel itself may write (which __ldg may not
// read), but one that the compiler may move: held where they stand, the loads
// of join_row32 wait behind the accumulator's and the last stores (8192 x 512 x
// 2048 onto a residual 54 us, 26 with these).  So it is for values that the
// reader alone overwrites, by stores that hang on what it read, and behind a
// branch on the wait for what came before, which it does not pass.
__device__ __forceinline__ uint4 ld_own(const uint4* a) {
  uint4 q;
  asm("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
      : "l"(reinterpret_cast<uint64_t>(a)));
  return q;
}

// 32 bf16 values of a row of which `cols` exist, added to v[0..31] or multiplied
// into them; the row may be the one the caller overwrites.
template <bool MUL>
__device__ __forceinline__ void join_row32(float* v, const uint16_t* a, int cols) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (8 * j < cols) {
      float f[8];
      unpack8x(ld_own(reinterpret_cast<const uint4*>(a) + j), f);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[8 * j + q] = MUL ? v[8 * j + q] * f[q] : v[8 * j + q] + f[q];
    }
  }
}

// v[0..31] += k * 32 bf16 values of a row of which `cols` exist (which nothing
// writes meanwhile).
__device__ __forceinline__ void add_row32(float* v, const uint16_t* a, float k, int cols) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (8 * j < cols) {
      float f[8];
      unpack8x(__ldg(reinterpret_cast<const uint4*>(a) + j), f);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[8 * j + q] = fmaf(k, f[q], v[8 * j + q]);
    }
  }
}

// The same with fp32 values and k = 1 (plain loads: the row may be the one
// the caller overwrites).
__device__ __forceinline__ void add_row32(float* v, const float* a, int cols) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (4 * j < cols) {
      const float4 q = *(reinterpret_cast<const float4*>(a) + j);
      v[4 * j] += q.x, v[4 * j + 1] += q.y, v[4 * j + 2] += q.z, v[4 * j + 3] += q.w;
    }
  }
}

// write_rows32 with fp32 values: 16 columns at a time fill the slab's rows.
__device__ __forceinline__ void write_rows32(uint32_t slab, int lane, const float* v, float* out, int64_t ld, int rows,
                                             int cols) {
  const int sw = (lane >> 1) & 3;
  const int j = lane & 3, r0 = lane >> 2;
  out += r0 * ld + 4 * j;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float* f = v + 16 * h + 4 * q;
      st_shared(slab + lane * 64 + ((q ^ sw) << 4), make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                                                              __float_as_uint(f[2]), __float_as_uint(f[3])));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + r0;
      const uint4 u = ld_shared(slab + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
      if (r < rows && 16 * h + 4 * j < cols) *reinterpret_cast<uint4*>(out + 8 * i * ld + 16 * h) = u;
    }
    __syncwarp();
  }
}

// One unit of work: a tile of one product over a range of K slices.
struct Item {
  int dx;      // gradients: dx's or dW's
  int m, c0;   // pair-tile row, first column
  int k0, k1;  // K slices
  int part;
  bool wide;   // the second sub-tile has columns (else it is left out)
};

// Tile t of a grid, in groups of `raster` pair rows with the columns outer
// and the rows inner: pairs working at the same time share B columns while
// the group's A rows stay in L2.
__device__ __forceinline__ void tile_at(const Grid& g, uint32_t t, Item& it) {
  uint32_t part = 0;
  if (g.parts > 1) {
    part = g.tiles(t);
    t -= part * g.tiles.d;
  }
  it.part = part;
  it.k0 = part * g.per_part;
  it.k1 = min(it.k0 + g.per_part, g.slices);
  const uint32_t q = g.group(t);
  const uint32_t l = t - q * g.group.d;
  const uint32_t r0 = q * g.raster;
  const bool last = r0 + g.raster > static_cast<uint32_t>(g.mt);
  const uint32_t n = last ? g.rest(l) : g.high(l);
  it.m = r0 + l - n * (last ? g.rest.d : g.high.d);
  it.c0 = n * g.tile;
  it.wide = g.tile > BN && it.c0 + BN < g.cols;
}

// The j-th item of unit u of U (false: none left).  The items of grid[0],
// the longer ones, are dealt round; the `early` units that get one fewer of
// them first take `extra` items of grid[1] each (about the length of one of
// grid[0]), then those are dealt round as well, so all units end within about
// one short item of each other.
template <class P>
__device__ __forceinline__ bool item_of(const P& p, int u, int U, int j, Item& it) {
  const int mine = p.full + (u < p.rem ? 1 : 0);
  if (j < mine) {
    it.dx = p.first_dx;
    tile_at(p.grid[0], u + j * U, it);
    return true;
  }
  j -= mine;
  int i;
  if (p.early > 0 && u >= p.rem && j < p.extra) {
    i = j * p.early + (u - p.rem);
  } else {
    if (u >= p.rem && p.early > 0) j -= p.extra;
    i = p.early * p.extra + j * U + u;
  }
  if (i >= p.grid[1].items) return false;
  it.dx = !p.first_dx;
  tile_at(p.grid[1], i, it);
  return true;
}

// ----------------------------------------------------------------- host side

// As dmoe::make_map (128-byte swizzle), of a [rows, cols] corner of a matrix
// whose rows lie ld elements apart: what lies past cols reads as zero.
inline bool map_pitched(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_cols,
                 uint32_t box_rows) {
  auto fn = dmoe::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows}, pitch[1] = {ld * 2};
  const cuuint32_t box[2] = {box_cols, box_rows}, step[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, pitch, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

inline Grid cut_grid(int M, int N, int K, int raster, int parts, int tile) {
  Grid g{};
  g.cols = N;
  g.tile = tile;
  g.mt = ceil_div(M, 2 * BM);
  g.nt = ceil_div(N, tile);
  g.raster = raster;
  g.slices = ceil_div(K, BK);
  g.per_part = ceil_div(g.slices, parts);
  g.parts = ceil_div(g.slices, g.per_part);  // none of them empty
  g.items = g.mt * g.nt * g.parts;
  g.tiles.set(static_cast<uint32_t>(g.mt) * g.nt);
  g.group.set(static_cast<uint32_t>(raster) * g.nt);
  g.high.set(raster);
  g.rest.set(g.mt % raster ? g.mt % raster : raster);
  return g;
}

// Deals the items of two grids (the second may have none) to U units: the
// longer ones into grid[0], and how many of the shorter ones the units with
// one long item fewer take first (item_of()).  busiest: the time of the unit
// that has most.
struct Dealt {
  int full, rem, early, extra;
  int64_t busiest;
};
inline Dealt dealt(int n0, int64_t l0, int n1, int64_t l1, int U) {  // the longer items first
  Dealt r{};
  r.full = n0 / U;
  r.rem = n0 % U;
  r.early = r.rem > 0 && n1 > 0 ? U - r.rem : 0;
  r.extra = r.early > 0 ? static_cast<int>((l0 + l1 / 2) / l1) : 0;
  const int64_t taken = std::min<int64_t>(n1, static_cast<int64_t>(r.early) * r.extra);
  const int64_t rest = n1 - taken, round = rest / U, left = rest % U;
  const int64_t a = (r.full + (r.rem > 0)) * l0 + (round + (left > 0)) * l1;
  const int64_t b = r.early == 0 ? 0 : r.full * l0 + (ceil_div(taken, r.early) + round + (left > r.rem)) * l1;
  r.busiest = std::max(a, b);
  return r;
}

}  // namespace tile
}  // namespace dmoe
