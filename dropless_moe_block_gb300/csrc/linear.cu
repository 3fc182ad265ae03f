// Dense linear layer beside the routed experts, and its backward:
//
//   z = x W + bias,  y = act(z) + residual,  deriv = act'(z)
//   dz = dy deriv,  dx = (dz W^T) factor,  dW = x^T dz,  dbias = sum_t dz_t
//
// x [M, K], W [K, N] as an expert's weights lie: no transposed copies, the
// tensor cores take each operand as it is (x and dz along K, W along N in the
// forward product; dz and W both along N for dx; x and dz both along their
// rows' width for dW).  deriv, in bf16, is all the backward needs of z, and
// `factor` puts the deriv of the layer before into dx's epilogue, so that a
// stack of layers never makes a pass over its rows in between.
//
// The products are bound by the tensor cores (2 M K N flops each) except for
// few rows, where W's bytes are.  They run as persistent CTA pairs (tcgen05
// cta_group::2, tile.cuh): warp 0 TMA producer, warp 1 TMEM allocator and
// (rank 0) MMA issuer, warps 2-17 epilogue.  Tiles are 256 x 512 (two
// sub-tiles that share each K slice's rows of the first operand), 256 x 256 or
// 256 x 128; both gradients' tiles go in one launch.  Where there are fewer
// tiles than pairs the sum is cut into parts, whose fp32 sums a second launch
// joins in a fixed order.  The forward product of few rows, and small ones, run
// turned round, on clusters (turned_kernel).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "act.cuh"
#include "tile.cuh"

namespace {

using namespace dmoe::tile;
using namespace dmoe::act;

constexpr int kEpiWarps = 16;  // four per TMEM lane quadrant, 64 columns of a sub-tile each
constexpr int kThreadsL = 64 + 32 * kEpiWarps;

template <int NS>
struct PlanL {
  static constexpr uint32_t SLAB_BYTES = kEpiWarps * SLAB32;
  static constexpr uint32_t STAGE = A_BYTES + NS * B_BYTES;
  static constexpr int FIT = static_cast<int>((kSmemMax - 1536 - SLAB_BYTES) / STAGE);
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr size_t SMEM = 1024 + STAGES * STAGE + SLAB_BYTES + 512;
  static_assert(STAGES >= 4 && SMEM <= kSmemMax, "shared-memory plan");
};

// What becomes of a product's sums on their way out.  Rows lie `cols` apart
// where nothing else is said.
struct Out {
  int rows, cols;
  const void* bias;          // [cols], bf16 or fp32 (NULL: none)
  int bias_f32;
  uint16_t* deriv;           // act'(z) (NULL: not kept)
  const uint16_t* residual;  // added, rows ld_res apart (NULL: none)
  int64_t ld_res;
  const uint16_t* factor;    // multiplied last (NULL: none)
  void* out;                 // bf16 or fp32
  int f32;
  float* part;               // fp32 sums of each part [parts][rows][cols] (NULL: one part)
};

struct ParamsL {
  CUtensorMap map_a[2], map_b[2];  // of kind 0 (y or dx) and 1 (dW)
  int b_mn;                        // kind 0: the second operand lies along its columns (y) or along the sum (dx)
  int a_rows;                      // kind 0: rows of map_a's box: what lies past the last row is not loaded
  int width[2];                    // columns of a sub-tile
  int first_dx, full, rem, early, extra;
  Grid grid[2];
  Out o[2];
  int32_t* err;
};

// 32 columns of one row: bias, activation, what is kept.  g receives act'.
template <int ACT>
__device__ __forceinline__ void activate(float* v, float* g, int n) {
#pragma unroll
  for (int q = 0; q < n; q += 2) {
    float2 y, s;
    if (ACT == DMOE_ACT_GELU) gelu_pair(make_float2(v[q], v[q + 1]), y, s);
    else silu_pair(make_float2(v[q], v[q + 1]), y, s);
    v[q] = y.x, v[q + 1] = y.y;
    g[q] = s.x, g[q + 1] = s.y;
  }
}

// Eight biases from column c on.
__device__ __forceinline__ void load_bias(const Out& o, int c, float* b) {
  if (o.bias_f32) {
    const float4* a = reinterpret_cast<const float4*>(static_cast<const float*>(o.bias) + c);
    const float4 u = __ldg(a), w = __ldg(a + 1);
    b[0] = u.x, b[1] = u.y, b[2] = u.z, b[3] = u.w;
    b[4] = w.x, b[5] = w.y, b[6] = w.z, b[7] = w.w;
  } else {
    unpack8x(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(o.bias) + c)), b);
  }
}

__device__ __forceinline__ void prefetch_l2(const void* a) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(a)) : "memory");
}

template <int ACT, int NS>
__global__ void __launch_bounds__(kThreadsL, 1) linear_kernel(const __grid_constant__ ParamsL p) {
  using PL = PlanL<NS>;
  constexpr int STAGES = PL::STAGES;
  constexpr uint32_t TMEM_COLS = 512;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* slab_mem = smem + STAGES * PL::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(slab_mem + PL::SLAB_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tempty + a, 2 * kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&p.map_a[0]);
    tma_prefetch_map(&p.map_b[0]);
    tma_prefetch_map(&p.map_a[1]);
    tma_prefetch_map(&p.map_b[1]);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, TMEM_COLS);
  fence_before_sync();
  cluster_sync();
  fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();

  const int U = static_cast<int>(gridDim.x >> 1);
  const int unit = static_cast<int>(blockIdx.x >> 1);

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t full_pair = dsmem_addr(smem_u32(full), 0);  // rank 0 counts both CTAs' bytes
      Item it;
      for (int j = 0; ok && item_of(p, unit, U, j, it); ++j) {
        const int kind = it.dx ? 0 : 1;
        const int m0 = it.m * 2 * BM + rank * BM;
        const int width = p.width[kind];
        const int n0 = it.c0 + rank * (width / 2);
        const bool a_mn = kind == 1, b_mn = kind == 1 || p.b_mn;
        // the bytes of both CTAs' rows of the first operand, and whether this one has any
        const bool a_none = !a_mn && m0 >= p.o[0].rows;
        const uint32_t a_bytes = a_mn || it.m * 2 * BM + BM < p.o[0].rows ? 2 * A_BYTES
                                                                          : static_cast<uint32_t>(p.a_rows) * BK * 2;
        const CUtensorMap* ma = &p.map_a[kind];
        const CUtensorMap* mb = &p.map_b[kind];
        const int subs = NS == 2 && it.wide ? 2 : 1;
        for (int i = it.k0; i < it.k1; ++i) {
          ok = mbar_wait(empty + stage, phase ^ 1u, abort_flag);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(full + stage, a_bytes + subs * width * BK * 2);
          const uint32_t bar = full_pair + 8u * stage;
          uint8_t* sa = smem + stage * PL::STAGE;
          uint8_t* sb = sa + A_BYTES;
          const int k0 = i * BK;
          if (a_mn) {
            tma_load_2d_pair(sa, ma, bar, m0, k0);
            tma_load_2d_pair(sa + ATOM, ma, bar, m0 + 64, k0);
          } else if (!a_none) {
            tma_load_2d_pair(sa, ma, bar, k0, m0);
          }
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            if (s == subs) break;
            if (b_mn) {
              tma_load_2d_pair(sb + s * B_BYTES, mb, bar, n0 + s * BN, k0);
              if (width == BN) tma_load_2d_pair(sb + s * B_BYTES + ATOM, mb, bar, n0 + s * BN + 64, k0);
            } else {
              tma_load_2d_pair(sb + s * B_BYTES, mb, bar, k0, n0 + s * BN);
            }
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every stage this CTA filled has been consumed before it may leave
      for (int s = 0; s < STAGES && ok; ++s) {
        ok = mbar_wait(empty + stage, phase ^ 1u, abort_flag);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        dmoe::raise_error(p.err, DMOE_SITE_GEMM_WAIT | DMOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ------------------------------------------------------------ MMA issue
      int stage = 0;
      uint32_t phase = 0;
      uint32_t acc = 0, acc_phase = 0;
      bool ok = true;
      // Of a descriptor only the start address (the low word) moves: by a
      // stage, a sub-tile or a K step, in 16-byte units.  The distance of
      // 64-column atoms (low word) goes by the operand's direction.
      constexpr uint32_t MN_STEP = (UMMA_K * 128) >> 4, K_STEP = (UMMA_K * 2) >> 4;
      const uint32_t hi = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem), 16, 1024) >> 32);
      uint32_t a_lo = 0, b_lo = 0, a_step = 0, b_step = 0, idesc = 0;
      // one K slice of sub-tile `s` from ring stage st into accumulator d
      auto mmas = [&](uint32_t d, int st, int s, bool first) {
        const uint32_t a = a_lo + st * (PL::STAGE >> 4);
        const uint32_t b = b_lo + st * (PL::STAGE >> 4) + s * (B_BYTES >> 4);
        mma_pair(d, a, hi, b, hi, idesc, first ? 0u : 1u);
#pragma unroll
        for (int kk = 1; kk < BK / UMMA_K; ++kk) mma_pair(d, a + a_step * kk, hi, b + b_step * kk, hi, idesc, 1u);
      };
      Item it;
      for (int j = 0; ok && item_of(p, unit, U, j, it); ++j) {
        const int kit = it.k1 - it.k0;
        const int kind = it.dx ? 0 : 1;
        const bool a_mn = kind == 1, b_mn = kind == 1 || p.b_mn;
        a_step = a_mn ? MN_STEP : K_STEP;
        b_step = b_mn ? MN_STEP : K_STEP;
        a_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem), a_mn ? ATOM : 16, 1024));
        b_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem) + A_BYTES, b_mn ? ATOM : 16, 1024));
        idesc = idesc_bf16(2 * BM, p.width[kind], a_mn, b_mn);
        if (NS == 2) {
          // both accumulators belong to this tile: sub-tile 0 starts once its
          // columns are drained, sub-tile 1's first slices stay in the ring
          // until its own are (without a second sub-tile its columns are
          // waited for all the same, so that the barrier's phases keep step)
          ok = mbar_wait_cluster(tempty, acc_phase ^ 1u, abort_flag);
          if (!ok) break;
          fence_after_sync();
          bool free1 = false;
          int held = 0;
          const int hstage = stage;
          auto catch_up = [&]() {
            for (int h = 0; h < held; ++h) {
              const int st = (hstage + h) % STAGES;
              mmas(tmem_base + BN, st, 1, h == 0);
              mma_commit_pair(empty + st);
            }
            held = 0;
          };
          for (int i = 0; i < kit; ++i) {
            ok = mbar_wait(full + stage, phase, abort_flag);
            if (!ok) break;
            fence_after_sync();
            mmas(tmem_base, stage, 0, i == 0);
            if (!it.wide) {
              mma_commit_pair(empty + stage);
            } else {
              if (!free1) free1 = mbar_try_wait_cluster(tempty + 1, acc_phase ^ 1u);
              if (!free1 && held + 1 == STAGES) {
                ok = mbar_wait_cluster(tempty + 1, acc_phase ^ 1u, abort_flag);
                if (!ok) break;
                free1 = true;
              }
              if (free1) {
                fence_after_sync();
                catch_up();
                mmas(tmem_base + BN, stage, 1, i == 0);
                mma_commit_pair(empty + stage);
              } else {
                ++held;
              }
            }
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (held > 0 || !it.wide) {
            ok = mbar_wait_cluster(tempty + 1, acc_phase ^ 1u, abort_flag);
            if (!ok) break;
            fence_after_sync();
            catch_up();
          }
          mma_commit_pair(tfull);
          acc_phase ^= 1u;
        } else {
          ok = mbar_wait_cluster(tempty + acc, acc_phase ^ 1u, abort_flag);
          if (!ok) break;
          fence_after_sync();
          for (int i = 0; i < kit; ++i) {
            ok = mbar_wait(full + stage, phase, abort_flag);
            if (!ok) break;
            fence_after_sync();
            mmas(tmem_base + acc * BN, stage, 0, i == 0);
            mma_commit_pair(empty + stage);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          mma_commit_pair(tfull + acc);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (!ok) {
        dmoe::raise_error(p.err, DMOE_SITE_GEMM_WAIT | DMOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int quad = warp & 3;         // TMEM lanes 32 quad .. 32 quad + 31
    const int part = (warp - 2) >> 2;  // columns 64 part .. + 63 of a sub-tile
    const uint32_t slab = smem_u32(slab_mem + (warp - 2) * SLAB32);
    const uint32_t tempty_pair = dsmem_addr(smem_u32(tempty), 0);
    uint32_t acc = 0, acc_phase = 0;
    bool ok = true;
    auto release = [&]() {  // this warp is done reading accumulator acc
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty_pair + 8u * acc);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    };
    Item it;
    for (int j = 0; ok && item_of(p, unit, U, j, it); ++j) {
      const int kind = it.dx ? 0 : 1;
      const Out& o = p.o[kind];
      const int width = p.width[kind];
      const int row0 = it.m * 2 * BM + rank * BM + quad * 32;  // this warp's 32 rows
      const int row = row0 + lane;
      const int rows = o.rows - row0;  // rows of them that exist (or fewer than 1)
      // what the epilogue reads of its row, on its way while the product runs
      if (row < o.rows && !o.part && (o.residual || o.factor)) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const int c = it.c0 + s * BN + part * 64;
          if (part * 64 < width && c < o.cols) {
            if (o.residual) prefetch_l2(o.residual + static_cast<int64_t>(row) * o.ld_res + c);
            if (o.factor) prefetch_l2(o.factor + static_cast<int64_t>(row) * o.cols + c);
          }
        }
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int c = it.c0 + s * BN + part * 64;  // this warp's first column
        if (NS == 1 || s == 0) {
          ok = mbar_wait_cluster(tfull + acc, acc_phase, abort_flag);
          if (!ok) break;
          __syncwarp();
        }
        if ((NS == 2 && s == 1 && !it.wide) || part * 64 >= width || rows <= 0 || c >= o.cols) {
          release();  // nothing here
          continue;
        }
        fence_after_sync();
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * BN + part * 64;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float v[32];
          __syncwarp();
          tmem_ld32(tb + 32 * h, v);
          tmem_wait(v);
          if (h == 1) release();  // the last of this warp's columns are in registers
          const int ch = c + 32 * h;
          const int cols = o.cols - ch;  // columns that exist from here on
          if (cols <= 0) continue;
          if (o.part) {
            write_rows32(slab, lane, v, o.part + (static_cast<int64_t>(it.part) * o.rows + row0) * o.cols + ch, o.cols,
                         rows, cols);
            continue;
          }
          if (o.bias) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float b[8];
              if (8 * q < cols) {
                load_bias(o, ch + 8 * q, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[8 * q + i] += b[i];
              }
            }
          }
          if (ACT != DMOE_ACT_NONE) {
            float g[32];
            activate<ACT>(v, g, 32);
            if (o.deriv)
              write_rows32(slab, lane, g, o.deriv + static_cast<int64_t>(row0) * o.cols + ch, o.cols, rows, cols);
          }
          // y may be residual and dx factor: each value is read by the warp that
          // overwrites it, before
          if (o.residual && row < o.rows)
            join_row32<false>(v, o.residual + static_cast<int64_t>(row) * o.ld_res + ch, cols);
          if (o.factor && row < o.rows) join_row32<true>(v, o.factor + static_cast<int64_t>(row) * o.cols + ch, cols);
          const int64_t at = static_cast<int64_t>(row0) * o.cols + ch;
          if (o.f32) write_rows32(slab, lane, v, static_cast<float*>(o.out) + at, o.cols, rows, cols);
          else write_rows32(slab, lane, v, static_cast<uint16_t*>(o.out) + at, o.cols, rows, cols);
        }
      }
    }
    if (!ok && lane == 0) {
      dmoe::raise_error(p.err, DMOE_SITE_GEMM_WAIT | DMOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }

  __syncwarp();
  if (*abort_flag) {  // a wait gave up: let copies and products under way land before their memory goes
    const uint64_t t0 = dmoe::globaltimer_ns();
    while (dmoe::globaltimer_ns() - t0 < kDrainNs) __nanosleep(1000);
  }
  fence_before_sync();
  // a CTA of a pair leaves only once the other no longer reads or signals
  // its shared memory
  cluster_sync();
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------- the product turned
// For few rows W's bytes are all there is to do, and a tile of 256 rows of x is
// nearly empty: its product takes as long as its loads.  So W takes the place
// of the first operand, 128 of its columns the rows of a tile, and the rows of
// x, 16 to 128 of them, are the columns: y^T = W^T x^T, and the product is a
// tenth of the loads.  One CTA a tile and part of K, a deep ring of 16 KB slices
// of W; the parts of a tile are a cluster, whose CTAs meet in each other's
// shared memory, in a fixed order.  More rows take blocks of 128: small
// products, too, are done sooner in 5 us of launch, first loads and epilogue
// than in the 8 of the pairs below.  (us, those and these: 1 x 14336 x 4096
// 26.5 and 22, 64 x 1024 x 1024 12.2 and 6.1, 128 x 4096 x 4096 18.5 and 13.2,
// 512 x 1024 x 1024 12.8 and 8.0.)  The gradients, of which one has a long sum or
// many tiles, gained nothing turned: with both in one launch of clusters 70 sizes
// from 8 x 512 x 512 on took the same or up to 19% more.
constexpr int kTurnedRows = 128;  // of a block
constexpr int kFewTile = 128;     // columns of W
constexpr int kFewStages = 11;
constexpr int kFewEpiWarps = 8;
constexpr int kFewThreads = 64 + 32 * kFewEpiWarps;  // with the TMA producer and the MMA issuer

struct ParamsF {
  CUtensorMap map_w, map_x;
  int box;  // rows of x that are loaded
  int cols;  // tiles over the columns
  int tiles, parts, log_parts, slices;  // tiles: over the columns, then over the blocks of rows
  Out o;
  int32_t* err;
};

template <int ROWS>
struct PlanF {
  static constexpr uint32_t W_BYTES = 2 * ATOM;
  static constexpr uint32_t STAGE = W_BYTES + ROWS * BK * 2;
  static constexpr int FIT = static_cast<int>((kSmemMax - 2048) / STAGE);
  static constexpr int STAGES = FIT < kFewStages ? FIT : kFewStages;
  static constexpr size_t SMEM = 1024 + STAGES * STAGE + 512;
  static_assert(SMEM <= kSmemMax && STAGE % 1024 == 0, "shared-memory plan");
  static_assert(ROWS * kFewTile * sizeof(float) <= STAGES * STAGE, "the parts' sums take the ring's place");
};

// 16 consecutive fp32 columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_load16(uint32_t ta, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(ta)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

__device__ __forceinline__ uint32_t bf16_pair(float2 v) {
  const __nv_bfloat162 h = __float22bfloat162_rn(v);
  return reinterpret_cast<const uint32_t&>(h);
}

__device__ __forceinline__ float2 pair_of(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

template <int ACT>
__device__ __forceinline__ void act_pair(float2 z, float2& y, float2& g) {
  if (ACT == DMOE_ACT_GELU) gelu_pair(z, y, g);
  else if (ACT == DMOE_ACT_SILU) silu_pair(z, y, g);
  else y = z, g = make_float2(1.f, 1.f);
}

__device__ __forceinline__ float2 dsmem_ld_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int ACT, int ROWS>
__global__ void __launch_bounds__(kFewThreads, 1) turned_kernel(const __grid_constant__ ParamsF p) {
  using PL = PlanF<ROWS>;
  constexpr int STAGES = PL::STAGES;
  constexpr uint32_t TMEM_COLS = 2 * ROWS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * PL::STAGE);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tempty + a, kFewEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&p.map_w);
    tma_prefetch_map(&p.map_x);
  }
  if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  // one tile a cluster, or where K is whole as many as it takes
  const int rank = p.parts > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = static_cast<int>(blockIdx.x) >> p.log_parts;
  const int next = p.parts > 1 ? p.tiles : static_cast<int>(gridDim.x);
  const int k0 = p.slices * rank >> p.log_parts, k1 = p.slices * (rank + 1) >> p.log_parts;  // below 2^31: 64 long
  const int quad = warp & 3;  // epilogue: TMEM lanes, and columns of W, 32 quad .. 32 quad + 31
  float* sums = reinterpret_cast<float*>(smem);  // parts > 1: [M][kFewTile], once the ring is done with
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int tile = first; ok && tile < p.tiles; tile += next) {
        const int block = tile / p.cols, c0 = (tile - block * p.cols) * kFewTile;
        for (int i = k0; i < k1; ++i) {
          ok = mbar_wait(empty + stage, phase ^ 1u, abort_flag);
          if (!ok) break;
          uint8_t* sw = smem + stage * PL::STAGE;
          mbar_arrive_expect_tx(full + stage, PL::W_BYTES + p.box * BK * 2);
          tma_load_2d(sw, &p.map_w, full + stage, c0, i * BK);
          tma_load_2d(sw + ATOM, &p.map_w, full + stage, c0 + 64, i * BK);
          tma_load_2d(sw + PL::W_BYTES, &p.map_x, full + stage, i * BK, block * ROWS);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every stage has been consumed before the CTA may leave
      for (int s = 0; s < STAGES && ok; ++s) {
        ok = mbar_wait(empty + stage, phase ^ 1u, abort_flag);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, acc = 0, acc_phase = 0;
      constexpr uint32_t MN_STEP = (UMMA_K * 128) >> 4, K_STEP = (UMMA_K * 2) >> 4;
      const uint64_t a0 = sdesc_sw128(smem_u32(smem), ATOM, 1024);
      const uint64_t b0 = sdesc_sw128(smem_u32(smem) + PL::W_BYTES, 16, 1024);
      constexpr uint32_t idesc = idesc_bf16(kFewTile, ROWS, true, false);
      for (int tile = first; ok && tile < p.tiles; tile += next) {
        ok = mbar_wait(tempty + acc, acc_phase ^ 1u, abort_flag);
        if (!ok) break;
        fence_after_sync();
        for (int i = k0; i < k1; ++i) {
          ok = mbar_wait(full + stage, phase, abort_flag);
          if (!ok) break;
          fence_after_sync();
          const uint64_t off = static_cast<uint64_t>(stage) * (PL::STAGE >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / UMMA_K; ++kk)
            mma_bf16(tmem_base + acc * ROWS, a0 + off + MN_STEP * kk, b0 + off + K_STEP * kk, idesc, i > k0 || kk > 0);
          mma_commit(empty + stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(tfull + acc);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
  } else {
    uint32_t acc = 0, acc_phase = 0;
    for (int tile = first; ok && tile < p.tiles; tile += next) {
      const int block = tile / p.cols, c = (tile - block * p.cols) * kFewTile + quad * 32 + lane;
      const int row0 = block * ROWS, rows = min(ROWS, p.o.rows - row0);
      float bias = 0.f;
      if (p.parts == 1 && p.o.bias && c < p.o.cols)
        bias = p.o.bias_f32 ? __ldg(static_cast<const float*>(p.o.bias) + c)
                            : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p.o.bias) + c)) << 16);
      ok = mbar_wait(tfull + acc, acc_phase, abort_flag);
      if (!ok) break;
      __syncwarp();
      fence_after_sync();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * ROWS;
#pragma unroll 1
      for (int r = (warp - 2) / 4 * 16; r < rows; r += kFewEpiWarps / 4 * 16) {
        float v[16];
        __syncwarp();
        tmem_load16(tb + r, v);
        if (p.parts > 1) {
#pragma unroll
          for (int q = 0; q < 16; ++q)
            if (r + q < rows) sums[(r + q) * kFewTile + quad * 32 + lane] = v[q];
        } else if (c < p.o.cols) {
          // what is added is fetched for all rows at once: y may be where it lies
          uint16_t add[16];
          if (p.o.residual) {
#pragma unroll
            for (int q = 0; q < 16; ++q) add[q] = r + q < rows ? p.o.residual[(row0 + r + q) * p.o.ld_res + c] : 0;
          }
          const int64_t at = static_cast<int64_t>(row0 + r) * p.o.cols + c;
#pragma unroll
          for (int q = 0; q < 16; q += 2) {
            float2 y, g;
            act_pair<ACT>(make_float2(v[q] + bias, v[q + 1] + bias), y, g);
            if (p.o.residual) y = dmoe::f2_add(y, make_float2(__uint_as_float(add[q] << 16), __uint_as_float(add[q + 1] << 16)));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (r + q + j >= rows) continue;
              if (ACT != DMOE_ACT_NONE && p.o.deriv) p.o.deriv[at + static_cast<int64_t>(q + j) * p.o.cols] = bf16_bits(j ? g.y : g.x);
              static_cast<uint16_t*>(p.o.out)[at + static_cast<int64_t>(q + j) * p.o.cols] = bf16_bits(j ? y.y : y.x);
            }
          }
        }
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty + acc);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  if (!ok && (warp > 1 ? lane == 0 : true)) {
    dmoe::raise_error(p.err, DMOE_SITE_GEMM_WAIT | DMOE_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  __syncwarp();
  if (*abort_flag) {  // a wait gave up: let copies and products under way land before their memory goes
    const uint64_t t0 = dmoe::globaltimer_ns();
    while (dmoe::globaltimer_ns() - t0 < kDrainNs) __nanosleep(1000);
  }
  if (p.parts > 1) {
    __syncwarp();
    cluster_sync();  // every part's sums are there
    // this CTA's share of the columns, of all rows, two columns at a time; four of
    // those pairs together, for the way to the other CTAs and to what is added
    const int log_pairs = 6 - p.log_parts, share = 2 << log_pairs;
    const int block = first / p.cols, c0 = (first - block * p.cols) * kFewTile;
    const int row0 = block * ROWS, rows = min(ROWS, p.o.rows - row0);
    const int from = rank * share, pairs = rows << log_pairs;
    for (int i0 = threadIdx.x; i0 < pairs; i0 += 4 * kFewThreads) {
      float2 v[4][8], bias[4];
      uint32_t add[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * kFewThreads;
        const int r = i >> log_pairs, col = from + 2 * (i & (share / 2 - 1)), c = c0 + col;
        bias[j] = make_float2(0.f, 0.f);
        add[j] = 0;
        if (i >= pairs || c >= p.o.cols) continue;
        const uint32_t at = smem_u32(sums + r * kFewTile + col);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[j][q] = q < p.parts ? dsmem_ld_f32x2(dsmem_addr(at, q)) : make_float2(0.f, 0.f);
        if (p.o.bias)
          bias[j] = p.o.bias_f32 ? __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(p.o.bias) + c))
                                 : pair_of(__ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.o.bias) + c)));
        if (p.o.residual) add[j] = *reinterpret_cast<const uint32_t*>(p.o.residual + (row0 + r) * p.o.ld_res + c);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * kFewThreads;
        const int r = i >> log_pairs, c = c0 + from + 2 * (i & (share / 2 - 1));
        if (i >= pairs || c >= p.o.cols) continue;
        float2 sum = v[j][0], y, g;
#pragma unroll
        for (int q = 1; q < 8; ++q) sum = dmoe::f2_add(sum, v[j][q]);
        act_pair<ACT>(dmoe::f2_add(sum, bias[j]), y, g);
        const int64_t to = static_cast<int64_t>(row0 + r) * p.o.cols + c;
        if (ACT != DMOE_ACT_NONE && p.o.deriv) *reinterpret_cast<uint32_t*>(p.o.deriv + to) = bf16_pair(g);
        if (p.o.residual) y = dmoe::f2_add(y, pair_of(add[j]));
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o.out) + to) = bf16_pair(y);
      }
    }
    __syncwarp();
    cluster_sync();  // the others have read this one's
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// Joins the parts of up to two products, eight columns a piece.  SHARE
// neighbouring lanes take every SHARE-th part of a piece and add theirs up, in
// a fixed order: where pieces are few the parts' loads go side by side.
struct Join {
  Out o[2];
  int parts[2];
  int64_t vecs[2];  // 8-column pieces (0: nothing to join)
};

template <int ACT, int SHARE>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Join p) {
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / SHARE;
  const int mine = threadIdx.x % SHARE;
  const int kind = i < p.vecs[0] ? 0 : 1;
  if (kind == 1) i -= p.vecs[0];
  const bool live = i < p.vecs[kind];
  const Out& o = p.o[kind];
  const int per_row = o.cols >> 3;
  const int64_t row = live ? i / per_row : 0;
  const int c = live ? static_cast<int>(i - row * per_row) * 8 : 0;
  const int64_t at = row * o.cols + c, step = static_cast<int64_t>(o.rows) * o.cols;
  float v[8] = {};
  if (live) {
#pragma unroll 8
    for (int s = mine; s < p.parts[kind]; s += SHARE) {
      const float4* a = reinterpret_cast<const float4*>(o.part + s * step + at);
      const float4 u = __ldg(a), w = __ldg(a + 1);
      v[0] += u.x, v[1] += u.y, v[2] += u.z, v[3] += u.w;
      v[4] += w.x, v[5] += w.y, v[6] += w.z, v[7] += w.w;
    }
  }
#pragma unroll
  for (int h = SHARE / 2; h > 0; h /= 2) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += __shfl_xor_sync(0xffffffffu, v[q], h);
  }
  if (!live || mine != 0) return;
  if (o.bias) {
    float b[8];
    load_bias(o, c, b);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += b[q];
  }
  if (ACT != DMOE_ACT_NONE) {
    float g[8];
    activate<ACT>(v, g, 8);
    if (o.deriv) *reinterpret_cast<uint4*>(o.deriv + at) = pack8x(g);
  }
  float f[8];
  if (o.residual) {
    unpack8x(*reinterpret_cast<const uint4*>(o.residual + row * o.ld_res + c), f);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += f[q];
  }
  if (o.factor) {
    unpack8x(*reinterpret_cast<const uint4*>(o.factor + at), f);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= f[q];
  }
  if (o.f32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(o.out) + at);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.out) + at) = pack8x(v);
  }
}

// dz = bf16(dy deriv) (dz NULL: dy is dz), and the sums over every gridDim.x-th
// stripe of rows of the unrounded products: one fp32 row of `sums` each, or,
// where the stripes are a cluster (JOINED), their sum in `sums` itself (sums NULL:
// none).  256 columns a block, eight rows at a time; JOINED, for fewer rows, 64
// columns and 32 rows, for more blocks (a whole backward of 1024 x 1024 x 1024
// takes 16.9 us so, 25 in 256 columns).  dz is in 16 bits because both
// products take it so: half a step of bf16 on each of a sum's terms.  HBM-bound:
// 4093 x 10240 37 us, 6.8 TB/s (in one wave: with eight rows in flight and three
// blocks an SM, in two, 70).
template <bool JOINED>
__global__ void __launch_bounds__(256) dz_kernel(const uint16_t* __restrict__ dy, int64_t lddy,
                                                 const uint16_t* __restrict__ deriv, int M, int N,
                                                 uint16_t* __restrict__ dz, float* __restrict__ sums) {
  constexpr int COLS = JOINED ? 64 : 256, ROWS = 2048 / COLS;  // of a block at a time
  __shared__ __align__(16) float sh[ROWS][COLS + 4];  // filled four columns at a time
  __shared__ float total[COLS];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int at = threadIdx.x % (COLS / 8) * 8, row = threadIdx.x / (COLS / 8);
  const int c = blockIdx.y * COLS + at;
  float s[8] = {};
  if (c < N) {
#pragma unroll 4
    for (int64_t r = blockIdx.x * ROWS + row; r < M; r += gridDim.x * ROWS) {
      float f[8];
      unpack8x(__ldg(reinterpret_cast<const uint4*>(dy + r * lddy + c)), f);
      if (deriv) {
        float g[8];
        unpack8x(__ldg(reinterpret_cast<const uint4*>(deriv + r * N + c)), g);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] *= g[q];
        if (dz) *reinterpret_cast<uint4*>(dz + r * N + c) = pack8x(f);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += f[q];
    }
  }
  if (!sums) return;
#pragma unroll
  for (int q = 0; q < 8; q += 4) *reinterpret_cast<float4*>(&sh[row][at + q]) = make_float4(s[q], s[q + 1], s[q + 2], s[q + 3]);
  __syncthreads();
  const int mine = threadIdx.x, col = blockIdx.y * COLS + mine;
  float t = 0.f;
  if (mine < COLS) {
#pragma unroll
    for (int w = 0; w < ROWS; ++w) t += sh[w][mine];
  }
  if (JOINED) {
    if (mine < COLS) total[mine] = t;
    cluster_sync();
    if (cluster_ctarank() == 0 && mine < COLS && col < N) {
      t = 0.f;
      for (unsigned q = 0; q < gridDim.x; ++q) t += dsmem_ld_f32(dsmem_addr(smem_u32(total + mine), q));
      sums[col] = t;
    }
    cluster_sync();  // the others' sums have been read
  } else if (col < N) {
    sums[static_cast<int64_t>(blockIdx.x) * N + col] = t;
  }
}

__global__ void __launch_bounds__(256) dbias_kernel(const float* __restrict__ sums, int n, int N,
                                                    float* __restrict__ dbias) {
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= N) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = 0; i < n; ++i) s += __ldg(sums + static_cast<int64_t>(i) * N + c);
  dbias[c] = s;
}

// ----------------------------------------------------------------- host side

constexpr int kMaxParts = 64;
constexpr int kMinSlices = 4;  // of a part

// What the items' times leave out: launch and first loads, and the last
// epilogue (with an activation more).  Single tiles of 264 columns of K, none
// and gelu: 7.0 and 9.1 us.
constexpr int64_t kTilesNs = 5000, kTurnedNs = 2500;
int64_t last_epilogue_ns(bool act) { return act ? 2700 : 1000; }

// Nanoseconds of an item: `busy` pairs at work, each with this many K slices
// of a tile.  A slice costs what its product or its loads from L2 take or,
// where no other pair reads the same columns (alone), what its bytes take from
// HBM at 6.5 TB/s.  A 512-wide tile, which fills the TMEM, also waits for part of
// its epilogue; of a narrower one the next product hides it, unless it is
// longer (several: pairs have more than one), as with an activation and its
// derivative over a short sum.
// Measured: 1024 x 2048 x 2048 in tiles of 128, 256 and 512 20, 24 and 41 us, in
// two parts 22, 19 and -; 8192 x 512 x 2048, gelu 44, 37 and 40; 8192 x 2048 x
// 512 28, 22 and 33; 8192 x 14336 x 4096 -, 610 and 572.
int64_t item_ns(int slices, int tile, bool alone, int busy, bool act, bool several) {
  const int64_t product = tile == 2 * BN ? 630 : tile == BN ? 400 : 310;
  const int64_t bytes = alone ? static_cast<int64_t>(tile) * BK * 2 * busy / 6500 : 0;
  const int64_t sums = slices * std::max(product, bytes);
  if (tile == 2 * BN) return sums + (act ? 11000 : 5500);
  return several ? std::max<int64_t>(sums, tile == BN ? (act ? 7000 : 4000) : (act ? 5000 : 2500)) : sums;
}

// A product [rows, cols] over K slices, and how it is cut.
struct Want {
  int rows, cols, slices;
  bool act;  // an activation in the epilogue
  int tile, parts;
  int items() const { return ceil_div(rows, 2 * BM) * ceil_div(cols, tile) * parts; }
  int64_t ns(int busy) const {
    return item_ns(ceil_div(slices, parts), tile, rows <= 2 * BM, std::min(busy, kUnits), act && parts == 1, busy > kUnits);
  }
  // the join: a launch, and the sums' way to memory and back
  int64_t join_ns() const {
    return parts > 1 ? static_cast<int64_t>(parts) * rows * cols * 8 / 6500 : 0;
  }
};

// Chooses tiles and parts of up to two products (b.rows == 0: one): the cut
// whose busiest pair is done first.  Parts only where there are at most two
// items a pair, which bounds the sums that they leave (part_bytes()).
int64_t choose(Want& a, Want& b) {
  Want best_a = a, best_b = b;
  int64_t least = -1;
  static constexpr int kParts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
  auto tries = [](const Want& w, int tile, int parts) {
    if (parts == 1) return true;
    Want t = w;
    t.tile = tile, t.parts = parts;
    return w.slices / parts >= kMinSlices && t.items() <= 2 * kUnits;
  };
  auto weigh = [&](const Want& x, const Want& y) {
    const int nx = x.items(), ny = y.rows ? y.items() : 0;
    const int64_t lx = x.ns(nx + ny), ly = ny ? y.ns(nx + ny) : 1;
    const int64_t busiest = (ny == 0 || lx >= ly ? dealt(nx, lx, ny, ly, kUnits) : dealt(ny, ly, nx, lx, kUnits)).busiest;
    const int64_t joins = x.join_ns() + (ny ? y.join_ns() : 0);
    const int64_t ns = busiest + joins + (x.parts > 1 || (ny && y.parts > 1) ? 2500 : 0);
    if (least < 0 || ns < least) {
      least = ns;
      best_a = x, best_b = y;
    }
  };
  a.parts = b.parts = 1;
  a.tile = b.tile = 2 * BN;
  weigh(a, b);
  for (const int ta : {BN, BN / 2})
    for (const int tb : {BN, BN / 2}) {
      if (!b.rows && tb != BN) continue;
      for (const int pa : kParts) {
        if (!tries(a, ta, pa)) break;
        if (b.rows && (pa & (pa - 1))) continue;  // of two products powers of two alone: each try takes the host 50 ns
        for (const int pb : kParts) {
          if (pb > 1 && (!b.rows || !tries(b, tb, pb))) break;
          if (pb & (pb - 1)) continue;
          a.tile = ta, a.parts = pa, b.tile = tb, b.parts = pb;
          weigh(a, b);
        }
      }
    }
  a = best_a, b = best_b;
  return least + kTilesNs + last_epilogue_ns(a.act);
}

// Bytes that the parts of a [rows, cols] product's sums need at most: 2 kUnits
// items of 256 x 256.  Never falls with rows.
constexpr int64_t kMostPartSums = static_cast<int64_t>(2 * kUnits) * 2 * BM * BN;
size_t part_bytes(int64_t rows, int64_t cols) {
  const int64_t most = std::min<int64_t>(kMostPartSums, kMaxParts * rows * cols);
  return static_cast<size_t>(round_up(most * sizeof(float), 256));
}

Grid grid_of(const Want& w, int busy, int raster) {
  Grid g = cut_grid(w.rows, w.cols, w.slices * BK, raster, w.parts, w.tile);
  g.time = std::max<int64_t>(1, w.ns(busy));
  return g;
}

template <int ACT, int NS>
dmoe_status launch_linear(ParamsL& p, const Grid& ga, const Grid& gb, const dmoe::DeviceInfo& di, cudaStream_t st) {
  auto kern = linear_kernel<ACT, NS>;
  const size_t smem = PlanL<NS>::SMEM;
  static std::atomic<int> clusters[64];
  int n = clusters[di.device].load(std::memory_order_acquire);
  if (n == 0) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(di.sm_count & ~1));
    cfg.blockDim = dim3(kThreadsL);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    if (n < 1) return DMOE_ERR_UNSUPPORTED;
    clusters[di.device].store(n, std::memory_order_release);
  }
  const int units = static_cast<int>(std::min<int64_t>(n, static_cast<int64_t>(ga.items) + gb.items));
  p.first_dx = ga.items > 0 && (gb.items == 0 || ga.time >= gb.time);
  p.grid[0] = p.first_dx ? ga : gb;
  p.grid[1] = p.first_dx ? gb : ga;
  const Dealt r = dealt(p.grid[0].items, p.grid[0].time, p.grid[1].items, std::max<int64_t>(1, p.grid[1].time), units);
  p.full = r.full, p.rem = r.rem, p.early = r.early, p.extra = r.extra;
  const cudaError_t e = dmoe::launch_pdl_cluster(kern, dim3(2 * units), dim3(kThreadsL), smem, st, 2, p);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

template <int ACT>
dmoe_status join(const Out* o, int parts_a, int parts_b, cudaStream_t st) {
  Join j{};
  for (int k = 0; k < 2; ++k) {
    j.o[k] = o[k];
    j.parts[k] = k ? parts_b : parts_a;
    j.vecs[k] = o[k].part ? static_cast<int64_t>(o[k].rows) * (o[k].cols >> 3) : 0;
  }
  const int64_t vecs = j.vecs[0] + j.vecs[1];
  if (vecs == 0) return DMOE_OK;
  // the parts side by side as long as that leaves no SM more than its threads
  const bool share = vecs * 8 <= 4 * kUnits * 1024;
  const int64_t blocks = (vecs * (share ? 8 : 1) + 255) / 256;
  const cudaError_t e = dmoe::launch_pdl(share ? join_kernel<ACT, 8> : join_kernel<ACT, 1>,
                                         dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, j);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

// Clusters of so many CTAs of a turned product that are resident together, as
// the device answers once (of 8 there are fewer than 16, however many SMs are
// free: 256 x 1024 x 1024 in 16 of them 14.2 us, in two waves; 0: it does not say).
int resident_clusters(int parts, const dmoe::DeviceInfo& di) {
  static std::atomic<int> kept[64][4];
  const int at = parts == 8 ? 3 : parts == 4 ? 2 : parts == 2 ? 1 : 0;
  int n = kept[di.device][at].load(std::memory_order_acquire);
  if (n == 0) {
    auto kern = turned_kernel<DMOE_ACT_NONE, kTurnedRows>;
    constexpr size_t smem = PlanF<kTurnedRows>::SMEM;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(parts));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(parts);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    kept[di.device][at].store(n, std::memory_order_release);
  }
  return n;
}

// The parts of a turned product (a cluster's CTAs: 1, 2, 4 or 8, as many as are
// resident together), and its nanoseconds.  A slice takes a CTA 0.27 us (0.30
// where K is whole), or its share of HBM's 6.5 TB/s; the epilogue, four pairs of
// columns a thread in 1 us behind the cluster's meeting, or of a whole tile 32
// rows in 0.2, 0.9 with an activation.  Of 132 sizes from 4 x 256 x 264 to 6000 x
// 4096 x 4096, which was quicker, this or pairs, is met but for 1% of the time
// with an activation and 0.4% without.
struct TurnedCut {
  int rows, parts;
  int64_t ns;
};
TurnedCut cut_turned(int M, int K, int N, bool act, const dmoe::DeviceInfo& di) {
  const int rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : kTurnedRows;
  const int cols = ceil_div(N, kFewTile), blocks = ceil_div(M, rows), slices = ceil_div(K, BK);
  const int64_t tiles = static_cast<int64_t>(cols) * blocks;
  int parts = 8;
  while (parts > 1 && (slices < 2 * parts || tiles > resident_clusters(parts, di))) parts /= 2;
  const int64_t busy = std::min<int64_t>(tiles * parts, 2 * kUnits);
  const int64_t bytes = static_cast<int64_t>(2 * ATOM) * busy / std::min<int64_t>(blocks, busy);
  const int64_t slice = std::max<int64_t>(parts > 1 ? 270 : 300, bytes / 6500);
  const int64_t live = std::min(M, rows);
  const int64_t epilogue = parts > 1 ? 1500 + ceil_div(live * (kFewTile / 2 / parts), 4 * kFewThreads) * 1000 + 10 * live
                                     : ceil_div(live, 4 * kFewEpiWarps) * (act ? 875 : 225);
  const int64_t waves = (tiles * parts + 2 * kUnits - 1) / (2 * kUnits);
  return TurnedCut{rows, parts, waves * (ceil_div(slices, parts) * slice + epilogue) + kTurnedNs};
}

template <int ACT, int ROWS>
cudaError_t launch_turned(const ParamsF& p, const dmoe::DeviceInfo& di, cudaStream_t st) {
  auto kern = turned_kernel<ACT, ROWS>;
  constexpr size_t smem = PlanF<ROWS>::SMEM;
  static std::atomic<uint64_t> opted{0};
  const uint64_t bit = uint64_t(1) << di.device;
  if (!(opted.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    opted.fetch_or(bit, std::memory_order_acq_rel);
  }
  if (p.parts == 1)
    return dmoe::launch_pdl(kern, dim3(static_cast<unsigned>(std::min(di.sm_count, p.tiles))), dim3(kFewThreads), smem, st, p);
  return dmoe::launch_pdl_cluster(kern, dim3(static_cast<unsigned>(p.tiles * p.parts)), dim3(kFewThreads), smem, st, p.parts,
                                  p);
}

template <int ACT>
dmoe_status run_turned(const uint16_t* x, int64_t ldx, const uint16_t* w, int K, const Out& o, const TurnedCut& cut,
                       const dmoe::DeviceInfo& di, cudaStream_t st) {
  ParamsF p{};
  p.box = std::min(o.rows, cut.rows);
  p.cols = ceil_div(o.cols, kFewTile);
  p.tiles = p.cols * ceil_div(o.rows, cut.rows);
  p.parts = cut.parts;
  p.log_parts = cut.parts == 8 ? 3 : cut.parts / 2;
  p.slices = ceil_div(K, BK);
  p.o = o;
  p.err = di.err_word;
  if (!map_pitched(&p.map_w, w, K, o.cols, o.cols, 64, BK) || !map_pitched(&p.map_x, x, o.rows, K, ldx, BK, p.box))
    return DMOE_ERR_CUDA;
  const cudaError_t e = cut.rows == 16   ? launch_turned<ACT, 16>(p, di, st)
                        : cut.rows == 32 ? launch_turned<ACT, 32>(p, di, st)
                        : cut.rows == 64 ? launch_turned<ACT, 64>(p, di, st) : launch_turned<ACT, kTurnedRows>(p, di, st);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

// Runs the products a (kind 0) and b (kind 1; b.rows == 0: none) as chosen,
// and joins what was cut.
template <int ACT>
dmoe_status run_products(ParamsL& p, const Want& a, const Want& b, float* part_a, float* part_b,
                         const dmoe::DeviceInfo& di, cudaStream_t st) {
  const int busy = (a.rows ? a.items() : 0) + (b.rows ? b.items() : 0);
  const bool wide = (a.rows ? a.tile : b.tile) == 2 * BN;
  Grid ga{}, gb{};
  if (a.rows) ga = grid_of(a, busy, 16);
  if (b.rows) gb = grid_of(b, busy, 16);
  p.width[0] = std::min(a.tile, BN);
  p.width[1] = std::min(b.tile, BN);
  if (ga.parts > 1) p.o[0].part = part_a;
  if (gb.parts > 1) p.o[1].part = part_b;
  const dmoe_status s = wide ? launch_linear<ACT, 2>(p, ga, gb, di, st) : launch_linear<ACT, 1>(p, ga, gb, di, st);
  if (s != DMOE_OK) return s;
  return join<ACT>(p.o, ga.parts, gb.parts, st);
}

bool sizes_ok(int M, int K, int N) {
  return M >= 0 && K >= 8 && N >= 8 && (K & 7) == 0 && (N & 7) == 0 && K <= (1 << 20) && N <= (1 << 20);
}
bool bad_pitch(int64_t ld, int cols) { return ld < cols || (ld & 7); }
bool off16(const void* a) { return !dmoe::aligned16(a); }

// Rows of the first operand's box: what lies past the last row is not loaded
// (it only reaches rows past it).
int box_rows(int rows) { return std::min(rows, BM); }

// Stripes of rows, a cluster, of a dz_kernel that joins its sums itself: up to
// 128 rows each (0: more rows, or more than some four blocks an SM, whose sums a
// launch of their own joins).  Us of a backward, joined and not: 400 x 264 x 264
// 9.7 and 11.7, 400 x 264 x 4096 (512 blocks) 19.7 and 21.4, 400 x 264 x 8192 27.9
// and 25.0, 2048 x 1024 x 1024 24.8 and 22.5.
int joined_stripes(int M, int N) {
  const int n = M > 256 ? 8 : M > 128 ? 4 : M > 64 ? 2 : 1;
  return M > 1024 || n * ceil_div(N, 64) > 4 * 2 * kUnits ? 0 : n;
}

// Stripes of rows whose sums dz_kernel leaves: some four blocks an SM.
int stripes(int M, int N) {
  const int cols = ceil_div(N, 256);
  return std::max(1, std::min(ceil_div(M, 32), 4 * 2 * kUnits / cols));
}

struct BackLayout {
  size_t dz, sums, part_x, part_w, bytes;
};
BackLayout back_layout(int M, int K, int N) {
  BackLayout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += static_cast<size_t>(round_up(static_cast<int64_t>(bytes), 256));
    return a;
  };
  l.dz = take(static_cast<size_t>(M) * N * 2);
  l.sums = take(static_cast<size_t>(std::max(1, 8 * kUnits / ceil_div(N, 256))) * N * sizeof(float));
  l.part_x = take(part_bytes(M, K));
  l.part_w = take(part_bytes(K, N));
  l.bytes = at;
  return l;
}

}  // namespace

DMOE_API size_t dmoe_linear_workspace_size(int M, int K, int N) {
  return sizes_ok(M, K, N) ? part_bytes(M, N) : 0;
}

DMOE_API dmoe_status dmoe_linear(const uint16_t* x, int64_t ldx, const uint16_t* w, const void* bias, int bias_f32,
                                 int act, const uint16_t* residual, int64_t ldr, int M, int K, int N, uint16_t* y,
                                 uint16_t* deriv, void* ws, size_t ws_bytes, dmoe_stream_t stream) {
  if (!sizes_ok(M, K, N) || act < DMOE_ACT_NONE || act > DMOE_ACT_SILU || (deriv && act == DMOE_ACT_NONE))
    return DMOE_ERR_INVALID_ARG;
  if (M == 0) return DMOE_OK;
  if (!x || !w || !y || bad_pitch(ldx, K) || (residual && bad_pitch(ldr, N))) return DMOE_ERR_INVALID_ARG;
  if (off16(x) || off16(w) || off16(bias) || off16(residual) || off16(y) || off16(deriv) ||
      (reinterpret_cast<uintptr_t>(ws) & 15))
    return DMOE_ERR_INVALID_ARG;
  if (y == x || y == w || y == deriv || (y == residual && M > 1 && ldr != N)) return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  const dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  Want a{M, N, ceil_div(K, BK), act != DMOE_ACT_NONE}, none{};
  const int64_t ns = choose(a, none);
  const TurnedCut cut = cut_turned(M, K, N, act != DMOE_ACT_NONE, di);
  const bool turned = cut.ns < ns;
  if (!turned && a.parts > 1 && (!ws || ws_bytes < part_bytes(M, N))) return DMOE_ERR_INVALID_ARG;
  const Out o{M, N, bias, bias_f32, deriv, residual, ldr, nullptr, y, 0, nullptr};
  float* part = static_cast<float*>(ws);
  cudaStream_t st = dmoe::as_stream(stream);
  if (turned) {
    if (act == DMOE_ACT_GELU) return run_turned<DMOE_ACT_GELU>(x, ldx, w, K, o, cut, di, st);
    if (act == DMOE_ACT_SILU) return run_turned<DMOE_ACT_SILU>(x, ldx, w, K, o, cut, di, st);
    return run_turned<DMOE_ACT_NONE>(x, ldx, w, K, o, cut, di, st);
  }
  ParamsL p{};
  if (!map_pitched(&p.map_a[0], x, M, K, ldx, BK, box_rows(M)) || !map_pitched(&p.map_b[0], w, K, N, N, 64, BK))
    return DMOE_ERR_CUDA;
  p.map_a[1] = p.map_a[0];
  p.map_b[1] = p.map_b[0];
  p.b_mn = 1;
  p.a_rows = box_rows(M);
  p.o[0] = o;
  p.err = di.err_word;
  if (act == DMOE_ACT_GELU) return run_products<DMOE_ACT_GELU>(p, a, none, part, nullptr, di, st);
  if (act == DMOE_ACT_SILU) return run_products<DMOE_ACT_SILU>(p, a, none, part, nullptr, di, st);
  return run_products<DMOE_ACT_NONE>(p, a, none, part, nullptr, di, st);
}

DMOE_API size_t dmoe_linear_backward_workspace_size(int M, int K, int N) {
  return sizes_ok(M, K, N) ? back_layout(M, K, N).bytes : 0;
}

DMOE_API dmoe_status dmoe_linear_backward(const uint16_t* dy, int64_t lddy, const uint16_t* deriv, const uint16_t* x,
                                          int64_t ldx, const uint16_t* w, const uint16_t* factor, int M, int K, int N,
                                          uint16_t* dx, void* dw, int dw_f32, float* dbias, void* ws, size_t ws_bytes,
                                          dmoe_stream_t stream) {
  if (!sizes_ok(M, K, N) || (factor && !dx)) return DMOE_ERR_INVALID_ARG;
  if (off16(dy) || off16(deriv) || off16(x) || off16(w) || off16(factor) || off16(dx) || off16(dw) ||
      (reinterpret_cast<uintptr_t>(dbias) & 3) || (reinterpret_cast<uintptr_t>(ws) & 15))
    return DMOE_ERR_INVALID_ARG;
  if (M > 0) {
    if (!dy || bad_pitch(lddy, N) || (dx && !w) || (dw && (!x || bad_pitch(ldx, K)))) return DMOE_ERR_INVALID_ARG;
    if ((dx && (dx == dy || dx == w || dx == x || dx == deriv || dx == dw)) || (dw && (dw == w || dw == x || dw == dy)))
      return DMOE_ERR_INVALID_ARG;
  }
  dmoe::DeviceInfo di;
  dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  cudaStream_t st = dmoe::as_stream(stream);
  if (M == 0) {  // no rows: the sums over them are zero
    cudaError_t e = cudaSuccess;
    if (dw) e = cudaMemsetAsync(dw, 0, static_cast<size_t>(K) * N * (dw_f32 ? 4 : 2), st);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * sizeof(float), st);
    return dmoe::cuda_status(e);
  }
  const BackLayout l = back_layout(M, K, N);
  if (!ws || ws_bytes < l.bytes) return DMOE_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(ws);
  const uint16_t* dz = dy;
  int64_t lddz = lddy;
  const int joined = joined_stripes(M, N), n = joined ? joined : stripes(M, N);
  const bool products = dx || dw;
  if ((deriv && products) || dbias) {
    uint16_t* out = deriv && products ? reinterpret_cast<uint16_t*>(base + l.dz) : nullptr;
    float* sums = !dbias ? nullptr : joined ? dbias : reinterpret_cast<float*>(base + l.sums);
    const dim3 grid(n, ceil_div(N, joined ? 64 : 256));
    const cudaError_t e =
        joined ? dmoe::launch_pdl_cluster(dz_kernel<true>, grid, dim3(256), 0, st, n, dy, lddy, deriv, M, N, out, sums)
               : dmoe::launch_pdl(dz_kernel<false>, grid, dim3(256), 0, st, dy, lddy, deriv, M, N, out, sums);
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    dmoe::count_launches(1);
    if (out) dz = out, lddz = N;
  }
  if (products) {
    Want a{dx ? M : 0, K, ceil_div(N, BK), false}, b{dw ? K : 0, N, ceil_div(M, BK), false};
    if (dx) {
      choose(a, b);
    } else {
      choose(b, a);
    }
    ParamsL p{};
    const int half = std::min(a.tile, BN) / 2;  // of a sub-tile's columns, each CTA's
    if (dx && (!map_pitched(&p.map_a[0], dz, M, N, lddz, BK, box_rows(M)) || !map_pitched(&p.map_b[0], w, K, N, N, BK, half)))
      return DMOE_ERR_CUDA;
    if (dw && (!map_pitched(&p.map_a[1], x, M, K, ldx, 64, BK) || !map_pitched(&p.map_b[1], dz, M, N, lddz, 64, BK)))
      return DMOE_ERR_CUDA;
    if (!dx) p.map_a[0] = p.map_a[1], p.map_b[0] = p.map_b[1];
    if (!dw) p.map_a[1] = p.map_a[0], p.map_b[1] = p.map_b[0];
    p.a_rows = box_rows(M);
    if (dx) p.o[0] = Out{M, K, nullptr, 0, nullptr, nullptr, 0, factor, dx, 0, nullptr};
    if (dw) p.o[1] = Out{K, N, nullptr, 0, nullptr, nullptr, 0, nullptr, dw, dw_f32 ? 1 : 0, nullptr};
    p.err = di.err_word;
    s = run_products<DMOE_ACT_NONE>(p, a, b, reinterpret_cast<float*>(base + l.part_x),
                                    reinterpret_cast<float*>(base + l.part_w), di, st);
    if (s != DMOE_OK) return s;
  }
  if (dbias && !joined) {
    const cudaError_t e = dmoe::launch_pdl(dbias_kernel, dim3(ceil_div(N, 256)), dim3(256), 0, st,
                                           reinterpret_cast<const float*>(base + l.sums), n, N, dbias);
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    dmoe::count_launches(1);
  }
  return DMOE_OK;
}
