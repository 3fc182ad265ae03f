// Softmax cross entropy of rows x [T, d] against a vocabulary head W [V, d],
// with the gradients of both, without the [T, V] logits in memory.
//
//   l_tv = <x_t, W_v>,  lse_t = log sum_v exp(l_tv),
//   loss_t = lse_t - l_t,target
//   G_tv = g_t (exp(l_tv - lse_t) - [v = target_t]),  dx = G W,  dW = G^T x
//
// Tokens go in pieces.  A piece's launches:
//   1 logits   P = x W^T on the tensor cores; the epilogue turns a tile's
//              accumulators into exp(l - ref) and, for each row and 128
//              columns, leaves the pair (ref, sum of exp(l - ref)).  With
//              gradients the exponentials go to a [piece, V] bf16 array, the
//              only thing of that size that ever exists; without, nothing is
//              written.
//   2 rows     the pairs of a row meet in lse_t; loss_t; the factor g_t
//   3 scale    the piece's array becomes G in place
//   4 dx, dW   two products with G
//
// ref is 0 while a row's 128 logits stay within +-kRefLimit, else their
// maximum: exp(l) of a moderate logit needs no maximum subtracted in fp32
// or bf16 (both reach 3e38), so in the usual case every pair of a row has
// the same reference.  What bf16 costs here is one rounding of G (2^-9 of
// an element), the rounding a bf16 gradient of the logits has anyway.
//
// The products are bound by the tensor cores (2 T V d flops each).  They run
// as persistent CTA pairs (tcgen05 cta_group::2): M = 256 x N = 256 NS tiles,
// a ring of TMA-filled K slices of 64, accumulators in TMEM.  Roles per CTA:
// warp 0 TMA producer, warp 1 TMEM allocator and (rank 0) MMA issuer, warps
// 2-9 epilogue.  Every ragged edge is the tensor maps': what lies past a
// matrix reads as zero, and the epilogue stores nothing there.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "tc.cuh"
#include "tmap.cuh"

namespace {

using namespace dmoe::tc;

constexpr int BM = 128;   // rows of a CTA's half of a pair tile
constexpr int BN = 256;   // columns of a sub-tile
constexpr int BK = 64;    // K slice per stage (one 128-byte swizzle row)
constexpr int UMMA_K = 16;
constexpr uint32_t A_BYTES = BM * BK * 2;        // this CTA's A rows
constexpr uint32_t B_BYTES = (BN / 2) * BK * 2;  // this CTA's half of a sub-tile's B
constexpr uint32_t ATOM = 64 * BK * 2;           // MN-major operands: 64 MN x 64 K boxes
constexpr int kEpiWarps = 8;
constexpr int kThreadsX = 64 + 32 * kEpiWarps;
constexpr uint32_t SLAB = 32 * 32 * 2;
constexpr uint32_t SLAB_BYTES = kEpiWarps * 2 * SLAB;
constexpr size_t kSmemMax = 232448;
constexpr int kGroup = 128;          // columns that share a (ref, sum) pair
constexpr float kRefLimit = 60.f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr int kPieceDefault = 8192;  // tokens per piece when the caller names none
constexpr int kPieceMax = 1 << 18;

enum Job : int { JOB_LOGITS = 0, JOB_DX = 1, JOB_DW = 2 };

template <int NS>
struct PlanX {
  static constexpr uint32_t STAGE = A_BYTES + NS * B_BYTES;
  static constexpr int FIT = static_cast<int>((kSmemMax - 1536 - SLAB_BYTES) / STAGE);
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr size_t SMEM = 1024 + STAGES * STAGE + SLAB_BYTES + 512;
  static_assert(STAGES >= 4 && SMEM <= kSmemMax, "shared-memory plan");
};

struct ParamsX {
  CUtensorMap map_a;
  CUtensorMap map_b;
  int M, N, K;       // product sizes
  int mt, nt;        // pair-tile rows, tile columns
  int raster;        // pair-tile rows per raster group
  uint16_t* out;     // bf16 result (dx, dW) or the exponentials
  float* out32;      // fp32 result (dW), instead of out
  const float* add;  // fp32 partial result added to the accumulators, or NULL
  int64_t ldo;       // row pitch of out / out32 / add
  // JOB_LOGITS
  const int32_t* targets;
  float2* pairs;     // [N / 128][ldp] (ref, sum)
  int64_t ldp;
  float* target_logit;
  int32_t* err;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

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

// 64 fp32 accumulator columns of this thread's TMEM lane, waited for in the
// same statement so that no use of a register can move above the wait.
__device__ __forceinline__ void tmem_load64(uint32_t ta, float* v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]),
        "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]),
        "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]),
        "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]),
        "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(ta)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// Writes 32 rows x 64 columns held one row per lane (v[0..63]) as coalesced
// 16-byte stores through the warp's two 2 KB slabs: each lane puts its row
// into both (16-byte piece j of row r at piece j ^ ((r >> 1) & 3)), then each
// store instruction writes 4 rows x 128 bytes.  Only rows below `rows` and
// 8-column pieces below `cols` exist (both counted from this corner).
__device__ __forceinline__ void write_rows64(uint8_t* slabs, int lane, const float* v, uint16_t* out, int64_t ld,
                                             int rows, int cols) {
  const int sw = (lane >> 1) & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    *reinterpret_cast<uint4*>(slabs + lane * 64 + ((j ^ sw) << 4)) = pack8x(v + 8 * j);
    // the second slab keeps its rows pairwise swapped: the two reads of one
    // instruction then hit different banks
    *reinterpret_cast<uint4*>(slabs + SLAB + (lane ^ 1) * 64 + ((j ^ sw) << 4)) = pack8x(v + 32 + 8 * j);
  }
  __syncwarp();
  const int j = lane & 7;
  const uint8_t* sl = slabs + (j >> 2) * SLAB;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    const uint4 q = *reinterpret_cast<const uint4*>(sl + (r ^ (j >> 2)) * 64 + (((j & 3) ^ ((r >> 1) & 3)) << 4));
    if (r < rows && 8 * j < cols) *reinterpret_cast<uint4*>(out + r * ld + 8 * j) = q;
  }
  __syncwarp();
}

// Tile t of the mt x nt grid, in groups of `raster` pair rows with the
// columns outer and the rows inner: pairs working at the same time share B
// columns while the group's A rows stay in L2.
__device__ __forceinline__ void tile_at(const ParamsX& p, int t, int& m, int& n) {
  const int per = p.raster * p.nt;
  const int g = t / per;
  const int r0 = g * p.raster;
  const int h = min(p.raster, p.mt - r0);
  const int l = t - g * per;
  n = l / h;
  m = r0 + l % h;
}

// K major of the operands: the logits' product has both K-major (x and W
// rows), dx has P K-major and W MN-major, dW has P and x MN-major.
template <int JOB, int NS>
__global__ void __launch_bounds__(kThreadsX, 1) head_kernel(const __grid_constant__ ParamsX p) {
  using PL = PlanX<NS>;
  constexpr int STAGES = PL::STAGES;
  constexpr bool A_MN = JOB == JOB_DW;
  constexpr bool B_MN = JOB != JOB_LOGITS;
  constexpr uint32_t IDESC = idesc_bf16(2 * BM, BN, A_MN, B_MN);
  constexpr uint64_t A_STEP = A_MN ? (UMMA_K * 128) >> 4 : (UMMA_K * 2) >> 4;
  constexpr uint64_t B_STEP = B_MN ? (UMMA_K * 128) >> 4 : (UMMA_K * 2) >> 4;
  constexpr uint32_t A_LBO = A_MN ? ATOM : 16;
  constexpr uint32_t B_LBO = B_MN ? ATOM : 16;
  constexpr uint32_t TMEM_COLS = 512;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* slab_mem = smem + STAGES * PL::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(slab_mem + SLAB_BYTES);
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
    tma_prefetch_map(&p.map_a);
    tma_prefetch_map(&p.map_b);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, TMEM_COLS);
  fence_before_sync();
  cluster_sync();
  fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();

  const int ntiles = p.mt * p.nt;
  const int G = static_cast<int>(gridDim.x >> 1);
  const int unit = static_cast<int>(blockIdx.x >> 1);
  const int kit = (p.K + BK - 1) / BK;

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t full_pair = dsmem_addr(smem_u32(full), 0);  // rank 0 counts both CTAs' bytes
      for (int t = unit; t < ntiles && ok; t += G) {
        int m, n;
        tile_at(p, t, m, n);
        const int m0 = m * 2 * BM + rank * BM;
        const int n0 = n * NS * BN + rank * (BN / 2);
        for (int i = 0; i < kit; ++i) {
          ok = mbar_wait(empty + stage, phase ^ 1u, abort_flag);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(full + stage, 2 * PL::STAGE);
          const uint32_t bar = full_pair + 8u * stage;
          uint8_t* sa = smem + stage * PL::STAGE;
          uint8_t* sb = sa + A_BYTES;
          const int k0 = i * BK;
          if (A_MN) {
            tma_load_2d_pair(sa, &p.map_a, bar, m0, k0);
            tma_load_2d_pair(sa + ATOM, &p.map_a, bar, m0 + 64, k0);
          } else {
            tma_load_2d_pair(sa, &p.map_a, bar, k0, m0);
          }
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            if (B_MN) {
              tma_load_2d_pair(sb + s * B_BYTES, &p.map_b, bar, n0 + s * BN, k0);
              tma_load_2d_pair(sb + s * B_BYTES + ATOM, &p.map_b, bar, n0 + s * BN + 64, k0);
            } else {
              tma_load_2d_pair(sb + s * B_BYTES, &p.map_b, bar, k0, n0 + s * BN);
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
      // one K slice of sub-tile `s` from ring stage st into accumulator d
      auto mmas = [&](uint32_t d, int st, int s, bool first) {
        const uint32_t sa = smem_u32(smem + st * PL::STAGE);
        const uint64_t adesc = sdesc_sw128(sa, A_LBO, 1024);
        const uint64_t bdesc = sdesc_sw128(sa + A_BYTES + s * B_BYTES, B_LBO, 1024);
#pragma unroll
        for (int kk = 0; kk < BK / UMMA_K; ++kk)
          mma_bf16_pair(d, adesc + A_STEP * kk, bdesc + B_STEP * kk, IDESC, (!first || kk > 0) ? 1u : 0u);
      };
      for (int t = unit; t < ntiles && ok; t += G) {
        if (NS == 2) {
          // both accumulators belong to this tile: sub-tile 0 starts once its
          // columns are drained, sub-tile 1's first slices stay in the ring
          // until its own are
          ok = mbar_wait_cluster(tempty, acc_phase ^ 1u, abort_flag);
          if (!ok) break;
          fence_after_sync();
          bool free1 = false;
          int held = 0;
          const int hstage = stage;
          auto catch_up = [&]() {
            for (int j = 0; j < held; ++j) {
              const int st = (hstage + j) % STAGES;
              mmas(tmem_base + BN, st, 1, j == 0);
              mma_commit_pair(empty + st);
            }
            held = 0;
          };
          for (int i = 0; i < kit; ++i) {
            ok = mbar_wait(full + stage, phase, abort_flag);
            if (!ok) break;
            fence_after_sync();
            mmas(tmem_base, stage, 0, i == 0);
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
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (held > 0) {
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
    const int quad = warp & 3;                 // TMEM lanes 32 quad .. 32 quad + 31
    const int half = (warp - 2) >> 2;          // columns 128 half .. + 127 of a sub-tile
    uint8_t* const slabs = slab_mem + (warp - 2) * 2 * SLAB;
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
    for (int t = unit; t < ntiles && ok; t += G) {
      int m, n;
      tile_at(p, t, m, n);
      const int row0 = m * 2 * BM + rank * BM + quad * 32;  // this warp's 32 rows
      const int row = row0 + lane;
      const int rows = p.M - row0;  // rows of them that exist (or fewer than 1)
      int target = -1;
      if (JOB == JOB_LOGITS && row < p.M) target = __ldg(p.targets + row);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int c0 = (n * NS + s) * BN + half * (BN / 2);  // this warp's first column
        if (NS == 1 || s == 0) {
          ok = mbar_wait_cluster(tfull + acc, acc_phase, abort_flag);
          if (!ok) break;
        }
        fence_after_sync();
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * BN + half * (BN / 2);
        if (JOB == JOB_LOGITS) {
          float v[128];
          tmem_load64(tb, v);
          tmem_load64(tb + 64, v + 64);
          release();
          if (c0 >= p.N) continue;  // past the vocabulary: no such group
          if (static_cast<unsigned>(target - c0) < 128u) {
            float l = 0.f;
#pragma unroll
            for (int j = 0; j < 128; ++j) l = j == target - c0 ? v[j] : l;
            p.target_logit[row] = l;
          }
          if (c0 + 128 > p.N) {
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (c0 + j >= p.N) v[j] = -INFINITY;
          }
          float top = v[0];
#pragma unroll
          for (int j = 1; j < 128; ++j) top = fmaxf(top, v[j]);
          const float ref = (fabsf(top) > kRefLimit && top != -INFINITY) ? top : 0.f;
          const float bias = -ref * kLog2e;
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int j = 0; j < 128; j += 4) {
            v[j] = ex2(fmaf(v[j], kLog2e, bias));
            v[j + 1] = ex2(fmaf(v[j + 1], kLog2e, bias));
            v[j + 2] = ex2(fmaf(v[j + 2], kLog2e, bias));
            v[j + 3] = ex2(fmaf(v[j + 3], kLog2e, bias));
            s0 += v[j];
            s1 += v[j + 1];
            s2 += v[j + 2];
            s3 += v[j + 3];
          }
          if (row < p.M) p.pairs[static_cast<int64_t>(c0 / kGroup) * p.ldp + row] = make_float2(ref, (s0 + s1) + (s2 + s3));
          if (p.out) {
            uint16_t* o = p.out + static_cast<int64_t>(row0) * p.ldo + c0;
            const int cols = static_cast<int>(p.ldo) - c0;
            write_rows64(slabs, lane, v, o, p.ldo, rows, cols);
            write_rows64(slabs, lane, v + 64, o + 64, p.ldo, rows, cols - 64);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[64];
            tmem_load64(tb + 64 * h, v);
            if (h == 1) release();
            const int c = c0 + 64 * h;
            if (p.add && row < p.M) {
              const float* a = p.add + static_cast<int64_t>(row) * p.ldo + c;
#pragma unroll
              for (int j = 0; j < 64; j += 4)
                if (c + j < p.N) {
                  const float4 q = *reinterpret_cast<const float4*>(a + j);
                  v[j] += q.x, v[j + 1] += q.y, v[j + 2] += q.z, v[j + 3] += q.w;
                }
            }
            if (p.out32) {
              float* o = p.out32 + static_cast<int64_t>(row) * p.ldo + c;
#pragma unroll
              for (int j = 0; j < 64; j += 4)
                if (row < p.M && c + j < p.N)
                  *reinterpret_cast<float4*>(o + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            } else {
              write_rows64(slabs, lane, v, p.out + static_cast<int64_t>(row0) * p.ldo + c, p.ldo, rows, p.N - c);
            }
          }
        }
      }
    }
    if (!ok && lane == 0) {
      dmoe::raise_error(p.err, DMOE_SITE_GEMM_WAIT | DMOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }

  __syncwarp();
  fence_before_sync();
  // a CTA of a pair leaves only once the other no longer reads or signals
  // its shared memory
  cluster_sync();
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------ row statistics

constexpr int kStatRows = 32, kStatSlices = 32;

// How many targets count: one block over all T.
__global__ void __launch_bounds__(1024) count_targets_kernel(const int32_t* __restrict__ targets, int T, int V,
                                                             int ignore, int32_t* __restrict__ count, int32_t* err) {
  __shared__ int sh[32];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  int n = 0;
  bool bad = false;
#pragma unroll 8
  for (int t = threadIdx.x; t < T; t += 1024) {
    const int32_t v = __ldg(targets + t);
    const bool in = static_cast<unsigned>(v) < static_cast<unsigned>(V);
    n += in && v != ignore;
    bad |= !in && v != ignore;
  }
  if (bad) dmoe::raise_error(err, DMOE_SITE_LOSS_TARGET | DMOE_ERR_DEVICE);
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = n;
  __syncthreads();
  if (threadIdx.x < 32) {
    n = __reduce_add_sync(0xffffffffu, sh[threadIdx.x]);
    if (threadIdx.x == 0) *count = n;
  }
}

// (R, S) <- the pair of the union: S counts exp(l - R).
__device__ __forceinline__ void join(float& R, float& S, float r, float s) {
  if (r == R) {
    S += s;
  } else if (r < R) {
    S += s * expf(r - R);
  } else {
    S = S * expf(R - r) + s;
    R = r;
  }
}

// 32 rows x 32 slices of the row's groups per block.
__global__ void __launch_bounds__(kStatRows * kStatSlices)
    row_stats_kernel(const float2* __restrict__ pairs, int64_t ldp, int groups, const float* __restrict__ target_logit,
                     const int32_t* __restrict__ targets, int n, int V, int ignore, const float* __restrict__ d_loss,
                     const int32_t* __restrict__ count, float* __restrict__ loss, float* __restrict__ lse,
                     float4* __restrict__ factor) {
  __shared__ float2 sh[kStatSlices][kStatRows];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int slice = threadIdx.x >> 5;
  const int t = blockIdx.x * kStatRows + lane;
  float R = -INFINITY, S = 0.f;
  if (t < n) {
#pragma unroll 4
    for (int g = slice; g < groups; g += kStatSlices) {
      const float2 q = __ldg(pairs + g * ldp + t);
      join(R, S, q.x, q.y);
    }
  }
  sh[slice][lane] = make_float2(R, S);
  __syncthreads();
  if (slice != 0 || t >= n) return;
  for (int i = 1; i < kStatSlices; ++i) {
    const float2 q = sh[i][lane];
    if (q.x != -INFINITY) join(R, S, q.x, q.y);  // a slice without groups
  }
  const float L = R + logf(S);
  const int32_t v = __ldg(targets + t);
  const bool counts = static_cast<unsigned>(v) < static_cast<unsigned>(V) && v != ignore;
  const float nll = counts ? L - __ldg(target_logit + t) : 0.f;
  loss[t] = nll;
  if (lse) lse[t] = L;
  if (factor) {
    float g = 0.f;
    if (counts) g = d_loss ? __ldg(d_loss + t) : 1.f / static_cast<float>(*count);
    // the target's own element from its fp32 logit: where the softmax is close
    // to 1, its rounded exponential minus 1 would be all rounding
    factor[t] = make_float4(L, g, g * expm1f(-nll), 0.f);
  }
}

// G in place of the exponentials: one warp per row and 1024 columns.
constexpr int kScaleCols = 1024;
__global__ void __launch_bounds__(256)
    scale_kernel(uint16_t* __restrict__ P, int64_t ld, int n, int V, const float2* __restrict__ pairs, int64_t ldp,
                 const float4* __restrict__ factor, const int32_t* __restrict__ targets) {
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (t >= n) return;
  const int c0 = blockIdx.x * kScaleCols;
  const float4 f = __ldg(factor + t);
  const int target = __ldg(targets + t);
  uint4* row = reinterpret_cast<uint4*>(P + t * ld + c0);
  uint4 u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + (i * 32 + lane) * 8;
    if (c < ld) u[i] = row[i * 32 + lane];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + (i * 32 + lane) * 8;
    if (c >= ld) continue;
    float v[8];
    unpack8x(u[i], v);
    // padding columns past the vocabulary have no pair, a row that does not
    // count stays zero whatever it holds
    const bool zero = c >= V || f.y == 0.f;
    const float k = zero ? 0.f : expf(__ldg(&pairs[(c / kGroup) * ldp + t].x) - f.x) * f.y;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = zero ? 0.f : v[j] * k;
      if (c + j == target) v[j] = f.z;
    }
    row[i * 32 + lane] = pack8x(v);
  }
}

// ----------------------------------------------------------------- host side

// Opt-in shared memory and the number of 2-CTA clusters that fit, once per
// instantiation and device.
template <int JOB, int NS>
dmoe_status launch_head(const ParamsX& p, const dmoe::DeviceInfo& di, cudaStream_t st) {
  auto kern = head_kernel<JOB, NS>;
  const size_t smem = PlanX<NS>::SMEM;
  static std::atomic<int> clusters[64];
  int n = clusters[di.device].load(std::memory_order_acquire);
  if (n == 0) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(di.sm_count & ~1));
    cfg.blockDim = dim3(kThreadsX);
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
  const int64_t tiles = static_cast<int64_t>(p.mt) * p.nt;
  const int grid = 2 * static_cast<int>(std::min<int64_t>(n, tiles));
  cudaError_t e = dmoe::launch_pdl_cluster(kern, dim3(grid), dim3(kThreadsX), smem, st, 2, p);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

// Bytes of a workspace, in order (each part 256-byte aligned).
struct Layout {
  int64_t piece;   // tokens per piece
  int64_t ldp;     // row pitch of the (ref, sum) pairs
  int64_t ldv;     // row pitch of the exponentials
  int64_t groups;
  size_t count, pairs, target_logit, factor, acc, P, total;
};

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

Layout layout_of(int T, int d, int V, bool grad, bool dw_bf16, int piece) {
  Layout l{};
  l.piece = std::min(round_up(std::min(piece > 0 ? piece : kPieceDefault, kPieceMax), 2 * BM),
                     round_up(std::max(T, 1), 2 * BM));
  l.ldp = l.piece;
  l.ldv = round_up(V, 64);
  l.groups = (V + kGroup - 1) / kGroup;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += static_cast<size_t>(round_up(static_cast<int64_t>(bytes), 256));
    return a;
  };
  l.count = take(256);
  l.pairs = take(static_cast<size_t>(l.groups * l.ldp) * sizeof(float2));
  l.target_logit = take(static_cast<size_t>(l.piece) * sizeof(float));
  if (grad) {
    l.factor = take(static_cast<size_t>(l.piece) * sizeof(float4));
    // dW of earlier pieces, when it does not fit the output's own type
    l.acc = take(dw_bf16 && T > l.piece ? static_cast<size_t>(V) * d * sizeof(float) : 0);
    l.P = take(static_cast<size_t>(l.piece * l.ldv) * 2);
  }
  l.total = at;
  return l;
}

bool sizes_ok(int T, int d, int V, int piece) {
  return T >= 0 && d >= 8 && (d & 7) == 0 && V >= 1 && V <= (1 << 24) && d <= (1 << 20) && piece >= 0;
}

#define DMOE_TRY(call)                 \
  do {                                 \
    const dmoe_status st__ = (call);   \
    if (st__ != DMOE_OK) return st__;  \
  } while (0)

}  // namespace

DMOE_API size_t dmoe_linear_cross_entropy_workspace_size(int T, int d, int V, int grad, int dw_f32, int piece) {
  if (!sizes_ok(T, d, V, piece)) return 0;
  return layout_of(T, d, V, grad != 0, !dw_f32, piece).total;
}

DMOE_API dmoe_status dmoe_linear_cross_entropy(const uint16_t* x, const uint16_t* w, const int32_t* targets, int T,
                                               int d, int V, int ignore_index, const float* d_loss, float* loss,
                                               float* lse, uint16_t* dx, void* dw, int dw_f32, int accumulate,
                                               int piece, void* ws, size_t ws_bytes, dmoe_stream_t stream) {
  if (!sizes_ok(T, d, V, piece) || (accumulate && !(dw && dw_f32))) return DMOE_ERR_INVALID_ARG;
  const bool grad = dx || dw;
  if (T > 0 && (!x || !w || !targets || !loss || !ws)) return DMOE_ERR_INVALID_ARG;
  if (!dmoe::aligned16(x) || !dmoe::aligned16(w) || !dmoe::aligned16(dx) || !dmoe::aligned16(dw) ||
      (reinterpret_cast<uintptr_t>(ws) & 255) ||
      ((reinterpret_cast<uintptr_t>(targets) | reinterpret_cast<uintptr_t>(d_loss) |
        reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(lse)) & 3))
    return DMOE_ERR_INVALID_ARG;
  const Layout l = layout_of(T, d, V, grad, dw && !dw_f32, piece);
  if (T > 0 && ws_bytes < l.total) return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  cudaStream_t st = dmoe::as_stream(stream);
  if (T == 0) {
    if (dw && !accumulate)
      return dmoe::cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * d * (dw_f32 ? 4 : 2), st));
    return DMOE_OK;
  }
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* count = reinterpret_cast<int32_t*>(base + l.count);
  float2* pairs = reinterpret_cast<float2*>(base + l.pairs);
  float* target_logit = reinterpret_cast<float*>(base + l.target_logit);
  float4* factor = grad ? reinterpret_cast<float4*>(base + l.factor) : nullptr;
  uint16_t* P = grad ? reinterpret_cast<uint16_t*>(base + l.P) : nullptr;
  float* acc = grad ? reinterpret_cast<float*>(base + l.acc) : nullptr;

  cudaError_t e = dmoe::launch_pdl(count_targets_kernel, dim3(1), dim3(1024), 0, st, targets, T, V, ignore_index,
                                   count, di.err_word);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);

  for (int64_t t0 = 0; t0 < T; t0 += l.piece) {
    const int n = static_cast<int>(std::min<int64_t>(l.piece, T - t0));
    const uint16_t* xp = x + t0 * d;
    {
      ParamsX p{};
      if (!dmoe::make_map(&p.map_a, xp, n, d, BK, BM) || !dmoe::make_map(&p.map_b, w, V, d, BK, BN / 2))
        return DMOE_ERR_CUDA;
      p.M = n, p.N = V, p.K = d;
      p.mt = (n + 2 * BM - 1) / (2 * BM);
      p.nt = (V + 2 * BN - 1) / (2 * BN);
      p.raster = 16;
      p.out = P;
      p.ldo = l.ldv;
      p.targets = targets + t0;
      p.pairs = pairs;
      p.ldp = l.ldp;
      p.target_logit = target_logit;
      p.err = di.err_word;
      DMOE_TRY((launch_head<JOB_LOGITS, 2>(p, di, st)));
    }
    e = dmoe::launch_pdl(row_stats_kernel, dim3((n + kStatRows - 1) / kStatRows), dim3(kStatRows * kStatSlices), 0, st,
                         static_cast<const float2*>(pairs), l.ldp, static_cast<int>(l.groups),
                         static_cast<const float*>(target_logit), targets + t0, n, V, ignore_index,
                         d_loss ? d_loss + t0 : nullptr, static_cast<const int32_t*>(count), loss + t0,
                         lse ? lse + t0 : nullptr, factor);
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    dmoe::count_launches(1);
    if (!grad) continue;
    e = dmoe::launch_pdl(scale_kernel, dim3(static_cast<unsigned>((l.ldv + kScaleCols - 1) / kScaleCols), (n + 7) / 8),
                         dim3(256), 0, st, P, l.ldv, n, V, static_cast<const float2*>(pairs), l.ldp,
                         static_cast<const float4*>(factor), targets + t0);
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    dmoe::count_launches(1);
    if (dx) {
      ParamsX p{};
      // P as [n, V] with row pitch ldv: the columns past V read as zero
      if (!dmoe::make_map_ld(&p.map_a, P, n, V, l.ldv, BK, BM) || !dmoe::make_map(&p.map_b, w, V, d, 64, BK))
        return DMOE_ERR_CUDA;
      p.M = n, p.N = d, p.K = V;
      p.mt = (n + 2 * BM - 1) / (2 * BM);
      p.nt = (d + 2 * BN - 1) / (2 * BN);
      p.raster = 16;
      p.out = dx + t0 * d;
      p.ldo = d;
      p.err = di.err_word;
      DMOE_TRY((launch_head<JOB_DX, 2>(p, di, st)));
    }
    if (dw) {
      ParamsX p{};
      if (!dmoe::make_map_ld(&p.map_a, P, n, V, l.ldv, 64, BK) || !dmoe::make_map(&p.map_b, xp, n, d, 64, BK))
        return DMOE_ERR_CUDA;
      p.M = V, p.N = d, p.K = n;
      p.mt = (V + 2 * BM - 1) / (2 * BM);
      p.nt = (d + 2 * BN - 1) / (2 * BN);
      p.raster = 1;
      p.ldo = d;
      p.err = di.err_word;
      const bool last = t0 + n >= T;
      if (dw_f32) {
        p.out32 = static_cast<float*>(dw);
        p.add = (accumulate || t0 > 0) ? static_cast<const float*>(dw) : nullptr;
      } else {
        // fp32 until the last piece, then one rounding
        p.add = t0 > 0 ? acc : nullptr;
        if (last) p.out = static_cast<uint16_t*>(dw);
        else p.out32 = acc;
      }
      DMOE_TRY((launch_head<JOB_DW, 2>(p, di, st)));
    }
  }
  return DMOE_OK;
}
