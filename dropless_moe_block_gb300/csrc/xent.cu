// Softmax cross entropy of rows x [T, d] against a vocabulary head W [V, d],
// with the gradients of both, without the [T, V] logits in memory.
//
//   l_tv = <x_t, W_v>,  lse_t = log sum_v exp(l_tv),
//   loss_t = lse_t - l_t,target
//   G_tv = g_t (exp(l_tv - lse_t) - [v = target_t]),  dx = G W,  dW = G^T x
//
// With a reference r_t of each row, E_tv = exp(l_tv - r_t) for v other than
// the target and 0 at the target, s_t = g_t exp(r_t - lse_t) and
// c_t = g_t (exp(-loss_t) - 1):
//
//   dx_t = s_t (E W)_t + c_t W_target        dW_v = (E^T (s x))_v + sum c_t x_t
//                                                   over the tokens whose target is v
//
// so the products need only the unnormalised exponentials, which the logits'
// product can leave behind before lse is known, and the target's element,
// the large one, never passes through 16 bits: it is added in fp32.
//
// Tokens go in pieces.  A piece's launches:
//   1 logits   x W^T on the tensor cores; the epilogue turns a tile's
//              accumulators into E and, for each row and 64 columns, leaves
//              the pair (ref, sum of exp(l - ref)).  With gradients E goes to a
//              [piece, V] bf16 array, the only thing of that size that ever
//              exists; without, nothing is written.
//   2 rows     the pairs of a row meet in lse_t; loss_t, s_t, c_t, s_t x_t; the
//              tokens ordered by target
//   3 targets  sums of c_t x_t by word, up to 32 tokens each
//   4 grads    the tiles of both products in one launch
//
// ref is 0 while the largest of a row's 64 logits lies in [kRefLow,
// kRefHigh], else that maximum: exp of a moderate logit needs no maximum
// subtracted, fp32 and bf16 reach from 1e-38 to 3e38, so in the usual case
// every pair of a row has the reference 0 and E needs no second pass.  A row
// whose groups disagree is brought to its largest reference by launch 2.
// What bf16 costs is one rounding of E, a second where launch 2 brings a row to
// one reference, and one of s x (2^-8 of an element at most each, independent
// from element to element): the products are of tensor-core operands, so a dW
// in fp32, too, sums terms known to 8 bits, only the target's part to 24.
//
// The tensor cores truncate where they add products to an accumulator, so a
// logit comes out too small by an amount that goes by how its sum grows.  In
// units of (d / 16) 2^-26 of the logit (d = 512 to 8192, measured): none where
// every partial sum fits (one-hot rows, small integers), 1.0 to 1.1 for Gaussian
// rows, 1.9 to 4.6 where all products have one sign.  The epilogue gives
// one unit back, an estimate for rows as a norm leaves them: the loss at d =
// 4096 is 3e-7 off with it and 1.3e-6 without; sums of one sign stay 0.9 to 3.6
// units too small, and exact logits come out one unit too large (3.8e-6 of
// themselves at d = 4096).  An fp32 sum in sequence may be off by 64 units.
//
// The products are bound by the tensor cores (2 T V d flops each).  They run
// as persistent CTA pairs (tcgen05 cta_group::2): M = 256 x N = 512 tiles (two
// sub-tiles of N = 256 that share each K slice's A; the logits also N = 256,
// 128 or 64, see logits_tile()), a ring of TMA-filled K slices of 64,
// accumulators in TMEM.  Roles per CTA: warp 0 TMA producer, warp 1 TMEM
// allocator and (rank 0) MMA issuer, warps 2-17 epilogue: sixteen warps,
// because exponentials, sums and stores of a tile take as long as its product
// over 512 columns, and eight left that time to latency (8192 x 512 x 32000:
// logits 231 us with eight, 195 with sixteen).  Every ragged edge is the
// tensor maps': what lies past a matrix reads as zero, and the epilogue stores
// nothing there.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "tc.cuh"
#include "tile.cuh"
#include "tmap.cuh"

namespace {

using namespace dmoe::tc;
using namespace dmoe::tile;
using dmoe::f2_add;
using dmoe::f2_fma;
using dmoe::f2_mul;

constexpr int kEpiWarps = 16;  // four per TMEM lane quadrant, 64 columns of a sub-tile each
constexpr int kThreadsX = 64 + 32 * kEpiWarps;
// One epilogue warp's output on its way out: 32 rows x 32 columns, or, where
// it leaves by TMA, all 64 of its columns.
constexpr uint32_t SLAB64 = 32 * 64 * 2;
constexpr int kGroup = 64;           // columns that share a (ref, sum) pair
// Above: 2^24 exponentials of kRefHigh, times any sensible weights, stay far
// below 3e38.  Below: what is 27 under kRefLow, 2e-12 of its group's largest
// exponential, reaches the denormals.
constexpr float kRefHigh = 40.f, kRefLow = -60.f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kTruncation = 1.f / 67108864.f;  // given back: 2^-26 of the sum per 16 products, see above
constexpr int kPieceDefault = 8192;  // tokens per piece when the caller names none
constexpr int kPieceMax = 1 << 18;
// Logits over at most so many columns run 256-wide tiles: their two
// accumulators let a tile's exponentials overlap the next tile's product,
// which 512-wide tiles, filling the TMEM, do only in part.  The logits of
// 8192 x 32000, 256-wide against 512-wide: d = 64 92 against 110 us, 256 119
// / 131, 512 193 / 215, 1024 322 / 325, 2048 562 / 570; at d = 4096, where the
// exponentials are a small part, the operands that 512-wide tiles save
// count: with its gradients 3828 / 3814 us.
constexpr int kNarrowD = 1024;

constexpr int kFewTokens = 8;        // dW of so few tokens has a form of its own
constexpr int kRun = 32;             // positions per partial sum of launch 3
// Words with at most so many tokens are summed by dW's epilogue itself, token
// by token.  From kDirectFrom tokens on that hides behind the tile's product,
// and keeps launch 3 from writing a row for every token (17 MB at 8192 x 512).
// With fewer tokens the product is short, and the epilogue adds launch 3's
// rows only (1216 x 736 x 41031: gradients 169 us with 4, 162 with 0).
constexpr int kDirect = 4;
constexpr int kDirectFrom = 4096;

template <bool GRAD, int NS>
struct PlanX {
  // the exponentials leave by TMA where the tiles' sums are short (NS = 1):
  // storing them is then as long as the product, see write_tile()
  static constexpr bool TMA_OUT = !GRAD && NS == 1;
  static constexpr uint32_t SLAB = TMA_OUT ? SLAB64 : SLAB32;
  static constexpr uint32_t SLAB_BYTES = kEpiWarps * SLAB;
  static constexpr uint32_t STAGE = A_BYTES + NS * B_BYTES;
  static constexpr int FIT = static_cast<int>((kSmemMax - 1536 - SLAB_BYTES) / STAGE);
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr size_t SMEM = 1024 + STAGES * STAGE + SLAB_BYTES + 512;
  static_assert(STAGES >= 4 && SMEM <= kSmemMax, "shared-memory plan");
};

struct ParamsX {
  CUtensorMap map_a;   // logits: x K-major;  gradients: E K-major (dx)
  CUtensorMap map_b;   // logits: W K-major;  gradients: W MN-major (dx)
  CUtensorMap map_a2;  // gradients: E MN-major (dW)
  CUtensorMap map_b2;  // gradients: s x MN-major (dW)
  CUtensorMap map_e;   // logits: E, as the epilogue stores it
  int n, d, V;         // tokens of the piece, columns, vocabulary
  int a_rows;          // rows of map_a's box: what lies past n is not loaded (it only reaches rows past n)
  int first_dx;        // gradients: grid[0] is dx's (else dW's)
  int full, rem;       // grid[0]'s items per unit, and the units that get one more
  int early, extra;    // see item_of()
  Grid grid[2];        // logits: one grid;  gradients: the longer items first
  const int32_t* targets;
  int32_t* err;
  // logits
  uint16_t* E;         // [n][ldv] exponentials (NULL: the loss alone)
  float* E32;          // the same unrounded, of few tokens (else NULL)
  int64_t ldv;
  float* sums;         // [V / 64][ldp] sums of exponentials, negative where the
  float* refs;         // reference is not 0 but this one
  int64_t ldp;
  float* target_logit;
  float unbias;        // 1 + the truncation given back
  const int32_t* all;  // the whole call's targets, to be counted (NULL: not here)
  int T, ignore;
  int32_t* count;
  // gradients
  const float2* coef;  // (s_t, c_t)
  const uint16_t* W;
  const uint16_t* x;
  uint16_t* dx;        // dx, or with parts > 1 the fp32 sums of each part:
  float* dx_part;      // [parts][n][d]
  uint16_t* dw;        // dW in bf16,
  float* dw32;         // or in fp32
  const float* dw_add; // fp32 dW of earlier pieces (or what the caller adds to)
  const int32_t* skey;   // targets in ascending order
  const int2* words;     // positions [x, y) of a word's tokens, for words that have some
  const int32_t* order;  // their tokens, ascending among equal targets
  int direct;            // words with more tokens have sums in runs
  const float* runs;     // launch 3's sums, at the position of their first token
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The largest of three (numbers before NaN).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

// The same for 64 columns at (x, y) of a tensor map with 64 x 32 boxes, by TMA
// out of the warp's 4 KB slab in the 128-byte swizzle (16-byte piece j of row
// r at piece j ^ (r & 7)): no second pass through registers.  The previous
// store has read the slab (a tile ago) before it is written again; rows and
// columns past the map are not written.  At d = 64 the logits of 8192 x 32000
// take 92 us this way, 110 us through registers.
__device__ __forceinline__ void write_tile(uint32_t slab, int lane, const float* v, const CUtensorMap* map, int x,
                                           int y) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j) st_shared(slab + lane * 128 + ((j ^ (lane & 7)) << 4), pack8x(v + 8 * j));
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(slab), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

__device__ __forceinline__ void prefetch_l1(const void* a) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<uint64_t>(a)) : "memory");
}

// A target's word, V for one that does not count.
__device__ __forceinline__ int key_of(int32_t target, int V, int ignore) {
  return static_cast<unsigned>(target) < static_cast<unsigned>(V) && target != ignore ? target : V;
}

// The logits' product has both operands K-major (rows of x and of W); dx has
// E K-major and W MN-major, dW has E and s x MN-major.
template <bool GRAD, int NS>
__global__ void __launch_bounds__(kThreadsX, 1) head_kernel(const __grid_constant__ ParamsX p) {
  using PL = PlanX<GRAD, NS>;
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
    tma_prefetch_map(&p.map_a);
    tma_prefetch_map(&p.map_b);
    if (GRAD) {
      tma_prefetch_map(&p.map_a2);
      tma_prefetch_map(&p.map_b2);
    }
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
        const int m0 = it.m * 2 * BM + rank * BM;
        const int width = GRAD || NS == 2 ? BN : p.grid[0].tile;  // of a sub-tile
        const int n0 = it.c0 + rank * (width / 2);
        const bool a_mn = GRAD && !it.dx;
        // the bytes of both CTAs' A rows, and whether this one has any
        const bool a_none = !a_mn && m0 >= p.n;
        const uint32_t a_bytes =
            a_mn || it.m * 2 * BM + BM < p.n ? 2 * A_BYTES : static_cast<uint32_t>(p.a_rows) * BK * 2;
        const CUtensorMap* ma = a_mn ? &p.map_a2 : &p.map_a;
        const CUtensorMap* mb = a_mn ? &p.map_b2 : &p.map_b;
        for (int i = it.k0; i < it.k1; ++i) {
          ok = mbar_wait(empty + stage, phase ^ 1u, abort_flag);
          if (!ok) break;
          const int subs = NS == 2 && it.wide ? 2 : 1;
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
            if (GRAD) {
              tma_load_2d_pair(sb + s * B_BYTES, mb, bar, n0 + s * BN, k0);
              tma_load_2d_pair(sb + s * B_BYTES + ATOM, mb, bar, n0 + s * BN + 64, k0);
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
    if (!GRAD && rank == 1 && unit == 0 && p.all) {
      // a warp without other work counts the targets that count
      int c = 0;
#pragma unroll 1
      for (int i0 = lane; i0 < p.T; i0 += 32 * 16) {
        int t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = i0 + 32 * i < p.T ? __ldg(p.all + i0 + 32 * i) : p.ignore;
#pragma unroll
        for (int i = 0; i < 16; ++i) c += key_of(t[i], p.V, p.ignore) < p.V;
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) *p.count = c;
    }
    if (lane == 0 && rank == 0) {
      // ------------------------------------------------------------ MMA issue
      int stage = 0;
      uint32_t phase = 0;
      uint32_t acc = 0, acc_phase = 0;
      bool ok = true;
      // operand majors of the current item; B is MN-major in both gradients.
      // Of a descriptor only the start address (the low word) moves: by a
      // stage, a sub-tile or a K step, in 16-byte units.  This thread shares
      // its scheduler with busy epilogue warps, so it adds little else.
      constexpr uint32_t MN_STEP = (UMMA_K * 128) >> 4, K_STEP = (UMMA_K * 2) >> 4;
      constexpr uint32_t B_STEP = GRAD ? MN_STEP : K_STEP;
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem) + A_BYTES, GRAD ? ATOM : 16, 1024);
      const uint32_t a_hi = static_cast<uint32_t>(adesc0 >> 32), b_hi = static_cast<uint32_t>(bdesc0 >> 32);
      uint32_t a_lo = static_cast<uint32_t>(adesc0);
      const uint32_t b_lo = static_cast<uint32_t>(bdesc0);
      uint32_t a_step = K_STEP, idesc = idesc_bf16(2 * BM, BN, false, GRAD);
      if (!GRAD && NS == 1)
        idesc = p.grid[0].tile == BN ? idesc_bf16(2 * BM, BN, false, false)
                                     : p.grid[0].tile == 128 ? idesc_bf16(2 * BM, 128, false, false)
                                                               : idesc_bf16(2 * BM, 64, false, false);
      // one K slice of sub-tile `s` from ring stage st into accumulator d
      auto mmas = [&](uint32_t d, int st, int s, bool first) {
        const uint32_t a = a_lo + st * (PL::STAGE >> 4);
        const uint32_t b = b_lo + st * (PL::STAGE >> 4) + s * (B_BYTES >> 4);
        mma_pair(d, a, a_hi, b, b_hi, idesc, first ? 0u : 1u);
#pragma unroll
        for (int kk = 1; kk < BK / UMMA_K; ++kk) mma_pair(d, a + a_step * kk, a_hi, b + B_STEP * kk, b_hi, idesc, 1u);
      };
      Item it;
      for (int j = 0; ok && item_of(p, unit, U, j, it); ++j) {
        const int kit = it.k1 - it.k0;
        if (GRAD) {
          a_step = it.dx ? K_STEP : MN_STEP;
          a_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem), it.dx ? 16 : ATOM, 1024));
          idesc = it.dx ? idesc_bf16(2 * BM, BN, false, true) : idesc_bf16(2 * BM, BN, true, true);
        }
        if (NS == 2) {
          // both accumulators belong to this tile: sub-tile 0 starts once its
          // columns are drained, sub-tile 1's first slices stay in the ring
          // until its own are
          ok = mbar_wait_cluster(tempty, acc_phase ^ 1u, abort_flag);
          if (!ok) break;
          fence_after_sync();
          // (without a second sub-tile its columns are still waited for below, so
          // that the barrier's phases keep step with the tiles)
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
            if (!it.wide) {
              mma_commit_pair(empty + stage);
              if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
              }
              continue;
            }
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
    const int quad = warp & 3;                 // TMEM lanes 32 quad .. 32 quad + 31
    const int part = (warp - 2) >> 2;          // columns 64 part .. + 63 of a sub-tile
    const uint32_t slab = smem_u32(slab_mem + (warp - 2) * PL::SLAB);
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
      const int row0 = it.m * 2 * BM + rank * BM + quad * 32;  // this warp's 32 rows
      const int row = row0 + lane;
      const int M = GRAD && !it.dx ? p.V : p.n;
      const int rows = M - row0;  // rows of them that exist (or fewer than 1)
      // what the epilogue adds to its row, fetched while the product runs
      int target = -1;
      float2 cf = make_float2(0.f, 0.f);
      int first = 0, tokens = 0;  // dW: the positions of this word's tokens
      if (row < M) {
        if (!GRAD || it.dx) {
          target = __ldg(p.targets + row);
          if (GRAD) cf = __ldg(p.coef + row);
        } else {
          // a word without tokens holds what an earlier call left there
          const int2 at = __ldg(p.words + row);
          if (static_cast<unsigned>(at.x) < static_cast<unsigned>(p.n) && __ldg(p.skey + at.x) == row) {
            first = at.x;
            tokens = at.y - at.x;
            // the sums it will add (1216 x 736 x 41031 in 512-wide tiles: 152 us
            // with two binary searches and no prefetch, 149 so; 126 without the
            // additions, which registers are too few to fetch earlier)
            if (tokens > p.direct) {
              const float* a = p.runs + static_cast<int64_t>(first) * p.d + it.c0 + part * 64;
              const int cols = p.d - (it.c0 + part * 64);
#pragma unroll
              for (int i = 0; i < 2 * NS; ++i)
                if ((i < 2 || it.wide) && (i >> 1) * BN + (i & 1) * 32 < cols) prefetch_l1(a + (i >> 1) * BN + (i & 1) * 32);
            }
          }
        }
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int width = GRAD || NS == 2 ? BN : p.grid[0].tile;
        const int c = it.c0 + s * BN + part * 64;  // this warp's first column
        if (NS == 1 || s == 0) {
          ok = mbar_wait_cluster(tfull + acc, acc_phase, abort_flag);
          if (!ok) break;
          __syncwarp();
        }
        if ((NS == 2 && s == 1 && !it.wide) || (NS == 1 && part * 64 >= width)) {
          release();  // no such columns
          continue;
        }
        fence_after_sync();
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * BN + part * 64;
        if (!GRAD) {
          float v[64];
          __syncwarp();  // the first sub-tile left lanes with a target or a reference of their own
          tmem_load64(tb, v);
          release();  // all of this warp's columns are in registers
          const int cols = p.V - c;  // words from here on
          if (cols <= 0) continue;
          const int mine = target - c;  // the target's column, if it is one of these
          const bool here = static_cast<unsigned>(mine) < 64u;
          if (here) {
            float l = 0.f;
#pragma unroll
            for (int q = 0; q < 64; ++q) l = q == mine ? v[q] : l;
            p.target_logit[row] = l * p.unbias;
          }
          if (cols < 64) {
#pragma unroll
            for (int q = 0; q < 64; ++q) v[q] = q < cols ? v[q] : -INFINITY;
          }
          float top = v[0], top2 = v[1];
#pragma unroll
          for (int q = 2; q < 62; q += 4) {
            top = max3(top, v[q], v[q + 1]);
            top2 = max3(top2, v[q + 2], v[q + 3]);
          }
          top = max3(top, max3(top2, v[62], v[63]), -INFINITY);
          const bool shift = top > kRefHigh || (top < kRefLow && top != -INFINITY);
          const float ref = shift ? top * p.unbias : 0.f;
          // The reference leaves before the scaling to powers of two: ref log2 e of a
          // logit near the type's limits (a mask by its lowest value) is infinite,
          // and of one of some hundreds loses digits of the difference.
          if (__any_sync(0xffffffffu, shift)) {
            const float less = shift ? top : 0.f;
#pragma unroll
            for (int q = 0; q < 64; ++q) v[q] -= less;
          }
          const float2 k2 = make_float2(kLog2e * p.unbias, kLog2e * p.unbias);
          float2 sum2 = make_float2(0.f, 0.f), sum3 = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 64; q += 4) {
            float2 a = f2_mul(make_float2(v[q], v[q + 1]), k2);
            float2 b = f2_mul(make_float2(v[q + 2], v[q + 3]), k2);
            a = make_float2(ex2(a.x), ex2(a.y));
            b = make_float2(ex2(b.x), ex2(b.y));
            sum2 = f2_add(sum2, a);
            sum3 = f2_add(sum3, b);
            v[q] = a.x, v[q + 1] = a.y, v[q + 2] = b.x, v[q + 3] = b.y;
          }
          if (row < p.n) {
            // a sum belongs to the reference 0, or, with its sign set, to one in refs
            const float sum = (sum2.x + sum2.y) + (sum3.x + sum3.y);
            const int64_t at = static_cast<int64_t>(c / kGroup) * p.ldp + row;
            p.sums[at] = shift ? -fabsf(sum) : fabsf(sum);
            if (shift) p.refs[at] = ref;
          }
          if (p.E32 && row < p.n) {
            float4* o = reinterpret_cast<float4*>(p.E32 + static_cast<int64_t>(row) * p.ldv + c);
#pragma unroll
            for (int q = 0; q < 16; ++q) o[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
          if (p.E) {
            if (here) {  // the target's own element is added in fp32 by the gradients
#pragma unroll
              for (int q = 0; q < 64; ++q) v[q] = q == mine ? 0.f : v[q];
            }
            if (PL::TMA_OUT) {
              if (rows > 0) write_tile(slab, lane, v, &p.map_e, c, row0);
            } else {
              uint16_t* o = p.E + static_cast<int64_t>(row0) * p.ldv + c;  // ldv is a multiple of 64
              write_rows32(slab, lane, v, o, p.ldv, rows, 32);
              write_rows32(slab, lane, v + 32, o + 32, p.ldv, rows, 32);
            }
          }
        } else {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            float v[32];
            __syncwarp();  // dW: the lanes took different numbers of tokens
            tmem_ld32(tb + 32 * h, v);
            tmem_wait(v);
            if (h == 1) release();  // the last of this warp's columns are in registers
            const int ch = c + 32 * h;
            const int cols = p.d - ch;  // columns that exist from here on
            if (cols <= 0) continue;
            if (it.dx) {
              if (p.dx_part) {
                write_rows32(slab, lane, v, p.dx_part + (static_cast<int64_t>(it.part) * p.n + row0) * p.d + ch, p.d,
                             rows, cols);
              } else {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = cf.x == 0.f ? 0.f : v[q] * cf.x;
                if (cf.y != 0.f) add_row32(v, p.W + static_cast<int64_t>(target) * p.d + ch, cf.y, cols);
                write_rows32(slab, lane, v, p.dx + static_cast<int64_t>(row0) * p.d + ch, p.d, rows, cols);
              }
            } else {
              if (tokens > p.direct) {
                for (int q = first; q < first + tokens; q = (q / kRun + 1) * kRun)
                  add_row32(v, p.runs + static_cast<int64_t>(q) * p.d + ch, cols);
              } else {
                for (int q = 0; q < tokens; ++q) {
                  const int t = __ldg(p.order + first + q);
                  const float k = __ldg(&p.coef[t].y);
                  if (k != 0.f) add_row32(v, p.x + static_cast<int64_t>(t) * p.d + ch, k, cols);
                }
              }
              if (p.dw_add && row < M) add_row32(v, p.dw_add + static_cast<int64_t>(row) * p.d + ch, cols);
              if (p.dw32) write_rows32(slab, lane, v, p.dw32 + static_cast<int64_t>(row0) * p.d + ch, p.d, rows, cols);
              else write_rows32(slab, lane, v, p.dw + static_cast<int64_t>(row0) * p.d + ch, p.d, rows, cols);
            }
          }
        }
      }
    }
    if (PL::TMA_OUT && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // all of it written
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

// ------------------------------------------------------- tokens by target


// Sums of c_t x_t by word, in blocks of kRun = 32 positions of the sorted
// order: runs[r], r a word's first position or a multiple of 32, sums its
// tokens from there to the end of the block; and words[v], where a word's
// tokens begin and end.  Words of at most `direct` tokens
// inside one block are left out.  One warp per block of positions and kRunCols
// columns, eight rows in flight.
constexpr int kRunCols = 256;
static_assert(kRun == 32, "a lane per position");
__global__ void __launch_bounds__(128)
    target_runs_kernel(const uint16_t* __restrict__ x, int n, int d, int V, int direct,
                       const int32_t* __restrict__ skey, const int32_t* __restrict__ order,
                       const float2* __restrict__ coef, float* __restrict__ runs, int2* __restrict__ words) {
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int base = (blockIdx.x * 4 + (threadIdx.x >> 5)) * kRun;
  if (base >= n) return;
  const int r = base + lane;
  const int key = r < n ? __ldg(skey + r) : -1;
  const int before = r > 0 && r <= n ? __ldg(skey + r - 1) : -1;  // (the end of the tokens starts a "word", too)
  const int after = base + kRun < n ? __ldg(skey + base + kRun) : -1;
  const bool word = r < n && key < V;
  const int token = word ? __ldg(order + r) : 0;
  const float weight = word ? __ldg(&coef[token].y) : 0.f;
  // this position's word: positions s .. e - 1 of the block
  const uint32_t starts = __ballot_sync(0xffffffffu, lane == 0 || key != before);
  const int s = 31 - __clz(starts & (0xffffffffu >> (31 - lane)));
  const uint32_t later = lane == 31 ? 0u : starts >> (lane + 1);
  const int e = later ? lane + __ffs(later) : 32;
  const int left = __shfl_sync(0xffffffffu, before, 0);  // the key before the block
  const bool crosses = (s == 0 && left == key) || (e == 32 && after == key);
  const uint32_t need = __ballot_sync(0xffffffffu, word && (e - s > direct || crosses));
  if (blockIdx.y == 0 && word) {  // where the word's tokens begin and end
    if (lane == s && !(s == 0 && left == key)) words[key].x = r;
    if (lane + 1 == e && !(e == 32 && after == key)) words[key].y = r + 1;
  }
  const int c = blockIdx.y * kRunCols + lane * 8;
  const uint16_t* col = x + (c < d ? c : 0);
  float acc[8] = {};
#pragma unroll 1
  for (int b = 0; b < 32; b += 8) {
    if (!((need >> b) & 0xffu)) continue;
    uint4 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = __shfl_sync(0xffffffffu, token, b + j);
      u[j] = __ldg(reinterpret_cast<const uint4*>(col + static_cast<int64_t>(t) * d));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float w = __shfl_sync(0xffffffffu, weight, b + j);
      const int from = __shfl_sync(0xffffffffu, s, b + j), end = __shfl_sync(0xffffffffu, e, b + j);
      if (!((need >> (b + j)) & 1u)) continue;
      float f[8];
      unpack8x(u[j], f);
      if (w != 0.f) {  // a token of no weight may hold what is not finite
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
      }
      if (b + j + 1 == end) {  // the word's last position here
        if (c < d) {
          float4* o = reinterpret_cast<float4*>(runs + static_cast<int64_t>(base + from) * d + c);
          o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
          o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      }
    }
  }
}

// ------------------------------------------------------------ row statistics


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

struct ParamsR {
  const float* sums;
  const float* refs;
  int64_t ldp;
  int groups;
  const float* target_logit;
  const int32_t* targets;
  int n, d, V, ignore;
  const float* d_loss;
  const int32_t* count;
  float* loss;
  float* lse;
  float2* coef;       // NULL: the loss alone
  const uint16_t* x;
  uint16_t* xs;       // s x in bf16 (NULL: no dW)
  uint16_t* E;
  float* E32;
  int64_t ldv;
  int sorting;        // blocks that sort
  int32_t* skey;
  int32_t* order;
  int32_t* err;
};

constexpr int kStatThreads = 1024;
constexpr int kSortTokens = 2 * kStatThreads / 32;  // per block
constexpr int kSortChunk = 2048;

// Stable sort of the piece's targets (those that do not count last) by
// counting: each warp counts the tokens that come before two of its own, n^2
// comparisons in all.  The keys are held in fp32 (exact to 2^24): a comparison
// is then saturate(limit - key), 1 or 0, and runs at the full rate of the
// FMA pipe, where integer comparisons have half.  skey[r], order[r]: the key
// and the token at position r.
__device__ void sort_targets(const ParamsR& p, int block, float4* keys) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int t0 = block * kSortTokens + 2 * warp, t1 = t0 + 1;  // in one group of four
  const int key0 = t0 < p.n ? key_of(__ldg(p.targets + t0), p.V, p.ignore) : 0;
  const int key1 = t1 < p.n ? key_of(__ldg(p.targets + t1), p.V, p.ignore) : 0;
  float f0 = 0.f, f1 = 0.f;
  for (int base = 0; base < p.n; base += kSortChunk) {
    const int groups = min(kSortChunk, (p.n - base + 3) & ~3) / 4;
    __syncthreads();
    for (int i = threadIdx.x; i < 4 * groups; i += kStatThreads)  // past the end: after every key
      reinterpret_cast<float*>(keys)[i] =
          base + i < p.n ? static_cast<float>(key_of(__ldg(p.targets + base + i), p.V, p.ignore)) : 3e7f;
    __syncthreads();
    const int split = (t0 - base) >> 2;  // groups before the tokens' own also count equal keys
#pragma unroll 4
    for (int i = lane; i < groups; i += 32) {
      const float4 k = keys[i];
      const float eq = i < split ? 1.f : 0.f;
      const float l0 = static_cast<float>(key0) + eq, l1 = static_cast<float>(key1) + eq;
      f0 += (__saturatef(l0 - k.x) + __saturatef(l0 - k.y)) + (__saturatef(l0 - k.z) + __saturatef(l0 - k.w));
      f1 += (__saturatef(l1 - k.x) + __saturatef(l1 - k.y)) + (__saturatef(l1 - k.z) + __saturatef(l1 - k.w));
    }
  }
  int r0 = static_cast<int>(f0), r1 = static_cast<int>(f1);
  // equal keys earlier in the tokens' own group of four
  const int u = (t0 & ~3) + lane;
  if (lane < 3 && u < p.n) {
    const int k = key_of(__ldg(p.targets + u), p.V, p.ignore);
    r0 += u < t0 && k == key0;
    r1 += u < t1 && k == key1;
  }
  r0 = __reduce_add_sync(0xffffffffu, r0);
  r1 = __reduce_add_sync(0xffffffffu, r1);
  if (lane == 0 && t0 < p.n) {
    p.skey[r0] = key0;
    p.order[r0] = t0;
    if (t1 < p.n) {
      p.skey[r1] = key1;
      p.order[r1] = t1;
    }
  }
}

// ROWS rows per block (32, or 8 where those leave SMs idle): 1024 / ROWS
// threads share a row's groups, then its warps write s x and, where the row's
// groups have different references, bring its E to one.  The first blocks, the
// longer ones, sort the targets.
constexpr int kStatFewRows = 2048;  // 26 rows of 85000 words: 12.8 us by 32, 6.2 by 8
template <int ROWS>
__global__ void __launch_bounds__(kStatThreads, 2) row_stats_kernel(const ParamsR p) {
  constexpr int SLICES = kStatThreads / ROWS;
  constexpr int WARPS = 32 / ROWS;  // per row, for the second half
  __shared__ float4 sh[SLICES][ROWS];
  __shared__ float sh_s[ROWS], sh_r[ROWS];
  __shared__ int sh_fix[ROWS];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) < p.sorting) {
    static_assert(sizeof(sh) >= kSortChunk * sizeof(float), "the keys share the rows' scratch");
    sort_targets(p, static_cast<int>(blockIdx.x), &sh[0][0]);
    return;
  }
  const int block = static_cast<int>(blockIdx.x) - p.sorting;
  const int r0 = threadIdx.x % ROWS;
  const int slice = threadIdx.x / ROWS;
  const int t = block * ROWS + r0;
  float R = -INFINITY, S = 0.f, low = INFINITY, high = -INFINITY;
  if (t < p.n) {
    for (int g0 = slice; g0 < p.groups; g0 += 4 * SLICES) {
      float s[4];  // four loads in flight
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = g0 + i * SLICES;
        s[i] = g < p.groups ? __ldg(p.sums + g * p.ldp + t) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = g0 + i * SLICES;
        if (g >= p.groups) break;
        if (s[i] == 0.f) continue;  // words that are all masked by minus infinity: no reference either
        const float r = signbit(s[i]) ? __ldg(p.refs + g * p.ldp + t) : 0.f;
        join(R, S, r, fabsf(s[i]));
        low = fminf(low, r);
        high = fmaxf(high, r);
      }
    }
  }
  sh[slice][r0] = make_float4(R, S, low, high);
#pragma unroll 1
  for (int half = SLICES / 2; half > 0; half /= 2) {
    __syncthreads();
    if (slice < half) {
      const float4 q = sh[slice + half][r0];
      if (q.x != -INFINITY) join(R, S, q.x, q.y);  // else no groups
      low = fminf(low, q.z);
      high = fmaxf(high, q.w);
      sh[slice][r0] = make_float4(R, S, low, high);
    }
  }
  if (slice == 0 && t < p.n) {
    const float L = R + logf(S);
    const int32_t v = __ldg(p.targets + t);
    const bool counts = key_of(v, p.V, p.ignore) < p.V;
    if (!counts && v != p.ignore) dmoe::raise_error(p.err, DMOE_SITE_LOSS_TARGET | DMOE_ERR_DEVICE);
    const float nll = counts ? L - __ldg(p.target_logit + t) : 0.f;
    p.loss[t] = nll;
    if (p.lse) p.lse[t] = L;
    if (p.coef) {
      float g = 0.f;
      if (counts) g = p.d_loss ? __ldg(p.d_loss + t) : 1.f / static_cast<float>(*p.count);
      const float s = g == 0.f ? 0.f : g * expf(R - L);
      // expm1: where the softmax at the target is close to 1 or to 0
      p.coef[t] = make_float2(s, g == 0.f ? 0.f : g * expm1f(-nll));
      sh_s[r0] = s;
      sh_r[r0] = R;
      // 1: bring the row's groups to one reference; 2: a row that does not
      // count holds what is not finite, which times 0 would still spread
      sh_fix[r0] = g == 0.f ? (isfinite(S) ? 0 : 2) : (low != high ? 1 : 0);
    }
  }
  if (!p.coef) return;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int rw = (threadIdx.x >> 5) / WARPS, sub = (threadIdx.x >> 5) % WARPS;
  const int row = block * ROWS + rw;
  if (row >= p.n) return;
  if (p.xs) {
    const float s = sh_s[rw];
    const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(row) * p.d);
    uint4* dst = reinterpret_cast<uint4*>(p.xs + static_cast<int64_t>(row) * p.d);
#pragma unroll 4
    for (int v = sub * 32 + lane; v < p.d / 8; v += 32 * WARPS) {
      float f[8];
      unpack8x(__ldg(src + v), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = s == 0.f ? 0.f : f[j] * s;
      dst[v] = pack8x(f);
    }
  }
  const int fix = sh_fix[rw];
  if (fix) {
    const float top = sh_r[rw];
    uint16_t* e = p.E + static_cast<int64_t>(row) * p.ldv;
    for (int g = sub; g < p.groups; g += WARPS) {
      const float s = __ldg(p.sums + g * p.ldp + row);
      const float r = signbit(s) ? __ldg(p.refs + g * p.ldp + row) : 0.f;
      if (fix == 1 && (r == top || s == 0.f)) continue;  // nothing to bring there (0 stays 0)
      const float k = fix == 2 ? 0.f : expf(r - top);
      __nv_bfloat162* u = reinterpret_cast<__nv_bfloat162*>(e + g * kGroup) + lane;
      float2 f = __bfloat1622float2(*u);
      f.x = fix == 2 ? 0.f : f.x * k;
      f.y = fix == 2 ? 0.f : f.y * k;
      *u = __floats2bfloat162_rn(f.x, f.y);
      if (p.E32) {
        float2* u32 = reinterpret_cast<float2*>(p.E32 + row * p.ldv + g * kGroup) + lane;
        *u32 = fix == 2 ? make_float2(0.f, 0.f) : make_float2(u32->x * k, u32->y * k);
      }
    }
  }
}

// dW of a few tokens (n <= NT <= kFewTokens): rows of dW are then sums of a few
// multiples of rows of x, bound by writing them, and need neither the tensor
// cores nor the sort, and E can stay in fp32 (with so few terms its rounding
// would not average out).  A block takes kFewRows words; their coefficients
// s_t E_tv (c_t at a token's target) meet in shared memory in fp32, every
// thread holds 8 columns of the n tokens' x.  32000 words, d = 4096: 54 us
// for 8 tokens beside 59 for dx; with 9 tokens the tensor cores take 115 us
// for both, and a launch before it.
constexpr int kFewRows = 64;
constexpr int kFewThreads = 128;
template <int NT>
__global__ void __launch_bounds__(kFewThreads)
    few_dw_kernel(const float* __restrict__ E32, int64_t ldv, const float2* __restrict__ coef,
                  const int32_t* __restrict__ targets, const uint16_t* __restrict__ x, int n, int d, int V,
                  int per_row, uint16_t* dw, float* dw32, const float* add) {
  __shared__ float a[kFewRows][NT];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  // The tokens of some weight: a row of none may hold anything, and 0 times what
  // is not finite is not 0.
  const int lane = threadIdx.x & 31;
  const float2 own = lane < n ? __ldg(coef + lane) : make_float2(0.f, 0.f);
  const uint32_t weighs = __ballot_sync(0xffffffffu, own.x != 0.f || own.y != 0.f);
  const int v0 = blockIdx.x * kFewRows;
  for (int i = threadIdx.x; i < kFewRows * NT; i += kFewThreads) {
    const int t = i / kFewRows, r = i % kFewRows, v = v0 + r;
    float k = 0.f;
    if (t < n && v < V) {
      const float2 cf = __ldg(coef + t);
      if (__ldg(targets + t) == v) k = cf.y;
      else if (cf.x != 0.f) k = cf.x * __ldg(E32 + t * ldv + v);
    }
    a[r][t] = k;
  }
  // per_row threads (a power of two) share a row, the others take further rows
  const int c = (blockIdx.y * per_row + threadIdx.x % per_row) * 8;
  float2 xf[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float f[8] = {};
    if ((weighs >> t & 1u) && c < d)
      unpack8x(__ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(t) * d + c)), f);
#pragma unroll
    for (int j = 0; j < 4; ++j) xf[t][j] = make_float2(f[2 * j], f[2 * j + 1]);
  }
  __syncthreads();
  if (c >= d) return;
  const int rows = min(kFewRows, V - v0);
#pragma unroll 2
  for (int r = threadIdx.x / per_row; r < rows; r += kFewThreads / per_row) {
    float2 o[4] = {};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float2 k = make_float2(a[r][t], a[r][t]);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = f2_fma(k, xf[t][j], o[j]);
    }
    const int64_t at = static_cast<int64_t>(v0 + r) * d + c;
    float f[8] = {o[0].x, o[0].y, o[1].x, o[1].y, o[2].x, o[2].y, o[3].x, o[3].y};
    if (add) {
      const float4 p = *reinterpret_cast<const float4*>(add + at), q = *reinterpret_cast<const float4*>(add + at + 4);
      f[0] += p.x, f[1] += p.y, f[2] += p.z, f[3] += p.w;
      f[4] += q.x, f[5] += q.y, f[6] += q.z, f[7] += q.w;
    }
    if (dw32) {
      *reinterpret_cast<float4*>(dw32 + at) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(dw32 + at + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(dw + at) = pack8x(f);
    }
  }
}

// dx from the fp32 sums of its parts: SHARE threads (1, or 8 where there are
// many parts) per 8 columns.
template <int SHARE>
__global__ void __launch_bounds__(256)
    join_dx_kernel(const float* __restrict__ part, int parts, int n, int d, const float2* __restrict__ coef,
                   const int32_t* __restrict__ targets, const uint16_t* __restrict__ W, uint16_t* __restrict__ dx) {
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int nvec = d / 8;
  const int64_t all = static_cast<int64_t>(n) * nvec;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / SHARE;
  const int mine = threadIdx.x % SHARE;
  const int64_t i = at < all ? at : all - 1;  // every lane takes part in the sum
  const int64_t t = i / nvec;
  const int c = static_cast<int>(i - t * nvec) * 8;
  const float2 cf = __ldg(coef + t);
  const int target = __ldg(targets + t);
  float acc[8] = {};
#pragma unroll 4
  for (int q = mine; q < parts; q += SHARE) {
    const float4* a = reinterpret_cast<const float4*>(part + (static_cast<int64_t>(q) * n + t) * d + c);
    const float4 u = __ldg(a), v = __ldg(a + 1);
    acc[0] += u.x, acc[1] += u.y, acc[2] += u.z, acc[3] += u.w;
    acc[4] += v.x, acc[5] += v.y, acc[6] += v.z, acc[7] += v.w;
  }
#pragma unroll
  for (int o = SHARE / 2; o > 0; o /= 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
  }
  if (mine != 0 || at >= all) return;
  float f[8] = {};
  if (cf.y != 0.f) unpack8x(__ldg(reinterpret_cast<const uint4*>(W + static_cast<int64_t>(target) * d + c)), f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = fmaf(cf.y, f[j], cf.x == 0.f ? 0.f : acc[j] * cf.x);
  *reinterpret_cast<uint4*>(dx + t * d + c) = pack8x(f);
}

// ----------------------------------------------------------------- host side

// Time of a gradient item in hundredths of a 512-wide K slice (0.57 us), as
// measured: the product, of whose operands a 256-wide tile loads a third more
// a column (8192 x 512 x 32000 all in 256-wide tiles: 0.69 a slice), and the
// part of the epilogue that the next product does not hide (dW alone, 64 and
// 19 slices: 10 to 12 slices an item).  alone: no other tile reads the same B,
// whose 64 KB (or 32) a slice then come from HBM, 0.73 us for 76 pairs
// together.
int64_t item_time(int slices, int tile, int cols, bool alone = false) {
  if (tile > BN && cols > BN) return (alone ? 128 : 100) * static_cast<int64_t>(slices) + 1000;
  return (alone ? 95 : 69) * static_cast<int64_t>(slices) + 560;
}

Grid make_grid(int M, int N, int K, int raster, int parts = 1, int tile = 2 * BN) {
  Grid g = cut_grid(M, N, K, raster, parts, tile);
  g.time = item_time(g.per_part, tile, N, g.mt == 1);
  return g;
}

// Columns of a logits tile.  Few tokens and words make few tiles; then narrower
// ones spread the reading of W over more SMs: the width whose busiest pair is
// shortest, in hundredths of a 256-wide slice.  A 512-wide one saves operands,
// of a narrower one the loads of x and the latency stay.  The loss, 512-, 256-,
// 128- and 64-wide: 1 x 4096 x 5000 words 47, 33, 31 and 47 us; 167 x 2640 x
// 24257 47, 51, 57 and 74; 313 x 3160 x 14191 48, 55, 62 and 96; 1024 x 3160 x
// 50645 217, 240, 328 and 582; 1024 x 4096 x 32000 168, 158, 256 and 473.
int logits_tile(int n, int d, int V) {
  const int64_t mt = ceil_div(n, 2 * BM);
  auto cost = [&](int tile, int per_slice) {
    return static_cast<int64_t>(ceil_div(mt * ceil_div(V, tile), kUnits)) * per_slice;
  };
  int best = d <= kNarrowD ? BN : 2 * BN;
  int64_t least = best == BN ? cost(BN, 100) : cost(2 * BN, 180);
  for (const auto& w : {std::pair<int, int>{BN, 100}, {128, 75}, {64, 60}})
    if (cost(w.first, w.second) < least) {
      best = w.first;
      least = cost(w.first, w.second);
    }
  return best;
}

void deal(ParamsX& p, const Grid& gx, const Grid& gw, int U) {
  p.first_dx = gx.items > 0 && (gw.items == 0 || gx.time >= gw.time);
  p.grid[0] = p.first_dx ? gx : gw;
  p.grid[1] = p.first_dx ? gw : gx;
  const Dealt r = dealt(p.grid[0].items, p.grid[0].time, p.grid[1].items, std::max<int64_t>(1, p.grid[1].time), U);
  p.full = r.full, p.rem = r.rem, p.early = r.early, p.extra = r.extra;
}

// How the gradients' tiles are cut: the widths of dx's and dW's tiles and the
// parts of dx's sum over the vocabulary.  512-wide tiles are the faster ones
// by operands, but few: dx has few tiles of V / 64 slices each, and the last
// of them can outlast everything else (512 tokens: 8 tiles for 76 pairs).
// Takes the cut whose busiest unit is shortest, charging the fp32 sums that
// parts write and read back: 12 bytes an element at 6.5 TB/s, and a launch.
// Times are compared as whole numbers, without a division: over the n of the
// same number of K slices only the charge changes, by parts * d each token, so
// that more tokens never mean more parts there (part_bytes_up_to() counts on it).
// Gradients with the join of the parts, 512-wide tiles throughout and as cut
// here: 2000 x 2048 x 32000 341 and 301 us, 1216 x 736 x 41031 167 and 144,
// 13 x 3984 x 48294 170 and 164; 8192 x 512 x 32000 317 us in the 512-wide
// tiles that it gets, 362 in 256-wide ones.
struct Cut {
  int parts, tile_x, tile_w;
};
Cut cut_grads(int n, int d, int V, bool dx, bool dw) {
  const int mx = ceil_div(n, 2 * BM), mw = ceil_div(V, 2 * BM), slices = ceil_div(V, BK);
  Cut best{1, 2 * BN, 2 * BN};
  int64_t least = -1;
  for (const int tx : {2 * BN, BN}) {
    for (const int tw : {2 * BN, BN}) {
      if ((tx == BN && (!dx || d <= BN)) || (tw == BN && (!dw || d <= BN))) continue;
      const int nw = dw ? mw * ceil_div(d, tw) : 0;
      const int64_t lw = item_time(ceil_div(n, BK), tw, d, mw == 1);
      for (const int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
        const int nx = dx ? mx * ceil_div(d, tx) * s : 0;
        if (s > 1 && (!dx || slices / s < 8 || nx > 16 * kUnits)) break;
        const int64_t lx = item_time(ceil_div(slices, s), tx, d, mx == 1);
        const int64_t busiest = (nw == 0 || (nx > 0 && lx >= lw) ? dealt(nx, lx, nw, lw, kUnits) : dealt(nw, lw, nx, lx, kUnits)).busiest;
        const int64_t time = 2700 * (busiest + (s > 1 ? 1000 : 0)) + (s > 1 ? static_cast<int64_t>(s) * n * d : 0);
        if (least < 0 || time < least) {
          best = Cut{s, tx, tw};
          least = time;
        }
      }
    }
  }
  return best;
}

// Opt-in shared memory and the number of 2-CTA clusters that fit, once per
// instantiation and device.
template <bool GRAD, int NS>
dmoe_status launch_head(ParamsX& p, const Grid& ga, const Grid& gb, const dmoe::DeviceInfo& di, cudaStream_t st) {
  auto kern = head_kernel<GRAD, NS>;
  const size_t smem = PlanX<GRAD, NS>::SMEM;
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
  const int units = static_cast<int>(std::min<int64_t>(n, static_cast<int64_t>(ga.items) + gb.items));
  deal(p, ga, gb, units);
  cudaError_t e = dmoe::launch_pdl_cluster(kern, dim3(2 * units), dim3(kThreadsX), smem, st, 2, p);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

// Bytes of a workspace, in order (each part 256-byte aligned).
struct Layout {
  int64_t piece;   // tokens per piece
  int64_t ldp;     // row pitch of sums and refs
  int64_t ldv;     // row pitch of the exponentials
  int64_t groups;
  size_t count, sums, refs, target_logit, coef, skey, order, words, xs, runs, acc, E32, E, part;
};

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
  const size_t rows = static_cast<size_t>(l.piece);
  l.count = take(256);
  l.sums = take(static_cast<size_t>(l.groups * l.ldp) * sizeof(float));
  l.refs = take(static_cast<size_t>(l.groups * l.ldp) * sizeof(float));
  l.target_logit = take(rows * sizeof(float));
  if (grad) {
    l.coef = take(rows * sizeof(float2));
    l.skey = take(rows * sizeof(int32_t));
    l.order = take(rows * sizeof(int32_t));
    l.words = take(static_cast<size_t>(V) * sizeof(int2));
    l.xs = take(rows * d * 2);
    l.runs = take(rows * d * sizeof(float));
    // dW of earlier pieces, when it does not fit the output's own type
    l.acc = take(dw_bf16 && T > l.piece ? static_cast<size_t>(V) * d * sizeof(float) : 0);
    l.E32 = take(static_cast<size_t>(kFewTokens * l.ldv) * sizeof(float));
    l.E = take(static_cast<size_t>(l.piece * l.ldv) * 2);
  }
  l.part = at;  // dx's parts come last, see part_bytes()
  return l;
}

// Bytes of dx's fp32 parts: the full pieces' or the last, shorter one's.
size_t part_bytes(const Layout& l, int T, int d, int V, bool dw) {
  size_t most = 0;
  for (const int64_t n : {std::min<int64_t>(l.piece, T), T % l.piece}) {
    const int s = n > 0 ? cut_grads(static_cast<int>(n), d, V, true, dw && n > kFewTokens).parts : 1;
    if (s > 1) most = std::max(most, static_cast<size_t>(n) * s * d * sizeof(float));
  }
  return most;
}

// The most of part_bytes() that T tokens or fewer need, with dw or without: the
// parts get more as the tokens get fewer, and a workspace for the longest batch
// has to do for a shorter one.  Counted from the first n of every K slice on, which
// has the most parts of its slice's, up to 63 tokens too many.
size_t part_bytes_up_to(const Layout& l, int T, int d, int V) {
  const int64_t most_n = std::min<int64_t>(l.piece, T);
  size_t most = 0;
  for (int64_t n = 0; n < most_n; n += BK)
    for (const bool dw : {false, true}) {
      const int s = cut_grads(static_cast<int>(n) + 1, d, V, true, dw).parts;
      if (s > 1) most = std::max(most, static_cast<size_t>(std::min(n + BK, most_n)) * s * d * sizeof(float));
    }
  return most;
}

bool sizes_ok(int T, int d, int V, int piece) {
  return T >= 0 && d >= 8 && (d & 7) == 0 && V >= 1 && V < (1 << 24) && d <= (1 << 20) && piece >= 0;
}

#define DMOE_TRY(call)                \
  do {                                \
    const dmoe_status st__ = (call);  \
    if (st__ != DMOE_OK) return st__; \
  } while (0)

#define DMOE_TRY_LAUNCH(call)                          \
  do {                                                 \
    const cudaError_t e__ = (call);                    \
    if (e__ != cudaSuccess) return dmoe::cuda_status(e__); \
    dmoe::count_launches(1);                           \
  } while (0)

}  // namespace

DMOE_API size_t dmoe_linear_cross_entropy_workspace_size(int T, int d, int V, int grad, int dw_f32, int piece) {
  if (!sizes_ok(T, d, V, piece)) return 0;
  const Layout l = layout_of(T, d, V, grad != 0, !dw_f32, piece);
  return l.part + (grad ? part_bytes_up_to(l, T, d, V) : 0);
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
  if (T > 0 && ws_bytes < l.part + (dx ? part_bytes(l, T, d, V, dw != nullptr) : 0)) return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  DMOE_TRY(dmoe::device_info(&di));
  cudaStream_t st = dmoe::as_stream(stream);
  if (T == 0) {
    if (dw && !accumulate)
      return dmoe::cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * d * (dw_f32 ? 4 : 2), st));
    return DMOE_OK;
  }
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto at = [&](size_t off) { return grad ? base + off : nullptr; };
  int32_t* count = reinterpret_cast<int32_t*>(base + l.count);
  float* sums = reinterpret_cast<float*>(base + l.sums);
  float* refs = reinterpret_cast<float*>(base + l.refs);
  float* target_logit = reinterpret_cast<float*>(base + l.target_logit);
  float2* coef = reinterpret_cast<float2*>(at(l.coef));
  int32_t* skey = reinterpret_cast<int32_t*>(at(l.skey));
  int32_t* order = reinterpret_cast<int32_t*>(at(l.order));
  int2* words = reinterpret_cast<int2*>(at(l.words));
  uint16_t* xs = reinterpret_cast<uint16_t*>(at(l.xs));
  float* runs = reinterpret_cast<float*>(at(l.runs));
  float* part = reinterpret_cast<float*>(at(l.part));
  float* acc = reinterpret_cast<float*>(at(l.acc));
  uint16_t* E = reinterpret_cast<uint16_t*>(at(l.E));
  float* E32 = reinterpret_cast<float*>(at(l.E32));

  for (int64_t t0 = 0; t0 < T; t0 += l.piece) {
    const int n = static_cast<int>(std::min<int64_t>(l.piece, T - t0));
    const uint16_t* xp = x + t0 * d;
    const int32_t* tp = targets + t0;
    ParamsX p{};
    p.n = n, p.d = d, p.V = V;
    p.direct = n >= kDirectFrom ? kDirect : 0;
    p.a_rows = static_cast<int>(std::min<int64_t>(BM, round_up(n, 8)));
    p.targets = tp;
    p.err = di.err_word;
    p.ldv = l.ldv;
    {
      ParamsX q = p;
      const int tile = logits_tile(n, d, V);
      if (!dmoe::make_map(&q.map_a, xp, n, d, BK, p.a_rows) ||
          !dmoe::make_map(&q.map_b, w, V, d, BK, std::min(tile, BN) / 2))
        return DMOE_ERR_CUDA;
      if (grad && !dmoe::make_map(&q.map_e, E, n, l.ldv, 64, 32)) return DMOE_ERR_CUDA;
      q.E = E;
      q.E32 = dw && n <= kFewTokens ? E32 : nullptr;
      q.sums = sums;
      q.refs = refs;
      q.ldp = l.ldp;
      q.target_logit = target_logit;
      q.all = grad && !d_loss && t0 == 0 ? targets : nullptr;
      q.T = T, q.ignore = ignore_index, q.count = count;
      q.unbias = 1.f + static_cast<float>(ceil_div(d, UMMA_K)) * kTruncation;
      const Grid g = make_grid(n, V, d, 16, 1, tile);
      if (tile > BN) DMOE_TRY((launch_head<false, 2>(q, g, Grid{}, di, st)));
      else DMOE_TRY((launch_head<false, 1>(q, g, Grid{}, di, st)));
    }
    ParamsR r{};
    r.sums = sums, r.refs = refs, r.ldp = l.ldp, r.groups = static_cast<int>(l.groups);
    r.target_logit = target_logit, r.targets = tp;
    r.n = n, r.d = d, r.V = V, r.ignore = ignore_index;
    r.d_loss = d_loss ? d_loss + t0 : nullptr;
    r.count = count;
    r.loss = loss + t0, r.lse = lse ? lse + t0 : nullptr;
    r.coef = coef;
    const bool few = n <= kFewTokens;
    r.x = xp, r.xs = dw && !few ? xs : nullptr;
    r.E = E, r.E32 = dw && few ? E32 : nullptr, r.ldv = l.ldv;
    r.skey = skey, r.order = order;
    r.err = di.err_word;
    r.sorting = dw && !few ? ceil_div(n, kSortTokens) : 0;
    if (n <= kStatFewRows)
      DMOE_TRY_LAUNCH(dmoe::launch_pdl(row_stats_kernel<8>, dim3(ceil_div(n, 8) + r.sorting), dim3(kStatThreads), 0, st, r));
    else
      DMOE_TRY_LAUNCH(dmoe::launch_pdl(row_stats_kernel<32>, dim3(ceil_div(n, 32) + r.sorting), dim3(kStatThreads), 0, st, r));
    if (!grad) continue;
    if (dw && !few)
      DMOE_TRY_LAUNCH(dmoe::launch_pdl(target_runs_kernel, dim3(ceil_div(n, 4 * kRun), ceil_div(d, kRunCols)),
                                       dim3(128), 0, st, xp, n, d, V, p.direct, static_cast<const int32_t*>(skey),
                                       static_cast<const int32_t*>(order), static_cast<const float2*>(coef), runs, words));
    const Cut cut = cut_grads(n, d, V, dx != nullptr, dw && !few);
    Grid gx{}, gw{};
    // E as [n, V] with row pitch ldv: the columns past V read as zero
    if (dx) {
      if (!map_pitched(&p.map_a, E, n, V, l.ldv, BK, p.a_rows) || !dmoe::make_map(&p.map_b, w, V, d, 64, BK))
        return DMOE_ERR_CUDA;
      gx = make_grid(n, d, V, 16, cut.parts, cut.tile_x);
    }
    if (dw && !few) {
      if (!map_pitched(&p.map_a2, E, n, V, l.ldv, 64, BK) || !dmoe::make_map(&p.map_b2, xs, n, d, 64, BK))
        return DMOE_ERR_CUDA;
      gw = make_grid(V, d, n, 1, 1, cut.tile_w);
    }
    p.coef = coef, p.W = w, p.x = xp;
    p.dx = dx ? dx + t0 * d : nullptr;
    p.dx_part = gx.parts > 1 ? part : nullptr;
    p.skey = skey, p.order = order, p.runs = runs, p.words = words;
    const bool last = t0 + n >= T;
    if (dw_f32) {
      p.dw32 = static_cast<float*>(dw);
      p.dw_add = (accumulate || t0 > 0) ? p.dw32 : nullptr;
    } else {  // fp32 until the last piece, then one rounding
      p.dw = static_cast<uint16_t*>(dw);
      p.dw32 = last ? nullptr : acc;
      p.dw_add = t0 > 0 ? acc : nullptr;
    }
    if (dw && few) {
      int per_row = 1;
      while (per_row < kFewThreads && per_row * 8 < d) per_row *= 2;
      const dim3 grid(ceil_div(V, kFewRows), ceil_div(d, per_row * 8));
      auto kern = n <= 2 ? few_dw_kernel<2> : n <= 4 ? few_dw_kernel<4> : few_dw_kernel<kFewTokens>;
      DMOE_TRY_LAUNCH(dmoe::launch_pdl(kern, grid, dim3(kFewThreads), 0, st, static_cast<const float*>(E32), l.ldv,
                                       static_cast<const float2*>(coef), tp, xp, n, d, V, per_row, p.dw, p.dw32,
                                       p.dw_add));
    }
    if (gx.items + gw.items > 0) DMOE_TRY((launch_head<true, 2>(p, gx, gw, di, st)));
    if (gx.parts > 1) {
      const int share = gx.parts >= 8 ? 8 : 1;
      auto kern = share == 8 ? join_dx_kernel<8> : join_dx_kernel<1>;
      DMOE_TRY_LAUNCH(dmoe::launch_pdl(kern, dim3(ceil_div(static_cast<int64_t>(n) * (d / 8) * share, 256)), dim3(256), 0,
                                       st, static_cast<const float*>(part), gx.parts, n, d,
                                       static_cast<const float2*>(coef), tp, w, dx + t0 * d));
    }
  }
  return DMOE_OK;
}
