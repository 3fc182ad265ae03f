// Residual addition + root-mean-square norm in front of an MoE layer, with
// rows in bf16 or in 8 bits, and its backward.
//
//   h      = bf16(x + residual)                       (h = x without residual)
//   rstd_t = 1 / sqrt(mean_c h_tc^2 + eps)
//   y_tc   = h_tc rstd_t w_c
// The residual stream is kept in bf16 and the norm reads the kept value: the
// backward has nothing else, so it is the gradient of exactly this forward.
//   backward:  u = dy w,  m_t = mean_c u_tc h_tc rstd_t^2
//              dx = dh + rstd (u - h m),   dw_c = sum_t dy_tc h_tc rstd_t
//
// Both are HBM-bound (8 bytes an element, ~10 flops), so each row is read
// once and stays in registers between its sum and its use: TPR threads hold
// a row, VPT 16-byte vectors each, the sum crossing the row's warps by
// shuffles and, above 32 threads, through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace {

using namespace dmoe::rows;

// Block sizes while a row takes fewer threads (up to 2048 columns): smaller
// blocks end sooner.  The kernel alone at 256 and 128 threads: forward 16384 x
// 512 11.3 and 11.0 us, backward 8192 x 512 13.0 and 10.8.
constexpr int kFwdThreads = 128;
constexpr int kNormThreads = 128;  // backward
constexpr int kMaxD = 32768;
constexpr int kQGroup = 128;       // columns that share a scale in the 8-bit rows
constexpr float kE4M3Max = 448.f;
constexpr int kMaxStages = 4;      // backward: units of rows in flight per block
constexpr size_t kRingBytes = 200 * 1024;  // of shared memory for them per SM

// a / b from inv = 1 / b: the product, then one step by what it leaves of a, which
// the fused multiply-add gives without a rounding (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  1 / b the
// same way, from an approximation.  4093 rows of 3584 in 8 bits, calls in a
// row: 19.5 us; 18.7 with values times the approximation, which puts some of
// them one step of e4m3 off; 22.9 with divisions.
__device__ __forceinline__ float quotient(float a, float inv, float b) {
  const float q = a * inv;
  return fmaf(fmaf(-q, b, a), inv, q);
}

__device__ __forceinline__ float2 quotient(float2 a, float inv, float b) {
  const float2 i = make_float2(inv, inv);
  const float2 q = dmoe::f2_mul(a, i);
  return dmoe::f2_fma(dmoe::f2_fma(q, make_float2(-b, -b), a), i, q);
}

__device__ __forceinline__ float reciprocal(float b, float back) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
  return fmaf(fmaf(-back, r, 1.f), r, r);
}

// One row per TPR threads; BLOCK / TPR rows per block.
template <int TPR, int VPT, bool WF32, bool Q8>
__global__ void __launch_bounds__(TPR > kFwdThreads ? TPR : kFwdThreads, 1536 / (TPR > kFwdThreads ? TPR : kFwdThreads))
    add_rms_norm_kernel(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
                        const void* __restrict__ weight, float eps, int T, int d, uint16_t* h, uint16_t* y,
                        float* __restrict__ rstd, uint8_t* __restrict__ q, float* __restrict__ q_scale) {
  constexpr int BLOCK = TPR > kFwdThreads ? TPR : kFwdThreads;
  constexpr int RPB = BLOCK / TPR;
  __shared__ float red[BLOCK / 32];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int c = threadIdx.x % TPR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool live = t < T;
  const int nvec = d >> 3;
  uint4 u[VPT];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = c + i * TPR;
    u[i] = make_uint4(0, 0, 0, 0);
    if (live && v < nvec) {
      u[i] = *(reinterpret_cast<const uint4*>(x + t * ldx) + v);
      if (residual) {
        const uint4 rv = *(reinterpret_cast<const uint4*>(residual + t * ldr) + v);
        float f[8], g[8];
        unpack8(u[i], f);
        unpack8(rv, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += g[j];
        u[i] = pack8(f);  // the kept stream: bf16, what the backward will read
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float f[8];
    unpack8(u[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
  }
  ss = row_sum<TPR>(ss, red);
  const float r = rsqrtf(ss / static_cast<float>(d) + eps);
  if (live && c == 0 && rstd) rstd[t] = r;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = c + i * TPR;
    const bool in = live && v < nvec;
    float f[8], w[8];
    unpack8(u[i], f);
    if (in) {
      if (h) *(reinterpret_cast<uint4*>(h + t * d) + v) = u[i];
      load_w<WF32>(weight, v, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * r * w[j];
      if (y) *(reinterpret_cast<uint4*>(y + t * d) + v) = pack8(f);
    }
    if (Q8) {
      // 16 neighbouring lanes hold the 128 columns of one scale (TPR and the
      // row's first vector are multiples of 16); lanes past the row hold 0
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // at least the smallest normal number: the scale of a group keeps its digits
      const float s = top == INFINITY ? top
                      : top > 0.f     ? fmaxf(quotient(top, 1.f / kE4M3Max, kE4M3Max), 1.17549435e-38f)
                                      : 1.f;
      if (in) {
        const float back = s < INFINITY ? s : 0.f;  // what is finite over an infinite scale is 0
        const float inv = reciprocal(s, back);
        // Two values an instruction, except where forty registers must hold four
        // vectors (4096 x 10240: 76.9 us in pairs, 66.8 one by one; 4093 x 3584,
        // with two vectors, 19.5 and 19.9).
        constexpr bool PAIRS = !(TPR == 512 && VPT == 4);
        uint2 b;
        uint16_t* p = reinterpret_cast<uint16_t*>(&b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 n = make_float2(f[2 * j], f[2 * j + 1]);
          p[j] = __nv_cvt_float2_to_fp8x2(
              PAIRS ? quotient(n, inv, back) : make_float2(quotient(n.x, inv, back), quotient(n.y, inv, back)),
              __NV_SATFINITE, __NV_E4M3);
        }
        *(reinterpret_cast<uint2*>(q + t * d) + v) = b;
        if ((v & 15) == 0) q_scale[t * ((d + kQGroup - 1) / kQGroup) + (v >> 4)] = s;
      }
    }
  }
}

// Backward.  A persistent block walks units of RPB rows (BLOCK / TPR), dealt
// round-robin; a ring of `stages` units of dy, h and dh is filled ahead by bulk
// copies (one per row and tensor), so that the loads in flight do not depend
// on registers or on the barrier each row's sum needs.  Between a row's sum and
// its use it stays packed in registers, 8 values in 4 (16381 x 4096, the kernel
// alone: 106 us with loads straight into registers, 100 with the ring, 82, 6.5
// TB/s, with the packed row).  Every thread keeps its columns of the weight and
// adds its columns of dw over its rows; a block's row groups meet in shared
// memory, and the block writes one fp32 row of partial[gridDim.x][d].
template <int TPR, int VPT, bool WF32>
__global__ void __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads, TPR > 256 ? 1 : TPR > kNormThreads ? 2 : 4)
    add_rms_norm_backward_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* h, const void* __restrict__ weight,
                                 const float* __restrict__ rstd, const uint16_t* dh, int64_t lddh, int T, int d,
                                 int stages, uint16_t* dx, float* __restrict__ partial, int32_t* err) {
  using namespace dmoe::tc;
  constexpr int BLOCK = TPR > kNormThreads ? TPR : kNormThreads;
  constexpr int RPB = BLOCK / TPR;
  __shared__ float red[2][BLOCK / 32];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int gave_up;
  extern __shared__ __align__(16) uint8_t ring[];  // [stages][dy, h, dh][RPB][d], then reused for dw
  const int c = threadIdx.x % TPR;
  const int rg = threadIdx.x / TPR;
  const int nvec = d >> 3;
  const uint32_t row_bytes = static_cast<uint32_t>(d) * 2;
  const uint32_t part_bytes = RPB * row_bytes;
  const int64_t units = (static_cast<int64_t>(T) + RPB - 1) / RPB;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(full + s, 1);
    gave_up = 0;
    fence_mbar_init();
  }
  __syncthreads();
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  // the weight's columns stay in registers, except where four vectors a thread
  // leave too few (they come from L1 then)
  constexpr bool KEEP = VPT == 2;
  float kept[KEEP ? VPT : 1][8], dw[VPT][8] = {};
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
#pragma unroll
      for (int j = 0; j < 8; ++j) kept[i][j] = 0.f;
      if (v < nvec) load_w<WF32>(weight, v, kept[i]);
    }
  }
  auto weights = [&](int i, float* w) {
    if (KEEP) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = kept[i][j];
    } else if (c + i * TPR < nvec) {
      load_w<WF32>(weight, c + i * TPR, w);
    }
  };
  // thread 0: the rows of unit u into stage s
  auto fill = [&](int64_t u, int s) {
    if (u >= units) return;
    const int64_t t0 = u * RPB;
    const int rows = static_cast<int>(min(static_cast<int64_t>(RPB), T - t0));
    uint8_t* at = ring + s * 3 * part_bytes;
    mbar_arrive_expect_tx(full + s, rows * row_bytes * (dh ? 3 : 2));
    for (int r = 0; r < rows; ++r) {
      bulk_load(at + r * row_bytes, dy + (t0 + r) * lddy, row_bytes, full + s);
      bulk_load(at + part_bytes + r * row_bytes, h + (t0 + r) * d, row_bytes, full + s);
      if (dh) bulk_load(at + 2 * part_bytes + r * row_bytes, dh + (t0 + r) * lddh, row_bytes, full + s);
    }
  };
  int64_t u = blockIdx.x;
  if (threadIdx.x == 0)
    for (int s = 0; s < stages; ++s) fill(u + static_cast<int64_t>(s) * gridDim.x, s);
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  for (; u < units; u += gridDim.x) {
    const int64_t t = u * RPB + rg;
    const bool live = t < T;
    const float r = live ? __ldg(rstd + t) : 0.f;
    if (!mbar_wait(full + stage, phase, &gave_up)) gave_up = 1;
    const uint8_t* at = ring + stage * 3 * part_bytes + rg * row_bytes;
    float s = 0.f;
    uint4 a[VPT], b[VPT];  // kept packed for the second use
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (live && v < nvec) {
        a[i] = *(reinterpret_cast<const uint4*>(at) + v);
        b[i] = *(reinterpret_cast<const uint4*>(at + part_bytes) + v);
      }
      float f[8], g[8], w[8] = {};
      unpack8(a[i], f);
      unpack8(b[i], g);
      weights(i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s = fmaf(f[j] * w[j], g[j], s);
        dw[i][j] = fmaf(f[j] * r, g[j], dw[i][j]);
      }
    }
    s = row_sum<TPR>(s, red[flip]);
    if (TPR == 32) __syncthreads();
    if (gave_up) break;
    // past this barrier every thread is done with the unit before this one
    if (stages > 1 && threadIdx.x == 0 && u != static_cast<int64_t>(blockIdx.x))
      fill(u + static_cast<int64_t>(stages - 1) * gridDim.x, stage == 0 ? stages - 1 : stage - 1);
    flip ^= 1;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    const float m = s / static_cast<float>(d) * r * r;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (!live || v >= nvec) continue;
      // unpacked anew (the compiler would carry 16 floats over the barrier instead)
      asm volatile("" : "+r"(a[i].x), "+r"(a[i].y), "+r"(a[i].z), "+r"(a[i].w));
      asm volatile("" : "+r"(b[i].x), "+r"(b[i].y), "+r"(b[i].z), "+r"(b[i].w));
      float f[8], g[8], w[8] = {}, o[8] = {};
      unpack8(a[i], f);
      unpack8(b[i], g);
      weights(i, w);
      if (dh) unpack8(*(reinterpret_cast<const uint4*>(at + 2 * part_bytes) + v), o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmaf(r, fmaf(f[j], w[j], -g[j] * m), o[j]);
      *(reinterpret_cast<uint4*>(dx + t * d) + v) = pack8(o);
    }
    if (stages == 1) {
      __syncthreads();
      if (threadIdx.x == 0) fill(u + gridDim.x, 0);
    }
  }
  __syncthreads();
  if (gave_up) {  // a copy that did not arrive: nothing more is written
    if (threadIdx.x == 0) {
      dmoe::raise_error(err, DMOE_SITE_NORM_WAIT | DMOE_ERR_TIMEOUT);
      volatile int go_on = 0;
      for (int i = 0; i < stages; ++i) {  // the copies still on their way, as far as they come
        mbar_wait(full + stage, phase, &go_on);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    return;
  }
  if (!partial) return;
  if (RPB > 1) {
    float* sh = reinterpret_cast<float*>(ring);  // [RPB - 1][d]: every unit has been read
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (rg > 0 && v < nvec) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sh[static_cast<int64_t>(rg - 1) * d + 8 * v + j] = dw[i][j];
      }
    }
    __syncthreads();
    if (rg == 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = c + i * TPR;
        if (v >= nvec) continue;
        for (int g = 1; g < RPB; ++g) {
#pragma unroll
          for (int j = 0; j < 8; ++j) dw[i][j] += sh[static_cast<int64_t>(g - 1) * d + 8 * v + j];
        }
      }
    }
  }
  if (rg == 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (v >= nvec) continue;
      float4* o = reinterpret_cast<float4*>(partial + static_cast<int64_t>(blockIdx.x) * d) + 2 * v;
      o[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      o[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// dw[c] = sum over the n partial rows, in a fixed order: 32 columns x 32 row
// slices per block.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ partial, int n, int d,
                                                          float* __restrict__ dw) {
  __shared__ float sh[32][33];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int i = slice; i < n; i += 32) s += __ldg(partial + static_cast<int64_t>(i) * d + c);
  }
  sh[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sh[i][lane];
    dw[c] = s;
  }
}

// Threads per row: the smallest power of two from 32 on that holds the row
// at two vectors a thread; over 8192 columns at four.
int threads_per_row(int d) {
  const int nvec = d >> 3;
  if (nvec > 2048) return 1024;
  int tpr = 32;
  while (tpr < 512 && 2 * tpr < nvec) tpr *= 2;
  return tpr;
}

int rows_per_block(int d) { return std::max(1, kNormThreads / threads_per_row(d)); }

// Bytes of one unit of the backward's ring, blocks per SM, and units per block:
// as many as fit, for wide rows two in what a block can have, or one.
size_t unit_bytes(int d) { return static_cast<size_t>(rows_per_block(d)) * d * 2 * 3; }
int blocks_per_sm(int d) {
  const int tpr = threads_per_row(d);
  return tpr <= kNormThreads ? 4 : tpr <= 256 ? 2 : 1;  // what their registers allow
}
int ring_stages(int d) {
  return static_cast<int>(std::clamp<size_t>(kRingBytes / blocks_per_sm(d) / unit_bytes(d), 1, kMaxStages));
}

// Blocks of the backward: what is resident, each leaving one partial row of dw.
int backward_blocks(int T, int d, int sms) {
  const int rpb = rows_per_block(d);
  const int64_t need = (static_cast<int64_t>(T) + rpb - 1) / rpb;
  return static_cast<int>(std::min<int64_t>(need, static_cast<int64_t>(sms) * blocks_per_sm(d)));
}

// Calls f.template operator()<TPR, VPT>() for rows of d columns.
template <typename F>
cudaError_t by_width(int d, F&& f) {
  switch (threads_per_row(d)) {
    case 32: return f.template operator()<32, 2>();
    case 64: return f.template operator()<64, 2>();
    case 128: return f.template operator()<128, 2>();
    case 256: return f.template operator()<256, 2>();
    case 512: return (d >> 3) <= 1024 ? f.template operator()<512, 2>() : f.template operator()<512, 4>();
    default: return f.template operator()<1024, 4>();
  }
}

struct Forward {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* residual;
  int64_t ldr;
  const void* weight;
  int wf32;
  float eps;
  int T, d;
  uint16_t *h, *y;
  float* rstd;
  uint8_t* q;
  float* q_scale;
  cudaStream_t st;

  template <int TPR, int VPT>
  cudaError_t operator()() const {
    constexpr int block = TPR > kFwdThreads ? TPR : kFwdThreads;
    const int rpb = block / TPR;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) + rpb - 1) / rpb));
    auto kern = wf32 ? (q ? add_rms_norm_kernel<TPR, VPT, true, true> : add_rms_norm_kernel<TPR, VPT, true, false>)
                     : (q ? add_rms_norm_kernel<TPR, VPT, false, true> : add_rms_norm_kernel<TPR, VPT, false, false>);
    return dmoe::launch_pdl(kern, grid, dim3(block), 0, st, x, ldx, residual, ldr, weight, eps, T, d, h, y, rstd, q,
                            q_scale);
  }
};

struct Backward {
  const uint16_t* dy;
  int64_t lddy;
  const uint16_t* h;
  const void* weight;
  int wf32;
  const float* rstd;
  const uint16_t* dh;
  int64_t lddh;
  int T, d;
  uint16_t* dx;
  float* partial;
  int blocks;
  int device;
  int32_t* err;
  cudaStream_t st;

  template <int TPR, int VPT, bool WF32>
  cudaError_t launch() const {
    constexpr int block = TPR > kNormThreads ? TPR : kNormThreads;
    auto kern = add_rms_norm_backward_kernel<TPR, VPT, WF32>;
    // the ring also holds the row groups' dw: (RPB - 1) fp32 rows in 3 RPB bf16 ones
    const size_t smem = ring_stages(d) * unit_bytes(d);
    static std::atomic<uint64_t> opted{0};
    const uint64_t bit = uint64_t(1) << device;
    if (!(opted.load(std::memory_order_acquire) & bit)) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kRingBytes));
      if (e != cudaSuccess) return e;
      opted.fetch_or(bit, std::memory_order_acq_rel);
    }
    return dmoe::launch_pdl(kern, dim3(blocks), dim3(block), smem, st, dy, lddy, h, weight, rstd, dh, lddh, T, d,
                            ring_stages(d), dx, partial, err);
  }

  template <int TPR, int VPT>
  cudaError_t operator()() const {
    return wf32 ? launch<TPR, VPT, true>() : launch<TPR, VPT, false>();
  }
};

}  // namespace

DMOE_API dmoe_status dmoe_add_rms_norm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
                                       const void* weight, int weight_f32, float eps, int T, int d, uint16_t* h,
                                       uint16_t* y, float* rstd, uint8_t* q, float* q_scale, dmoe_stream_t stream) {
  if (T < 0 || d < 8 || (d & 7) || d > kMaxD || !(eps >= 0.f)) return DMOE_ERR_INVALID_ARG;
  if (T == 0) return DMOE_OK;
  if (!x || !weight || (!y && !q) || (q && !q_scale) || (residual && !h)) return DMOE_ERR_INVALID_ARG;
  if (bad_ld(ldx, d) || (residual && bad_ld(ldr, d))) return DMOE_ERR_INVALID_ARG;
  if (bad_ptr(x) || bad_ptr(residual) || bad_ptr(weight) || bad_ptr(h) || bad_ptr(y) ||
      (reinterpret_cast<uintptr_t>(q) & 7) ||
      ((reinterpret_cast<uintptr_t>(rstd) | reinterpret_cast<uintptr_t>(q_scale)) & 3))
    return DMOE_ERR_INVALID_ARG;
  if (bad_alias(h, x, ldx, T, d) || bad_alias(y, x, ldx, T, d) || bad_alias(h, residual, ldr, T, d) ||
      bad_alias(y, residual, ldr, T, d))
    return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  const Forward f{x, ldx, residual, ldr, weight, weight_f32, eps, T, d, h, y, rstd, q, q_scale, dmoe::as_stream(stream)};
  cudaError_t e = by_width(d, f);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

DMOE_API size_t dmoe_add_rms_norm_backward_workspace_size(int T, int d) {
  dmoe::DeviceInfo di;
  if (T < 0 || d < 8 || (d & 7) || d > kMaxD || dmoe::device_info(&di) != DMOE_OK) return 0;
  return static_cast<size_t>(backward_blocks(T, d, di.sm_count)) * d * sizeof(float);
}

DMOE_API dmoe_status dmoe_add_rms_norm_backward(const uint16_t* dy, int64_t lddy, const uint16_t* h,
                                                const void* weight, int weight_f32, const float* rstd,
                                                const uint16_t* dh, int64_t lddh, int T, int d, uint16_t* dx,
                                                float* dw, void* ws, size_t ws_bytes, dmoe_stream_t stream) {
  if (T < 0 || d < 8 || (d & 7) || d > kMaxD) return DMOE_ERR_INVALID_ARG;
  if (T > 0 && (!dy || !h || !weight || !rstd || !dx)) return DMOE_ERR_INVALID_ARG;
  if (T > 0 && (bad_ld(lddy, d) || (dh && bad_ld(lddh, d)))) return DMOE_ERR_INVALID_ARG;
  if (bad_ptr(dy) || bad_ptr(h) || bad_ptr(weight) || bad_ptr(dh) || bad_ptr(dx) || bad_ptr(ws) ||
      ((reinterpret_cast<uintptr_t>(rstd) | reinterpret_cast<uintptr_t>(dw)) & 3))
    return DMOE_ERR_INVALID_ARG;
  if (bad_alias(dx, dy, lddy, T, d) || bad_alias(dx, dh, lddh, T, d)) return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  cudaStream_t st = dmoe::as_stream(stream);
  if (T == 0) {  // no rows: their sum over nothing is zero
    return dw ? dmoe::cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(d) * sizeof(float), st)) : DMOE_OK;
  }
  const int blocks = backward_blocks(T, d, di.sm_count);
  if (dw && (!ws || ws_bytes < static_cast<size_t>(blocks) * d * sizeof(float))) return DMOE_ERR_INVALID_ARG;
  const Backward b{dy, lddy, h, weight, weight_f32, rstd, dh, lddh, T, d, dx, dw ? static_cast<float*>(ws) : nullptr,
                   blocks, di.device, di.err_word, st};
  cudaError_t e = by_width(d, b);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  if (dw) {
    e = dmoe::launch_pdl(column_sum_kernel, dim3((d + 31) / 32), dim3(1024), 0, st,
                         static_cast<const float*>(ws), blocks, d, dw);
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    dmoe::count_launches(1);
  }
  return DMOE_OK;
}
