// The norm after a block, its gate, the scaled residual stream and the norm
// before the next block in one pass, and the backward.
//
//   n = u ru a,  ru = 1 / sqrt(mean u^2 + eps)      (a: weight after the block)
//   h = bf16(scale x + gate n)
//   y = h rh b,  rh = 1 / sqrt(mean h^2 + eps)      (b: weight before the next)
// The stream is kept in bf16 and its norm reads the kept value, which is all
// the backward has.  The gate is one number a row, or one for all.
//
//   backward, with g = dy b:
//     dH = dh + rh (g - h rh^2 mean(g h)),  dx = scale dH
//     du = gate ru (a dH - u ru^2 mean(a dH u))
//     d_gate = ru sum_c a dH u,  da = sum_t gate ru dH u,  db = sum_t rh dy h
// The second mean needs dH, which needs the first; but dH is linear in it:
//     sum a u dH = sum a u (dh + rh g) - rh^3 mean(g h) sum a u h
// so one meeting of the row's threads gives all three sums.
//
// Both are HBM-bound (8 and 12 bytes an element, some 10 and 24 flops): a row
// is read once.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace {

using namespace dmoe::rows;

constexpr int kMaxD = 16384;
constexpr int kMinThreads = 128;           // of a block, while a row takes fewer
constexpr int kMaxStages = 4;              // backward: units of rows in flight per block
constexpr size_t kRingBytes = 200 * 1024;  // of shared memory for them per SM
constexpr int kBackThreads = 512;          // backward: threads per SM, 128 registers each

template <int TPR, int VPT, bool WF32>
__global__ void __launch_bounds__(TPR > kMinThreads ? TPR : kMinThreads, 1024 / (TPR > kMinThreads ? TPR : kMinThreads))
    sandwich_norm_kernel(const uint16_t* u, int64_t ldu, const uint16_t* x, int64_t ldx,
                         const void* __restrict__ w_post, const void* __restrict__ w_pre,
                         const float* __restrict__ gate, int gate_step, float scale, float eps, int T, int d,
                         uint16_t* h, uint16_t* y, float* __restrict__ rstd_u, float* __restrict__ rstd_h) {
  constexpr int BLOCK = TPR > kMinThreads ? TPR : kMinThreads;
  constexpr int RPB = BLOCK / TPR;
  __shared__ float red[2][BLOCK / 32];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int c = threadIdx.x % TPR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool live = t < T;
  const int nvec = d >> 3;
  uint4 a[VPT], b[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = c + i * TPR;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (live && v < nvec) {
      a[i] = *(reinterpret_cast<const uint4*>(u + t * ldu) + v);
      b[i] = *(reinterpret_cast<const uint4*>(x + t * ldx) + v);
    }
  }
  const float gt = gate && live ? __ldg(gate + t * gate_step) : 1.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float f[8];
    unpack8(a[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(f[j], f[j], s);
  }
  s = row_sum<TPR>(s, red[0]);
  const float ru = rsqrtf(s / static_cast<float>(d) + eps);
  const float k = ru * gt;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = c + i * TPR;
    float f[8], g[8], w[8] = {};
    unpack8(a[i], f);
    unpack8(b[i], g);
    if (v < nvec) load_w<WF32>(w_post, v, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = fmaf(scale, g[j], f[j] * k * w[j]);
    b[i] = pack8(f);  // the kept stream: bf16, what the backward will read
    if (live && v < nvec) *(reinterpret_cast<uint4*>(h + t * d) + v) = b[i];
    else b[i] = make_uint4(0, 0, 0, 0);
    unpack8(b[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(f[j], f[j], s);
  }
  s = row_sum<TPR>(s, red[1]);
  const float rh = rsqrtf(s / static_cast<float>(d) + eps);
  if (live && c == 0) {
    if (rstd_u) rstd_u[t] = ru;
    if (rstd_h) rstd_h[t] = rh;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = c + i * TPR;
    if (!live || v >= nvec) continue;
    float f[8], w[8];
    unpack8(b[i], f);
    load_w<WF32>(w_pre, v, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * rh * w[j];
    *(reinterpret_cast<uint4*>(y + t * d) + v) = pack8(f);
  }
}

struct Back {
  const uint16_t *dy, *u, *h, *dh;
  int64_t lddy, ldu, lddh;
  const void *w_post, *w_pre;
  const float *rstd_u, *rstd_h, *gate;
  int gate_step;
  float scale;
  int T, d, stages;
  uint16_t *du, *dx;
  float* d_gate;   // [T] (NULL: none)
  float* partial;  // [gridDim.x][2 d] of dw_post and dw_pre (NULL: neither)
  int32_t* err;
};

// A persistent block walks units of RPB rows, dealt round-robin; a ring of
// `stages` units of dy, u, h and dh is filled ahead by bulk copies, one per
// row and tensor.  Every thread keeps its columns' sums of both weights'
// gradients over its rows; a block's row groups meet in shared memory, and the
// block writes one fp32 row of `partial`.
template <int TPR, int VPT, bool WF32>
__global__ void __launch_bounds__(TPR > kMinThreads ? TPR : kMinThreads, kBackThreads / (TPR > kMinThreads ? TPR : kMinThreads))
    sandwich_norm_backward_kernel(const Back p) {
  using namespace dmoe::tc;
  constexpr int BLOCK = TPR > kMinThreads ? TPR : kMinThreads;
  constexpr int RPB = BLOCK / TPR;
  constexpr int WPR = TPR / 32;
  constexpr bool KEEP = VPT == 1;  // the row between its sums and their use, and the weights, in registers
  __shared__ float4 red[2][BLOCK / 32];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int gave_up;
  extern __shared__ __align__(16) uint8_t ring[];  // [stages][dy, u, h, dh][RPB][d], then reused for the weights' sums
  const int c = threadIdx.x % TPR;
  const int rg = threadIdx.x / TPR;
  const int d = p.d, nvec = d >> 3;
  const uint32_t row_bytes = static_cast<uint32_t>(d) * 2;
  const uint32_t part_bytes = RPB * row_bytes;
  const int64_t units = (static_cast<int64_t>(p.T) + RPB - 1) / RPB;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(full + s, 1);
    gave_up = 0;
    fence_mbar_init();
  }
  __syncthreads();
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  float wa[KEEP ? 8 : 1], wb[KEEP ? 8 : 1];
  float da[VPT][8] = {}, db[VPT][8] = {};
  if (KEEP) {
#pragma unroll
    for (int j = 0; j < 8; ++j) wa[j] = wb[j] = 0.f;
    if (c < nvec) {
      load_w<WF32>(p.w_post, c, wa);
      load_w<WF32>(p.w_pre, c, wb);
    }
  }
  auto weights = [&](int v, float* a, float* b) {
    if (KEEP) {
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = wa[j], b[j] = wb[j];
    } else {
      load_w<WF32>(p.w_post, v, a);
      load_w<WF32>(p.w_pre, v, b);
    }
  };
  // thread 0: the rows of unit n into stage s
  auto fill = [&](int64_t n, int s) {
    if (n >= units) return;
    const int64_t t0 = n * RPB;
    const int rows = static_cast<int>(min(static_cast<int64_t>(RPB), p.T - t0));
    uint8_t* at = ring + s * 4 * part_bytes;
    mbar_arrive_expect_tx(full + s, rows * row_bytes * (p.dh ? 4 : 3));
    for (int r = 0; r < rows; ++r) {
      bulk_load(at + r * row_bytes, p.dy + (t0 + r) * p.lddy, row_bytes, full + s);
      bulk_load(at + part_bytes + r * row_bytes, p.u + (t0 + r) * p.ldu, row_bytes, full + s);
      bulk_load(at + 2 * part_bytes + r * row_bytes, p.h + (t0 + r) * d, row_bytes, full + s);
      if (p.dh) bulk_load(at + 3 * part_bytes + r * row_bytes, p.dh + (t0 + r) * p.lddh, row_bytes, full + s);
    }
  };
  int64_t n = blockIdx.x;
  if (threadIdx.x == 0)
    for (int s = 0; s < p.stages; ++s) fill(n + static_cast<int64_t>(s) * gridDim.x, s);
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  const float per = 1.f / static_cast<float>(d);
  for (; n < units; n += gridDim.x) {
    const int64_t t = n * RPB + rg;
    const bool live = t < p.T;
    const float ru = live ? __ldg(p.rstd_u + t) : 0.f;
    const float rh = live ? __ldg(p.rstd_h + t) : 0.f;
    const float gt = live && p.gate ? __ldg(p.gate + t * p.gate_step) : 1.f;
    if (!mbar_wait(full + stage, phase, &gave_up)) gave_up = 1;
    const uint4* at = reinterpret_cast<const uint4*>(ring + stage * 4 * part_bytes + rg * row_bytes);
    const int next = RPB * nvec;  // from one tensor's rows to the next one's
    uint4 q[KEEP ? 4 : 1];        // the row's dy, u, h and dh, kept packed
    float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (KEEP) q[0] = q[KEEP ? 1 : 0] = q[KEEP ? 2 : 0] = q[KEEP ? 3 : 0] = make_uint4(0, 0, 0, 0);
      if (!live || v >= nvec) continue;
      const uint4 q0 = at[v], q1 = at[next + v], q2 = at[2 * next + v];
      const uint4 q3 = p.dh ? at[3 * next + v] : make_uint4(0, 0, 0, 0);
      if (KEEP) q[0] = q0, q[KEEP ? 1 : 0] = q1, q[KEEP ? 2 : 0] = q2, q[KEEP ? 3 : 0] = q3;
      float f[8], g[8], w[8], o[8], a[8], b[8];
      unpack8(q0, f);
      unpack8(q1, g);
      unpack8(q2, w);
      unpack8(q3, o);
      weights(v, a, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gy = f[j] * b[j], au = a[j] * g[j];
        s1 = fmaf(gy, w[j], s1);
        s2 = fmaf(au, fmaf(rh, gy, o[j]), s2);
        s3 = fmaf(au, w[j], s3);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      s3 += __shfl_xor_sync(0xffffffffu, s3, o);
    }
    if (WPR > 1) {
      if ((threadIdx.x & 31) == 0) red[flip][threadIdx.x >> 5] = make_float4(s1, s2, s3, 0.f);
      __syncthreads();
      s1 = s2 = s3 = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        const float4 r = red[flip][rg * WPR + i];
        s1 += r.x, s2 += r.y, s3 += r.z;
      }
    } else {
      __syncthreads();
    }
    if (gave_up) break;
    // past this barrier every thread is done with the unit before this one
    if (p.stages > 1 && threadIdx.x == 0 && n != static_cast<int64_t>(blockIdx.x))
      fill(n + static_cast<int64_t>(p.stages - 1) * gridDim.x, stage == 0 ? p.stages - 1 : stage - 1);
    const float m1 = s1 * per * rh * rh;                    // dH = dh + rh (g - h m1)
    const float along = ru * fmaf(-rh * m1, s3, s2);        // sum a dH u ru
    const float m2 = along * per * ru;                      // du = gate ru (a dH - u m2)
    if (live && c == 0 && p.d_gate) p.d_gate[t] = along;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (!live || v >= nvec) continue;
      float f[8], g[8], w[8], o[8], a[8], b[8];
      if (KEEP) {
        // unpacked anew (the compiler would carry 32 floats over the barrier instead)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          asm volatile("" : "+r"(q[KEEP ? k : 0].x), "+r"(q[KEEP ? k : 0].y), "+r"(q[KEEP ? k : 0].z),
                       "+r"(q[KEEP ? k : 0].w));
        unpack8(q[0], f);
        unpack8(q[KEEP ? 1 : 0], g);
        unpack8(q[KEEP ? 2 : 0], w);
        unpack8(q[KEEP ? 3 : 0], o);
      } else {
        unpack8(at[v], f);
        unpack8(at[next + v], g);
        unpack8(at[2 * next + v], w);
        unpack8(p.dh ? at[3 * next + v] : make_uint4(0, 0, 0, 0), o);
      }
      weights(v, a, b);
      const float gr = gt * ru;
      float du[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dH = fmaf(rh, fmaf(f[j], b[j], -w[j] * m1), o[j]);
        db[i][j] = fmaf(f[j] * rh, w[j], db[i][j]);
        da[i][j] = fmaf(dH * gr, g[j], da[i][j]);
        du[j] = gr * fmaf(a[j], dH, -g[j] * m2);
        o[j] = p.scale * dH;
      }
      *(reinterpret_cast<uint4*>(p.du + t * d) + v) = pack8(du);
      *(reinterpret_cast<uint4*>(p.dx + t * d) + v) = pack8(o);
    }
    if (p.stages == 1) {
      __syncthreads();
      if (threadIdx.x == 0) fill(n + gridDim.x, 0);
    }
    flip ^= 1;
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  __syncthreads();
  if (gave_up) {  // a copy that did not arrive: nothing more is written
    if (threadIdx.x == 0) {
      dmoe::raise_error(p.err, DMOE_SITE_NORM_WAIT | DMOE_ERR_TIMEOUT);
      volatile int go_on = 0;
      for (int i = 0; i < p.stages; ++i) {  // the copies still on their way, as far as they come
        mbar_wait(full + stage, phase, &go_on);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    return;
  }
  if (!p.partial) return;
  if (RPB > 1) {
    float* sh = reinterpret_cast<float*>(ring);  // [RPB - 1][2 d]: every unit has been read
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (rg > 0 && v < nvec) {
        float* o = sh + static_cast<int64_t>(rg - 1) * 2 * d + 8 * v;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = da[i][j], o[d + j] = db[i][j];
      }
    }
    __syncthreads();
    if (rg == 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = c + i * TPR;
        if (v >= nvec) continue;
        for (int g = 1; g < RPB; ++g) {
          const float* o = sh + static_cast<int64_t>(g - 1) * 2 * d + 8 * v;
#pragma unroll
          for (int j = 0; j < 8; ++j) da[i][j] += o[j], db[i][j] += o[d + j];
        }
      }
    }
  }
  if (rg == 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (v >= nvec) continue;
      float* o = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * d + 8 * v;
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        *reinterpret_cast<float4*>(o + j) = make_float4(da[i][j], da[i][j + 1], da[i][j + 2], da[i][j + 3]);
        *reinterpret_cast<float4*>(o + d + j) = make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
      }
    }
  }
}

// What the rows left, summed in a fixed order: both weights' gradients over
// the n partial rows (32 columns x 32 slices of rows per block), and in the
// last block the gradient of a gate that all rows share.
__global__ void __launch_bounds__(1024) sandwich_sums_kernel(const float* __restrict__ partial, int n, int d,
                                                             float* __restrict__ dw_post, float* __restrict__ dw_pre,
                                                             const float* __restrict__ row_gate, int T,
                                                             float* __restrict__ d_gate, int col_blocks) {
  __shared__ float sh[32][33];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int slice = threadIdx.x >> 5;
  float s = 0.f;
  if (static_cast<int>(blockIdx.x) == col_blocks) {
#pragma unroll 8
    for (int t = threadIdx.x; t < T; t += 1024) s += __ldg(row_gate + t);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sh[0][slice] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) s += sh[0][i];
      d_gate[0] = s;
    }
    return;
  }
  const int c = blockIdx.x * 32 + lane;
  if (c < 2 * d) {
#pragma unroll 8
    for (int i = slice; i < n; i += 32) s += __ldg(partial + static_cast<int64_t>(i) * 2 * d + c);
  }
  sh[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < 2 * d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sh[i][lane];
    float* o = c < d ? dw_post : dw_pre;
    if (o) o[c < d ? c : c - d] = s;
  }
}

// Threads per row, forward: the smallest power of two that holds it at two
// vectors a thread (four above 8192 columns); backward: at one vector, which
// leaves room for both weights' sums (two and four above 4096 and 8192).
int threads_per_row(int d, int vectors) {
  int tpr = 32;
  while (tpr < 512 && vectors * tpr < (d >> 3)) tpr *= 2;
  return tpr;
}

template <typename F>
cudaError_t by_width(int d, const F& f) {
  const int nvec = d >> 3;
  switch (threads_per_row(d, F::kVectors)) {
    case 32: return f.template operator()<32, F::kVectors>();
    case 64: return f.template operator()<64, F::kVectors>();
    case 128: return f.template operator()<128, F::kVectors>();
    case 256: return f.template operator()<256, F::kVectors>();
    default:
      if (nvec <= 512 * F::kVectors) return f.template operator()<512, F::kVectors>();
      if (nvec <= 1024) return f.template operator()<512, 2>();
      return f.template operator()<512, 4>();
  }
}

int back_block(int d) { return std::max(kMinThreads, threads_per_row(d, 1)); }
int back_rows(int d) { return back_block(d) / threads_per_row(d, 1); }
size_t unit_bytes(int d) { return static_cast<size_t>(back_rows(d)) * d * 2 * 4; }
int blocks_per_sm(int d) { return kBackThreads / back_block(d); }
int ring_stages(int d) {
  return static_cast<int>(std::clamp<size_t>(kRingBytes / blocks_per_sm(d) / unit_bytes(d), 1, kMaxStages));
}

// Blocks of the backward: what is resident, each leaving one partial row.
int backward_blocks(int T, int d, int sms) {
  const int rpb = back_rows(d);
  const int64_t need = (static_cast<int64_t>(T) + rpb - 1) / rpb;
  return static_cast<int>(std::min<int64_t>(need, static_cast<int64_t>(sms) * blocks_per_sm(d)));
}

struct Forward {
  static constexpr int kVectors = 2;
  const uint16_t* u;
  int64_t ldu;
  const uint16_t* x;
  int64_t ldx;
  const void *w_post, *w_pre;
  int wf32;
  const float* gate;
  int gate_step;
  float scale, eps;
  int T, d;
  uint16_t *h, *y;
  float *rstd_u, *rstd_h;
  cudaStream_t st;

  template <int TPR, int VPT>
  cudaError_t operator()() const {
    constexpr int block = TPR > kMinThreads ? TPR : kMinThreads;
    const int rpb = block / TPR;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) + rpb - 1) / rpb));
    auto kern = wf32 ? sandwich_norm_kernel<TPR, VPT, true> : sandwich_norm_kernel<TPR, VPT, false>;
    return dmoe::launch_pdl(kern, grid, dim3(block), 0, st, u, ldu, x, ldx, w_post, w_pre, gate, gate_step, scale, eps,
                            T, d, h, y, rstd_u, rstd_h);
  }
};

struct Backward {
  static constexpr int kVectors = 1;
  Back p;
  int wf32;
  int blocks;
  int device;
  cudaStream_t st;

  template <int TPR, int VPT, bool WF32>
  cudaError_t launch() const {
    constexpr int block = TPR > kMinThreads ? TPR : kMinThreads;
    auto kern = sandwich_norm_backward_kernel<TPR, VPT, WF32>;
    // the ring also holds the row groups' sums: (RPB - 1) x 2 fp32 rows in 4 RPB bf16 ones
    static std::atomic<uint64_t> opted{0};
    const uint64_t bit = uint64_t(1) << device;
    if (!(opted.load(std::memory_order_acquire) & bit)) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kRingBytes));
      if (e != cudaSuccess) return e;
      opted.fetch_or(bit, std::memory_order_acq_rel);
    }
    return dmoe::launch_pdl(kern, dim3(blocks), dim3(block), p.stages * unit_bytes(p.d), st, p);
  }

  template <int TPR, int VPT>
  cudaError_t operator()() const {
    return wf32 ? launch<TPR, VPT, true>() : launch<TPR, VPT, false>();
  }
};

bool misaligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) & 3u; }

}  // namespace

DMOE_API dmoe_status dmoe_sandwich_norm(const uint16_t* u, int64_t ldu, const uint16_t* residual, int64_t ldr,
                                        const void* w_post, const void* w_pre, int weight_f32, const float* gate,
                                        int gate_rows, float scale, float eps, int T, int d, uint16_t* h, uint16_t* y,
                                        float* rstd_u, float* rstd_h, dmoe_stream_t stream) {
  if (T < 0 || d < 8 || (d & 7) || d > kMaxD || !(eps >= 0.f)) return DMOE_ERR_INVALID_ARG;
  if (T == 0) return DMOE_OK;
  if (!u || !residual || !w_post || !w_pre || !h || !y || h == y) return DMOE_ERR_INVALID_ARG;
  if (gate && gate_rows != 1 && gate_rows != T) return DMOE_ERR_INVALID_ARG;
  if (bad_ld(ldu, d) || bad_ld(ldr, d)) return DMOE_ERR_INVALID_ARG;
  if (bad_ptr(u) || bad_ptr(residual) || bad_ptr(w_post) || bad_ptr(w_pre) || bad_ptr(h) || bad_ptr(y) ||
      misaligned4(gate) || misaligned4(rstd_u) || misaligned4(rstd_h))
    return DMOE_ERR_INVALID_ARG;
  if (bad_alias(h, u, ldu, T, d) || bad_alias(y, u, ldu, T, d) || bad_alias(h, residual, ldr, T, d) ||
      bad_alias(y, residual, ldr, T, d))
    return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  const Forward f{u, ldu, residual, ldr, w_post, w_pre, weight_f32, gate, gate_rows == 1 ? 0 : 1, scale, eps, T, d,
                  h, y, rstd_u, rstd_h, dmoe::as_stream(stream)};
  const cudaError_t e = by_width(d, f);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

DMOE_API size_t dmoe_sandwich_norm_backward_workspace_size(int T, int d) {
  dmoe::DeviceInfo di;
  if (T < 0 || d < 8 || (d & 7) || d > kMaxD || dmoe::device_info(&di) != DMOE_OK) return 0;
  return (static_cast<size_t>(backward_blocks(T, d, di.sm_count)) * 2 * d + T) * sizeof(float);
}

DMOE_API dmoe_status dmoe_sandwich_norm_backward(const uint16_t* dy, int64_t lddy, const uint16_t* u, int64_t ldu,
                                                 const uint16_t* h, const void* w_post, const void* w_pre,
                                                 int weight_f32, const float* gate, int gate_rows, float scale,
                                                 const float* rstd_u, const float* rstd_h, const uint16_t* dh,
                                                 int64_t lddh, int T, int d, uint16_t* du, uint16_t* dx, float* dw_post,
                                                 float* dw_pre, float* d_gate, void* ws, size_t ws_bytes,
                                                 dmoe_stream_t stream) {
  if (T < 0 || d < 8 || (d & 7) || d > kMaxD) return DMOE_ERR_INVALID_ARG;
  if (gate && gate_rows != 1 && gate_rows != T) return DMOE_ERR_INVALID_ARG;
  if (d_gate && !gate) return DMOE_ERR_INVALID_ARG;
  if (T > 0) {
    if (!dy || !u || !h || !w_post || !w_pre || !rstd_u || !rstd_h || !du || !dx || du == dx) return DMOE_ERR_INVALID_ARG;
    if (bad_ld(lddy, d) || bad_ld(ldu, d) || (dh && bad_ld(lddh, d))) return DMOE_ERR_INVALID_ARG;
  }
  if (bad_ptr(dy) || bad_ptr(u) || bad_ptr(h) || bad_ptr(dh) || bad_ptr(w_post) || bad_ptr(w_pre) || bad_ptr(du) ||
      bad_ptr(dx) || bad_ptr(ws) || misaligned4(rstd_u) || misaligned4(rstd_h) || misaligned4(gate) ||
      misaligned4(dw_post) || misaligned4(dw_pre) || misaligned4(d_gate))
    return DMOE_ERR_INVALID_ARG;
  if (bad_alias(du, dy, lddy, T, d) || bad_alias(dx, dy, lddy, T, d) || bad_alias(du, u, ldu, T, d) ||
      bad_alias(dx, u, ldu, T, d) || bad_alias(du, dh, lddh, T, d) || bad_alias(dx, dh, lddh, T, d))
    return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  cudaStream_t st = dmoe::as_stream(stream);
  const bool shared = d_gate && gate_rows == 1;  // one gate for all rows: its gradient is their sum
  if (T == 0) {  // no rows: the sums over them are zero
    cudaError_t e = cudaSuccess;
    if (dw_post) e = cudaMemsetAsync(dw_post, 0, static_cast<size_t>(d) * sizeof(float), st);
    if (e == cudaSuccess && dw_pre) e = cudaMemsetAsync(dw_pre, 0, static_cast<size_t>(d) * sizeof(float), st);
    if (e == cudaSuccess && shared) e = cudaMemsetAsync(d_gate, 0, sizeof(float), st);
    return dmoe::cuda_status(e);
  }
  const int blocks = backward_blocks(T, d, di.sm_count);
  const size_t part = static_cast<size_t>(blocks) * 2 * d;
  const bool sums = dw_post || dw_pre;
  if ((sums || shared) && (!ws || ws_bytes < (part + T) * sizeof(float))) return DMOE_ERR_INVALID_ARG;
  float* row_gate = static_cast<float*>(ws) + part;
  Back p{dy, u, h, dh, lddy, ldu, lddh, w_post, w_pre, rstd_u, rstd_h, gate, gate_rows == 1 ? 0 : 1, scale, T, d,
         ring_stages(d), du, dx, shared ? row_gate : d_gate, sums ? static_cast<float*>(ws) : nullptr, di.err_word};
  cudaError_t e = by_width(d, Backward{p, weight_f32, blocks, di.device, st});
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  if (sums || shared) {
    const int cols = sums ? (2 * d + 31) / 32 : 0;
    e = dmoe::launch_pdl(sandwich_sums_kernel, dim3(cols + (shared ? 1 : 0)), dim3(1024), 0, st,
                         static_cast<const float*>(ws), blocks, d, dw_post, dw_pre, static_cast<const float*>(row_gate), T,
                         d_gate, cols);
    if (e != cudaSuccess) return dmoe::cuda_status(e);
    dmoe::count_launches(1);
  }
  return DMOE_OK;
}
