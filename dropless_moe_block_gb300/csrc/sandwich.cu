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
constexpr int kMaxStages = 4;              // backward: rows in flight per group of threads
constexpr size_t kRingBytes = 200 * 1024;  // of shared memory for them per SM

// Forward: threads of a block, whole rows of TPR threads, and blocks an SM.
// Five blocks of 256 threads (48 registers): 8192 x 4096 42.2 us, 45.4 with
// four, 48.2 with six; 320 threads, 4093 x 5120, likewise (29.6 us, 31.5 with
// three).  Narrower rows are better off with registers (8192 x 512: 7.8 us with
// 1024 threads an SM, 8.7 with 1280; 192 threads, 8192 x 3000, 33.2 with 1152,
// 39.3 with 1344).
__host__ __device__ constexpr int forward_block(int tpr) { return tpr == 96 ? 192 : tpr > 128 ? tpr : 128; }
__host__ __device__ constexpr int forward_blocks(int tpr) {
  return (tpr == 256 || tpr == 320 ? 1280 : tpr % 96 == 0 ? 1152 : 1024) / forward_block(tpr);
}

template <int TPR, int VPT, bool WF32>
__global__ void __launch_bounds__(forward_block(TPR), forward_blocks(TPR))
    sandwich_norm_kernel(const uint16_t* u, int64_t ldu, const uint16_t* x, int64_t ldx,
                         const void* __restrict__ w_post, const void* __restrict__ w_pre,
                         const float* __restrict__ gate, int gate_step, float scale, float eps, int T, int d,
                         uint16_t* h, uint16_t* y, float* __restrict__ rstd_u, float* __restrict__ rstd_h) {
  constexpr int BLOCK = forward_block(TPR);
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
    for (int j = 0; j < 8; ++j) f[j] = fmaf(f[j] * w[j], k, scale * g[j]);  // two bf16 values' product is exact
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
    for (int j = 0; j < 8; ++j) f[j] = f[j] * w[j] * rh;
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

// Eight bf16 values as four pairs.
__device__ __forceinline__ void unpack4(const uint4& u, float2* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __bfloat1622float2(h[i]);
}

__device__ __forceinline__ uint4 pack4(const float2* f) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(f[i]);
  return u;
}

template <bool WF32>
__device__ __forceinline__ void load_w4(const void* w, int v, float2* f) {
  float a[8];
  load_w<WF32>(w, v, a);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(a[2 * i], a[2 * i + 1]);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The sums of s[0..2] over a warp: of s[q] in lanes 8 q .. 8 q + 7.  Lanes
// that part with half of the sums at a step send fewer numbers than three sums
// of their own would: 6 exchanges instead of 15.
__device__ __forceinline__ float three_sums(const float* s, int lane) {
  const bool high = lane & 16;
  // the upper half keeps s[2], the lower one s[0] and s[1]
  const float x = __shfl_xor_sync(0xffffffffu, high ? s[0] : s[2], 16);
  const float y = __shfl_xor_sync(0xffffffffu, high ? s[1] : 0.f, 16);
  const float k0 = (high ? s[2] : s[0]) + x, k1 = (high ? 0.f : s[1]) + y;
  const bool odd = lane & 8;
  float k = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
  return k;
}

// One block an SM, in groups of the TPR threads that share a row; the groups
// walk their rows without meeting one another.  Each fills a ring of `stages`
// rows ahead by bulk copies, one per tensor, and reads a row twice from there:
// before its sums and after.  Every thread keeps its columns of both weights (up
// to two vectors) and of both weights' gradients; the groups' meet in shared
// memory at the end, and the block writes one fp32 row of `partial`.
// Instructions come close to being the bound: pairs of values an instruction,
// and two vectors a thread, so that the sums' meeting costs a quarter of them
// (8192 x 4096: 99 us with one vector and value by value, 71 so; 8191 x 512,
// with blocks of four rows that wait for one another and leave 608 partial
// rows, 19 us, 17.7 with groups).
// Its threads, one block an SM: whole groups of a row's threads, 128 registers each.
__host__ __device__ constexpr int back_threads(int tpr) { return 512 / tpr * tpr; }

template <int TPR, int VPT, bool WF32>
__global__ void __launch_bounds__(back_threads(TPR), 1) sandwich_norm_backward_kernel(const __grid_constant__ Back p) {
  using namespace dmoe::tc;
  using dmoe::f2_fma;
  using dmoe::f2_mul;
  constexpr int THREADS = back_threads(TPR);
  constexpr int GROUPS = THREADS / TPR;
  constexpr int WPR = TPR / 32;
  constexpr bool KEEP = VPT <= 2;  // the weights in registers
  __shared__ float red[2][THREADS / 32 * 4];
  __shared__ uint64_t full[GROUPS][kMaxStages];
  __shared__ int gave_up[GROUPS];
  extern __shared__ __align__(16) uint8_t ring[];  // [GROUPS][stages][dy, u, h, dh][d], then the weights' sums
  const int c = threadIdx.x % TPR;
  const int rg = threadIdx.x / TPR;
  const int lane = threadIdx.x & 31;
  const int d = p.d, nvec = d >> 3;
  const uint32_t row_bytes = static_cast<uint32_t>(d) * 2;
  const uint32_t stage_bytes = 4 * row_bytes;
  uint8_t* mine = ring + static_cast<size_t>(rg) * p.stages * stage_bytes;
  auto meet = [&]() {  // of the group
    if (TPR == 32) __syncwarp();
    else if (GROUPS == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(rg + 1), "n"(TPR) : "memory");
  };
  if (c == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&full[rg][s], 1);
    gave_up[rg] = 0;
    fence_mbar_init();
  }
  __syncthreads();
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  float2 wa[KEEP ? VPT : 1][4], wb[KEEP ? VPT : 1][4];
  float2 da[VPT][4], db[VPT][4];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = c + i * TPR;
#pragma unroll
    for (int j = 0; j < 4; ++j) da[i][j] = db[i][j] = both(0.f);
    if (KEEP) {
#pragma unroll
      for (int j = 0; j < 4; ++j) wa[i][j] = wb[i][j] = both(0.f);
      if (v < nvec) {
        load_w4<WF32>(p.w_post, v, wa[i]);
        load_w4<WF32>(p.w_pre, v, wb[i]);
      }
    }
  }
  auto weights = [&](int i, float2* a, float2* b) {
    if (KEEP) {
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = wa[KEEP ? i : 0][j], b[j] = wb[KEEP ? i : 0][j];
    } else {
      load_w4<WF32>(p.w_post, c + i * TPR, a);
      load_w4<WF32>(p.w_pre, c + i * TPR, b);
    }
  };
  // the group's first thread: row t into stage s
  auto fill = [&](int64_t t, int s) {
    if (t >= p.T) return;
    uint8_t* at = mine + s * stage_bytes;
    uint64_t* bar = &full[rg][s];
    mbar_arrive_expect_tx(bar, row_bytes * (p.dh ? 4 : 3));
    bulk_load(at, p.dy + t * p.lddy, row_bytes, bar);
    bulk_load(at + row_bytes, p.u + t * p.ldu, row_bytes, bar);
    bulk_load(at + 2 * row_bytes, p.h + t * d, row_bytes, bar);
    if (p.dh) bulk_load(at + 3 * row_bytes, p.dh + t * p.lddh, row_bytes, bar);
  };
  // rows are dealt round the blocks, then the groups: few rows take many SMs
  const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
  const int64_t t0 = blockIdx.x + static_cast<int64_t>(gridDim.x) * rg;
  if (c == 0)
    for (int s = 0; s < p.stages; ++s) fill(t0 + s * step, s);
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  const float per = 1.f / static_cast<float>(d);
  for (int64_t t = t0; t < p.T; t += step) {
    const float ru = __ldg(p.rstd_u + t);
    const float rh = __ldg(p.rstd_h + t);
    const float gt = p.gate ? __ldg(p.gate + t * p.gate_step) : 1.f;
    if (!mbar_wait(&full[rg][stage], phase, &gave_up[rg])) gave_up[rg] = 1;
    const uint4* at = reinterpret_cast<const uint4*>(mine + stage * stage_bytes);
    float2 s1 = both(0.f), s2 = both(0.f), s3 = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (v >= nvec) continue;
      float2 f[4], g[4], w[4], o[4], a[4], b[4];
      unpack4(at[v], f);
      unpack4(at[nvec + v], g);
      unpack4(at[2 * nvec + v], w);
      unpack4(p.dh ? at[3 * nvec + v] : make_uint4(0, 0, 0, 0), o);
      weights(i, a, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 gy = f2_mul(f[j], b[j]), au = f2_mul(a[j], g[j]);
        s1 = f2_fma(gy, w[j], s1);
        s2 = f2_fma(au, f2_fma(both(rh), gy, o[j]), s2);
        s3 = f2_fma(au, w[j], s3);
      }
    }
    __syncwarp();
    const float part[3] = {s1.x + s1.y, s2.x + s2.y, s3.x + s3.y};
    float sum = three_sums(part, lane);  // of number lane / 8
    if (WPR > 1) {
      // sum q of warp w at 4 w + q; each lane brings together those of one q
      if ((lane & 7) == 0) red[flip][(threadIdx.x >> 5) * 4 + (lane >> 3)] = sum;
      meet();
      const float* r = red[flip] + rg * WPR * 4;
      sum = lane < 4 * WPR ? r[lane] : 0.f;
#pragma unroll
      for (int k = 32; k < 4 * WPR; k += 32)
        if (lane + k < 4 * WPR) sum += r[lane + k];
#pragma unroll
      for (int o = 16; o > 2; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const int span = WPR > 1 ? 1 : 8;  // lanes from one sum to the next
    const float t1 = __shfl_sync(0xffffffffu, sum, 0), t2 = __shfl_sync(0xffffffffu, sum, span),
                t3 = __shfl_sync(0xffffffffu, sum, 2 * span);
    if (*reinterpret_cast<volatile int*>(&gave_up[rg])) break;
    // past this meeting every thread of the group is done with the row before this one
    if (p.stages > 1 && c == 0 && t != t0) fill(t + (p.stages - 1) * step, stage == 0 ? p.stages - 1 : stage - 1);
    const float m1 = t1 * per * rh * rh;              // dH = dh + rh (g - h m1)
    const float along = ru * fmaf(-rh * m1, t3, t2);  // sum a dH u ru
    const float m2 = along * per * ru;                // du = gate ru (a dH - u m2)
    if (c == 0 && p.d_gate) p.d_gate[t] = along;
    const float gr = gt * ru;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = c + i * TPR;
      if (v >= nvec) continue;
      float2 f[4], g[4], w[4], o[4], a[4], b[4];
      unpack4(at[v], f);
      unpack4(at[nvec + v], g);
      unpack4(at[2 * nvec + v], w);
      unpack4(p.dh ? at[3 * nvec + v] : make_uint4(0, 0, 0, 0), o);
      weights(i, a, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 dH = f2_fma(both(rh), f2_fma(f[j], b[j], f2_mul(w[j], both(-m1))), o[j]);
        db[i][j] = f2_fma(f2_mul(f[j], both(rh)), w[j], db[i][j]);
        da[i][j] = f2_fma(f2_mul(dH, both(gr)), g[j], da[i][j]);
        f[j] = f2_mul(f2_fma(a[j], dH, f2_mul(g[j], both(-m2))), both(gr));
        o[j] = f2_mul(dH, both(p.scale));
      }
      *(reinterpret_cast<uint4*>(p.du + t * d) + v) = pack4(f);
      *(reinterpret_cast<uint4*>(p.dx + t * d) + v) = pack4(o);
    }
    if (p.stages == 1) {
      meet();
      if (c == 0) fill(t + step, 0);
    }
    flip ^= 1;
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  __syncwarp();
  if (gave_up[rg] && c == 0) {  // a copy that did not arrive
    dmoe::raise_error(p.err, DMOE_SITE_NORM_WAIT | DMOE_ERR_TIMEOUT);
    volatile int go_on = 0;
    for (int i = 0; i < p.stages; ++i) {  // the copies still on their way, as far as they come
      mbar_wait(&full[rg][stage], phase, &go_on);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (!p.partial) return;
  __syncthreads();  // every row has been read
  float* sums = reinterpret_cast<float*>(ring);  // [GROUPS][2 d]
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = c + i * TPR;
    if (v >= nvec) continue;
    float* o = sums + static_cast<size_t>(rg) * 2 * d + 8 * v;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      *reinterpret_cast<float4*>(o + 2 * j) = make_float4(da[i][j].x, da[i][j].y, da[i][j + 1].x, da[i][j + 1].y);
      *reinterpret_cast<float4*>(o + d + 2 * j) = make_float4(db[i][j].x, db[i][j].y, db[i][j + 1].x, db[i][j + 1].y);
    }
  }
  __syncthreads();
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * d;
  for (int i = threadIdx.x; i < d / 2; i += THREADS) {  // four columns of 2 d
    float4 a = reinterpret_cast<const float4*>(sums)[i];
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) {
      const float4 q = reinterpret_cast<const float4*>(sums + static_cast<size_t>(g) * 2 * d)[i];
      a.x += q.x, a.y += q.y, a.z += q.z, a.w += q.w;
    }
    reinterpret_cast<float4*>(out)[i] = a;
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

// Forward: the fewest threads of these that hold a row at two vectors each; above
// 8192 columns four.  (Where powers of two alone would leave up to half of
// them without a second vector: 8192 x 2560 34 us in 256 threads, 28 in 160;
// 8192 x 6144 87 in 512, 64 in 384.)
template <typename F>
cudaError_t forward_by_width(int d, const F& f) {
  const int nvec = d >> 3;
  if (nvec <= 2 * 32) return f.template operator()<32, 2>();
  if (nvec <= 2 * 64) return f.template operator()<64, 2>();
  if (nvec <= 2 * 96) return f.template operator()<96, 2>();
  if (nvec <= 2 * 128) return f.template operator()<128, 2>();
  if (nvec <= 2 * 160) return f.template operator()<160, 2>();
  if (nvec <= 2 * 192) return f.template operator()<192, 2>();
  if (nvec <= 2 * 256) return f.template operator()<256, 2>();
  if (nvec <= 2 * 320) return f.template operator()<320, 2>();
  if (nvec <= 2 * 384) return f.template operator()<384, 2>();
  if (nvec <= 2 * 512) return f.template operator()<512, 2>();
  return f.template operator()<512, 4>();
}

// Backward: threads per row, likewise (8192 x 1280 35 us in 128 threads, 29 in 96;
// 8192 x 2560 56 in 256, 47 in 160; 192 and 384 gain nothing, as fewer than 480
// threads an SM are left).
int threads_per_row(int d) {
  for (const int tpr : {32, 64, 96, 128, 160, 256})
    if ((d >> 3) <= 2 * tpr) return tpr;
  return 512;
}

template <typename F>
cudaError_t by_width(int d, const F& f) {
  switch (threads_per_row(d)) {
    case 32: return f.template operator()<32, 2>();
    case 64: return f.template operator()<64, 2>();
    case 96: return f.template operator()<96, 2>();
    case 128: return f.template operator()<128, 2>();
    case 160: return f.template operator()<160, 2>();
    case 256: return f.template operator()<256, 2>();
    default: return (d >> 3) <= 1024 ? f.template operator()<512, 2>() : f.template operator()<512, 4>();
  }
}

size_t back_stage_bytes(int d) { return static_cast<size_t>(back_threads(threads_per_row(d)) / threads_per_row(d)) * d * 2 * 4; }
int ring_stages(int d) { return static_cast<int>(std::clamp<size_t>(kRingBytes / back_stage_bytes(d), 1, kMaxStages)); }

// Blocks of the backward: one an SM, each leaving one partial row.
int backward_blocks(int T, int sms) { return std::min(T, sms); }

struct Forward {
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
    constexpr int block = forward_block(TPR), rpb = block / TPR;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) + rpb - 1) / rpb));
    auto kern = wf32 ? sandwich_norm_kernel<TPR, VPT, true> : sandwich_norm_kernel<TPR, VPT, false>;
    return dmoe::launch_pdl(kern, grid, dim3(block), 0, st, u, ldu, x, ldx, w_post, w_pre, gate, gate_step, scale, eps,
                            T, d, h, y, rstd_u, rstd_h);
  }
};

struct Backward {
  Back p;
  int wf32;
  int blocks;
  int device;
  cudaStream_t st;

  template <int TPR, int VPT, bool WF32>
  cudaError_t launch() const {
    auto kern = sandwich_norm_backward_kernel<TPR, VPT, WF32>;
    // the ring also holds the groups' sums: two fp32 rows each where four bf16 ones were
    static std::atomic<uint64_t> opted{0};
    const uint64_t bit = uint64_t(1) << device;
    if (!(opted.load(std::memory_order_acquire) & bit)) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kRingBytes));
      if (e != cudaSuccess) return e;
      opted.fetch_or(bit, std::memory_order_acq_rel);
    }
    return dmoe::launch_pdl(kern, dim3(blocks), dim3(back_threads(TPR)), p.stages * back_stage_bytes(p.d), st, p);
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
  const cudaError_t e = forward_by_width(d, f);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

DMOE_API size_t dmoe_sandwich_norm_backward_workspace_size(int T, int d) {
  dmoe::DeviceInfo di;
  if (T < 0 || d < 8 || (d & 7) || d > kMaxD || dmoe::device_info(&di) != DMOE_OK) return 0;
  return (static_cast<size_t>(backward_blocks(T, di.sm_count)) * 2 * d + T) * sizeof(float);
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
  if (T == 0) {  // no rows: the sums over them are zero
    cudaError_t e = cudaSuccess;
    if (dw_post) e = cudaMemsetAsync(dw_post, 0, static_cast<size_t>(d) * sizeof(float), st);
    if (e == cudaSuccess && dw_pre) e = cudaMemsetAsync(dw_pre, 0, static_cast<size_t>(d) * sizeof(float), st);
    if (e == cudaSuccess && d_gate && gate_rows == 1) e = cudaMemsetAsync(d_gate, 0, sizeof(float), st);
    return dmoe::cuda_status(e);
  }
  const int blocks = backward_blocks(T, di.sm_count);
  const size_t part = static_cast<size_t>(blocks) * 2 * d;
  const bool sums = dw_post || dw_pre;
  const bool shared = d_gate && gate_rows != T;  // one gate for all rows: its gradient is their sum
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
