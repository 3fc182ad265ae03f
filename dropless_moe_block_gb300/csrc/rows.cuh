// Rows of bf16 values in registers and on their way there: what the norms'
// kernels share.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "tc.cuh"

namespace dmoe {
namespace rows {

// Copies bytes (a multiple of 16) between 16-byte aligned addresses,
// asynchronously; completes them on bar.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   dmoe::tc::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(dmoe::tc::smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __bfloat1622float2(h[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return u;
}

// Eight weights from column 8 v on, bf16 or fp32.
template <bool WF32>
__device__ __forceinline__ void load_w(const void* w, int v, float* f) {
  if (WF32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w) + 2 * v);
    const float4 b = __ldg(reinterpret_cast<const float4*>(w) + 2 * v + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + v), f);
  }
}

// Sum of v over the TPR threads of this thread's row; red: one float per
// warp of the block.  Every thread of the block takes part when TPR > 32.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR > 32) {
    constexpr int WPR = TPR / 32;  // warps per row
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const float* r = red + warp / WPR * WPR;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) v += r[i];
  }
  return v;
}

// ----------------------------------------------------------------- host side

inline bool bad_ptr(const void* p) { return !dmoe::aligned16(p); }
inline bool bad_ld(int64_t ld, int d) { return ld < d || (ld & 7); }
// Rows written over rows of another pitch: over some that another block has yet
// to read.
inline bool bad_alias(const void* out, const void* in, int64_t ld, int T, int d) { return out && out == in && T > 1 && ld != d; }

}  // namespace rows
}  // namespace dmoe
