// The global norm of many gradients, and their clipping.
//
//   n = sqrt(sum_i sum_e g_i[e]^2),  c = min(1, max_norm / (n + eps)),
//   out_i = c g_i
//
// HBM-bound: every gradient is read, and written once.  A set larger than
// the L2 cache has to be read twice (the factor is known only after the
// last element), so the floor is 3 passes over the bytes, 2 when the set
// stays in L2.  Two launches.  The first sums squares, one double per block;
// the last of its blocks to finish (an atomic ticket says which) adds the
// blocks' sums in the order of the blocks, so the result does not depend on
// who was last, and leaves the norm and the factor.  The second scales, one
// chunk per block: short-lived blocks in the order of the addresses take 785 us
// for 2.8 GB (7.2 TB/s of reads and writes), persistent ones 991 to 1023 (5.5
// to 5.7 TB/s; the kernel alone).
//
// The tensors are cut into chunks of kChunk elements, counted from each
// tensor's address rounded down to 16 bytes: chunks then load whole vectors
// wherever a tensor begins, and only a tensor's two ragged ends go by
// elements.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"

namespace {

constexpr int kClipThreads = 128;
constexpr int kChunk = DMOE_GRAD_CHUNK;
constexpr int kBlocksPerSm = 8;  // of the sums
constexpr int kMaxBlocks = 2048;

// The workspace: zero before its first use, ready for the next call after each.
struct Scratch {
  unsigned int ticket;
  float factor;
  double pad;
  double sums[kMaxBlocks];
};

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (F32) return reinterpret_cast<const float*>(p)[i];
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

template <bool F32>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (F32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// The 4 (fp32) or 8 (bf16) values of a 16-byte vector.
template <bool F32>
__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  if (F32) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  } else {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __bfloat1622float2(h[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}

template <bool F32>
__device__ __forceinline__ uint4 pack(const float* f) {
  uint4 u;
  if (F32) {
    u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  }
  return u;
}

// A chunk of one tensor: elements [lo, hi), of which [vlo, vhi) are whole
// 16-byte vectors.
struct Span {
  int64_t lo, hi, vlo, vhi;
};

template <bool F32>
__device__ __forceinline__ Span span_of(const dmoe_grad& g, int64_t chunk) {
  constexpr int V = F32 ? 4 : 8;
  const int64_t off = (reinterpret_cast<uintptr_t>(g.in) & 15u) / (F32 ? 4 : 2);
  Span s;
  s.lo = max(chunk * kChunk - off, int64_t(0));
  s.hi = min((chunk + 1) * kChunk - off, g.n);
  s.vlo = min(((s.lo + off + V - 1) / V) * V - off, s.hi);
  s.vhi = max(((s.hi + off) / V) * V - off, s.vlo);
  return s;
}

// Vectors of a whole chunk per thread.
template <bool F32>
__host__ __device__ constexpr int whole() {
  return kChunk / (F32 ? 4 : 8) / kClipThreads;
}

template <bool F32>
__device__ float chunk_squares(const dmoe_grad& g, int64_t chunk) {
  constexpr int V = F32 ? 4 : 8, N = whole<F32>();
  const Span s = span_of<F32>(g, chunk);
  float acc = 0.f;
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(g.in) + s.vlo * (F32 ? 4 : 2));
  const int nv = static_cast<int>((s.vhi - s.vlo) / V);
  // eight loads in flight, also of a chunk that is not whole (400 small
  // tensors 10.8 us; 13.0 by a loop with a remainder, which in turn takes 391
  // instead of 396 us for 2.8 GB; the kernel alone)
#pragma unroll
  for (int b = 0; b < N; b += 8) {
    uint4 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = threadIdx.x + (b + j) * kClipThreads;
      u[j] = i < nv ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float f[V];
      unpack<F32>(u[j], f);
#pragma unroll
      for (int q = 0; q < V; ++q) acc = fmaf(f[q], f[q], acc);
    }
  }
  for (int64_t i = s.lo + threadIdx.x; i < s.vlo; i += kClipThreads) {
    const float f = load1<F32>(g.in, i);
    acc = fmaf(f, f, acc);
  }
  for (int64_t i = s.vhi + threadIdx.x; i < s.hi; i += kClipThreads) {
    const float f = load1<F32>(g.in, i);
    acc = fmaf(f, f, acc);
  }
  return acc;
}

template <bool F32>
__device__ void chunk_scale(const dmoe_grad& g, int64_t chunk, float c) {
  constexpr int V = F32 ? 4 : 8, N = whole<F32>();
  constexpr int ES = F32 ? 4 : 2;
  Span s = span_of<F32>(g, chunk);
  // vectors only where source and destination begin alike
  if ((reinterpret_cast<uintptr_t>(g.in) ^ reinterpret_cast<uintptr_t>(g.out)) & 15u) s.vlo = s.vhi = s.lo;
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(g.in) + s.vlo * ES);
  uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<char*>(g.out) + s.vlo * ES);
  const int nv = static_cast<int>((s.vhi - s.vlo) / V);
#pragma unroll
  for (int b = 0; b < N; b += 8) {
    // loaded before the first is stored: source and destination may be the same
    uint4 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = threadIdx.x + (b + j) * kClipThreads;
      if (i < nv) u[j] = p[i];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = threadIdx.x + (b + j) * kClipThreads;
      if (i >= nv) continue;
      float f[V];
      unpack<F32>(u[j], f);
#pragma unroll
      for (int q = 0; q < V; ++q) f[q] *= c;
      o[i] = pack<F32>(f);
    }
  }
  for (int64_t i = s.lo + threadIdx.x; i < s.vlo; i += kClipThreads) store1<F32>(g.out, i, load1<F32>(g.in, i) * c);
#pragma unroll 8
  for (int64_t i = s.vhi + threadIdx.x; i < s.hi; i += kClipThreads) store1<F32>(g.out, i, load1<F32>(g.in, i) * c);
}

// The tensor of a chunk, kept from one chunk to the next.
struct Cursor {
  dmoe_grad g;
  int64_t end;  // first chunk after it

  // Moves to the tensor that holds chunk ch: the last one whose first chunk is
  // <= ch (tensors without elements own no chunk and are passed over).  The
  // warp looks at 32 tensors at a time.
  __device__ __forceinline__ void seek(const dmoe_grad* __restrict__ grads, int n, int64_t chunks, int64_t ch) {
    const int lane = threadIdx.x & 31;
    int lo = 0, count = n;
    while (count > 1) {
      const int step = (count + 31) / 32;
      const int at = lane * step;
      const bool below = at < count && __ldg(&grads[lo + at].first_chunk) <= ch;
      const int k = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // lane 0's always is
      lo += k * step;
      count = min(step, count - k * step);
    }
    g = grads[lo];
    end = lo + 1 < n ? __ldg(&grads[lo + 1].first_chunk) : chunks;
  }
  __device__ __forceinline__ bool holds(int64_t ch) const { return ch >= g.first_chunk && ch < end; }
};

__device__ __forceinline__ double block_sum(double v, double* sh) {
  __syncthreads();  // sh may still be read from a sum before
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < kClipThreads / 32; ++i) t += sh[i];
  return t;
}

__global__ void __launch_bounds__(kClipThreads, kBlocksPerSm)
    grad_squares_kernel(const dmoe_grad* __restrict__ grads, int n, int64_t chunks, Scratch* ws, float max_norm,
                        float eps, float* __restrict__ norm) {
  __shared__ double sh[kClipThreads / 32];
  __shared__ bool last;
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  // a thread's sum of at most kChunk / kClipThreads squares (and two ragged
  // ends) in fp32, the sums of chunks, threads and blocks in fp64
  double acc = 0.0;
  Cursor at{};
  for (int64_t ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    if (!at.holds(ch)) at.seek(grads, n, chunks, ch);
    acc += at.g.f32 ? chunk_squares<true>(at.g, ch - at.g.first_chunk) : chunk_squares<false>(at.g, ch - at.g.first_chunk);
  }
  acc = block_sum(acc, sh);
  if (threadIdx.x == 0) {
    ws->sums[blockIdx.x] = acc;
    __threadfence();
    last = atomicInc(&ws->ticket, gridDim.x - 1) == gridDim.x - 1;  // back to 0 with the last block
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double v = 0.0;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kClipThreads) v += __ldcg(&ws->sums[i]);
  const float nrm = static_cast<float>(sqrt(block_sum(v, sh)));
  if (threadIdx.x == 0) {
    *norm = nrm;
    // 0 / 0 is the factor of zeros, which need none; without a limit no norm
    // asks for one.  A norm that is not a number stays one, and reaches every
    // gradient.
    const float c = nrm + eps == 0.f || (max_norm == INFINITY && nrm == nrm) ? 1.f : max_norm / (nrm + eps);
    ws->factor = c > 1.f ? 1.f : c;
  }
}

__global__ void __launch_bounds__(kClipThreads)
    grad_scale_kernel(const dmoe_grad* __restrict__ grads, int n, int64_t chunks, const Scratch* ws) {
  const int64_t ch = blockIdx.x;
  Cursor at{};
  at.seek(grads, n, chunks, ch);  // the table is the caller's: nothing in flight writes it
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const float c = ws->factor;
  if (c == 1.f && at.g.in == at.g.out) return;  // in place and within the limit: nothing changes
  if (at.g.f32) chunk_scale<true>(at.g, ch - at.g.first_chunk, c);
  else chunk_scale<false>(at.g, ch - at.g.first_chunk, c);
}

int clip_blocks(int64_t chunks, int sms) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({chunks, int64_t(sms) * kBlocksPerSm, kMaxBlocks})));
}

}  // namespace

DMOE_API int64_t dmoe_grad_chunks(const void* in, int64_t n, int f32) {
  if (n <= 0) return 0;
  const int64_t off = static_cast<int64_t>((reinterpret_cast<uintptr_t>(in) & 15u) / (f32 ? 4 : 2));
  return (n + off + kChunk - 1) / kChunk;
}

DMOE_API size_t dmoe_clip_grad_norm_workspace_size(void) { return sizeof(Scratch); }

DMOE_API dmoe_status dmoe_clip_grad_norm(const dmoe_grad* grads, int n, int64_t chunks, float max_norm, float eps,
                                         float* norm, void* ws, size_t ws_bytes, dmoe_stream_t stream) {
  if (n < 0 || chunks < 0 || chunks > INT32_MAX || !(max_norm >= 0.f) || !(eps >= 0.f) || !norm || (reinterpret_cast<uintptr_t>(norm) & 3))
    return DMOE_ERR_INVALID_ARG;
  if (chunks > 0 && (n == 0 || !grads || !dmoe::aligned16(grads))) return DMOE_ERR_INVALID_ARG;
  if (!ws || !dmoe::aligned16(ws) || ws_bytes < dmoe_clip_grad_norm_workspace_size()) return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  cudaStream_t st = dmoe::as_stream(stream);
  const int blocks = clip_blocks(chunks, di.sm_count);
  Scratch* scratch = static_cast<Scratch*>(ws);
  cudaError_t e = dmoe::launch_pdl(grad_squares_kernel, dim3(blocks), dim3(kClipThreads), 0, st, grads, n, chunks,
                                   scratch, max_norm, eps, norm);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  if (chunks == 0) return DMOE_OK;
  e = dmoe::launch_pdl(grad_scale_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kClipThreads), 0, st, grads, n,
                       chunks, static_cast<const Scratch*>(scratch));
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}
