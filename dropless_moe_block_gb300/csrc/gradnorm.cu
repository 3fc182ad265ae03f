// The global norm of many gradients, and their clipping.
//
//   n = sqrt(sum_i sum_e g_i[e]^2),  c = min(1, max_norm / (n + eps)),
//   out_i = c g_i
//
// HBM-bound: every gradient is read, and written once.  A set larger than
// the L2 cache has to be read twice (the factor is known only after the
// last element), so the floor is 3 passes over the bytes, 2 when the set
// stays in L2.  Two launches: sums of squares, one double per block; then
// every block adds the blocks' sums in the same order (the result does not
// depend on which block ran when) and scales.  The chunks are walked forwards
// in the first launch and backwards in the second, so that what was read last
// is still in L2 when it is read again, and both times by all blocks side by
// side (runs of their own per block: DISCARD).
//
// The tensors are cut into chunks of kChunk elements, counted from each
// tensor's address rounded down to 16 bytes: chunks then load whole vectors
// wherever a tensor begins, and only a tensor's two ragged ends go by
// elements.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"

namespace {

constexpr int kClipThreads = 128;  // eight 16-byte vectors of a bf16 chunk each, all in flight
constexpr int kChunk = DMOE_GRAD_CHUNK;
constexpr int kBlocksPerSm = 8;
constexpr int kMaxBlocks = 2048;

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

template <bool F32>
__device__ float chunk_squares(const dmoe_grad& g, int64_t chunk) {
  constexpr int V = F32 ? 4 : 8;
  const Span s = span_of<F32>(g, chunk);
  float acc = 0.f;
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(g.in) + s.vlo * (F32 ? 4 : 2));
  const int nv = static_cast<int>((s.vhi - s.vlo) / V);
#pragma unroll 8
  for (int i = threadIdx.x; i < nv; i += kClipThreads) {
    float f[V];
    unpack<F32>(__ldg(p + i), f);
#pragma unroll
    for (int j = 0; j < V; ++j) acc = fmaf(f[j], f[j], acc);
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
  constexpr int V = F32 ? 4 : 8;
  constexpr int ES = F32 ? 4 : 2;
  Span s = span_of<F32>(g, chunk);
  // vectors only where source and destination begin alike
  if ((reinterpret_cast<uintptr_t>(g.in) ^ reinterpret_cast<uintptr_t>(g.out)) & 15u) s.vlo = s.vhi = s.lo;
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(g.in) + s.vlo * ES);
  uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<char*>(g.out) + s.vlo * ES);
  const int nv = static_cast<int>((s.vhi - s.vlo) / V);
#pragma unroll 8
  for (int i = threadIdx.x; i < nv; i += kClipThreads) {
    float f[V];
    unpack<F32>(p[i], f);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] *= c;
    o[i] = pack<F32>(f);
  }
  for (int64_t i = s.lo + threadIdx.x; i < s.vlo; i += kClipThreads) store1<F32>(g.out, i, load1<F32>(g.in, i) * c);
  for (int64_t i = s.vhi + threadIdx.x; i < s.hi; i += kClipThreads) store1<F32>(g.out, i, load1<F32>(g.in, i) * c);
}

// The tensor of a chunk, kept from one chunk to the next.
struct Cursor {
  dmoe_grad g;
  int64_t end;  // first chunk after it

  // Moves to the tensor that holds chunk ch: the last one whose first chunk is
  // <= ch (tensors without elements own no chunk and are passed over).
  __device__ __forceinline__ void seek(const dmoe_grad* __restrict__ grads, int n, int64_t chunks, int64_t ch) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(&grads[mid].first_chunk) <= ch) lo = mid;
      else hi = mid - 1;
    }
    g = grads[lo];
    end = lo + 1 < n ? grads[lo + 1].first_chunk : chunks;
  }
  __device__ __forceinline__ bool holds(int64_t ch) const { return ch >= g.first_chunk && ch < end; }
};

__device__ __forceinline__ double block_sum(double v, double* sh) {
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
    grad_squares_kernel(const dmoe_grad* __restrict__ grads, int n, int64_t chunks, double* __restrict__ partial) {
  __shared__ double sh[kClipThreads / 32];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  // a thread's sum of at most kChunk / kClipThreads squares in fp32, the sums
  // of chunks, threads and blocks in fp64
  double acc = 0.0;
  Cursor at{};
  for (int64_t ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    if (!at.holds(ch)) at.seek(grads, n, chunks, ch);
    acc += at.g.f32 ? chunk_squares<true>(at.g, ch - at.g.first_chunk) : chunk_squares<false>(at.g, ch - at.g.first_chunk);
  }
  acc = block_sum(acc, sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

__global__ void __launch_bounds__(kClipThreads, kBlocksPerSm)
    grad_scale_kernel(const dmoe_grad* __restrict__ grads, int n, int64_t chunks, const double* __restrict__ partial,
                      int nsums, float max_norm, float eps, float* __restrict__ norm) {
  __shared__ double sh[kClipThreads / 32];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  double v = 0.0;
  for (int i = threadIdx.x; i < nsums; i += kClipThreads) v += partial[i];
  const float nrm = static_cast<float>(sqrt(block_sum(v, sh)));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = nrm;
  float c = max_norm / (nrm + eps);
  if (c > 1.f) c = 1.f;  // (a norm that is not a number stays one, and reaches every gradient)
  Cursor at{};
  for (int64_t ch = chunks - 1 - blockIdx.x; ch >= 0; ch -= gridDim.x) {
    if (!at.holds(ch)) at.seek(grads, n, chunks, ch);
    if (c == 1.f && at.g.in == at.g.out) continue;  // in place and within the limit: nothing changes
    if (at.g.f32) chunk_scale<true>(at.g, ch - at.g.first_chunk, c);
    else chunk_scale<false>(at.g, ch - at.g.first_chunk, c);
  }
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

DMOE_API size_t dmoe_clip_grad_norm_workspace_size(void) { return kMaxBlocks * sizeof(double); }

DMOE_API dmoe_status dmoe_clip_grad_norm(const dmoe_grad* grads, int n, int64_t chunks, float max_norm, float eps,
                                         float* norm, void* ws, size_t ws_bytes, dmoe_stream_t stream) {
  if (n < 0 || chunks < 0 || !(max_norm >= 0.f) || !(eps >= 0.f) || !norm || (reinterpret_cast<uintptr_t>(norm) & 3))
    return DMOE_ERR_INVALID_ARG;
  if (chunks > 0 && (n == 0 || !grads || !dmoe::aligned16(grads))) return DMOE_ERR_INVALID_ARG;
  if (!ws || !dmoe::aligned16(ws) || ws_bytes < dmoe_clip_grad_norm_workspace_size()) return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status s = dmoe::device_info(&di);
  if (s != DMOE_OK) return s;
  cudaStream_t st = dmoe::as_stream(stream);
  const int blocks = clip_blocks(chunks, di.sm_count);
  double* partial = static_cast<double*>(ws);
  cudaError_t e = dmoe::launch_pdl(grad_squares_kernel, dim3(blocks), dim3(kClipThreads), 0, st, grads, n, chunks,
                                   partial);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  e = dmoe::launch_pdl(grad_scale_kernel, dim3(blocks), dim3(kClipThreads), 0, st, grads, n, chunks,
                       static_cast<const double*>(partial), blocks, max_norm, eps, norm);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(2);
  return DMOE_OK;
}
