// Routing with a bias for balance: softmax or sigmoid scores, groups of
// experts, top-k, weights renormalised and scaled; its backward, and the bias'
// update.
//
//   s_e = softmax(z)_e or sigmoid(z_e)           c_e = s_e + bias_e
//   a group's worth: its two largest c summed; the best groups stay
//   of their experts the k largest c;  w = s (/ their sum) * scale
//
// One warp per token, the row of logits in registers (lane l: experts l, l +
// 32, ...).  A round of the top-k is two integer reductions over the warp:
// the largest of order-preserving keys, and the lowest expert that has it.
//
// Which experts are chosen must not hang on how fp32 rounds s + bias: c is
// known to `tol`, and where two neighbours of the descending order (or the
// last group that stays and the first that goes) are closer than that, the
// token is decided again by c in 64 bits, of those candidates alone.  With
// 256 sigmoid scores that is one token in some hundred.  Without a bias the
// order is that of the logits, which is exact.
#include <float.h>
#include <math.h>

#include "common.cuh"

namespace {

constexpr int kWarps = 8;  // tokens per block
constexpr int kMaxGroups = 32;
constexpr uint32_t kFull = 0xffffffffu;

// Larger key, larger number; 0 is below every number's.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);  // -0 is 0
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float float_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) { return float_of(__reduce_max_sync(kFull, key_of(v))); }

// NaN counts as minus infinity, which no score comes of; plus infinity as the
// largest number.
__device__ __forceinline__ float clean(float z) { return isnan(z) ? -INFINITY : fminf(z, FLT_MAX); }

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// What the chosen scores are proportional to, `top` being the largest chosen
// logit: scores that would vanish in fp32 (all chosen sigmoids below e^-30,
// where they are exponentials to 13 digits) keep their ratios.
__device__ __forceinline__ float proportion(float z, float top, bool sig) {
  return sig && top >= -30.f ? sigmoid(z) : expf(z - top);
}

struct Choice {
  const float* logits;
  const float* bias;  // NULL: by the logits
  int T, E, k;
  int sig, renorm;
  float scale;
  int groups, top_groups;  // top_groups == groups: no groups
  int size;                // experts of a group
  uint32_t inv_size;       // ceil(2^20 / size): e / size = e inv_size >> 20 for e < 1024
  int lanes;               // per group, a power of two
  int stride;              // of a group's scores in shared memory
  int32_t* expert_idx;
  float* gate_w;
};

// c in 64 bits; m, total: the softmax's reference and sum.
__device__ double exact_choice(float z, float b, bool sig, float m, double total) {
  if (z == -INFINITY) return -INFINITY;
  const double s = sig ? 1.0 / (1.0 + exp(-static_cast<double>(z))) : exp(static_cast<double>(z) - m) / total;
  const double c = s + b;
  return isnan(c) ? -INFINITY : c;
}

template <class F>
__device__ __forceinline__ void top_two(F a, F& first, F& second) {
  if (a > first) {
    second = first;
    first = a;
  } else if (a > second) {
    second = a;
  }
}

template <class F>
__device__ __forceinline__ F group_worth(F first, F second, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) {
    const F f = __shfl_xor_sync(kFull, first, o), s = __shfl_xor_sync(kFull, second, o);
    top_two(f, first, second);
    top_two(s, first, second);
  }
  return second == -INFINITY ? first : first + second;
}

// How many of the groups (one every `lanes` lanes) are better than this lane's.
template <class F>
__device__ __forceinline__ int group_rank(F worth, int g, int groups, int lanes) {
  int rank = 0;
  for (int h = 0; h < groups; ++h) {
    const F w = __shfl_sync(kFull, worth, h * lanes);
    rank += w > worth || (w == worth && h < g);
  }
  return rank;
}

template <int NPL, bool GROUPS>
__global__ void __launch_bounds__(kWarps * 32) route_balanced_kernel(const Choice p) {
  extern __shared__ float group_mem[];  // [kWarps][groups * stride]
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const float* row = p.logits + t * p.E;
  const bool sig = p.sig;
  float z[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = i * 32 + lane;
    z[i] = e < p.E ? __ldg(row + e) : -INFINITY;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    z[i] = clean(z[i]);
    m = fmaxf(m, z[i]);
  }
  m = warp_max(m);
  const bool scored = GROUPS || p.bias || (!sig && !p.renorm);  // else the logits alone decide and weigh
  float inv = 1.f;  // of the softmax's sum
  float s[NPL];
  if (scored) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      s[i] = z[i] == -INFINITY ? 0.f : sig ? sigmoid(z[i]) : expf(z[i] - m);
      sum += s[i];
    }
    if (!sig) {
      sum = warp_sum(sum);
      inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) s[i] *= inv;
    }
  }

  // choices; how far fp32 may be off between two of them: a score is off by
  // 2^-22 (expf) and three roundings, a softmax also by its sum's roundings
  // (in the worst case one for every term a lane adds, and five), s + bias
  // by 2^-24 of itself; both sides counted
  float b[NPL];
  uint32_t key[NPL], alive = 0;
  float tol = 0.f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = i * 32 + lane;
    b[i] = p.bias && e < p.E ? __ldg(p.bias + e) : 0.f;
    if (e < p.E) alive |= 1u << i;
  }
  if (GROUPS || p.bias) {
    float size = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      size = fmaxf(size, s[i] + (fabsf(b[i]) < INFINITY ? fabsf(b[i]) : 0.f));
      const float c = z[i] == -INFINITY ? -INFINITY : s[i] + b[i];
      s[i] = isnan(c) ? -INFINITY : c;  // from here on the choice
    }
    tol = warp_max(size) * (8.f + (sig ? 0.f : 2.f * NPL + 10.f)) * 1.1920929e-7f;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) key[i] = key_of(p.bias ? s[i] : z[i]);

  double total = -1.0;  // the softmax's sum in 64 bits, once it is needed
  auto need_total = [&]() {
    if (sig || total >= 0.0) return;
    total = 0.0;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) {
      const float v = clean(__ldg(row + e));
      if (v > -INFINITY) total += exp(static_cast<double>(v) - m);
    }
    total = warp_sum(total);
  };

  if (GROUPS) {
    float* mem = group_mem + (threadIdx.x >> 5) * p.groups * p.stride;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = i * 32 + lane;
      const int g = static_cast<int>((e * p.inv_size) >> 20);
      if (e < p.E) mem[g * p.stride + (e - g * p.size)] = s[i];
    }
    __syncwarp();
    const int g = lane / p.lanes, r = lane & (p.lanes - 1);
    float first = -INFINITY, second = -INFINITY;
    if (g < p.groups)
      for (int o = r; o < p.size; o += p.lanes) top_two(mem[g * p.stride + o], first, second);
    const float worth = group_worth(first, second, p.lanes);
    // every lane takes part in the ranks' shuffles, those of no group too
    bool stays = group_rank(worth, g, p.groups, p.lanes) < p.top_groups;
    stays = stays && g < p.groups;
    // the worst that stays against the best that goes
    const float low = float_of(__reduce_min_sync(kFull, stays ? key_of(worth) : kFull));
    const float high = float_of(__reduce_max_sync(kFull, g < p.groups && !stays ? key_of(worth) : 0u));
    if (low - high <= 2.f * tol) {
      // rows whose experts are all alike (padding) need no digits
      bool alike = true;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const float z0 = __shfl_sync(kFull, z[0], 0), b0 = __shfl_sync(kFull, b[0], 0);
        alike &= i * 32 + lane >= p.E || (z[i] == z0 && b[i] == b0);
      }
      if (!__all_sync(kFull, alike)) {
        need_total();
        double f = -INFINITY, n = -INFINITY;
        if (g < p.groups) {
#pragma unroll 1
          for (int o = r; o < p.size; o += p.lanes) {
            const int e = g * p.size + o;
            top_two(exact_choice(clean(__ldg(row + e)), p.bias ? __ldg(p.bias + e) : 0.f, sig, m, total), f, n);
          }
        }
        const double exact = group_worth(f, n, p.lanes);
        stays = group_rank(exact, g, p.groups, p.lanes) < p.top_groups;
        stays = stays && g < p.groups;
      }
    }
    const uint32_t lanes_in = __ballot_sync(kFull, stays);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = i * 32 + lane;
      const int ge = static_cast<int>((e * p.inv_size) >> 20);
      if (e < p.E && !((lanes_in >> (ge * p.lanes)) & 1u)) alive &= ~(1u << i);
    }
  }

  int32_t* out_i = p.expert_idx + t * p.k;
  float* out_w = p.gate_w + t * p.k;
  // the best of what is left: its key, and the lowest expert that has it
  auto best_of = [&](uint32_t left, uint32_t& best) {
    uint32_t own = 0;
    int at = 0;
#pragma unroll
    for (int i = NPL - 1; i >= 0; --i) {
      const uint32_t v = (left >> i) & 1u ? key[i] : 0u;
      if (v >= own) own = v, at = i;
    }
    best = __reduce_max_sync(kFull, own);
    return static_cast<int>(__reduce_min_sync(kFull, own == best && own != 0 ? at * 32 + lane : 0x7fffffff));
  };
  uint32_t left = alive;
  bool near = false;
  float last = INFINITY;
  int mine = 0;  // slot `lane`'s expert
  for (int j = 0; j < p.k; ++j) {
    uint32_t best;
    const int e = best_of(left, best);
    if ((e & 31) == lane) left &= ~(1u << (e >> 5));
    if (lane == (j & 31)) {
      if (j < 32) mine = e;
      else out_i[j] = e;
    }
    const float c = float_of(best);
    near |= last - c <= tol;
    last = c;
  }
  if (p.bias) {  // the first that is not chosen
    uint32_t best;
    best_of(left, best);
    near |= best != 0 && last - float_of(best) <= tol;
    if (near) {
      left = alive;
#pragma unroll 1
      for (int j = 0; j < p.k; ++j) {
        uint32_t best;
        int e = best_of(left, best);
        const float least = float_of(best) - tol;
        uint32_t close = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (((left >> i) & 1u) && s[i] >= least) close |= 1u << i;
        const int n = static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(__popc(close))));
        if (n > 1) {
          // exactly alike: the lowest, as found
          float ze = 0.f, be = 0.f;
#pragma unroll
          for (int i = 0; i < NPL; ++i)
            if (i == (e >> 5)) ze = z[i], be = b[i];
          ze = __shfl_sync(kFull, ze, e & 31);
          be = __shfl_sync(kFull, be, e & 31);
          bool alike = true;
#pragma unroll
          for (int i = 0; i < NPL; ++i) alike &= !((close >> i) & 1u) || (z[i] == ze && b[i] == be);
          if (!__all_sync(kFull, alike)) {
            need_total();
            double top = -INFINITY;
            int at = 0x7fffffff;
#pragma unroll 1
            for (int i = 0; i < NPL; ++i) {
              if (!__any_sync(kFull, (close >> i) & 1u)) continue;
              const int q = i * 32 + lane;
              if ((close >> i) & 1u) {
                const double c = exact_choice(clean(__ldg(row + q)), __ldg(p.bias + q), sig, m, total);
                if (c > top || at == 0x7fffffff) top = c, at = q;
              }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              const double c = __shfl_xor_sync(kFull, top, o);
              const int q = __shfl_xor_sync(kFull, at, o);
              if (q != 0x7fffffff && (at == 0x7fffffff || c > top || (c == top && q < at))) top = c, at = q;
            }
            e = at;
          }
        }
        if ((e & 31) == lane) left &= ~(1u << (e >> 5));
        if (lane == (j & 31)) {
          if (j < 32) mine = e;
          else out_i[j] = e;
        }
      }
    }
  }

  // slot j's weight in lane j mod 32, which wrote its expert
  float top = -INFINITY;
  if (p.renorm) {
    for (int j = lane; j < p.k; j += 32) top = fmaxf(top, clean(__ldg(row + (j < 32 ? mine : out_i[j]))));
    top = warp_max(top);
  }
  float sum = 0.f;
  for (int j = lane; j < p.k; j += 32) {
    const int e = j < 32 ? mine : out_i[j];
    if (j < 32) out_i[j] = e;
    const float v = clean(__ldg(row + e));
    float w = 0.f;
    if (v > -INFINITY) w = p.renorm ? proportion(v, top, sig) : sig ? sigmoid(v) : expf(v - m) * inv;
    sum += w;
    if (!p.renorm) out_w[j] = w * p.scale;
    else if (p.k > 32) out_w[j] = w;
    else last = w;
  }
  if (p.renorm) {
    sum = warp_sum(sum);
    const float f = sum > 0.f ? p.scale / sum : 0.f;
    for (int j = lane; j < p.k; j += 32) out_w[j] = (p.k > 32 ? out_w[j] : last) * f;
  }
}

// With G_e the d_gate of the slot that holds expert e (0 where none does) and,
// for renormalised weights, r the weights before their scaling:
//   softmax  dz = scale p (G - sum G p)       renormalised  scale r (G - sum G r)
//   sigmoid  dz = scale G s (1 - s)           renormalised  scale r (1 - s) (G - sum G r)
template <int NPL>
__global__ void __launch_bounds__(kWarps * 32)
    route_balanced_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ expert_idx,
                                   const float* __restrict__ d_gate, int T, int E, int k, int sig, int renorm,
                                   float scale, float* __restrict__ d_logits, int32_t* err) {
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const float* row = logits + t * E;
  float z[NPL], G[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = i * 32 + lane;
    z[i] = e < E ? __ldg(row + e) : -INFINITY;
    G[i] = 0.f;
  }
  uint32_t on = 0;
  for (int j0 = 0; j0 < k; j0 += 32) {
    int ej = -1;
    float gj = 0.f;
    if (j0 + lane < k) {
      ej = __ldg(expert_idx + t * k + j0 + lane);
      gj = __ldg(d_gate + t * k + j0 + lane);
      if (ej < 0 || ej >= E) dmoe::raise_error(err, DMOE_SITE_ROUTE_INDEX | DMOE_ERR_DEVICE);
    }
    for (int j = 0; j < min(32, k - j0); ++j) {
      const int e = __shfl_sync(kFull, ej, j);
      const float g = __shfl_sync(kFull, gj, j);
      if (e < 0 || e >= E || (e & 31) != lane) continue;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == (e >> 5)) {
          G[i] = g;
          on |= 1u << i;
        }
    }
  }
  // what a weight is proportional to, over the experts that share a sum
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    z[i] = clean(z[i]);
    if (!renorm || ((on >> i) & 1u)) m = fmaxf(m, z[i]);
  }
  m = warp_max(m);
  float r[NPL], sum = 0.f, dot = 0.f;
  const bool shared = renorm || !sig;
  if (shared) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      r[i] = 0.f;
      if (z[i] > -INFINITY && (!renorm || ((on >> i) & 1u))) r[i] = renorm ? proportion(z[i], m, sig) : expf(z[i] - m);
      sum += r[i];
      if ((on >> i) & 1u) dot = fmaf(G[i], r[i], dot);
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const float mean = dot * inv;
  float* out = d_logits + t * E;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = i * 32 + lane;
    float d = 0.f;
    if (shared) d = r[i] == 0.f ? 0.f : scale * (r[i] * inv) * (G[i] - mean);
    if (sig && ((on >> i) & 1u)) {
      const float q = expf(-fabsf(z[i])), half = 1.f / (1.f + q);
      const float rest = z[i] > 0.f ? q * half : half;  // 1 - s
      d = renorm ? d * rest : scale * G[i] * (q * half) * half;
    }
    if (e < E) out[e] = d;
  }
}

// bias += rate * sign(mean load - load): what draws tokens to experts that got few.
__global__ void __launch_bounds__(1024) balance_bias_kernel(float* bias, const int32_t* __restrict__ counts, int E,
                                                            float rate) {
  __shared__ long long part[32];
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int e = threadIdx.x;
  const long long n = e < E ? counts[e] : 0;
  long long sum = n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if ((e & 31) == 0) part[e >> 5] = sum;
  __syncthreads();
  sum = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) sum += part[i];
  if (e >= E) return;
  const long long over = n * E - sum;  // E times the load above the mean
  if (over != 0) bias[e] += over < 0 ? rate : -rate;
}

// Calls f.template operator()<NPL>() for E experts.
template <class F>
cudaError_t by_experts(int E, F&& f) {
  if (E <= 32) return f.template operator()<1>();
  if (E <= 64) return f.template operator()<2>();
  if (E <= 128) return f.template operator()<4>();
  if (E <= 256) return f.template operator()<8>();
  if (E <= 512) return f.template operator()<16>();
  return f.template operator()<32>();
}

bool misaligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) & 3u; }

dim3 grid_of(int T) { return dim3(static_cast<unsigned>((static_cast<int64_t>(T) + kWarps - 1) / kWarps)); }

struct ForwardCall {
  Choice p;
  cudaStream_t st;
  template <int NPL>
  cudaError_t operator()() const {
    const dim3 grid = grid_of(p.T), block(kWarps * 32);
    if (p.top_groups == p.groups) return dmoe::launch_pdl(route_balanced_kernel<NPL, false>, grid, block, 0, st, p);
    const size_t smem = sizeof(float) * kWarps * p.groups * p.stride;  // at most (1024 + 32) * 32 bytes
    return dmoe::launch_pdl(route_balanced_kernel<NPL, true>, grid, block, smem, st, p);
  }
};

struct BackwardCall {
  const float* logits;
  const int32_t* ei;
  const float* dg;
  int T, E, k, sig, renorm;
  float scale;
  float* dl;
  int32_t* err;
  cudaStream_t st;
  template <int NPL>
  cudaError_t operator()() const {
    return dmoe::launch_pdl(route_balanced_backward_kernel<NPL>, grid_of(T), dim3(kWarps * 32), 0, st, logits, ei, dg, T,
                            E, k, sig, renorm, scale, dl, err);
  }
};

bool bad_scores(int scores) { return scores != DMOE_SCORES_SOFTMAX && scores != DMOE_SCORES_SIGMOID; }

}  // namespace

DMOE_API dmoe_status dmoe_route_balanced(const float* logits, const float* bias, int T, int E, int k, int scores,
                                         int groups, int top_groups, int renormalize, float scale, int32_t* expert_idx,
                                         float* gate_w, dmoe_stream_t stream) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || bad_scores(scores) || groups < 1 || groups > kMaxGroups || E % groups ||
      top_groups < 1 || top_groups > groups || k > top_groups * (E / groups) || !isfinite(scale))
    return DMOE_ERR_INVALID_ARG;
  if (T == 0) return DMOE_OK;
  if (!logits || !expert_idx || !gate_w) return DMOE_ERR_INVALID_ARG;
  if (misaligned4(logits) || misaligned4(bias) || misaligned4(expert_idx) || misaligned4(gate_w))
    return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status st = dmoe::device_info(&di);
  if (st != DMOE_OK) return st;
  Choice p{logits, bias, T, E, k, scores == DMOE_SCORES_SIGMOID, renormalize ? 1 : 0, scale, groups, top_groups};
  p.size = E / groups;
  p.inv_size = ((1u << 20) + p.size - 1) / p.size;
  p.lanes = 1;
  while (2 * p.lanes * groups <= 32) p.lanes *= 2;
  // groups of a multiple of 8 scores would meet in the same banks
  p.stride = p.size % 8 ? p.size : p.size + p.lanes;
  p.expert_idx = expert_idx;
  p.gate_w = gate_w;
  const cudaError_t e = by_experts(E, ForwardCall{p, dmoe::as_stream(stream)});
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

DMOE_API dmoe_status dmoe_route_balanced_backward(const float* logits, const int32_t* expert_idx, const float* d_gate,
                                                  int T, int E, int k, int scores, int renormalize, float scale,
                                                  float* d_logits, dmoe_stream_t stream) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > E || bad_scores(scores) || !isfinite(scale)) return DMOE_ERR_INVALID_ARG;
  if (T == 0) return DMOE_OK;
  if (!logits || !expert_idx || !d_gate || !d_logits) return DMOE_ERR_INVALID_ARG;
  if (misaligned4(logits) || misaligned4(expert_idx) || misaligned4(d_gate) || misaligned4(d_logits))
    return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status st = dmoe::device_info(&di);
  if (st != DMOE_OK) return st;
  const cudaError_t e =
      by_experts(E, BackwardCall{logits, expert_idx, d_gate, T, E, k, scores == DMOE_SCORES_SIGMOID,
                                 renormalize ? 1 : 0, scale, d_logits, di.err_word, dmoe::as_stream(stream)});
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

DMOE_API dmoe_status dmoe_balance_bias(float* bias, const int32_t* tokens_per_expert, int E, float rate,
                                       dmoe_stream_t stream) {
  if (E < 1 || E > 1024 || !isfinite(rate) || !bias || !tokens_per_expert || misaligned4(bias) ||
      misaligned4(tokens_per_expert))
    return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status st = dmoe::device_info(&di);
  if (st != DMOE_OK) return st;
  const cudaError_t e = dmoe::launch_pdl(balance_bias_kernel, dim3(1), dim3((E + 31) / 32 * 32), 0,
                                         dmoe::as_stream(stream), bias, tokens_per_expert, E, rate);
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}
