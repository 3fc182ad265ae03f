// Routing with a bias for balance: softmax or sigmoid scores, groups of
// experts, top-k, weights renormalised and scaled; its backward, and the bias'
// update.
//
//   s_e = softmax(z)_e or sigmoid(z_e)           c_e = s_e + bias_e
//   a group's worth: its two largest c summed; the best groups stay
//   of their experts the k largest c;  w = s (/ their sum) * scale
//
// A warp per token, lane l with experts l, l + 32, ..., for any number of
// experts; of 64, 128 or 256, and where there are tokens enough, four tokens a
// warp (route_eighths_kernel).  16381 tokens of 256 experts in groups are 17 MB,
// 3 us of HBM, and take four a warp 19 to 24: 450 instructions a token, whose
// latency bounds it, and behind them the last of the tokens decided twice.  A
// warp a token takes some 1080, and is bound by them (70% of the issue slots
// while an SM is busy, 25 to 27 us).  So the choice works on 31-bit keys, a
// choice's place in its range and under it the expert's register, or number,
// such that one integer reduction finds the best and where it lies.
//
// Which experts are chosen must not hang on how the keys, or fp32, round: a
// key is known to `tol` steps, and a token where two neighbours of the
// descending order (or the last group that stays and the first that goes) are
// closer than that is decided again by c in 64 bits, of those that come into
// question alone.  With 256 sigmoid scores that is one token in a thousand;
// what it takes, some microseconds, is the fetching of code that was not run
// before, so that code is small and one (all of a token's scores in 64 bits,
// everything inlined: 50 us).
#include <float.h>
#include <math.h>

#include <algorithm>

#include "act.cuh"
#include "common.cuh"

namespace {

using namespace dmoe::act;

constexpr int kWarps = 8;  // tokens per block
constexpr int kMaxGroups = 32;
// Four tokens go to a warp from so many tokens on, or where each takes one
// expert: then few orders are open.  What is left to the whole warp costs its
// 6 us however few they are (us, whole warps and four tokens: 64 experts, top-1
// softmax, 1024 tokens 2.7 and 2.5, 8192 5.5 and 3.5, 32768 17.0 and 7.5; top-8
// sigmoid, 4096 6.5 and 7.9, 8192 9.1 and 8.2, 32768 24.8 and 12.3; 256 experts
// in 8 groups, 4096 9.7 and 14.1, 8192 15.3 and 15.5, 16381 24.5 and 21.6, 32768
// 42.8 and 29.7).
constexpr int kEighthsFrom = 8192;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896341f;

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
__device__ __forceinline__ float clean(float z) { return fminf(fmaxf(z, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// What the chosen scores are proportional to, `top` being the largest chosen
// logit: scores that would vanish in fp32 keep their ratios.  Where all chosen
// sigmoids lie below e^-30 they are exponentials to 13 digits; above it they are
// taken 2^48 times, which their quotients do not show, and those that fp32 holds
// no longer in full (below e^-80) from the square of their root.
__device__ __forceinline__ float proportion(float z, float top, bool sig) {
  if (!sig || top < -30.f) return expf(z - top);
  constexpr float up = 281474976710656.f;  // 2^48
  if (z >= -80.f) return sigmoid(z) * up;
  const float root = expf(0.5f * z);
  return root * up * root;
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

__device__ __forceinline__ float lower(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ float upper(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double lower(double a, double b) { return a < b ? a : b; }
__device__ __forceinline__ double upper(double a, double b) { return a > b ? a : b; }

template <class F>
__device__ __forceinline__ void top_two(F a, F& first, F& second) {
  second = upper(second, lower(first, a));
  first = upper(first, a);
}

// Half a group's worth, which passes no type's end where its two terms do not.
template <class F>
__device__ __forceinline__ F half_worth(F first, F second) {
  const F half = static_cast<F>(0.5);
  return second == -INFINITY ? half * first : half * first + half * second;
}

// That of the lanes that share a group, `lanes` neighbours (a power of two).
template <class F>
__device__ __forceinline__ F group_worth(F first, F second, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) {
    const F f = __shfl_xor_sync(kFull, first, o), s = __shfl_xor_sync(kFull, second, o);
    top_two(f, first, second);
    top_two(s, first, second);
  }
  return half_worth(first, second);
}

// How many of the groups (one every `lanes` lanes, a power of two) are better
// than this lane's group g.  Every lane of the warp takes part; those of a
// group share its comparisons.
template <class F>
__device__ __forceinline__ int group_rank(F worth, int g, int groups, int lanes, int lane) {
  int rank = 0;
  for (int h = lane & (lanes - 1), n = 0; n < groups; h += lanes, n += lanes) {
    const F w = __shfl_sync(kFull, worth, (h * lanes) & 31);
    rank += h < groups && (w > worth || (w == worth && h < g));
  }
  for (int o = 1; o < lanes; o <<= 1) rank += __shfl_xor_sync(kFull, rank, o);
  return rank;
}

// c in 64 bits; m and total: the softmax's reference and sum.
__device__ __noinline__ double exact_choice(float z, float b, int sig, float m, double total) {
  if (z == -INFINITY) return -INFINITY;
  const double e = exp(sig ? -static_cast<double>(z) : static_cast<double>(z) - m);
  const double c = (sig ? 1.0 : e) / (sig ? 1.0 + e : total) + b;
  return isnan(c) ? -static_cast<double>(INFINITY) : c;
}

// The softmax's sum in 64 bits.
__device__ __noinline__ double exact_total(const float* row, int E, int lane, float m) {
  double sum = 0.0;
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const float z = clean(row[e]);
    if (z > -INFINITY) sum += exp(static_cast<double>(z) - m);
  }
  return warp_sum(sum);
}

// The whole choice by the definition, in 64 bits, where more than a warp's
// lanes come into question: slot j's expert from lane j mod 32.
__device__ __noinline__ void choose_exactly(const Choice& p, const float* row, int lane, float m, int32_t* out_i) {
  const int n = (p.E + 31) >> 5;
  double c[32];
  const double total = p.sig ? 1.0 : exact_total(row, p.E, lane, m);
  for (int i = 0; i < n; ++i) c[i] = i * 32 + lane < p.E ? clean(row[i * 32 + lane]) : -INFINITY;
  uint32_t left = 0;  // of this lane's experts
  for (int i = 0; i < n; ++i)
    if (i * 32 + lane < p.E) left |= 1u << i;
  const bool groups = p.top_groups < p.groups;
  auto choice = [&](int i) {
    return exact_choice(static_cast<float>(c[i]), p.bias ? p.bias[i * 32 + lane] : 0.f, p.sig, m, total);
  };
  if (p.bias)  // else the logits order the experts, and the scores the groups
    for (int i = 0; i < n; ++i)
      if ((left >> i) & 1u) c[i] = choice(i);
  if (groups) {
    double worth = -INFINITY;  // of group `lane`
    for (int g = 0; g < p.groups; ++g) {
      double first = -INFINITY, second = -INFINITY;
      for (int i = 0; i < n; ++i)
        if (((left >> i) & 1u) && (i * 32 + lane) / p.size == g) top_two(p.bias ? c[i] : choice(i), first, second);
      const double w = group_worth(first, second, 32);
      if (lane == g) worth = w;
    }
    const int rank = group_rank(worth, lane, p.groups, 1, lane);
    const uint32_t stay = __ballot_sync(kFull, rank < p.top_groups && lane < p.groups);
    for (int i = 0; i < n; ++i) {
      const int e = i * 32 + lane;
      if (e < p.E && !((stay >> (e / p.size)) & 1u)) left &= ~(1u << i);
    }
  }
  for (int j = 0; j < p.k; ++j) {
    double top = -INFINITY;
    int at = 0x7fffffff;
    for (int i = 0; i < n; ++i)
      if (((left >> i) & 1u) && (at == 0x7fffffff || c[i] > top)) top = c[i], at = i * 32 + lane;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double v = __shfl_xor_sync(kFull, top, o);
      const int q = __shfl_xor_sync(kFull, at, o);
      if (q != 0x7fffffff && (at == 0x7fffffff || v > top || (v == top && q < at))) top = v, at = q;
    }
    if ((at & 31) == lane) left &= ~(1u << (at >> 5));
    if (lane == (j & 31)) out_i[j] = at;
  }
}

// A choice's key: its place v in [1, 2], whose 23 bits of fraction are steps of
// the range, above the register i that holds it (a lower one is the larger
// key).  Minus infinity, at the place just below 1, is below all numbers; 0 is
// no expert.
constexpr uint32_t kMasked = 1u << 5;
constexpr float kMaskedPlace = 0.99999994f;
__device__ __forceinline__ uint32_t pack(float v, int i) {
  return ((__float_as_uint(v) - 0x3f800000u + 2u) << 5) + (31 - i);
}

// One token by one warp; b: the bias of the lane's experts, most: the largest
// finite one in magnitude, mem: room for the groups' scores.  FULL: E is 32 NPL.
template <int NPL, bool GROUPS, bool FULL>
__device__ __forceinline__ void route_by_warp(const Choice& p, int64_t t, const float (&b)[NPL], float most, float* mem,
                                              int lane) {
  const bool sig = p.sig, biased = p.bias != nullptr;
  auto there = [&](int i) { return FULL || i * 32 + lane < p.E; };
  // Steps that two keys may be off by together.  Without a bias: places by the
  // logit's distance from the largest, monotone, so only equal ones are open.
  // With one, in steps of 2^-22 of the range: a sigmoid is off by 1 (its
  // exponential's argument, ex2 and rcp to 2^-22.5 and 2^-23), the sum and its
  // place by 0.7, for each of the two; a softmax also by its sum's roundings (a
  // lane's NPL terms, five more, and its inverse).
  const float open_steps = sig ? 6.f : 10.f + NPL / 4;
  const uint32_t tol = (biased ? (sig ? 6u : 10u + NPL / 4) << 5 : 0u) + 31;
  const float* row = p.logits + t * p.E;
  float z[NPL], m = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < NPL; ++i) z[i] = there(i) ? __ldg(row + i * 32 + lane) : -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    z[i] = clean(z[i]);
    m = fmaxf(m, z[i]);
  }
  if (!sig || !biased) m = warp_max(m);
  float weigh = 0.f;  // what exponentials become weights by, where the whole softmax does
  if (!sig && !p.renorm) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) sum += expf(z[i] - m);
    sum = warp_sum(sum);
    weigh = sum > 0.f ? p.scale / sum : 0.f;
  }
  uint32_t key[NPL];
  float step = 0.f, s[NPL];
  if (GROUPS || biased) {
    float inv = 1.f;  // of the softmax's sum
    if (sig) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) s[i] = rcp_approx(1.f + ex2_approx(z[i] * -kLog2e));
    } else {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        s[i] = ex2_approx((z[i] - m) * kLog2e);
        sum += s[i];
      }
      sum = warp_sum(sum);
      inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) s[i] *= inv;
    }
    const float range = most + inv;  // a softmax's largest score is its largest exponential's, 1
    step = range * 2.3841858e-7f;
    const float half = 0.49999f / range;  // all numbers' places lie above 1
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      s[i] = z[i] == -INFINITY ? -INFINITY : fmaxf(s[i] + b[i], -INFINITY);  // the choice; NaN is minus infinity
      key[i] = pack(fmaxf(fminf(fmaf(s[i], half, 1.5f), 2.f), kMaskedPlace), i);
    }
  }
  if (!biased) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      key[i] = pack(z[i] == -INFINITY ? kMaskedPlace : fmaxf(fmaf(z[i] - m, 1.f / 32.f, 2.f), 1.f), i);
  }
  if (!FULL) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (!there(i)) key[i] = 0;
  }

  double total = -1.0;  // the softmax's sum in 64 bits, once it is needed
  // Rows whose experts are all alike (padding) are in order already.
  auto rows_alike = [&]() {
    bool alike = true;
    const float z0 = clean(__ldg(row)), b0 = biased ? __ldg(p.bias) : 0.f;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) alike &= clean(__ldg(row + e)) == z0 && (!biased || __ldg(p.bias + e) == b0);
    return __all_sync(kFull, alike) != 0;
  };
  auto exactly = [&](int e) {
    return exact_choice(clean(__ldg(row + e)), biased ? __ldg(p.bias + e) : 0.f, sig, m, total);
  };
  auto need_total = [&]() {
    if (!sig && total < 0.0) total = exact_total(row, p.E, lane, m);
  };
  if (GROUPS) {
    const int pad = p.stride - p.size;
    int at[NPL];
    __syncwarp();  // the last token's have been read
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = i * 32 + lane;
      at[i] = static_cast<int>((e * p.inv_size) >> 20);
      if (there(i)) mem[e + at[i] * pad] = s[i];
    }
    __syncwarp();
    const int g = lane / p.lanes, r = lane & (p.lanes - 1);
    const float* mine = mem + g * p.stride;
    float first = -INFINITY, second = -INFINITY;
    if (g < p.groups) {
#pragma unroll 4
      for (int o = r; o < p.size; o += p.lanes) top_two(mine[o], first, second);
    }
    const float worth = group_worth(first, second, p.lanes);
    int rank = group_rank(worth, g, p.groups, p.lanes, lane);
    bool stays = rank < p.top_groups && g < p.groups;
    // the worst that stays against the best that goes
    const float low = float_of(__reduce_min_sync(kFull, stays ? key_of(worth) : kFull));
    const float high = float_of(__reduce_max_sync(kFull, g < p.groups && !stays ? key_of(worth) : 0u));
    const float open = open_steps * step;  // as far as two choices may be off, and two halves of two choices
    if (low - high <= open && !rows_alike()) {
      // the groups' two best in 64 bits: of those that may be among them
      need_total();
      const float least = second - open;
      double f = -INFINITY, n = -INFINITY;
      int o = g < p.groups ? r : p.size;
      for (;;) {
        while (o < p.size && !(mine[o] >= least)) o += p.lanes;
        if (!__any_sync(kFull, o < p.size)) break;
        if (o < p.size) {
          top_two(exactly(g * p.size + o), f, n);
          o += p.lanes;
        }
      }
      rank = group_rank(group_worth(f, n, p.lanes), g, p.groups, p.lanes, lane);
      stays = rank < p.top_groups && g < p.groups;
    }
    const uint32_t lanes_in = __ballot_sync(kFull, stays);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (!((lanes_in >> ((at[i] * p.lanes) & 31)) & 1u)) key[i] = 0;  // (past the last expert it is 0 already)
  }

  int32_t* out_i = p.expert_idx + t * p.k;
  float* out_w = p.gate_w + t * p.k;
  uint32_t own = 0, second = 0;  // this lane's best two
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    second = max(second, min(own, key[i]));
    own = max(own, key[i]);
  }
  uint32_t used = 0;  // lanes whose second one has come up: behind it they look again
  uint32_t last = kFull, gap = kFull;  // gap: the smallest between neighbours
  int mine = 0;                        // slot `lane`'s expert
  int n = 0;                           // slots taken: k, and those behind whose order with the last is open
  uint32_t best = __reduce_max_sync(kFull, own);
  auto take = [&]() {
    last = best;
    const int src = __ffs(__ballot_sync(kFull, own == best)) - 1;  // equal keys: the lowest lane has the lowest expert
    const int e = static_cast<int>(31 - (best & 31)) * 32 + src;
    if (n < 32) mine = lane == n ? e : mine;
    else if (lane == (n & 31)) out_i[n] = e;
    if ((used >> src) & 1u) {
      uint32_t next = 0;  // the lane's best below: of the differences that wrap the largest
#pragma unroll
      for (int i = 0; i < NPL; ++i) next = max(next, key[i] - best);
      next = next & 0x80000000u ? next + best : 0u;
      own = lane == src ? next : own;
    } else {
      own = lane == src ? second : own;
      used |= 1u << src;
    }
    best = __reduce_max_sync(kFull, own);
    gap = min(gap, last - best);
    ++n;
  };
  while (n < p.k) take();
  // an order is open between numbers within tol (masked ones go by their place, which the slots below show, too)
  const bool near = gap <= tol;
  while (last - best <= tol && best >= 2 * kMasked && n < 32) take();
  if (near && !rows_alike()) {
    if (n < 32) {  // one slot a lane: their order in 64 bits
      if (biased) need_total();
      double c = -INFINITY;
      if (lane < n) c = biased ? exactly(mine) : static_cast<double>(clean(__ldg(row + mine)));
      int rank = 0;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const double v = __shfl_sync(kFull, c, j);
        const int e = __shfl_sync(kFull, mine, j);
        rank += v > c || (v == c && e < mine);
      }
      if (lane < n && rank < p.k) out_i[rank] = mine;
      __syncwarp();
    } else {
      choose_exactly(p, row, lane, m, out_i);
    }
    if (lane < p.k) mine = out_i[lane];
  }

  // slot j's weight in lane j mod 32, which wrote its expert
  float top = -INFINITY;
  if (p.renorm) {
    for (int j = lane; j < p.k; j += 32) top = fmaxf(top, clean(__ldg(row + (j < 32 ? mine : out_i[j]))));
    top = warp_max(top);
  }
  float sum = 0.f, only = 0.f;
  for (int j = lane; j < p.k; j += 32) {
    const int e = j < 32 ? mine : out_i[j];
    if (j < 32) out_i[j] = e;
    const float v = clean(__ldg(row + e));
    float w = 0.f;
    if (v > -INFINITY) w = p.renorm ? proportion(v, top, sig) : sig ? sigmoid(v) * p.scale : expf(v - m) * weigh;
    sum += w;
    if (!p.renorm) out_w[j] = w;
    else if (p.k > 32) out_w[j] = w;
    else only = w;
  }
  if (p.renorm) {
    sum = warp_sum(sum);
    const float f = sum > 0.f ? p.scale / sum : 0.f;
    for (int j = lane; j < p.k; j += 32) out_w[j] = (p.k > 32 ? out_w[j] : only) * f;
  }
}

template <int NPL, bool FULL>
__device__ __forceinline__ float load_bias(const Choice& p, float (&b)[NPL], int lane) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    b[i] = p.bias && (FULL || i * 32 + lane < p.E) ? __ldg(p.bias + i * 32 + lane) : 0.f;
    most = fmaxf(most, fabsf(b[i]) < INFINITY ? fabsf(b[i]) : 0.f);
  }
  return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(most)));
}

// A warp walks its tokens with the bias in registers.
template <int NPL, bool GROUPS, bool FULL>
__global__ void __launch_bounds__(kWarps * 32, NPL <= 8 ? 4 : NPL <= 16 ? 3 : 2)
    route_balanced_kernel(const __grid_constant__ Choice p) {
  extern __shared__ float group_mem[];  // [kWarps][groups * stride]
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  float b[NPL];
  const float most = load_bias<NPL, FULL>(p, b, lane);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < p.T;
       t += static_cast<int64_t>(gridDim.x) * kWarps)
    route_by_warp<NPL, GROUPS, FULL>(p, t, b, most, group_mem + (threadIdx.x >> 5) * p.groups * p.stride, lane);
}

// Four tokens a warp, eight lanes each: what is done once a token, the groups'
// merging, the slots and their weights, then serves four.  For E = 32 NI up to
// 256, k up to 8 and groups of whole 32s (G of them, 1: none), rows 16 bytes
// apart; lane q of a token has experts 32 i + 4 q + r.  Keys hold the expert's
// number itself, under a place of 22 bits, and a token whose order is open, or
// with experts ruled out among its best, is left to the whole warp.  (Settling
// it among the eight lanes took longer, 15 us against 11 at 1024 x 256: it is
// more code that was not run before.)
template <int NI, int G>
__device__ __noinline__ void route_again(const Choice& p, int64_t t, float* mem, int lane) {
  float b[NI];
  const float most = load_bias<NI, true>(p, b, lane);
  route_by_warp<NI, (G > 1), true>(p, t, b, most, mem, lane);
}

// The segment's largest: of eight neighbouring lanes.
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ uint32_t max8(uint32_t v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

constexpr uint32_t kLive8 = 2u << 8;  // the lowest key of a number
__device__ __forceinline__ uint32_t pack8(float place, int e) {
  return ((__float_as_uint(place) - 0x3f800000u + 2u) << 8) + (255 - e);
}

template <int NI, int G>
__global__ void __launch_bounds__(kWarps * 32, 4) route_eighths_kernel(const __grid_constant__ Choice p) {
  extern __shared__ float group_mem[];  // [kWarps][groups * stride], for route_again()
  dmoe::pdl_wait();
  dmoe::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, q = lane & 7, seg = lane >> 3;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * 4;
  if (t0 >= p.T) return;
  const bool there = t0 + seg < p.T;
  const int64_t t = there ? t0 + seg : p.T - 1;  // (the last token again, and written by none)
  const float* row = p.logits + t * p.E;
  const bool sig = p.sig, biased = p.bias != nullptr;
  float s[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(row) + 8 * i + q);
    s[i][0] = clean(v.x), s[i][1] = clean(v.y), s[i][2] = clean(v.z), s[i][3] = clean(v.w);
  }
  float m = -FLT_MAX;
  if (!sig || !biased) {
#pragma unroll
    for (int i = 0; i < NI; ++i) m = fmaxf(m, fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3])));
    m = max8(m);
  }
  float weigh = 0.f;  // what exponentials become weights by, where the whole softmax does
  if (!sig && !p.renorm) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) sum += expf(s[i][r] - m);
    sum = sum8(sum);
    weigh = sum > 0.f ? p.scale / sum : 0.f;
  }
  // In steps of 2^-21 of the range, half as many as the whole warp's, and one
  // for the coarser places; a lane adds 4 NI terms of a softmax's sum, and three
  // more.
  uint32_t tol = 255;
  float open = 0.f, quarter = 0.f;
  bool near = false;
  if (G > 1 || biased) {
    float inv = 1.f;
    if (!sig) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum += ex2_approx((s[i][r] - m) * kLog2e);
      sum = sum8(sum);
      inv = sum > 0.f ? 1.f / sum : 0.f;
    }
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
      if (biased) b = __ldg(reinterpret_cast<const float4*>(p.bias) + 8 * i + q);
      const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        most = fmaxf(most, fabsf(bb[r]) < INFINITY ? fabsf(bb[r]) : 0.f);  // (an infinite one's place is the range's end)
        const float z = s[i][r];
        const float v = sig ? rcp_approx(1.f + ex2_approx(z * -kLog2e)) : ex2_approx((z - m) * kLog2e) * inv;
        s[i][r] = z == -INFINITY ? -INFINITY : fmaxf(v + bb[r], -INFINITY);  // the choice; NaN is minus infinity
      }
    }
    most = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(most)));
    const float range = most + inv;
    open = (sig ? 5.f : 12.f) * 4.7683716e-7f * range;
    quarter = 0.24999f / range;  // all numbers' places lie above 1
    if (biased) tol += (sig ? 5u : 12u) << 8;
  }
  uint32_t in = 255;  // the groups that stay, a bit at lane h 8 / G
  if (G > 1) {
    constexpr int PER = NI / G;  // rows of 32 experts of a group
    float f[G], g[G];            // the best two of each group: the lane's, then of more and more lanes
#pragma unroll
    for (int h = 0; h < G; ++h) {
      f[h] = g[h] = -INFINITY;
#pragma unroll
      for (int i = h * PER; i < (h + 1) * PER; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) top_two(s[i][r], f[h], g[h]);
    }
    // lanes that part with half of the groups at a step: lane q ends with group q G / 8
#pragma unroll
    for (int o = 4, n = G; o > 0; o >>= 1) {
      const bool high = (q & o) != 0;
      if (n > 1) {
        n /= 2;
#pragma unroll
        for (int h = 0; h < n; ++h) {
          const float f2 = __shfl_xor_sync(kFull, high ? f[h] : f[h + n], o);
          const float g2 = __shfl_xor_sync(kFull, high ? g[h] : g[h + n], o);
          const float f1 = high ? f[h + n] : f[h], g1 = high ? g[h + n] : g[h];
          f[h] = fmaxf(f1, f2);
          g[h] = fmaxf(fminf(f1, f2), fmaxf(g1, g2));
        }
      } else {
        const float f2 = __shfl_xor_sync(kFull, f[0], o), g2 = __shfl_xor_sync(kFull, g[0], o);
        const float f1 = f[0];
        f[0] = fmaxf(f1, f2);
        g[0] = fmaxf(fminf(f1, f2), fmaxf(g[0], g2));
      }
    }
    const float worth = half_worth(f[0], g[0]);
    const int mine = q / (8 / G);
    int rank = 0;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float w = __shfl_sync(kFull, worth, (lane & 24) + h * (8 / G));
      rank += w > worth || (w == worth && h < mine);
    }
    const bool stays = rank < p.top_groups;
    const float low = -max8(stays ? -worth : -INFINITY), high = max8(stays ? -INFINITY : worth);
    near |= low - high <= open;
    in = __ballot_sync(kFull, stays) >> (lane & 24);
  }
  uint32_t key[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const bool here = G == 1 || ((in >> (i / (NI / G) * (8 / G))) & 1u);
    if (G > 1 && !biased) {  // the logits, whose place the groups' scores have taken
      const float4 v = __ldg(reinterpret_cast<const float4*>(row) + 8 * i + q);
      s[i][0] = clean(v.x), s[i][1] = clean(v.y), s[i][2] = clean(v.z), s[i][3] = clean(v.w);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float c = s[i][r];
      const float place = biased ? fminf(fmaxf(fmaf(c, quarter, 1.25f), kMaskedPlace), 1.5f)
                          : c == -INFINITY ? kMaskedPlace : fmaxf(fmaf(c - m, 1.f / 64.f, 1.5f), 1.f);
      key[i][r] = here ? pack8(place, 32 * i + 4 * q + r) : 0u;
    }
  }
  uint32_t own = 0, second = 0;  // the lane's best two
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      second = max(second, min(own, key[i][r]));
      own = max(own, key[i][r]);
    }
  bool used = false;  // the second one has come up: behind it the lane looks again
  uint32_t slot = 0, gap = kFull;
  uint32_t best = max8(own);
  for (int j = 0; j < p.k; ++j) {
    slot = q == j ? best : slot;
    const uint32_t last = best;
    const bool owner = own == best;  // keys are all different
    if (__any_sync(kFull, owner && used)) {
      uint32_t next = 0;  // the lane's best below: of the differences that wrap the largest
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) next = max(next, key[i][r] - best);
      second = owner && used ? (next & 0x80000000u ? next + best : 0u) : second;
    }
    own = owner ? second : own;
    used |= owner;
    best = max8(own);
    gap = min(gap, last - best);
    near |= last < kLive8;
  }
  near |= gap <= tol;
  // the slots' weights, one a lane
  const int e = static_cast<int>(255 - (slot & 255));
  const bool mine = q < p.k && slot != 0;
  const float v = mine ? clean(__ldg(row + e)) : -INFINITY;
  float w = 0.f;
  if (p.renorm) {
    const float top = max8(v);
    if (v > -INFINITY) w = proportion(v, top, sig);
    const float sum = sum8(w);
    w *= sum > 0.f ? p.scale / sum : 0.f;
  } else if (v > -INFINITY) {
    w = sig ? sigmoid(v) * p.scale : expf(v - m) * weigh;
  }
  if (mine && there && !near) {
    p.expert_idx[t * p.k + q] = e;
    p.gate_w[t * p.k + q] = w;
  }
  uint32_t again = __ballot_sync(kFull, near && there && q == 0);
  float* mem = group_mem + (threadIdx.x >> 5) * p.groups * p.stride;
  while (again) {
    const int at = __ffs(again) - 1;
    again &= again - 1;
    route_again<NI, G>(p, t0 + (at >> 3), mem, lane);
  }
}

// With G_e the d_gate of the slot that holds expert e (0 where none does) and,
// for renormalised weights, r the weights before their scaling:
//   softmax  dz = scale p (G - sum G p)       renormalised  scale r (G - sum G r)
//   sigmoid  dz = scale G s (1 - s)           renormalised  scale r (1 - s) (G - sum G r)
// Only the softmax without renormalisation reaches experts that were not
// chosen: elsewhere the slots' logits are all that is read, and the row is
// zeros but for them.  Slot j is lane j mod 32's.
template <bool ALL>
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
  float* out = d_logits + t * E;
  const int32_t* idx = expert_idx + t * k;
  const float* dg = d_gate + t * k;
  auto slot = [&](int j, float& z, float& g) {  // a slot's expert, -1 for none
    const int e = __ldg(idx + j);
    if (e < 0 || e >= E) {
      dmoe::raise_error(err, DMOE_SITE_ROUTE_INDEX | DMOE_ERR_DEVICE);
      return -1;
    }
    z = clean(__ldg(row + e));
    g = __ldg(dg + j);
    return e;
  };
  if (!ALL) {
    if (((E | static_cast<int>(reinterpret_cast<uintptr_t>(d_logits) >> 2)) & 3) == 0) {
      for (int e = lane; e < E / 4; e += 32) reinterpret_cast<float4*>(out)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int e = lane; e < E; e += 32) out[e] = 0.f;
    }
  }
  // the first 32 slots stay in registers
  float z0 = -INFINITY, g0 = 0.f;
  const int e0 = lane < k ? slot(lane, z0, g0) : -1;
  float m = -FLT_MAX, sum = 0.f, dot = 0.f;
  if (ALL) {
    for (int e = lane; e < E; e += 32) m = fmaxf(m, clean(__ldg(row + e)));
    m = warp_max(m);
    for (int e = lane; e < E; e += 32) sum += expf(clean(__ldg(row + e)) - m);
  } else if (renorm) {
    m = z0;
    for (int j = lane + 32; j < k; j += 32) {
      float z = -INFINITY, g;
      slot(j, z, g);
      m = fmaxf(m, z);
    }
    m = warp_max(m);
  }
  auto weight = [&](float z) { return z == -INFINITY ? 0.f : ALL ? expf(z - m) : proportion(z, m, sig); };
  float mean = 0.f, inv = 0.f;
  if (ALL || renorm) {
    const float w = e0 >= 0 ? weight(z0) : 0.f;
    dot = g0 * w;
    if (!ALL) sum = w;
    for (int j = lane + 32; j < k; j += 32) {
      float z, g;
      if (slot(j, z, g) < 0) continue;
      const float w1 = weight(z);
      dot = fmaf(g, w1, dot);
      if (!ALL) sum += w1;
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot);
    inv = sum > 0.f ? 1.f / sum : 0.f;
    mean = dot * inv;
  }
  if (ALL) {
    const float f = -scale * inv * mean;
    for (int e = lane; e < E; e += 32) out[e] = expf(clean(__ldg(row + e)) - m) * f;
  }
  __syncwarp();  // the row is there before its slots
  for (int j = lane; j < k; j += 32) {
    float z = z0, g = g0;
    const int e = j < 32 ? e0 : slot(j, z, g);
    if (e < 0) continue;
    float d;
    const float q = expf(-fabsf(z)), half = 1.f / (1.f + q);
    if (ALL || renorm) {
      const float w = weight(z);
      d = w == 0.f ? 0.f : scale * (w * inv) * (g - mean);
      if (sig) d *= z > 0.f ? q * half : half;  // 1 - s
    } else {
      d = scale * g * (q * half) * half;
    }
    out[e] = d;
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
  int sms;
  cudaStream_t st;
  template <int NPL>
  cudaError_t operator()() const {
    if constexpr (NPL >= 2 && NPL <= 8) {
      // four tokens a warp where it has that many
      const bool even = p.E == 32 * NPL && p.k <= 8 && dmoe::aligned16(p.logits) && dmoe::aligned16(p.bias);
      const int groups = p.top_groups == p.groups ? 1 : p.groups;
      if (even && (p.k == 1 || p.T >= kEighthsFrom)) {
        if (groups == 1) return eighths<NPL, 1>();
        if (groups == 2) return eighths<NPL, 2>();
        if constexpr (NPL >= 4)
          if (groups == 4) return eighths<NPL, 4>();
        if constexpr (NPL >= 8)
          if (groups == 8) return eighths<NPL, 8>();
      }
    }
    return p.E == 32 * NPL ? launch<NPL, true>() : launch<NPL, false>();
  }
  template <int NI, int G>
  cudaError_t eighths() const {
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.T) + 4 * kWarps - 1) / (4 * kWarps)));
    const size_t smem = G > 1 ? sizeof(float) * kWarps * p.groups * p.stride : 0;
    return dmoe::launch_pdl(route_eighths_kernel<NI, G>, grid, dim3(kWarps * 32), smem, st, p);
  }
  template <int NPL, bool FULL>
  cudaError_t launch() const {
    const unsigned resident = static_cast<unsigned>(sms * (NPL <= 8 ? 4 : NPL <= 16 ? 3 : 2));
    const dim3 grid(std::min(grid_of(p.T).x, resident)), block(kWarps * 32);
    if (p.top_groups == p.groups) return dmoe::launch_pdl(route_balanced_kernel<NPL, false, FULL>, grid, block, 0, st, p);
    const size_t smem = sizeof(float) * kWarps * p.groups * p.stride;  // at most (1024 + 32) * 32 bytes
    return dmoe::launch_pdl(route_balanced_kernel<NPL, true, FULL>, grid, block, smem, st, p);
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
  if (!logits || !expert_idx || !gate_w || gate_w == logits) return DMOE_ERR_INVALID_ARG;
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
  const cudaError_t e = by_experts(E, ForwardCall{p, di.sm_count, dmoe::as_stream(stream)});
  if (e != cudaSuccess) return dmoe::cuda_status(e);
  dmoe::count_launches(1);
  return DMOE_OK;
}

DMOE_API dmoe_status dmoe_route_balanced_backward(const float* logits, const int32_t* expert_idx, const float* d_gate,
                                                  int T, int E, int k, int scores, int renormalize, float scale,
                                                  float* d_logits, dmoe_stream_t stream) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > E || bad_scores(scores) || !isfinite(scale)) return DMOE_ERR_INVALID_ARG;
  if (T == 0) return DMOE_OK;
  if (!logits || !expert_idx || !d_gate || !d_logits || d_logits == logits || d_logits == d_gate) return DMOE_ERR_INVALID_ARG;
  if (misaligned4(logits) || misaligned4(expert_idx) || misaligned4(d_gate) || misaligned4(d_logits))
    return DMOE_ERR_INVALID_ARG;
  dmoe::DeviceInfo di;
  dmoe_status st = dmoe::device_info(&di);
  if (st != DMOE_OK) return st;
  const int sig = scores == DMOE_SCORES_SIGMOID, renorm = renormalize ? 1 : 0;
  auto kern = sig || renorm ? route_balanced_backward_kernel<false> : route_balanced_backward_kernel<true>;
  const cudaError_t e = dmoe::launch_pdl(kern, grid_of(T), dim3(kWarps * 32), 0, dmoe::as_stream(stream), logits,
                                         expert_idx, d_gate, T, E, k, sig, renorm, scale, d_logits, di.err_word);
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
