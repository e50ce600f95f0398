// Group-limited routing on given logits, and its gradient.
//
// For every token with logits l [E] (gate, selection bias, top-k and
// renormalisation as in SigmoidRouter.forward of the "moe-200m-qwen3-100b"
// README and the qwen3 preset of SpecForge PR #930; groups and the score-space
// bias of the "noaux_tc" router named on the page-3 model card, which prints
// no code for it):
//   s = sigmoid(l) or softmax_E(l);  key = (l or s) + bias;
//   an expert is eligible when l > -inf, s is a number and key > -inf;
//   group score = largest key, or the sum of the two largest;
//   the topk_group best groups stay, then the top_k best of their experts;
//   w = scale s / (sum of the chosen s + 1e-9), or scale s.
// The selection is the one fp64 keys give, ties to the lower id.  Keys are
// compared in fp32 first.  Groups, and picks, whose fp32 values are closer than
// their error are put in order by fp64 values of theirs alone (a few tokens
// in a thousand; deciding such a token anew as a whole, 10 us, showed as the
// tail of every launch); a token with values fp32 cannot rank is decided
// again as a whole in fp64.
//
// Bound by the selection's instructions for many tokens: 4 tokens per warp, 8
// lanes each, so that the cross-lane steps of the top-k serve four tokens at a
// time.  [131072, 256] fp32, 8 groups of which 4, top-8: 76 us, 1.8 TB/s of
// logits, about 1950 instructions a warp (of 82 us with blocks of four warps,
// the rounds of the top-k took 25, the groups 18, the keys 12, the margins 1).
// [16384, 128]: 9.8 us.  One token: 4 us, of which the launch is half.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kMaxE = 256;
constexpr int kMaxK = 32;
constexpr unsigned kFull = 0xffffffffu;

template <typename L>
__device__ __forceinline__ double to_f64(L v) { return static_cast<double>(v); }
template <>
__device__ __forceinline__ double to_f64<__nv_bfloat16>(__nv_bfloat16 v) {
  return static_cast<double>(__bfloat162float(v));
}
template <typename L>
__device__ __forceinline__ float to_f32(L v) { return static_cast<float>(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// Shared-memory position of expert e: 4 floats of padding per 32, so that
// the 8 lanes of a token, a group or E/8 experts apart, read 16-byte pieces
// from different banks.
__device__ __forceinline__ int at(int e) { return e + ((e >> 5) << 2); }
// The expert of a pick: positions are below 36 * 8, and p / 36 is taken by way
// of a multiplication; a pick's position is its block's place and, from bit 16, the
// expert in the block.
__device__ __forceinline__ int expert_at(int x) {
  const int p = (x & 0xffff) + (x >> 16);
  return p - 4 * ((p * 1821) >> 16);
}

// A key above -inf as an integer in the keys' order, never 0.
__device__ __forceinline__ unsigned long long ordered(double v) {
  const long long b = __double_as_longlong(v + 0.0);   // -0 as 0
  return static_cast<unsigned long long>(b < 0 ? ~b : b | (1ll << 63));
}

// The softmax of a row in fp64, by one warp: its maximum, the divisor, and
// e^(l - m) of the lane's experts lane + 32 i.  All loads, then all exponentials
// are in flight together: this runs for single tokens, where latency counts.
template <typename L>
__device__ __forceinline__ void softmax_f64(const RouteShape& a, const L* __restrict__ row,
                                            int lane, double& m, double& sum, double (&x)[8]) {
  double l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    l[i] = lane + 32 * i < a.E ? to_f64(row[lane + 32 * i]) : -INFINITY;
  m = l[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmax(m, l[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, o));
  if (m == -INFINITY) m = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = exp(l[i] - m);   // 0 past E
  sum = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
}

// The fp64 key of expert e (-inf where it is not eligible).
template <typename L>
__device__ __forceinline__ double key_f64(const RouteShape& a, const L* __restrict__ row,
                                          const float* __restrict__ bias, int e, double m,
                                          double sum) {
  const double l = to_f64(row[e]);
  double key = l;
  if (a.space == 1) {
    const double x = exp(a.gate == 0 ? l - m : -l);
    key = a.gate == 0 ? x / sum : 1.0 / (1.0 + x);
  }
  if (bias != nullptr) key += static_cast<double>(bias[e]);
  return l > -INFINITY && key > -INFINITY ? key : -INFINITY;
}

// The two largest of (m1 >= m2) and another pair.
__device__ __forceinline__ void top2(double& m1, double& m2, double o1, double o2) {
  m2 = fmax(fmin(m1, o1), fmax(m2, o2));
  m1 = fmax(m1, o1);
}

// The groups of one token whose fp32 scores (picks: error, score) overlap the
// border [lo, hi] between the chosen and the others, by fp64 scores; returns the
// chosen groups.  By the whole warp: one group after another.
template <typename L>
__device__ __noinline__ unsigned choose_groups_f64(const RouteShape& a, const L* __restrict__ row,
                                                   const float* __restrict__ bias, int lane,
                                                   float lo, float hi, const int2* picks) {
  double m = 0.0, sum = 1.0;
  if (a.gate == 0 && a.space == 1) {
    double x[8];
    softmax_f64(a, row, lane, m, sum, x);
  }
  bool open = false, in = false;
  if (lane < a.groups) {
    const float err = __int_as_float(picks[lane].x), sc = __int_as_float(picks[lane].y);
    open = sc > -INFINITY && sc + err >= lo && sc - err <= hi;
    in = sc > -INFINITY && sc - err > hi;
  }
  const unsigned todo = __ballot_sync(kFull, open);
  unsigned chosen = __ballot_sync(kFull, in);
  double score = -INFINITY;
  for (unsigned g = todo; g != 0u; g &= g - 1u) {
    const int gi = __ffs(g) - 1;
    double m1 = -INFINITY, m2 = -INFINITY;
    for (int e = lane; e < a.per; e += 32)
      top2(m1, m2, key_f64(a, row, bias, gi * a.per + e, m, sum), -INFINITY);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      top2(m1, m2, __shfl_xor_sync(kFull, m1, o), __shfl_xor_sync(kFull, m2, o));
    if (lane == gi) score = a.group_score == 2 && m2 > -INFINITY ? m1 + m2 : m1;
  }
  int rank = __popc(chosen);
  for (unsigned g = todo; g != 0u; g &= g - 1u) {
    const int h = __ffs(g) - 1;
    const double o = __shfl_sync(kFull, score, h);
    rank += (o > score || (o == score && h < lane)) ? 1 : 0;
  }
  chosen |= __ballot_sync(kFull, open && rank < a.topk_group);
  return chosen;
}

// The `count` <= 32 best experts of one token by fp32 keys (picks: position,
// key), put into the order of their fp64 keys by the whole warp: each lane
// counts the better ones.
template <typename L>
__device__ __noinline__ void order_picks_f64(const RouteShape& a, const L* __restrict__ row,
                                             const float* __restrict__ bias, int lane, int count,
                                             int2* picks) {
  double m = 0.0, sum = 1.0;
  if (a.gate == 0 && a.space == 1) {
    double x[8];
    softmax_f64(a, row, lane, m, sum, x);
  }
  int2 p = make_int2(0, 0);
  double key = -INFINITY;
  int e = kMaxE;
  if (lane < count) {
    p = picks[lane];
    e = expert_at(p.x);
    key = key_f64(a, row, bias, e, m, sum);
  }
  int rank = 0;
  for (int j = 0; j < count; ++j) {
    const double o = __shfl_sync(kFull, key, j);
    const int oe = __shfl_sync(kFull, e, j);
    rank += (o > key || (o == key && oe < e)) ? 1 : 0;
  }
  __syncwarp();
  if (lane < count) picks[rank] = p;
  __syncwarp();
}

// One token by one warp, in fp64.  skey: E doubles of shared memory.
template <typename L>
__device__ __noinline__ void route_token_f64(const RouteShape& a, const L* __restrict__ row,
                                             const float* __restrict__ bias, int t, int lane,
                                             double* skey, int32_t* __restrict__ topk_idx,
                                             float* __restrict__ topk_w) {
  const double ninf = -INFINITY;
  double m = 0.0, sum = 1.0;
  double key[8];                           // of the experts lane + 32 i
  if (a.gate == 0) {
    softmax_f64(a, row, lane, m, sum, key);
#pragma unroll
    for (int i = 0; i < 8; ++i) key[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      key[i] = lane + 32 * i < a.E ? 1.0 / (1.0 + exp(-to_f64(row[lane + 32 * i]))) : 0.0;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    const double l = e < a.E ? to_f64(row[e]) : ninf;
    const bool ok = l > ninf && key[i] == key[i];
    if (a.space == 0) key[i] = l;
    if (bias != nullptr && e < a.E) key[i] += static_cast<double>(bias[e]);
    key[i] = ok && key[i] > ninf ? key[i] : ninf;
  }
  if (a.topk_group < a.groups) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < a.E) skey[lane + 32 * i] = key[i];
    __syncwarp();
    double m1 = ninf, m2 = ninf;
    if (lane < a.groups) {
#pragma unroll 8
      for (int e = lane * a.per; e < (lane + 1) * a.per; ++e) top2(m1, m2, skey[e], ninf);
    }
    const double sc = a.group_score == 2 && m2 > ninf ? m1 + m2 : m1;
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const double o = __shfl_sync(kFull, sc, h);
      rank += (o > sc || (o == sc && h < lane)) ? 1 : 0;
    }
    const unsigned use = __ballot_sync(kFull, lane < a.groups && rank < a.topk_group);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < a.E && !((use >> ((lane + 32 * i) / a.per)) & 1u)) key[i] = ninf;
    __syncwarp();
  }
  // a round: each lane's best as an ordered integer
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    double best = ninf;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (key[i] > best) { best = key[i]; bi = i; }
    const unsigned long long ob = best > ninf ? ordered(best) : 0ull;
    const unsigned h = static_cast<unsigned>(ob >> 32);
    const unsigned mh = __reduce_max_sync(kFull, h);
    if (mh == 0u) break;                 // nothing eligible is left
    const unsigned l = h == mh ? static_cast<unsigned>(ob) : 0u;
    const unsigned ml = __reduce_max_sync(kFull, l);
    const int be = lane + 32 * bi;
    const int e = __reduce_min_sync(kFull, h == mh && l == ml ? be : kMaxE);
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i == e) key[i] = ninf;
  }
  double s = 0.0;
  if (mine >= 0) {
    const double x = exp(a.gate == 0 ? to_f64(row[mine]) - m : -to_f64(row[mine]));
    s = a.gate == 0 ? x / sum : 1.0 / (1.0 + x);
  }
  double tot = s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(kFull, tot, o);
  if (a.norm) s /= tot + 1e-9;
  if (lane < a.k) {
    topk_idx[static_cast<size_t>(t) * a.k + lane] = mine;
    topk_w[static_cast<size_t>(t) * a.k + lane] =
        mine >= 0 ? static_cast<float>(s * static_cast<double>(a.scale)) : 0.f;
  }
  __syncwarp();
}

// Every token in fp64 (the fp64 logits of fp32 layers).
template <typename L>
__global__ void __launch_bounds__(128)
route_f64_kernel(const RouteShape a, const L* __restrict__ logits, const float* __restrict__ bias,
                 const uint8_t* __restrict__ mask, int32_t* __restrict__ topk_idx,
                 float* __restrict__ topk_w) {
  pdl_trigger();
  pdl_wait();
  __shared__ double skey[4][kMaxE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * 4 + warp;
  if (t >= a.T) return;
  if (mask != nullptr && mask[t] == 0) {
    if (lane < a.k) {
      topk_idx[static_cast<size_t>(t) * a.k + lane] = -1;
      topk_w[static_cast<size_t>(t) * a.k + lane] = 0.f;
    }
    return;
  }
  route_token_f64<L>(a, logits + static_cast<size_t>(t) * a.ld, bias, t, lane, skey[warp],
                     topk_idx, topk_w);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// e^x within (2 + 1.16 |x|) 2^-23 of itself, below 2^-126 as 0.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}

// Within 2.5e-7 of the sigmoid: s (1 - s) turns the exponential's error into
// 7e-8; sum and reciprocal add 1.8e-7 s.
__device__ __forceinline__ float fast_sigmoid(float l) {
  return rcp_approx(1.0f + fast_exp(-l));
}

// Four consecutive logits of a row; VEC: one aligned load.
template <typename L, bool VEC>
__device__ __forceinline__ float4 load4(const L* __restrict__ row, int e, int E) {
  const float ninf = -INFINITY;
  if constexpr (VEC) {
    if (e >= E) return make_float4(ninf, ninf, ninf, ninf);
    if constexpr (sizeof(L) == 4) {
      return __ldg(reinterpret_cast<const float4*>(row + e));
    } else {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(row + e));
      const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q.x));
      const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q.y));
      return make_float4(lo.x, lo.y, hi.x, hi.y);
    }
  } else {
    return make_float4(e < E ? to_f32<L>(row[e]) : ninf, e + 1 < E ? to_f32<L>(row[e + 1]) : ninf,
                       e + 2 < E ? to_f32<L>(row[e + 2]) : ninf,
                       e + 3 < E ? to_f32<L>(row[e + 3]) : ninf);
  }
}

constexpr int kRouteWarps = 4;
constexpr int kMorePicks = 8;   // looked at where the last chosen one's lead is not clear
constexpr int kPickRow = kMaxK + 2 + kMorePicks;

// 4 tokens per warp, 8 lanes per token (`sub` of `tok`).
//   1  the 8 lanes read their token's row, 128 bytes at a time, form the keys
//      and leave them in shared memory
//   2  lane `sub` scans the groups sub, sub + 8, ..: two largest, score; the
//      groups are ranked by counting the better ones
//   3  the chosen groups' experts are dealt out to the 8 lanes in ascending
//      order; each 4 experts' keys sit sorted in registers, and a round of the
//      top-k is the maximum over a lane's heads, three shuffles, and the
//      winner's list moved up; which expert a key belongs to is looked up
//      after the rounds
//   4  weights
// NB: blocks of 4 experts of a lane in step 3, rounded up to a power of two.
// WARPS: at most, of a block.
template <typename L, int NB, bool VEC, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == kRouteWarps ? 7 : 4)
route_kernel(const RouteShape a, const L* __restrict__ logits, const float* __restrict__ bias,
             const uint8_t* __restrict__ mask, int32_t* __restrict__ topk_idx,
             float* __restrict__ topk_w) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & 7, tok = lane >> 3;
  const int nb = (a.E + 31) >> 5;
  const int ROW = 36 * nb;                   // floats of a token's keys
  float* sbias = smem;                       // laid out as a row of keys
  float* keys = smem + ROW + warp * (4 * ROW + 8 * kPickRow);
  int2* picks = reinterpret_cast<int2*>(keys + 4 * ROW) + tok * kPickRow;
  const float ninf = -INFINITY;
  // what is compared in fp32: the logits themselves where the keys' order is
  // theirs (no bias), else the biased keys
  const bool biased = bias != nullptr;
  const bool by_score = a.space == 1 && biased;   // keys = s + bias
  if (biased) {
    for (int e = threadIdx.x; e < 32 * nb; e += blockDim.x) {
      float v = 0.f;
      if (e < a.E) {
        v = bias[e];
        if (!(v == v)) v = ninf;                  // a NaN switches the expert off
      }
      sbias[at(e)] = v;
    }
    __syncthreads();
  }
  const int t0 = (blockIdx.x * (blockDim.x >> 5) + warp) * 4;
  if (t0 >= a.T) return;
  const int t = t0 + tok;
  // ---------------------------------------------------------------- 1 keys
  const bool on = t < a.T && (mask == nullptr || mask[t] != 0);
  float row_m = 0.f, row_inv = 1.f;               // softmax of this lane's token
  bool odd = false;                               // values only fp64 decides
  {
    const L* row = logits + static_cast<size_t>(t) * a.ld;
    float4 l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 4 * sub + 32 * i;
      l[i] = make_float4(ninf, ninf, ninf, ninf);
      if (i < nb && on && e < a.E) l[i] = load4<L, VEC>(row, e, a.E);
    }
    if (a.gate == 0) {
      float m = ninf, s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nb) m = fmaxf(fmaxf(m, fmaxf(l[i].x, l[i].y)), fmaxf(l[i].z, l[i].w));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      row_m = m;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nb)
          s += (fast_exp(l[i].x - m) + fast_exp(l[i].y - m)) +
               (fast_exp(l[i].z - m) + fast_exp(l[i].w - m));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
      odd = !(s >= 0.5f && s <= 1024.f);          // NaN, +inf, or no finite logit
      row_inv = rcp_approx(s);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= nb) break;
      float* v = reinterpret_cast<float*>(&l[i]);
      if (biased) {
        const float4 bq = *reinterpret_cast<const float4*>(sbias + 36 * i + 4 * sub);
        const float* bv = reinterpret_cast<const float*>(&bq);
        if (by_score) {
          if (a.gate == 0) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              v[c] = v[c] > ninf ? fmaf(fast_exp(v[c] - row_m), row_inv, bv[c]) : ninf;
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = v[c] > ninf ? fast_sigmoid(v[c]) + bv[c] : ninf;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            odd = odd || !(v[c] <= 1e30f);        // NaN or +inf
            // rounded towards zero, two finite terms make a finite key
            v[c] = v[c] > ninf ? __fadd_rz(v[c], bv[c]) : ninf;
          }
        }
      } else {
        // beyond 16 distinct logits may have equal fp64 sigmoids
        const float most = a.space == 1 && a.gate == 1 ? 16.f : 1e30f;
#pragma unroll
        for (int c = 0; c < 4; ++c) odd = odd || !(v[c] <= most);
      }
      *reinterpret_cast<float4*>(keys + tok * ROW + 36 * i + 4 * sub) = l[i];
    }
  }
  const unsigned live = __ballot_sync(kFull, on);         // bytes: tokens
  // byte r, not 0: token r is decided by fp64 as a whole
  unsigned slow = __ballot_sync(kFull, odd && on);
  __syncwarp();
  float* mykeys = keys + tok * ROW;
  // A score's fp32 error: 2.5e-7 of a sigmoid; of a softmax, whose largest
  // term is row_inv, 9e-7 row_inv (the exponential 4e-7, the divisor 5e-7).  The
  // sum with the bias rounds once more, 2^-24 of the key (2^-23 of a logit's).
  const float key_err = !by_score ? 0.f : a.gate == 0 ? 9e-7f * row_inv : 2.5e-7f;
  const int per = a.per;
  const bool limited = a.topk_group < a.groups;
  const bool whole = (per & 3) == 0;              // groups are whole blocks of 4
  const float inv_per = rcp_approx(static_cast<float>(per));   // of small integers only
  unsigned use = kFull;                           // groups this lane's token may use
  // -------------------------------------------------------------- 2 groups
  if (limited) {
    // a score's fp32 error: none for the largest of unbiased logits, relative
    // for sums of exponentials (down to the subnormal ones), else that of keys
    // formed from fp32 scores
#pragma unroll 1
    for (int g = sub; g < a.groups; g += 8) {
      float m1 = ninf, m2 = ninf;
      if (whole) {
#pragma unroll 2
        for (int e = g * per; e < (g + 1) * per; e += 4) {
          const float4 q = *reinterpret_cast<const float4*>(mykeys + at(e));
          const float h1 = fmaxf(q.x, q.y), l1 = fminf(q.x, q.y);
          const float h2 = fmaxf(q.z, q.w), l2 = fminf(q.z, q.w);
          const float h = fmaxf(h1, h2);
          const float second = fmaxf(fmaxf(fminf(h1, h2), l1), l2);
          m2 = fmaxf(fmaxf(fminf(m1, h), second), m2);
          m1 = fmaxf(m1, h);
        }
      } else {
        for (int e = g * per; e < (g + 1) * per; ++e) {
          const float v = mykeys[at(e)];
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
      }
      float sc = m1, err = 0.f;
      const bool two = a.group_score == 2 && m2 > ninf;
      if (a.group_score == 2 && a.space == 1 && !biased) {
        // sums of scores; the softmax's divisor is common to all groups
        if (m1 > ninf) {
          if (a.gate == 0) {
            sc = expf(m1 - row_m) + expf(m2 - row_m);
            err = 1e-5f * sc + 1e-42f;   // subnormal sums: steps of 1.4e-45
          } else {
            sc = fast_sigmoid(m1) + (two ? fast_sigmoid(m2) : 0.f);
            err = 7e-7f;
          }
        }
      } else if (biased || two) {
        // Beyond fp32's range a score is its lowest number, or inf, with a finite
        // error: in order, or within its error of the border.  A key may have
        // been cut to the lowest number already, in front of a large first one.
        if (two) sc = fmaxf(m1 + m2, -FLT_MAX);
        err = 2.f * key_err + (by_score ? 1.5e-7f : 2e-7f) * (fabsf(m1) + (two ? fabsf(m2) : 0.f));
        err = m2 == -FLT_MAX && !by_score ? FLT_MAX : fminf(err, FLT_MAX);
      }
      picks[g] = make_int2(__float_as_int(err), __float_as_int(sc));
    }
    __syncwarp();
    use = 0;
    float lo = INFINITY, hi = ninf;
#pragma unroll 1
    for (int i = 0; 8 * i < a.groups; ++i) {
      const int g = sub + 8 * i;
      const int2 own = picks[g < a.groups ? g : 0];
      const float sc = __int_as_float(own.y), err = __int_as_float(own.x);
      int rank = 0;
#pragma unroll 4
      for (int h = 0; h < a.groups; ++h) {
        const float o = __int_as_float(picks[h].y);
        rank += (o > sc || (o == sc && h < g)) ? 1 : 0;
      }
      const bool in = g < a.groups && rank < a.topk_group;
      const unsigned bits = __ballot_sync(kFull, in);
      use |= ((bits >> (tok << 3)) & 0xffu) << (8 * i);
      if (g < a.groups && sc > ninf) {
        if (in) lo = fminf(lo, sc - err); else hi = fmaxf(hi, sc + err);
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
    }
    bool near = hi > ninf && !(lo > hi);
    if (!biased && a.group_score == 1) {
      // largest logits: equal ones are equal keys and the lower group is
      // right; others may be equal as fp64 scores next to zero, and where
      // the scores leave fp64's range
      near = a.space == 1 && hi > ninf &&
             ((lo - hi <= 1e-12f && fabsf(lo) < 1e-6f) ||
              lo < (a.gate == 0 ? row_m - 700.f : -700.f));
    }
    const unsigned close_calls = __ballot_sync(kFull, near) & live & ~slow;
    if (close_calls != 0u) {                      // warp-uniform
      if (!biased && a.group_score == 1) {
        slow |= close_calls;                      // differences fp32 logits do not show
      } else {
#pragma unroll 1
        for (int r = 0; r < 4; ++r) {
          if (!((close_calls >> (8 * r)) & 0xffu)) continue;
          const unsigned u = choose_groups_f64<L>(
              a, logits + static_cast<size_t>(t0 + r) * a.ld, bias, lane,
              __shfl_sync(kFull, lo, 8 * r), __shfl_sync(kFull, hi, 8 * r),
              picks + (r - tok) * kPickRow);
          if (tok == r && __popc(u) == a.topk_group) use = u;   // as many as are read below
        }
      }
    }
    __syncwarp();                                 // the scores have been read
    if (whole) {
      // the chosen groups in ascending order
#pragma unroll 1
      for (int g = sub; g < a.groups; g += 8)
        if ((use >> g) & 1u) picks[__popc(use & ((1u << g) - 1u))].x = g * per;
    } else {
      for (int e = sub; e < a.E; e += 8) {
        const int g = static_cast<int>((e + 0.5f) * inv_per);
        if (!((use >> g) & 1u)) mykeys[at(e)] = ninf;
      }
    }
    __syncwarp();
  }

  // --------------------------------------------------------------- 3 top-k
  const bool alive = on && ((slow >> (8 * tok)) & 0xffu) == 0u;
  const int total = limited && whole ? a.topk_group * per : a.E;   // experts to choose from
  const int nbr = (total + 31) >> 5;               // blocks of 4 of a lane
  // The lane's blocks: where they lie in the token's keys, and their keys in
  // descending order (a block that is not there holds none).
  int base[NB];
  float h[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int p = 4 * (nbr * sub + i);
    base[i] = 0;
    float4 q = make_float4(ninf, ninf, ninf, ninf);
    if (alive && i < nbr && p < total) {
      int e = p;
      if (limited && whole) {
        const int gi = static_cast<int>((p + 0.5f) * inv_per);
        e = picks[gi].x + p - gi * per;
      }
      base[i] = at(e);
      q = *reinterpret_cast<const float4*>(mykeys + base[i]);
    }
    const float x1 = fmaxf(q.x, q.y), x2 = fminf(q.x, q.y);
    const float y1 = fmaxf(q.z, q.w), y2 = fminf(q.z, q.w);
    h[i][0] = fmaxf(x1, y1);
    h[i][3] = fminf(x2, y2);
    const float u = fminf(x1, y1), v = fmaxf(x2, y2);
    h[i][1] = fmaxf(u, v);
    h[i][2] = fminf(u, v);
  }
  __syncwarp();
  const unsigned lower = (0xffu << (tok << 3)) & ((1u << lane) - 1u);   // this token's lower lanes
  int count = 0;
  // pick j: (place of its block, key).  Without branches: the four tokens'
  // winners sit at different places.
  auto round = [&](int j) {
    float lm = h[0][0];
#pragma unroll
    for (int i = 1; i < NB; ++i) lm = fmaxf(lm, h[i][0]);
    float best = lm;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(kFull, best, o));
    const bool any = best > ninf;
    // lanes own ascending experts, so the lowest lane has the lowest id
    const unsigned who = __ballot_sync(kFull, lm == best);
    const bool win = any && lm == best && (who & lower) == 0u;
    count += any ? 1 : 0;
    bool open = win;
    int place = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const bool hit = open && h[i][0] == best;
      open = open && !hit;
      place = hit ? base[i] : place;
      h[i][0] = hit ? h[i][1] : h[i][0];
      h[i][1] = hit ? h[i][2] : h[i][1];
      h[i][2] = hit ? h[i][3] : h[i][2];
      h[i][3] = hit ? ninf : h[i][3];
    }
    if (win) picks[j] = make_int2(place, __float_as_int(best));
  };
  // The expert of pick j: the first in its block with that key, or as many
  // further as earlier picks share block and key.  Kept beside the place
  // (bits 16 and 17), which other lanes may still be reading.
  auto resolve = [&](int j) {
    const int2 p = picks[j];
    const float key = __int_as_float(p.y);
    const float4 q = *reinterpret_cast<const float4*>(mykeys + p.x);
    unsigned eq = (q.x == key ? 1u : 0u) | (q.y == key ? 2u : 0u) | (q.z == key ? 4u : 0u) |
                  (q.w == key ? 8u : 0u);
    if (eq & (eq - 1u)) {
      for (int i = 0; i < j; ++i) {
        const int2 o = picks[i];
        if ((o.x & 0xffff) == p.x && __int_as_float(o.y) == key) eq &= eq - 1u;   // -0 is 0
      }
    }
    picks[j].x = p.x | ((__ffs(eq) - 1) << 16);
  };
  for (int j = 0; j <= a.k; ++j) round(j);   // one more than k: is the last one's lead clear
  __syncwarp();
  for (int j = sub; j < count; j += 8) resolve(j);
  __syncwarp();
  // the logit of the lane's first pick, asked for before it is needed
  float first = 0.f;
  bool moved = false;
  if (biased && sub < count)
    first = to_f32<L>(logits[static_cast<size_t>(t) * a.ld + expert_at(picks[sub].x)]);
  // ---------------------------------------------- are the leads clear in fp32
  if (biased || a.space == 1) {
    const L* row = logits + static_cast<size_t>(t) * a.ld;
    // Keys closer than this may be in the wrong order.  Without a bias they are
    // the logits: distinct ones have distinct fp64 scores, but next to zero
    // (below 1e-15 apart) and below `floor`, where the scores leave fp64's range.
    auto margin = [&](float key) {
      return !biased ? 1e-12f
                     : 2.f * key_err + (by_score ? 2e-7f : 2.6e-7f) * (fabsf(key) + 1e-3f);
    };
    const float floor = biased ? ninf : a.gate == 0 ? row_m - 700.f : -700.f;
    // equal inputs make equal keys: an exact tie, ordered by id as it should be
    auto same = [&](int e, int f) {
      return to_f32<L>(row[e]) == to_f32<L>(row[f]) && bias[e] == bias[f];
    };
    bool near = false;   // two neighbours of the chosen ones
    bool edge = false;   // the last of them and the best one left out
    for (int j = sub; j + 1 < count; j += 8) {
      const int2 p = picks[j], n = picks[j + 1];
      const float best = __int_as_float(p.y), gap = best - __int_as_float(n.y);
      const bool c = !(gap > margin(best)) || best < floor;
      if (j + 1 == a.k)
        edge = c && (biased || fabsf(best) < 1e-6f || best < floor);
      else if (c)
        near = near || (biased ? !same(expert_at(p.x), expert_at(n.x)) : gap > 0.f);
    }
    if (__any_sync(kFull, near || edge)) {
      moved = true;
      // keys of +inf, whose gaps and margins say nothing (and count as close)
      slow |= __ballot_sync(kFull, count > 0 && __int_as_float(picks[0].y) > FLT_MAX);
      if ((slow >> (8 * tok)) & 0xffu) near = edge = false;
      const unsigned edges = __ballot_sync(kFull, edge);
      bool open = ((edges >> (8 * tok)) & 0xffu) != 0u;
      unsigned fix = __ballot_sync(kFull, near), again = 0;
      if (edges != 0u) {
        const int2 last = open ? picks[a.k - 1] : make_int2(0, 0);
        const float lk = __int_as_float(last.y);
        if (open) {
          // is any expert that close to the last chosen one not an exact tie
          // with it (it may be hidden behind ties)
          bool differs = false;
          for (int e = 4 * sub; e < a.E; e += 32) {
            if (limited && whole && !((use >> static_cast<int>((e + 0.5f) * inv_per)) & 1u))
              continue;
            const float4 q = *reinterpret_cast<const float4*>(mykeys + at(e));
            const float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (biased)
                differs = differs || (v[c] > ninf && fabsf(v[c] - lk) <= margin(lk) &&
                                      !same(e + c, expert_at(last.x)));
              else
                differs = differs || (v[c] != lk && v[c] > ninf &&
                                      (fabsf(v[c] - lk) <= margin(lk) ||
                                       (lk < floor && v[c] < floor)));
          }
          open = differs;
        }
        const unsigned any = __ballot_sync(kFull, open);
        open = ((any >> (8 * tok)) & 0xffu) != 0u;
        fix |= any;
        // the next ones, until one is clearly behind
#pragma unroll 1
        for (int x = 1; x <= kMorePicks && __any_sync(kFull, open); ++x) {
          const int before = count;
          round(a.k + x);
          __syncwarp();
          if (count > before && sub == 0) resolve(before);
          __syncwarp();
          if (open) {
            const float next = __int_as_float(picks[before].y);
            open = count > before && (!(lk - next > margin(lk)) || next < floor);
          }
        }
        again = __ballot_sync(kFull, open);
      }
      const unsigned many = __ballot_sync(kFull, count > 32);
#pragma unroll 1
      for (int r = 0; r < 4; ++r) {
        if (!((fix >> (8 * r)) & 0xffu)) continue;
        if (((again | many) >> (8 * r)) & 0xffu)
          slow |= 0xffu << (8 * r);
        else
          order_picks_f64<L>(a, logits + static_cast<size_t>(t0 + r) * a.ld, bias, lane,
                             __shfl_sync(kFull, count, 8 * r), picks + (r - tok) * kPickRow);
      }
    }
  }
  slow &= live;   // padding tokens are not decided at all

  // ------------------------------------------------------------- 4 weights
  const int n = count < a.k ? count : a.k;
  float tot = 0.f;
#pragma unroll 1
  for (int j = sub; j < n; j += 8) {
    const int2 p = picks[j];
    const int e = expert_at(p.x);
    // without a bias the key is the logit
    float l = __int_as_float(p.y);
    if (biased)
      l = j == sub && !moved ? first : to_f32<L>(logits[static_cast<size_t>(t) * a.ld + e]);
    const float s =
        a.gate == 0 ? expf(l - row_m) * row_inv : rcp_approx(1.0f + expf(-l));
    picks[j] = make_int2(e, __float_as_int(s));
    tot += s;
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) tot += __shfl_xor_sync(kFull, tot, o);
  if (t < a.T && ((slow >> (8 * tok)) & 0xffu) == 0u) {
    const float f = a.norm ? __fdividef(a.scale, tot + 1e-9f) : a.scale;
    int32_t* idx_row = topk_idx + static_cast<size_t>(t) * a.k;
    float* w_row = topk_w + static_cast<size_t>(t) * a.k;
#pragma unroll 1
    for (int j = sub; j < a.k; j += 8) {
      const int2 p = picks[j];
      idx_row[j] = j < n ? p.x : -1;
      w_row[j] = j < n ? __int_as_float(p.y) * f : 0.f;
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int r = 0; r < 4; ++r)   // warp-uniform
    if ((slow >> (8 * r)) & 0xffu)
      route_token_f64<L>(a, logits + static_cast<size_t>(t0 + r) * a.ld, bias, t0 + r, lane,
                         reinterpret_cast<double*>(keys), topk_idx, topk_w);
}

// dlogits, 4 tokens per warp.  For the chosen experts with scores s_j and
// incoming dw_j:  ds_j = c (dw_j - sum_i dw_i s_i / D) / D with
// D = sum_i s_i + 1e-9, or c dw_j;  sigmoid: dl = ds s (1 - s);  softmax:
// dl_e = p_e (ds_e - sum_j ds_j p_j).  The sums over the chosen experts are in
// fp64: with one expert a token the difference is 1e-9 of its terms.
//   1  (softmax) the warp reads one token's row after another and leaves the
//      exponentials in shared memory
//   2  lane `sub` of a token takes the pairs sub, sub + 8, ..
//      and leaves their elements in the row in shared memory
//   3  the rows: those elements, the exponentials' multiples (sigmoid: zeros)
//      elsewhere, each row written once
// Memory bound: a row is read (softmax) and written once.
// NP: pairs of a lane, rounded up to a power of two.
// No early trigger: blocks of the next launch that wait beside this one's leave
// its blocks uneven over the SMs ([16384, 128] softmax: 6.9 us with, 6.15
// without).  [131072, 256] fp32 sigmoid: 33 to 35 us, 134 MB written and a
// sector read for each pair, 0.75 of the copy bandwidth.
template <typename L, int NP, bool VEC>
__global__ void __launch_bounds__(32 * kRouteWarps)
route_bwd_kernel(const RouteShape a, const L* __restrict__ logits,
                 const int32_t* __restrict__ topk_idx, const float* __restrict__ dw,
                 L* __restrict__ dlogits, long long dld) {
  pdl_wait();
  extern __shared__ __align__(16) float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & 7, tok = lane >> 3;
  const int ROW = (a.E + 3) & ~3;
  float* rows = smem + warp * (4 * ROW + 32);
  unsigned* seen = reinterpret_cast<unsigned*>(rows + 4 * ROW);   // 256 bits per token
  const int t0 = (blockIdx.x * (blockDim.x >> 5) + warp) * 4;
  if (t0 >= a.T) return;
  const float ninf = -INFINITY;
  const bool soft = a.gate == 0;
  float row_m = 0.f, row_inv = 0.f;               // softmax of this lane's token
  // ------------------------------------------------------------ 1 softmax
  if (soft) {
#pragma unroll 1
    for (int r2 = 0; r2 < 4; r2 += 2) {
      float4 lv[2][2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lv[q][i] = make_float4(ninf, ninf, ninf, ninf);
          if (t0 + r2 + q < a.T && 128 * i < a.E)
            lv[q][i] = load4<L, VEC>(logits + static_cast<size_t>(t0 + r2 + q) * a.ld,
                                     4 * lane + 128 * i, a.E);
        }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float* l = reinterpret_cast<float*>(lv[q]);
        float m = ninf, s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, l[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        if (m == ninf) m = 0.f;                    // no finite logit: all zero
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          l[i] = __expf(l[i] - m);
          s += l[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int e = 4 * lane + 128 * i;
          if (e < ROW) *reinterpret_cast<float4*>(rows + (r2 + q) * ROW + e) = lv[q][i];
        }
        if (tok == r2 + q) {
          row_m = m;
          row_inv = s == 0.f ? 0.f : 1.0f / s;
        }
      }
    }
  }
  seen[lane] = 0u;
  __syncwarp();
  // -------------------------------------------------------------- 2 pairs
  const int t = t0 + tok;
  int e[NP];
  float d[NP], sj[NP], v[NP];
  double D = 0.0, Q = 0.0;
  bool twice = false;
  bool some = false;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int j = sub + 8 * i;
    e[i] = -1;
    d[i] = 0.f;
    sj[i] = 0.f;
    v[i] = 0.f;
    if (8 * i >= a.k) continue;
    if (t < a.T && j < a.k) e[i] = topk_idx[static_cast<size_t>(t) * a.k + j];
    if (e[i] < 0 || e[i] >= a.E) e[i] = -1;
    if (e[i] >= 0) {
      some = true;
      d[i] = dw[static_cast<size_t>(t) * a.k + j];
      const float l = to_f32<L>(logits[static_cast<size_t>(t) * a.ld + e[i]]);
      if (soft) {
        sj[i] = expf(l - row_m) * row_inv;
        v[i] = sj[i];                              // d score / d ds
      } else {
        const float x = expf(-fabsf(l)), r = 1.0f / (1.0f + x);
        sj[i] = l >= 0.f ? r : x * r;
        v[i] = x * r * r;                          // s (1 - s)
      }
      const unsigned bit = 1u << (e[i] & 31);
      twice = twice || (atomicOr(seen + 8 * tok + (e[i] >> 5), bit) & bit);
    }
    D += sj[i];
    Q += static_cast<double>(d[i]) * static_cast<double>(sj[i]);
  }
  double f = a.scale, q = 0.0;                     // ds = f (dw - q)
  if (a.norm) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      D += __shfl_xor_sync(kFull, D, o);
      Q += __shfl_xor_sync(kFull, Q, o);
    }
    D += 1e-9;
    f = static_cast<double>(a.scale) / (D * D);
  }
  double dot = 0.0;
  float ds[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    ds[i] = 0.f;
    if (8 * i >= a.k || e[i] < 0) continue;
    q = a.norm ? f * (static_cast<double>(d[i]) * D - Q) : f * static_cast<double>(d[i]);
    ds[i] = static_cast<float>(q);
    dot += q * static_cast<double>(sj[i]);
  }
  if (soft) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
  }
  if (__any_sync(kFull, twice)) {
    // an expert listed twice: the sum of its pairs, in pair order, at each
    float sum[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) sum[i] = 0.f;
#pragma unroll
    for (int ih = 0; ih < NP; ++ih) {
      if (8 * ih >= a.k) continue;
      for (int hl = 0; hl < 8; ++hl) {
        const int eh = __shfl_sync(kFull, e[ih], (tok << 3) | hl);
        const float dh = __shfl_sync(kFull, ds[ih], (tok << 3) | hl);
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (eh == e[i]) sum[i] += dh;
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) ds[i] = sum[i];
  }
  const unsigned with = __ballot_sync(kFull, some);
  const float fdot = soft ? static_cast<float>(dot) : 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (e[i] >= 0) rows[tok * ROW + e[i]] = v[i] * (ds[i] - fdot);
  __syncwarp();
  // --------------------------------------------------------------- 3 rows
  const float neg = -fdot * row_inv;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (t0 + r >= a.T) break;
    // a token without experts has a row of zeros, whatever its logits
    const bool dense = soft && ((with >> (8 * r)) & 0xffu);
    const float c = __shfl_sync(kFull, neg, 8 * r);
    L* out = dlogits + static_cast<size_t>(t0 + r) * dld;
    const float* row = rows + r * ROW;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int x = 4 * lane + 128 * i;
        if (x >= a.E) break;
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
        const unsigned own = seen[8 * r + (x >> 5)] >> (x & 31);   // chosen ones: as they are
        if (dense || (own & 15u)) {
          const float4 q = *reinterpret_cast<const float4*>(row + x);
          g.x = own & 1u ? q.x : dense ? q.x * c : 0.f;
          g.y = own & 2u ? q.y : dense ? q.y * c : 0.f;
          g.z = own & 4u ? q.z : dense ? q.z * c : 0.f;
          g.w = own & 8u ? q.w : dense ? q.w * c : 0.f;
        }
        if constexpr (sizeof(L) == 2) {
          const __nv_bfloat162 h0 = __floats2bfloat162_rn(g.x, g.y);
          const __nv_bfloat162 h1 = __floats2bfloat162_rn(g.z, g.w);
          *reinterpret_cast<uint2*>(out + x) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&h0),
                         *reinterpret_cast<const uint32_t*>(&h1));
        } else {
          *reinterpret_cast<float4*>(out + x) = g;
        }
      }
    } else {
      for (int x = lane; x < a.E; x += 32) {
        const bool own = (seen[8 * r + (x >> 5)] >> lane) & 1u;
        const float g = own ? row[x] : dense ? row[x] * c : 0.f;
        if constexpr (sizeof(L) == 2) out[x] = __float2bfloat16_rn(g); else out[x] = g;
      }
    }
  }
}

// Rows [offsets[E], offsets[E] + 64) of two bf16 matrices of R rows set to
// zero (block: one row), when tokens without experts left rows behind the
// last expert's: the weight gradients' last k-block reaches into them.
__global__ void __launch_bounds__(256)
zero_tail_kernel(const int32_t* __restrict__ offsets, int E, long long R, uint4* __restrict__ a,
                 int a_vecs, uint4* __restrict__ b, int b_vecs) {
  pdl_trigger();
  pdl_wait();
  const long long r = static_cast<long long>(offsets[E]) + blockIdx.x;
  if (r < 0 || r >= R) return;
  for (int c = threadIdx.x; c < a_vecs; c += blockDim.x) a[r * a_vecs + c] = make_uint4(0, 0, 0, 0);
  for (int c = threadIdx.x; c < b_vecs; c += blockDim.x) b[r * b_vecs + c] = make_uint4(0, 0, 0, 0);
}

template <typename L>
cudaError_t route_launch(const RouteShape& a, const L* logits, const float* bias,
                         const uint8_t* mask, int32_t* topk_idx, float* topk_w,
                         cudaStream_t stream) {
  const int per = a.per;
  const int total = a.topk_group < a.groups && per % 4 == 0 ? a.topk_group * per : a.E;
  // One warp per block until there are enough tokens for four on every SM.
  // Eight, which share the bias and keep 32 warps on an SM instead of 28, for
  // three rounds of tokens and more ([131072, 256] 80.3 us with four, 74.1 with
  // eight; below, the coarser last round costs more: [16384, 128] 9.6 and 10.2),
  // but for more than 4 blocks a lane, whose registers that leaves too few
  // ([131072, 160] without groups 75.9 and 78.5).
  const int warps = a.T <= 148 * 16 ? 1
                    : a.T <= 3 * 148 * 28 * 4 || total > 128 ? kRouteWarps : 2 * kRouteWarps;
  const unsigned grid = static_cast<unsigned>((a.T + 4 * warps - 1) / (4 * warps));
  const size_t row = 36 * ((a.E + 31) / 32);   // floats of a token's keys, and of the bias
  const size_t smem = (row + warps * (4 * row + 8 * kPickRow)) * sizeof(float);
  static_assert((288 + 2 * kRouteWarps * (4 * 288 + 8 * kPickRow)) * sizeof(float) <= 49152,
                "shared memory of a block without asking");
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 &&
                   (reinterpret_cast<uintptr_t>(logits) & (4 * sizeof(L) - 1)) == 0;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(grid), dim3(32 * warps), smem, stream, a, logits, bias, mask,
                      topk_idx, topk_w);
  };
  constexpr int W = kRouteWarps;
  auto best = [&](auto nb) {
    constexpr int NB = decltype(nb)::value;
    if (warps > W)
      return vec ? go(route_kernel<L, NB, true, 2 * W>) : go(route_kernel<L, NB, false, 2 * W>);
    return vec ? go(route_kernel<L, NB, true, W>) : go(route_kernel<L, NB, false, W>);
  };
  if (total <= 32) return best(std::integral_constant<int, 1>{});
  if (total <= 64) return best(std::integral_constant<int, 2>{});
  if (total <= 128) return best(std::integral_constant<int, 4>{});
  return vec ? go(route_kernel<L, 8, true, W>) : go(route_kernel<L, 8, false, W>);
}

template <typename L>
cudaError_t route_bwd_launch(const RouteShape& a, const L* logits, const int32_t* topk_idx,
                             const float* dw, L* dlogits, long long dld, cudaStream_t stream) {
  const int warps = a.T <= 148 * 16 ? 1 : kRouteWarps;
  const unsigned grid = static_cast<unsigned>((a.T + 4 * warps - 1) / (4 * warps));
  // the rows of the softmax's exponentials, and the seen bits
  const size_t smem = static_cast<size_t>(warps) * (4 * ((a.E + 3) & ~3) + 32) * sizeof(float);
  const uintptr_t align = 4 * sizeof(L) - 1;
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && dld % 4 == 0 &&
                   (reinterpret_cast<uintptr_t>(logits) & align) == 0 &&
                   (reinterpret_cast<uintptr_t>(dlogits) & align) == 0;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(grid), dim3(32 * warps), smem, stream, a, logits, topk_idx, dw,
                      dlogits, dld);
  };
  if (a.k <= 8) return vec ? go(route_bwd_kernel<L, 1, true>) : go(route_bwd_kernel<L, 1, false>);
  if (a.k <= 16) return vec ? go(route_bwd_kernel<L, 2, true>) : go(route_bwd_kernel<L, 2, false>);
  return vec ? go(route_bwd_kernel<L, 4, true>) : go(route_bwd_kernel<L, 4, false>);
}

}  // namespace

cudaError_t route_groups(const RouteShape& a, RouteLogits type, const void* logits,
                         const float* bias, const uint8_t* mask, int32_t* topk_idx,
                         float* topk_w, cudaStream_t stream) {
  if (type == RouteLogits::f64)
    return launch_pdl(route_f64_kernel<double>, dim3((a.T + 3) / 4), dim3(128), 0, stream, a,
                      static_cast<const double*>(logits), bias, mask, topk_idx, topk_w);
  if (type == RouteLogits::bf16)
    return route_launch(a, static_cast<const __nv_bfloat16*>(logits), bias, mask, topk_idx,
                        topk_w, stream);
  return route_launch(a, static_cast<const float*>(logits), bias, mask, topk_idx, topk_w, stream);
}

cudaError_t route_groups_backward(const RouteShape& a, RouteLogits type, const void* logits,
                                  const int32_t* topk_idx, const float* dw, void* dlogits,
                                  long long dld, cudaStream_t stream) {
  if (type == RouteLogits::bf16)
    return route_bwd_launch(a, static_cast<const __nv_bfloat16*>(logits), topk_idx, dw,
                            static_cast<__nv_bfloat16*>(dlogits), dld, stream);
  return route_bwd_launch(a, static_cast<const float*>(logits), topk_idx, dw,
                          static_cast<float*>(dlogits), dld, stream);
}

cudaError_t zero_tail_rows(const int32_t* offsets, int E, long long R, void* a, int a_cols,
                           void* b, int b_cols, cudaStream_t stream) {
  return launch_pdl(zero_tail_kernel, dim3(64), dim3(256), 0, stream, offsets, E, R,
                    static_cast<uint4*>(a), a_cols / 8, static_cast<uint4*>(b), b_cols / 8);
}

}  // namespace moe
