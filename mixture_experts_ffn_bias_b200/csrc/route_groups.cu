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
// compared in fp32 first; a token where two compared values are closer than
// their fp32 error is decided again in fp64 (a few in a thousand).
//
// Bound by memory for many tokens (the logits are read once), by the
// selection's instructions close behind: 4 tokens per warp, 8 lanes each, so
// that the cross-lane steps of the top-k serve four tokens at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

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

// One token by one warp, in fp64.  skey: E doubles of shared memory.
template <typename L>
__device__ __noinline__ void route_token_f64(const RouteShape& a, const L* __restrict__ row,
                                             const float* __restrict__ bias, int t, int lane,
                                             double* skey, int32_t* __restrict__ topk_idx,
                                             float* __restrict__ topk_w) {
  const double ninf = -INFINITY;
  double m = 0.0, sum = 1.0;
  if (a.gate == 0) {
    m = ninf;
    for (int e = lane; e < a.E; e += 32) m = fmax(m, to_f64(row[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, o));
    if (m == ninf) m = 0.0;
    sum = 0.0;
    for (int e = lane; e < a.E; e += 32) sum += exp(to_f64(row[e]) - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  auto score = [&](double l) {
    return a.gate == 0 ? exp(l - m) / sum : 1.0 / (1.0 + exp(-l));
  };
  for (int e = lane; e < a.E; e += 32) {
    const double l = to_f64(row[e]);
    const double s = score(l);
    double key = a.space == 1 ? s : l;
    if (bias != nullptr) key += static_cast<double>(bias[e]);
    const bool ok = l > ninf && s == s && key > ninf;
    skey[e] = ok ? key : ninf;
  }
  __syncwarp();
  const int per = a.E / a.groups;
  unsigned use = kFull;
  if (a.topk_group < a.groups) {
    double sc = ninf;
    if (lane < a.groups) {
      double m1 = ninf, m2 = ninf;
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        const double v = skey[e];
        if (v > m1) { m2 = m1; m1 = v; } else if (v > m2) { m2 = v; }
      }
      sc = a.group_score == 2 && m2 > ninf ? m1 + m2 : m1;
    }
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const double o = __shfl_sync(kFull, sc, h);
      rank += (o > sc || (o == sc && h < lane)) ? 1 : 0;
    }
    use = __ballot_sync(kFull, lane < a.groups && rank < a.topk_group);
  }
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    double best = ninf;
    int be = kMaxE;
    for (int e = lane; e < a.E; e += 32) {
      const double v = skey[e];
      if (v > best && ((use >> (a.topk_group < a.groups ? e / per : 0)) & 1u)) { best = v; be = e; }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double v = __shfl_xor_sync(kFull, best, o);
      const int e = __shfl_xor_sync(kFull, be, o);
      if (v > best || (v == best && e < be)) { best = v; be = e; }
    }
    if (be >= kMaxE) break;              // nothing eligible is left
    if (lane == j) mine = be;
    if ((be & 31) == lane) skey[be] = ninf;
  }
  double s = mine >= 0 ? score(to_f64(row[mine])) : 0.0;
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

__device__ __forceinline__ float fast_sigmoid(float l) {
  return __fdividef(1.0f, 1.0f + __expf(-l));
}

// Shared-memory position of expert e: 4 floats of padding per 32, so that
// the 8 lanes of a token, E/8 experts apart, read 16-byte pieces from
// different banks.
__device__ __forceinline__ int at(int e) { return e + ((e >> 5) << 2); }

// 4 tokens per warp, 8 lanes per token.  NB = ceil(E / 32): lane `sub` of a
// token owns the experts [4 NB sub, 4 NB (sub + 1)).
template <typename L, int NB>
__global__ void __launch_bounds__(256)
route_kernel(const RouteShape a, const L* __restrict__ logits, const float* __restrict__ bias,
             const uint8_t* __restrict__ mask, int32_t* __restrict__ topk_idx,
             float* __restrict__ topk_w) {
  pdl_trigger();
  pdl_wait();
  constexpr int ROW = 36 * NB;               // floats of a token's keys in shared memory
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & 7, tok = lane >> 3;
  float* keys = smem + warp * 4 * ROW;
  const int t0 = (blockIdx.x * (blockDim.x >> 5) + warp) * 4;
  if (t0 >= a.T) return;
  const float ninf = -INFINITY;
  // what is compared in fp32: the logits themselves where the keys' order is
  // theirs (no bias), else the biased keys
  const bool biased = bias != nullptr;
  const bool by_score = a.space == 1 && biased;   // keys = s + bias
  unsigned slow = 0;                              // bit r: token r of the four
  unsigned live = 0;
  float row_m = 0.f, row_inv = 1.f;               // softmax of this lane's token
#pragma unroll 1
  for (int r = 0; r < 4; ++r) {
    const int t = t0 + r;
    const bool on = t < a.T && (mask == nullptr || mask[t] != 0);   // warp-uniform
    if (!on) continue;
    live |= 1u << r;
    const L* row = logits + static_cast<size_t>(t) * a.ld;
    float l[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < a.E ? to_f32<L>(row[e]) : ninf;
    }
    bool odd = false;                             // a value only fp64 decides
    float m = 0.f, inv = 1.f;
    if (a.gate == 0) {
      m = ninf;
#pragma unroll
      for (int i = 0; i < NB; ++i) m = fmaxf(m, l[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NB; ++i) s += __expf(l[i] - m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
      odd = !(s >= 0.5f && s <= 1024.f);          // NaN, +inf, or no finite logit
      inv = 1.0f / s;
    } else if (!by_score) {
      // NaN or +inf; beyond 16 distinct logits may have equal fp64 sigmoids
      const float most = a.space == 1 ? 16.f : 1e30f;
#pragma unroll
      for (int i = 0; i < NB; ++i) odd = odd || !(l[i] <= most);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int e = lane + 32 * i;
      float key = l[i];
      if (by_score) key = a.gate == 0 ? __expf(l[i] - m) * inv : fast_sigmoid(l[i]);
      if (biased && e < a.E) key += bias[e];
      if (!(key > ninf) || !(l[i] > ninf)) key = ninf;
      keys[r * ROW + at(e)] = key;
    }
    if (__any_sync(kFull, odd)) slow |= 1u << r;
    if (tok == r) { row_m = m; row_inv = inv; }
  }
  __syncwarp();
  float* mykeys = keys + tok * ROW;
  const int per = a.E / a.groups;
  const bool limited = a.topk_group < a.groups;
  unsigned use = kFull;                           // groups this lane's token may use
  if (limited) {
    // a score's fp32 error: none for the largest of unbiased logits, relative
    // for sums of exponentials, else that of keys formed from fp32 scores
    float sc[4], err[4];
    float lo = INFINITY, hi = ninf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g = sub + 8 * i;
      sc[i] = ninf;
      err[i] = 0.f;
      if (8 * i >= a.groups) continue;            // warp-uniform
      if (g < a.groups) {
        float m1 = ninf, m2 = ninf;
        if ((per & 3) == 0) {
          for (int e = g * per; e < (g + 1) * per; e += 4) {
            const float4 q = *reinterpret_cast<const float4*>(mykeys + at(e));
            m2 = fmaxf(m2, fminf(m1, q.x)); m1 = fmaxf(m1, q.x);
            m2 = fmaxf(m2, fminf(m1, q.y)); m1 = fmaxf(m1, q.y);
            m2 = fmaxf(m2, fminf(m1, q.z)); m1 = fmaxf(m1, q.z);
            m2 = fmaxf(m2, fminf(m1, q.w)); m1 = fmaxf(m1, q.w);
          }
        } else {
          for (int e = g * per; e < (g + 1) * per; ++e) {
            const float v = mykeys[at(e)];
            m2 = fmaxf(m2, fminf(m1, v));
            m1 = fmaxf(m1, v);
          }
        }
        sc[i] = m1;
        const bool two = a.group_score == 2 && m2 > ninf;
        if (a.group_score == 2 && a.space == 1 && !biased && m1 > ninf) {
          // sums of scores; the softmax's divisor is common to all groups
          if (a.gate == 0) {
            sc[i] = expf(m1 - row_m) + expf(m2 - row_m);
            err[i] = 1e-5f * sc[i];
          } else {
            sc[i] = 1.0f / (1.0f + expf(-m1)) + (two ? 1.0f / (1.0f + expf(-m2)) : 0.f);
            err[i] = 2e-6f;
          }
        } else if (biased || two) {
          if (two) sc[i] = m1 + m2;
          err[i] = 4e-6f * (1.f + fabsf(m1) + (two ? fabsf(m2) : 0.f));
        }
      }
    }
    use = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (8 * i >= a.groups) continue;
      const int g = sub + 8 * i;
      int rank = 0;
#pragma unroll
      for (int ih = 0; ih < 4; ++ih) {
        if (8 * ih >= a.groups) continue;
#pragma unroll
        for (int hl = 0; hl < 8; ++hl) {
          const int h = hl + 8 * ih;
          const float o = __shfl_sync(kFull, sc[ih], (tok << 3) | hl);
          if (h < a.groups) rank += (o > sc[i] || (o == sc[i] && h < g)) ? 1 : 0;
        }
      }
      const bool in = g < a.groups && rank < a.topk_group;
      const unsigned bits = __ballot_sync(kFull, in);
      use |= ((bits >> (tok << 3)) & 0xffu) << (8 * i);
      if (g < a.groups && sc[i] > ninf) {
        if (in) lo = fminf(lo, sc[i] - err[i]); else hi = fmaxf(hi, sc[i] + err[i]);
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
      // right; close ones, and ones whose scores leave fp64, may be equal
      // as scores only
      near = a.space == 1 && hi > ninf &&
             ((lo > hi && lo - hi < 1e-7f) || lo < (a.gate == 0 ? row_m - 700.f : -700.f));
    }
    const unsigned nb = __ballot_sync(kFull, near);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if ((nb >> (8 * r)) & 0xffu) slow |= 1u << r;
  }

  // top-k: the maximum of each 4 experts in registers
  const bool alive = (live >> tok) & 1u;
  const float inv_per = 1.0f / static_cast<float>(per);
  float bm[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int e = 4 * (NB * sub + i);
    float4 q = *reinterpret_cast<const float4*>(mykeys + at(e));
    if (limited) {
      float* f = reinterpret_cast<float*>(&q);
      if ((per & 3) == 0) {
        const int g = static_cast<int>((e + 0.5f) * inv_per);
        if (!((use >> (g & 31)) & 1u)) q = make_float4(ninf, ninf, ninf, ninf);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int g = static_cast<int>((e + c + 0.5f) * inv_per);
          if (!((use >> (g & 31)) & 1u)) f[c] = ninf;
        }
        *reinterpret_cast<float4*>(mykeys + at(e)) = q;
      }
    }
    bm[i] = alive ? fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)) : ninf;
  }
  __syncwarp();
  int pick[kMaxK / 8];
#pragma unroll
  for (int i = 0; i < kMaxK / 8; ++i) pick[i] = -1;
  float prev = INFINITY;
  int prev_e = 0;
  bool near = false;
  const bool check = biased || a.space == 1;
  for (int j = 0; j <= a.k; ++j) {   // one more than k: is the last one's lead clear
    float lm = bm[0];
#pragma unroll
    for (int i = 1; i < NB; ++i) lm = fmaxf(lm, bm[i]);
    float best = lm;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(kFull, best, o));
    const bool any = best > ninf;
    const unsigned who = (__ballot_sync(kFull, lm == best) >> (tok << 3)) & 0xffu;
    const int wsub = __ffs(who) - 1;         // lanes own ascending experts
    int e = 0;
    if (any && sub == wsub) {
      int blk = 0;
#pragma unroll
      for (int i = NB - 1; i >= 0; --i)
        if (bm[i] == best) blk = i;
      const int e0 = 4 * (NB * sub + blk);
      float* kp = mykeys + at(e0);
      float4 q = *reinterpret_cast<const float4*>(kp);
      int c = 3;
      if (q.z == best) c = 2;
      if (q.y == best) c = 1;
      if (q.x == best) c = 0;
      e = e0 + c;
      kp[c] = ninf;
      if (c == 0) q.x = ninf;
      if (c == 1) q.y = ninf;
      if (c == 2) q.z = ninf;
      if (c == 3) q.w = ninf;
      const float nm = fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w));
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (i == blk) bm[i] = nm;
    }
    e = __shfl_sync(kFull, e, (tok << 3) | (any ? wsub : 0));
    if (any && check) {
      const float gap = prev - best;
      if (biased) {
        // keys formed in fp32; equal inputs are an exact tie
        if (!(gap > 2e-6f * (1.f + fabsf(best)))) {
          const L* row = logits + static_cast<size_t>(t0 + tok) * a.ld;
          near = near || !(to_f32<L>(row[e]) == to_f32<L>(row[prev_e]) &&
                           bias[e] == bias[prev_e]);
        }
      } else if ((gap > 0.f && gap < 1e-7f) || prev < (a.gate == 0 ? row_m - 700.f : -700.f)) {
        near = true;
      }
    }
    prev = best;
    prev_e = e;
#pragma unroll
    for (int i = 0; i < kMaxK / 8; ++i)
      if (any && j < a.k && j == sub + 8 * i) pick[i] = e;
    if (!__any_sync(kFull, any)) break;
  }
  const unsigned nb = __ballot_sync(kFull, near);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if ((nb >> (8 * r)) & 0xffu) slow |= 1u << r;
  slow &= live;

  // weights: lane `sub` has the picks sub, sub + 8, ..
  const int t = t0 + tok;
  float s[kMaxK / 8];
  float tot = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxK / 8; ++i) {
    s[i] = 0.f;
    if (pick[i] >= 0) {
      const float l = to_f32<L>(logits[static_cast<size_t>(t) * a.ld + pick[i]]);
      s[i] = a.gate == 0 ? expf(l - row_m) * row_inv : 1.0f / (1.0f + expf(-l));
    }
    tot += s[i];
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) tot += __shfl_xor_sync(kFull, tot, o);
  if (t < a.T && !((slow >> tok) & 1u)) {
    const float f = a.norm ? a.scale / (tot + 1e-9f) : a.scale;
#pragma unroll
    for (int i = 0; i < kMaxK / 8; ++i) {
      const int j = sub + 8 * i;
      if (j < a.k) {
        topk_idx[static_cast<size_t>(t) * a.k + j] = pick[i];
        topk_w[static_cast<size_t>(t) * a.k + j] = pick[i] >= 0 ? s[i] * f : 0.f;
      }
    }
  }
  __syncwarp();
  while (slow != 0) {   // warp-uniform
    const int r = __ffs(slow) - 1;
    slow &= slow - 1;
    route_token_f64<L>(a, logits + static_cast<size_t>(t0 + r) * a.ld, bias, t0 + r, lane,
                       reinterpret_cast<double*>(keys), topk_idx, topk_w);
  }
}

// dlogits of one token per warp.  For the chosen experts with scores s_j and
// incoming dw_j:  ds_j = c (dw_j - sum_i dw_i s_i / D) / D with
// D = sum_i s_i + 1e-9, or c dw_j;  sigmoid: dl = ds s (1 - s);  softmax:
// dl_e = p_e (ds_e - sum_j ds_j p_j).  The sums over the chosen experts are in
// fp64: with one expert a token the difference is 1e-9 of its terms.
template <typename L, int NB>
__global__ void __launch_bounds__(256)
route_bwd_kernel(const RouteShape a, const L* __restrict__ logits,
                 const int32_t* __restrict__ topk_idx, const float* __restrict__ dw,
                 L* __restrict__ dlogits, long long dld) {
  pdl_trigger();
  pdl_wait();
  __shared__ float rowbuf[8][32 * NB];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  float* buf = rowbuf[warp];
  const L* row = logits + static_cast<size_t>(t) * a.ld;
  int e = -1;
  float d = 0.f;
  if (lane < a.k) {
    e = topk_idx[static_cast<size_t>(t) * a.k + lane];
    if (e < 0 || e >= a.E) e = -1;
    if (e >= 0) d = dw[static_cast<size_t>(t) * a.k + lane];
  }
  float l[NB], p[NB];
  float m = 0.f, inv = 1.f;
  if (a.gate == 0) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int c = lane + 32 * i;
      l[i] = c < a.E ? to_f32<L>(row[c]) : -INFINITY;
      m = fmaxf(m, l[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (m == -INFINITY) m = 0.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      p[i] = expf(l[i] - m);
      s += p[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    inv = s > 0.f || !(s == s) ? 1.0f / s : 0.f;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) buf[lane + 32 * i] = 0.f;
  float sj = 0.f, slope = 0.f;   // the score and d score / d logit (sigmoid)
  if (e >= 0) {
    const float le = to_f32<L>(row[e]);
    if (a.gate == 0) {
      sj = expf(le - m) * inv;
    } else {
      const float x = expf(-fabsf(le));
      const float r = 1.0f / (1.0f + x);
      sj = le >= 0.f ? r : x * r;
      slope = x * r * r;
    }
  }
  double D = sj, Q = static_cast<double>(d) * static_cast<double>(sj);
  double ds = static_cast<double>(d) * static_cast<double>(a.scale);
  if (a.norm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      D += __shfl_xor_sync(kFull, D, o);
      Q += __shfl_xor_sync(kFull, Q, o);
    }
    D += 1e-9;
    ds = static_cast<double>(a.scale) * (static_cast<double>(d) * D - Q) / (D * D);
  }
  if (e < 0) ds = 0.0;
  double dot = 0.0;
  if (a.gate == 0) {
    dot = ds * static_cast<double>(sj);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
  }
  __syncwarp();
  // the same expert twice adds up, in pair order
  const float v = static_cast<float>(a.gate == 0 ? ds : ds * static_cast<double>(slope));
  const unsigned same = __match_any_sync(kFull, e);
  if (__any_sync(kFull, e >= 0 && (same & (same - 1)))) {
    for (int j = 0; j < a.k; ++j) {
      if (lane == j && e >= 0) buf[e] += v;
      __syncwarp();
    }
  } else if (e >= 0) {
    buf[e] = v;
  }
  __syncwarp();
  L* out = dlogits + static_cast<size_t>(t) * dld;
  const float fdot = static_cast<float>(dot);
  const bool chosen = __any_sync(kFull, e >= 0);   // a token without experts: zeros
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int c = lane + 32 * i;
    if (c >= a.E) break;
    float g = buf[c];
    if (a.gate == 0) g = chosen ? p[i] * inv * (g - fdot) : 0.f;
    if constexpr (sizeof(L) == 2)
      out[c] = __float2bfloat16_rn(g);
    else
      out[c] = g;
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
  // one warp per block until there are enough tokens for eight on every SM
  const int warps = a.T <= 148 * 32 ? 1 : 8;
  const int nb = (a.E + 31) / 32;
  const unsigned grid = static_cast<unsigned>((a.T + 4 * warps - 1) / (4 * warps));
  const size_t smem = static_cast<size_t>(warps) * 4 * 36 * nb * sizeof(float);
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(grid), dim3(32 * warps), smem, stream, a, logits, bias, mask,
                      topk_idx, topk_w);
  };
  switch (nb) {
    case 1: return go(route_kernel<L, 1>);
    case 2: return go(route_kernel<L, 2>);
    case 3: return go(route_kernel<L, 3>);
    case 4: return go(route_kernel<L, 4>);
    case 5: return go(route_kernel<L, 5>);
    case 6: return go(route_kernel<L, 6>);
    case 7: return go(route_kernel<L, 7>);
    default: return go(route_kernel<L, 8>);
  }
}

template <typename L>
cudaError_t route_bwd_launch(const RouteShape& a, const L* logits, const int32_t* topk_idx,
                             const float* dw, L* dlogits, long long dld, cudaStream_t stream) {
  const int warps = a.T <= 148 * 8 ? 1 : 8;
  const unsigned grid = static_cast<unsigned>((a.T + warps - 1) / warps);
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(grid), dim3(32 * warps), 0, stream, a, logits, topk_idx, dw,
                      dlogits, dld);
  };
  switch ((a.E + 31) / 32) {
    case 1: return go(route_bwd_kernel<L, 1>);
    case 2: return go(route_bwd_kernel<L, 2>);
    case 3: return go(route_bwd_kernel<L, 3>);
    case 4: return go(route_bwd_kernel<L, 4>);
    case 5: return go(route_bwd_kernel<L, 5>);
    case 6: return go(route_bwd_kernel<L, 6>);
    case 7: return go(route_bwd_kernel<L, 7>);
    default: return go(route_bwd_kernel<L, 8>);
  }
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
