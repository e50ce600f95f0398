// Newton-Schulz orthogonalisation of a batch of matrices (the update
// direction of the Muon optimiser the "moe-200m-qwen3-100b" README trains its
// matrix weights with), on 5th-generation tensor cores (tcgen05).
//
// For every matrix G [rows, cols], with X = G / (|G|_F + eps), transposed
// when rows > cols so that X is [m, n] with m <= n, each step does
//     A = X X^T          [m, m]   gram
//     B = b A + c A A    [m, m]   poly   (A is symmetric: A A = A A^T)
//     X = a X + B X      [m, n]   apply
// and the result is scale * X, transposed back.  The flops are the products':
// m^2 n + m^3 (A and B are symmetric, tiles below the diagonal are mirrored
// instead of computed) + 2 m^2 n per step.
//
// Precision.  Operands are fp16 planes with a fixed power-of-two scale (X
// times 2^10, A and B times 2^12: the singular values stay below about 1.3, so
// nothing overflows, and the small elements of early iterates stay out of
// fp16's subnormals); products accumulate in fp32.  Each value v is kept as
// hi = fp16(v) and, where it counts, lo = fp16(v - hi), 22 bits together.
//   TERMS = 3  (fp32 results) every product is hi lo + lo hi + hi hi and all
//              of X, A, B are pairs.  The tensor cores' accumulator does not
//              round to nearest, and its error grows with the inner
//              dimension (1.7e-5 of the result at n = 2048), so it takes 256
//              of it at a time and the epilogue adds those sums in fp32
//              registers: errors near fp32's own.
//   TERMS = 1  (bf16 results) products of the hi planes alone, A and B
//              without lo.  X keeps its lo plane for the a X term, except in
//              the last step: the directions whose singular values are still
//              tiny grow by a = 3.44 per step through that term, and fp16's
//              11 bits there would grow with them (relative error 3e-2 on
//              matrices of low rank against 1e-3 with the pair, simulated);
//              in the last step they grow no further, and lo times a without
//              lo times B would add error to the large ones.  The error of
//              the result, 1e-3, is below the rounding to bf16, 1.7e-3.
//              Matrices with m < 64 take three terms all the same: few
//              elements do not average the 11 bits' roundings out (7e-3 seen
//              on a 1 x 1 matrix), and their products cost next to nothing.
//
// The GEMM is persistent over CTA pairs (cluster of two, cta_group::2, tiles
// of 256 x 256): warp 0 loads (TMA, 128-byte swizzle, a ring of stages), one
// lane of warp 1 of rank 0 issues the MMAs, warps 2..9 run the epilogue from
// a double-buffered TMEM accumulator while the next tile's MMAs run.  No
// load uses cluster multicast; every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "launch.cuh"
#include "sm100.cuh"

namespace moe {
namespace {

constexpr float kScaleX = 1024.f;
constexpr float kScaleA = 4096.f;

constexpr int MODE_GRAM = 0;
constexpr int MODE_POLY = 1;
constexpr int MODE_APPLY = 2;    // X' as fp16 planes
constexpr int MODE_LAST = 3;     // the result, in the caller's type and layout

constexpr int TM = 256;          // tile rows (128 per CTA of the pair)
constexpr int TN = 256;          // tile columns
constexpr int BK = 64;
constexpr int OP_BYTES = 128 * BK * 2;    // one CTA's half of an operand tile
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int STAGES = 6;
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 64 + 32 * EPI_WARPS;
constexpr int CHUNK_KB = 4;               // TERMS 3: k-blocks of an accumulator
constexpr int TMEM_COLS = 512;            // two accumulators of 256 columns
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 256;

struct NsArgs {
  int batch, m, n;
  int tm, tn;               // tiles of a matrix (gram, poly: tm x tm, upper triangle)
  int tiles;                // tiles of a matrix that are computed
  int kblocks;              // BK-wide blocks of the inner dimension
  float alpha;              // factor of the accumulator
  float beta;               // factor of the added matrix
  const __half* add_hi;     // poly: A, apply: X (planes of the output's shape)
  const __half* add_lo;     // or null
  long long add_ld, add_bs;
  __half* out_hi;
  __half* out_lo;           // or null
  long long out_ld, out_bs;
  void* out;                // MODE_LAST
  int out_bf16, out_trans;
  long long o_ld, o_bs;     // row and matrix stride of out, in elements
  uint32_t* status;
};

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? (1u << 16) : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint64_t* bar,
                                                 int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32_rank0(bar)),
        "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(__half a, __half b) {
  __half2 v = __halves2half2(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Tile t of a matrix: (i, j), for the symmetric products of the upper
// triangle (j >= i), row by row.
template <int MODE>
__device__ __forceinline__ void tile_of(const NsArgs& a, int t, int& i, int& j) {
  if (MODE == MODE_GRAM || MODE == MODE_POLY) {
    i = 0;
    while (t >= a.tm - i) {
      t -= a.tm - i;
      ++i;
    }
    j = i + t;
  } else {
    i = t / a.tn;
    j = t - i * a.tn;
  }
}

// 32 values of one accumulator row, columns c0 .. c0 + 31 of the tile's row r:
// the added matrix's part and the stores.
template <int MODE>
__device__ __forceinline__ void finish32(const NsArgs& a, const float (&acc)[32], int b, int r,
                                         int c0, bool mirror, int lane) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = a.alpha * acc[i];
  const bool row_ok = r < a.m;
  if (MODE != MODE_GRAM) {
    if (row_ok) {
      const size_t at = static_cast<size_t>(b) * a.add_bs + static_cast<size_t>(r) * a.add_ld + c0;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const __half* src = p == 0 ? a.add_hi : a.add_lo;
        if (src == nullptr) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c0 + 8 * i >= a.add_ld) break;
          const uint4 q = *reinterpret_cast<const uint4*>(src + at + 8 * i);
          const __half2* h = reinterpret_cast<const __half2*>(&q);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(h[e]);
            v[8 * i + 2 * e] = fmaf(a.beta, f.x, v[8 * i + 2 * e]);
            v[8 * i + 2 * e + 1] = fmaf(a.beta, f.y, v[8 * i + 2 * e + 1]);
          }
        }
      }
    }
  }
  if (MODE == MODE_LAST) {
    // the caller's rows and columns: X[r][c] is out[r][c], or out[c][r]
    if (!row_ok) return;
    const size_t base = static_cast<size_t>(b) * a.o_bs;
    const int nc = a.n - c0 < 32 ? a.n - c0 : 32;
    if (a.out_bf16) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + base;
      if (a.out_trans) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < nc) o[static_cast<size_t>(c0 + i) * a.o_ld + r] = __float2bfloat16_rn(v[i]);
      } else {
        __nv_bfloat16* p = o + static_cast<size_t>(r) * a.o_ld + c0;
        if (nc == 32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 q;
            uint32_t* w = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]);
              w[e] = *reinterpret_cast<uint32_t*>(&h);
            }
            reinterpret_cast<uint4*>(p)[i] = q;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < nc) p[i] = __float2bfloat16_rn(v[i]);
        }
      }
    } else {
      float* o = static_cast<float*>(a.out) + base;
      if (a.out_trans) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < nc) o[static_cast<size_t>(c0 + i) * a.o_ld + r] = v[i];
      } else {
        float* p = o + static_cast<size_t>(r) * a.o_ld + c0;
        if (nc == 32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            reinterpret_cast<float4*>(p)[i] =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < nc) p[i] = v[i];
        }
      }
    }
    return;
  }
  const size_t obase = static_cast<size_t>(b) * a.out_bs;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    __half* plane = p == 0 ? a.out_hi : a.out_lo;
    if (plane == nullptr) break;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __half h0 = __float2half_rn(v[2 * i]), h1 = __float2half_rn(v[2 * i + 1]);
      w[i] = half2_bits(h0, h1);
      if (p == 0) {   // what the high plane leaves
        v[2 * i] -= __half2float(h0);
        v[2 * i + 1] -= __half2float(h1);
      }
    }
    if (row_ok) {
      __half* dst = plane + obase + static_cast<size_t>(r) * a.out_ld + c0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + 8 * i < a.out_ld)
          reinterpret_cast<uint4*>(dst)[i] =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    if (MODE == MODE_GRAM || MODE == MODE_POLY) {
      if (mirror) {
        // the mirrored tile: two lanes exchange a column pair, so that each
        // stores two neighbouring rows' values of one column
        const int odd = lane & 1;
        const int rr = r - odd;              // even, and out_ld is a multiple of 64
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, w[i], 1);
          const uint32_t st = odd ? __byte_perm(other, w[i], 0x7632)
                                  : __byte_perm(w[i], other, 0x5410);
          const int c = c0 + 2 * i + odd;
          if (c < a.m && rr < a.m)
            *reinterpret_cast<uint32_t*>(plane + obase + static_cast<size_t>(c) * a.out_ld + rr) =
                st;
        }
      }
    }
  }
}

template <int MODE, int TERMS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
ns_gemm_kernel(const __grid_constant__ CUtensorMap a_hi, const __grid_constant__ CUtensorMap a_lo,
               const __grid_constant__ CUtensorMap b_hi, const __grid_constant__ CUtensorMap b_lo,
               const NsArgs args) {
  constexpr bool BMN = MODE == MODE_APPLY || MODE == MODE_LAST;
  constexpr uint32_t IDESC = idesc_f16_f32(TM, TN, BMN);
  constexpr int BOX_MN = 64 * 128;   // 64 columns of 64 k-rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * OP_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  uint64_t* full_bar = bars;                      // rank 0's copy is used
  uint64_t* empty_bar = bars + STAGES;            // both copies
  uint64_t* tfull_bar = bars + 2 * STAGES;        // both copies
  uint64_t* tempty_bar = bars + 2 * STAGES + 2;   // rank 0's copy
  uint64_t* drain_bar = bars + 2 * STAGES + 4;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const long long total = static_cast<long long>(args.batch) * args.tiles;
  const int chunk_kb = TERMS == 3 ? CHUNK_KB : args.kblocks;

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 2 * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&a_hi);
    tma_prefetch_desc(&b_hi);
    if (TERMS == 3) {
      tma_prefetch_desc(&a_lo);
      tma_prefetch_desc(&b_lo);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem_base, TMEM_COLS);
    tmem_relinquish_pair();
  }
  pdl_wait();   // everything above touches no global memory
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  volatile int* abort_flag = &s_abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
      bool ok = true;
      for (long long t = pair; t < total && ok; t += npairs) {
        const int b = static_cast<int>(t / args.tiles);
        int ti, tj;
        tile_of<MODE>(args, static_cast<int>(t - static_cast<long long>(b) * args.tiles), ti, tj);
        const int arow = ti * TM + static_cast<int>(rank) * 128;
        const int bcol = tj * TN + static_cast<int>(rank) * 128;
        for (int k0 = 0; k0 < args.kblocks && ok; k0 += chunk_kb) {
          const int k1 = min(k0 + chunk_kb, args.kblocks);
          // TERMS 3: hi lo, lo hi, hi hi (the small products first)
          for (int term = TERMS == 3 ? 0 : 2; term < 3 && ok; ++term) {
            const CUtensorMap* ma = term == 1 ? &a_lo : &a_hi;
            const CUtensorMap* mb = term == 0 ? &b_lo : &b_hi;
            for (int kb = k0; kb < k1; ++kb) {
              if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
              if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * STAGE_BYTES);
              const int k = kb * BK;
              tma_load_3d_pair(sA + stage * OP_BYTES, ma, &full_bar[stage], k, arow, b);
              if (BMN) {
                tma_load_3d_pair(sB + stage * OP_BYTES, mb, &full_bar[stage], bcol, k, b);
                tma_load_3d_pair(sB + stage * OP_BYTES + BOX_MN, mb, &full_bar[stage], bcol + 64,
                                 k, b);
              } else {
                tma_load_3d_pair(sB + stage * OP_BYTES, mb, &full_bar[stage], k, bcol, b);
              }
              issued_mask |= 1u << stage;
              issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
              if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
          }
        }
      }
      pdl_trigger();   // all loads issued: the next kernel may launch
      if (!ok && rank == 0) {
        // rank 0's stage barriers count both CTAs' copies: let them all land
        for (int s = 0; s < STAGES; ++s) {
          if (!(issued_mask & (1u << s))) continue;
          const uint32_t par = (issued_phase >> s) & 1u;
          const unsigned long long t0 = globaltimer_ns();
          while (!mbar_try_wait(&full_bar[s], par))
            if (globaltimer_ns() - t0 > kWaitLimitNs) break;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer (rank 0)
    if (lane == 0 && rank == 0) {
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true, issued_any = false;
      for (long long t = pair; t < total && ok; t += npairs) {
        for (int k0 = 0; k0 < args.kblocks && ok; k0 += chunk_kb, ++it) {
          const int nkb = TERMS * (min(k0 + chunk_kb, args.kblocks) - k0);
          const int acc = it & 1;
          if (!mbar_wait(&tempty_bar[acc], ((it >> 1) & 1) ^ 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * TN;
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait(&full_bar[stage], phase, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a_addr = smem_u32(sA + stage * OP_BYTES);
            const uint32_t b_addr = smem_u32(sB + stage * OP_BYTES);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              const uint64_t bd = BMN ? smem_desc_sw128_mn(b_addr + kk * 16 * 128, BOX_MN)
                                      : smem_desc_sw128(b_addr + kk * 32);
              tc_mma_f16_pair(d_tmem, smem_desc_sw128(a_addr + kk * 32), bd, IDESC,
                              (kb | kk) != 0 ? 1u : 0u);
            }
            issued_any = true;
            tc_commit_pair(&empty_bar[stage]);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          tc_commit_pair(&tfull_bar[acc]);
        }
      }
      if (!ok && issued_any) {
        tc_commit_pair(drain_bar);
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0))
          if (globaltimer_ns() - t0 > kWaitLimitNs) break;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;              // the TMEM lanes this warp may read
    const int half = (warp - 2) >> 2;    // and its 128 of the 256 columns
    int it = 0;
    bool ok = true;
    for (long long t = pair; t < total && ok; t += npairs) {
      const int b = static_cast<int>(t / args.tiles);
      int ti, tj;
      tile_of<MODE>(args, static_cast<int>(t - static_cast<long long>(b) * args.tiles), ti, tj);
      const int warp_r0 = ti * TM + static_cast<int>(rank) * 128 + q * 32;
      const int c0 = tj * TN + half * 128;
      const int ncols = (MODE == MODE_GRAM || MODE == MODE_POLY) ? args.m : args.n;
      const uint32_t lane_addr = (static_cast<uint32_t>(q * 32) << 16) + half * 128;
      if constexpr (TERMS == 1) {
        const int acc = it & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull_bar[acc], (it >> 1) & 1, abort_flag));
        if (!ok) break;
        ++it;
        tc_fence_after();
        const uint32_t t_addr = tmem_base + acc * TN + lane_addr;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          if (warp_r0 >= args.m || c0 + c >= ncols) break;   // warp-uniform
          uint32_t v[32];
          tmem_ld16(t_addr + c, *reinterpret_cast<uint32_t(*)[16]>(&v[0]));
          tmem_ld16(t_addr + c + 16, *reinterpret_cast<uint32_t(*)[16]>(&v[16]));
          tmem_ld_wait();
          float f[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
          finish32<MODE>(args, f, b, warp_r0 + lane, c0 + c, ti != tj, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_rank0(&tempty_bar[acc]);
      } else {
        // the chunks' accumulators, added in fp32
        float sum[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) sum[i] = 0.f;
        for (int k0 = 0; k0 < args.kblocks; k0 += chunk_kb, ++it) {
          const int acc = it & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&tfull_bar[acc], (it >> 1) & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
          const uint32_t t_addr = tmem_base + acc * TN + lane_addr;
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            uint32_t v[16];
            tmem_ld16(t_addr + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_rank0(&tempty_bar[acc]);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 128; c += 32)
          if (warp_r0 < args.m && c0 + c < ncols)
            finish32<MODE>(args, *reinterpret_cast<const float(*)[32]>(&sum[c]), b,
                           warp_r0 + lane, c0 + c, ti != tj, lane);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();        // neither CTA leaves while the other still uses the pair
  if (threadIdx.x == 0 && s_abort) atomicOr(args.status, kDevTimeout);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ----------------------------------------------------- norm and first iterate
constexpr int kSumThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// Partial sums of squares in fp64 (squares of large or tiny gradients leave
// fp32's range): block (chunk, matrix) takes every nchunk-th row.
template <typename T>
__global__ void __launch_bounds__(kSumThreads)
ortho_sumsq_kernel(const T* __restrict__ g, int rows, int cols, long long ld, long long bs,
                   double* __restrict__ partial, uint32_t* __restrict__ status) {
  pdl_trigger();
  pdl_wait();
  __shared__ double s[kSumThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* base = g + static_cast<size_t>(blockIdx.y) * bs;
  constexpr int V = 16 / sizeof(T);
  const bool vec = cols % V == 0 && ld % V == 0 &&
                   (reinterpret_cast<uintptr_t>(base) & 15) == 0;
  double acc = 0.0;
  for (int r = blockIdx.x * (kSumThreads / 32) + warp; r < rows;
       r += gridDim.x * (kSumThreads / 32)) {
    const T* row = base + static_cast<size_t>(r) * ld;
    if (vec) {
      for (int c = lane * V; c < cols; c += 32 * V) {
        const uint4 q = *reinterpret_cast<const uint4*>(row + c);
        const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const double d = to_f32<T>(e[i]);
          acc = fma(d, d, acc);
        }
      }
    } else {
#pragma unroll 4
      for (int c = lane; c < cols; c += 32) {
        const double d = to_f32<T>(row[c]);
        acc = fma(d, d, acc);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) s[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < kSumThreads / 32; ++w) t += s[w];
    partial[static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x] = t;
    if (blockIdx.x == 0 && blockIdx.y == 0) *status = 0u;   // the call's status starts clear
  }
}

// X0 = G / (|G|_F + eps), scaled, as two fp16 planes [m, n]; TRANS: of G^T.
// One block per 64 x 64 tile of X0.
template <typename T, bool TRANS>
__global__ void __launch_bounds__(256)
ortho_init_kernel(const T* __restrict__ g, long long ld, long long bs,
                  const double* __restrict__ partial, int nchunk, double eps, int m, int n,
                  __half* __restrict__ hi, __half* __restrict__ lo, long long out_ld,
                  long long out_bs) {
  pdl_trigger();
  pdl_wait();
  __shared__ float s_inv;
  __shared__ float tile[64][65];
  const int b = blockIdx.z;
  if (threadIdx.x < 32) {
    double t = 0.0;
    for (int i = threadIdx.x; i < nchunk; i += 32) t += partial[static_cast<size_t>(b) * nchunk + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (threadIdx.x == 0)
      s_inv = static_cast<float>(static_cast<double>(kScaleX) / (sqrt(t) + eps));
  }
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of X0
  const T* base = g + static_cast<size_t>(b) * bs;
  // 64 x 64 elements, 16 per thread, along G's rows
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int y = (threadIdx.x >> 6) + 4 * i, x = threadIdx.x & 63;
    const int gr = (TRANS ? c0 : r0) + y, gc = (TRANS ? r0 : c0) + x;
    const int rows = TRANS ? n : m, cols = TRANS ? m : n;
    const float v = gr < rows && gc < cols ? to_f32<T>(base[static_cast<size_t>(gr) * ld + gc])
                                           : 0.f;
    if (TRANS) tile[x][y] = v; else tile[y][x] = v;
  }
  __syncthreads();
  const float inv = s_inv;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int y = (threadIdx.x >> 3) + 32 * i, x = (threadIdx.x & 7) * 8;
    const int r = r0 + y, c = c0 + x;
    if (r >= m || c >= out_ld) continue;
    uint4 qh, ql;
    uint32_t* wh = reinterpret_cast<uint32_t*>(&qh);
    uint32_t* wl = reinterpret_cast<uint32_t*>(&ql);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v0 = tile[y][x + 2 * e] * inv, v1 = tile[y][x + 2 * e + 1] * inv;
      const __half h0 = __float2half_rn(v0), h1 = __float2half_rn(v1);
      wh[e] = half2_bits(h0, h1);
      wl[e] = half2_bits(__float2half_rn(v0 - __half2float(h0)),
                         __float2half_rn(v1 - __half2float(h1)));
    }
    const size_t at = static_cast<size_t>(b) * out_bs + static_cast<size_t>(r) * out_ld + c;
    *reinterpret_cast<uint4*>(hi + at) = qh;
    *reinterpret_cast<uint4*>(lo + at) = ql;
  }
}

// ----------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return nullptr;
  }();
  return fn;
}

// A batch of row-major fp16 matrices [rows, cols], rows of ld elements, read
// in boxes of box_rows x 64; rows and columns past the matrix read as zero.
bool make_map3(CUtensorMap* map, const void* base, int rows, int cols, long long ld, int batch,
               long long bs, int box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(batch)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(bs) * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

int num_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

template <int MODE, int TERMS>
cudaError_t launch_ns(const CUtensorMap& ah, const CUtensorMap& al, const CUtensorMap& bh,
                      const CUtensorMap& bl, const NsArgs& args, cudaStream_t stream) {
  auto kern = ns_gemm_kernel<MODE, TERMS>;
  static std::atomic<unsigned long long> attr_done{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const long long total = static_cast<long long>(args.batch) * args.tiles;
  const int max_pairs = num_sms() / 2;
  const int pairs = static_cast<int>(total < max_pairs ? total : max_pairs);
  return launch_pdl(kern, dim3(2 * pairs), dim3(NUM_THREADS), SMEM_BYTES, stream, ah, al, bh, bl,
                    args);
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
inline long long pad64(int v) { return (static_cast<long long>(v) + 63) / 64 * 64; }

// Products of three terms (pairs of planes) or of the high planes alone.
bool three_terms(const OrthoShape& s) {
  return !s.out_bf16 || (s.rows < s.cols ? s.rows : s.cols) < 64;
}

struct OrthoLayout {
  size_t status, partial, xh[2], xl[2], ah, al, bh, bl, total;
};

int sum_chunks(int rows) {
  const int c = (rows + 8 - 1) / 8;   // eight rows (one per warp) at least
  return c < 64 ? c : 64;
}

OrthoLayout ortho_layout(const OrthoShape& s) {
  const int m = s.rows < s.cols ? s.rows : s.cols, n = s.rows < s.cols ? s.cols : s.rows;
  const size_t x = static_cast<size_t>(s.batch) * m * pad64(n) * 2;
  const size_t a = static_cast<size_t>(s.batch) * m * pad64(m) * 2;
  const bool pairs = three_terms(s);
  OrthoLayout L{};
  size_t o = 0;
  L.status = o;  o += 256;
  L.partial = o; o += up256(static_cast<size_t>(s.batch) * sum_chunks(s.rows) * 8);
  for (int i = 0; i < 2; ++i) {
    L.xh[i] = o; o += up256(x);
    L.xl[i] = o; o += up256(x);
  }
  L.ah = o; o += up256(a);
  L.al = o; o += pairs ? up256(a) : 0;
  L.bh = o; o += up256(a);
  L.bl = o; o += pairs ? up256(a) : 0;
  L.total = o;
  return L;
}

template <int TERMS>
cudaError_t run_steps(const OrthoShape& s, void* out, void* ws, cudaStream_t stream) {
  const OrthoLayout L = ortho_layout(s);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool trans = s.rows > s.cols;
  const int m = trans ? s.cols : s.rows, n = trans ? s.rows : s.cols;
  const long long ldx = pad64(n), lda = pad64(m);
  const long long bsx = ldx * m, bsa = lda * m;
  __half* ah = reinterpret_cast<__half*>(w + L.ah);
  __half* al = TERMS == 3 ? reinterpret_cast<__half*>(w + L.al) : nullptr;
  __half* bh = reinterpret_cast<__half*>(w + L.bh);
  __half* bl = TERMS == 3 ? reinterpret_cast<__half*>(w + L.bl) : nullptr;
  CUtensorMap xk[2][2], xn[2][2], ma[2], mb[2];   // [buffer][plane]
  for (int i = 0; i < 2; ++i)
    for (int p = 0; p < 2; ++p) {
      const void* base = w + (p ? L.xl[i] : L.xh[i]);
      if (!make_map3(&xk[i][p], base, m, n, ldx, s.batch, bsx, 128) ||
          !make_map3(&xn[i][p], base, m, n, ldx, s.batch, bsx, BK))
        return cudaErrorInvalidValue;
    }
  for (int p = 0; p < 2; ++p)
    if (!make_map3(&ma[p], p && al ? al : ah, m, m, lda, s.batch, bsa, 128) ||
        !make_map3(&mb[p], p && bl ? bl : bh, m, m, lda, s.batch, bsa, 128))
      return cudaErrorInvalidValue;
  const int tm = (m + TM - 1) / TM, tn = (n + TN - 1) / TN;
  NsArgs base{};
  base.batch = s.batch;
  base.m = m;
  base.n = n;
  base.tm = tm;
  base.tn = tn;
  base.status = reinterpret_cast<uint32_t*>(w + L.status);
  for (int step = 0; step < s.steps; ++step) {
    const int cur = step & 1;
    const bool last = step + 1 == s.steps;
    cudaError_t e;
    // A = X X^T
    NsArgs g = base;
    g.tiles = tm * (tm + 1) / 2;
    g.kblocks = (n + BK - 1) / BK;
    g.alpha = kScaleA / (kScaleX * kScaleX);
    g.out_hi = ah;
    g.out_lo = al;
    g.out_ld = lda;
    g.out_bs = bsa;
    e = launch_ns<MODE_GRAM, TERMS>(xk[cur][0], xk[cur][1], xk[cur][0], xk[cur][1], g, stream);
    if (e != cudaSuccess) return e;
    // B = b A + c A A
    NsArgs p = g;
    p.kblocks = (m + BK - 1) / BK;
    p.alpha = s.c / kScaleA;
    p.beta = s.b;
    p.add_hi = ah;
    p.add_lo = al;
    p.add_ld = lda;
    p.add_bs = bsa;
    p.out_hi = bh;
    p.out_lo = bl;
    e = launch_ns<MODE_POLY, TERMS>(ma[0], ma[1], ma[0], ma[1], p, stream);
    if (e != cudaSuccess) return e;
    // X = a X + B X
    NsArgs x = base;
    x.tiles = tm * tn;
    x.kblocks = (m + BK - 1) / BK;
    x.alpha = 1.f / kScaleA;
    x.beta = s.a;
    x.add_hi = reinterpret_cast<__half*>(w + L.xh[cur]);
    x.add_lo = TERMS == 3 || !last ? reinterpret_cast<__half*>(w + L.xl[cur]) : nullptr;
    x.add_ld = ldx;
    x.add_bs = bsx;
    if (last) {
      x.alpha *= s.scale / kScaleX;
      x.beta *= s.scale / kScaleX;
      x.out = out;
      x.out_bf16 = s.out_bf16;
      x.out_trans = trans;
      x.o_ld = s.out_ld;
      x.o_bs = s.out_bs;
      e = launch_ns<MODE_LAST, TERMS>(mb[0], mb[1], xn[cur][0], xn[cur][1], x, stream);
    } else {
      // the last step of bf16 results adds X's high plane alone
      const bool lo = TERMS == 3 || step + 2 < s.steps;
      x.out_hi = reinterpret_cast<__half*>(w + L.xh[cur ^ 1]);
      x.out_lo = lo ? reinterpret_cast<__half*>(w + L.xl[cur ^ 1]) : nullptr;
      x.out_ld = ldx;
      x.out_bs = bsx;
      e = launch_ns<MODE_APPLY, TERMS>(mb[0], mb[1], xn[cur][0], xn[cur][1], x, stream);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t run_init(const OrthoShape& s, const T* g, void* ws, cudaStream_t stream) {
  const OrthoLayout L = ortho_layout(s);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool trans = s.rows > s.cols;
  const int m = trans ? s.cols : s.rows, n = trans ? s.rows : s.cols;
  const int nchunk = sum_chunks(s.rows);
  double* partial = reinterpret_cast<double*>(w + L.partial);
  cudaError_t e =
      launch_pdl(ortho_sumsq_kernel<T>, dim3(nchunk, s.batch), dim3(kSumThreads), 0, stream, g,
                 s.rows, s.cols, s.g_ld, s.g_bs, partial,
                 reinterpret_cast<uint32_t*>(w + L.status));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(pad64(n) / 64), static_cast<unsigned>(pad64(m) / 64),
                  s.batch);
  __half* hi = reinterpret_cast<__half*>(w + L.xh[0]);
  __half* lo = reinterpret_cast<__half*>(w + L.xl[0]);
  const long long ldx = pad64(n);
  return launch_pdl(trans ? ortho_init_kernel<T, true> : ortho_init_kernel<T, false>, grid,
                    dim3(256), 0, stream, g, s.g_ld, s.g_bs,
                    static_cast<const double*>(partial), nchunk, static_cast<double>(s.eps), m, n,
                    hi, lo, ldx, ldx * m);
}

}  // namespace

size_t ortho_workspace(const OrthoShape& s) { return ortho_layout(s).total; }

cudaError_t orthogonalize(const OrthoShape& s, const void* g, void* out, void* ws,
                          cudaStream_t stream) {
  cudaError_t e = s.in_bf16 ? run_init(s, static_cast<const __nv_bfloat16*>(g), ws, stream)
                            : run_init(s, static_cast<const float*>(g), ws, stream);
  if (e != cudaSuccess) return e;
  return three_terms(s) ? run_steps<3>(s, out, ws, stream) : run_steps<1>(s, out, ws, stream);
}

// The polynomial p(x) = a x + b x^3 + c x^5 keeps the fp16 planes in range
// when, from x in [0, 1], every iterate's singular values square to at most
// 8 and |b y + c y^2| <= 8 for y = x^2 in range.  |p| is largest at an end of
// the interval or where p' = a + 3 b y + 5 c y^2 is zero.
bool ortho_coeffs_ok(float a, float b, float c, int steps) {
  double top = 1.0;   // bound of |x|
  for (int i = 0; i < steps; ++i) {
    const double y = top * top;
    if (!(y <= 8.0)) return false;
    double q = std::fabs(b * y + c * y * y);
    if (c != 0.0) {
      const double v = -b / (2.0 * c);
      if (v > 0.0 && v < y) q = std::fmax(q, std::fabs(b * v + c * v * v));
    }
    if (!(q <= 8.0)) return false;
    auto p = [&](double x) { return std::fabs(x * (a + b * x * x + c * x * x * x * x)); };
    double next = p(top);
    const double disc = 9.0 * b * b - 20.0 * a * c;
    if (c != 0.0 && disc >= 0.0) {
      for (int sgn = -1; sgn <= 1; sgn += 2) {
        const double r = (-3.0 * b + sgn * std::sqrt(disc)) / (10.0 * c);
        if (r > 0.0 && r < y) next = std::fmax(next, p(std::sqrt(r)));
      }
    } else if (c == 0.0 && b != 0.0) {
      const double r = -a / (3.0 * b);
      if (r > 0.0 && r < y) next = std::fmax(next, p(std::sqrt(r)));
    }
    top = next;
  }
  return true;
}

}  // namespace moe
