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
//   TERMS = 3  (fp32 results, and bf16 ones of more steps) every product is
//              hi lo + lo hi + hi hi and all of X, A, B are pairs.  The
//              tensor cores' accumulator does not round to nearest, and its
//              error grows with the inner dimension (1.7e-5 of the result at
//              n = 2048), so it takes 256 of it at a time and the epilogue
//              adds those sums in fp32 registers: errors near fp32's own.
//   TERMS = 1  (bf16 results) products of the hi planes alone, A and B
//              without lo.  X keeps its lo plane for the a X term, except in
//              the last step: the directions whose singular values are still
//              tiny grow by a = 3.44 per step through that term, and fp16's
//              11 bits there would grow with them (relative error 3e-2 on
//              matrices of low rank against 1e-3 with the pair, simulated);
//              in the last step they grow no further, and lo times a without
//              lo times B would add error to the large ones.  Simulated with
//              exact sums, Muon's polynomial, five steps, ten spectra from 64 x
//              64 to 640 x 1024: 0.2e-3 to 2.9e-3 of the result before its
//              rounding to bf16 (1.7e-3); six steps 4.6e-3, nine 1.3e-2, 32
//              steps 3.9e-2.  Roundings average out less where singular
//              vectors are sparse: a scaled identity of rank 43 1.2e-2 at five
//              steps.  Muon's polynomial moves the values near 1 about for
//              ever and multiplies errors as it goes, so one term is for
//              polynomials and steps that one_term_holds() accepts: Muon's up
//              to five steps, converging ones at any number.
//              Matrices with m < 64 take three terms all the same: few
//              elements do not average the 11 bits' roundings out (7e-3 seen
//              on a 1 x 1 matrix), and their products cost next to nothing.
//
// The GEMM is persistent: warp 0 loads operand tiles (TMA, 128-byte swizzle, a
// ring of stages), one lane of warp 1 issues the MMAs, warp 2 moves the added
// matrix's chunks in and the result's out (TMA, 128 rows x 64 columns), warps
// 3..10 run the epilogue from a double-buffered TMEM accumulator while the
// next tile's MMAs run.  No load uses cluster multicast; every wait is
// bounded.
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

constexpr int BK = 64;
constexpr int CHUNK_KB = 4;               // TERMS 3: k-blocks of an accumulator
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 32 * (3 + EPI_WARPS);
constexpr int PLANE_BYTES = 128 * 64 * 2; // a chunk: 128 rows x 64 columns of fp16
constexpr int BOX_MN = 64 * 128;          // 64 columns of 64 k-rows, MN-major

// Tile shapes: CG CTAs (1, or a cta_group::2 pair) per tile of 128 CG x TN.
template <int TERMS, int CG, int TN>
struct Cfg {
  static constexpr int TM = 128 * CG;
  static constexpr int PLANES = TERMS == 3 ? 2 : 1;
  static constexpr int A_BYTES = 128 * BK * 2;              // one plane, one CTA
  static constexpr int B_BYTES = TN / CG * BK * 2;
  static constexpr int STAGE_BYTES = PLANES * (A_BYTES + B_BYTES);
  // chunk planes: 3 chunks of two planes where a tile has several chunks and
  // the stages leave the room (96 KB of planes)
  static constexpr int EPI_PLANES =
      STAGE_BYTES >= 65536 ? 2 : (STAGE_BYTES >= 49152 || TN == 64) ? 4 : 6;
  static constexpr int EPI_BYTES = EPI_PLANES * PLANE_BYTES;
  static constexpr int STAGES_MAX = (232448 - 1280 - EPI_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_MAX > 8 ? 8 : STAGES_MAX;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + 1024 + 256;
  static constexpr int TMEM_COLS = 2 * TN;                  // two accumulators
  static_assert(STAGES >= 2 && SMEM_BYTES <= 232448, "shared memory");
};

// Chunk buffers of a launch: planes of one, and how many there are.
template <int MODE, int TERMS, int CG, int TN>
struct Chunks {
  static constexpr int OWN = TERMS == 3 || MODE == MODE_APPLY ? 2 : 1;
  // gram, poly: as many again for the mirrored tile, where there is room
  // (else it is stored from the registers)
  static constexpr bool STAGED = (MODE == MODE_GRAM || MODE == MODE_POLY) &&
                                 Cfg<TERMS, CG, TN>::EPI_PLANES >= 2 * OWN;
  static constexpr int PLANES = STAGED ? 2 * OWN : OWN;
  static constexpr int BUFS = Cfg<TERMS, CG, TN>::EPI_PLANES / PLANES;
  static constexpr int BYTES = PLANES * PLANE_BYTES;
};
constexpr int MAX_BUFS = 6;

struct NsArgs {
  int batch, m, n;
  int tm, tn;               // tiles of a matrix along its rows and columns
  int tiles;                // tiles of a matrix that are computed
  int full;                 // gram, poly: all tiles are, none is mirrored
  int kblocks;              // BK-wide blocks of the inner dimension
  float alpha;              // factor of the accumulator
  float beta;               // factor of the added matrix (poly: A, apply: X)
  int add_planes;           // its planes, 0 for gram
  int out_planes;           // planes written (not MODE_LAST)
  __half* out_hi;           // gram, poly: for the mirrored tiles
  __half* out_lo;
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

// 3-D tile load into this CTA's shared memory; CG 2: counted on the pair's
// rank-0 barrier.
template <int CG>
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z) {
  if constexpr (CG == 2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32_rank0(bar)),
          "r"(x), "r"(y), "r"(z)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)),
          "r"(x), "r"(y), "r"(z)
        : "memory");
  }
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int32_t x,
                                             int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
      ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Wait until at most N of this thread's committed bulk stores still read
// their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  if constexpr (CG == 2)
    tc_mma_f16_pair(d, a, b, idesc, accumulate);
  else
    tc_mma_f16(d, a, b, idesc, accumulate);
}
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CG == 2) tc_commit_pair(bar); else tc_commit(bar);
}

// Distributed shared memory: a variable's address in another CTA of the
// cluster, stores to it, and barriers across it.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// The two halves of cluster_sync_all.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_cluster() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}
// mbar_wait that also acquires what other CTAs of the cluster wrote.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity,
                                                  volatile int* abort_flag) {
  const bool ok = mbar_wait(bar, parity, abort_flag);
  fence_cluster();
  return ok;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}

// Tile t of a matrix: rows i, columns j.  The symmetric products compute the
// tiles that reach the diagonal or lie above it, j >= i TM / TN, row by row
// (all tiles where every one has a CTA of its own: mirroring would only add
// to the launch's last microseconds).
template <int MODE, int RATIO>
__device__ __forceinline__ void tile_of(const NsArgs& a, int t, int& i, int& j) {
  if ((MODE == MODE_GRAM || MODE == MODE_POLY) && !a.full) {
    i = 0;
    while (t >= a.tn - RATIO * i) {
      t -= a.tn - RATIO * i;
      ++i;
    }
    j = RATIO * i + t;
  } else {
    i = t / a.tn;
    j = t - i * a.tn;
  }
}

// 16-byte piece c (0..7) of a chunk's row, 128-byte swizzle.
__device__ __forceinline__ uint4* piece(uint8_t* plane, int row, int c) {
  return reinterpret_cast<uint4*>(plane + row * 128 + ((c ^ (row & 7)) << 4));
}

// 32 accumulator values of tile row `row` (matrix row r), columns c0 .. c0 + 31
// of the matrix: the added planes' part, read from the chunk buffer, and the
// result's planes, left in their place there.  `half`: which 32 columns of
// the chunk.
template <int MODE, bool STAGED>
__device__ __forceinline__ void finish32(const NsArgs& a, const float (&acc)[32], uint8_t* buf,
                                         int b, int row, int r, int c0, int half, bool mirror,
                                         int lane) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = a.alpha * acc[i];
  if (MODE != MODE_GRAM) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (p >= a.add_planes) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 q = *piece(buf + p * PLANE_BYTES, row, half * 4 + i);
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
  if (MODE == MODE_LAST) {
    const size_t base = static_cast<size_t>(b) * a.o_bs;
    if (a.out_trans) {
      // X[r][c] is out[c][r]: neighbouring lanes store neighbouring elements
      if (r >= a.m) return;
      const int nc = a.n - c0 < 32 ? a.n - c0 : 32;
      if (a.out_bf16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + base;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < nc) o[static_cast<size_t>(c0 + i) * a.o_ld + r] = __float2bfloat16_rn(v[i]);
      } else {
        float* o = static_cast<float*>(a.out) + base;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < nc) o[static_cast<size_t>(c0 + i) * a.o_ld + r] = v[i];
      }
      return;
    }
    // staged in the chunk (fp32: columns 0-15 in the first plane's place,
    // 16-31 in the second's), then stored along the rows
    const int row0 = row - lane, r0 = r - lane;
    if (a.out_bf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *piece(buf, row, half * 4 + i) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + base + c0;
      if (c0 + 32 <= a.n && a.o_ld % 8 == 0 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int y = 8 * i + (lane >> 2);
          if (r0 + y < a.m)
            *reinterpret_cast<uint4*>(o + static_cast<size_t>(r0 + y) * a.o_ld + (lane & 3) * 8) =
                *piece(buf, row0 + y, half * 4 + (lane & 3));
        }
      } else if (c0 + lane < a.n) {
        for (int y = 0; y < 32 && r0 + y < a.m; ++y)
          o[static_cast<size_t>(r0 + y) * a.o_ld + lane] =
              reinterpret_cast<const __nv_bfloat16*>(
                  piece(buf, row0 + y, half * 4 + (lane >> 3)))[lane & 7];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *piece(buf + (i >> 2) * PLANE_BYTES, row, half * 4 + (i & 3)) =
            make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                       __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
      __syncwarp();
      float* o = static_cast<float*>(a.out) + base + c0;
      if (c0 + 32 <= a.n && a.o_ld % 4 == 0 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int y = 4 * i + (lane >> 3), c = lane & 7;
          if (r0 + y < a.m)
            *reinterpret_cast<uint4*>(o + static_cast<size_t>(r0 + y) * a.o_ld + c * 4) =
                *piece(buf + (c >> 2) * PLANE_BYTES, row0 + y, half * 4 + (c & 3));
        }
      } else if (c0 + lane < a.n) {
        for (int y = 0; y < 32 && r0 + y < a.m; ++y)
          o[static_cast<size_t>(r0 + y) * a.o_ld + lane] = reinterpret_cast<const float*>(
              piece(buf + (lane >> 4) * PLANE_BYTES, row0 + y,
                    half * 4 + ((lane >> 2) & 3)))[lane & 3];
      }
    }
    return;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (p >= a.out_planes) break;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      // two at a time: the packed conversion runs at full rate
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = half2_bits(h);
      if (p == 0) {   // what the high plane leaves
        const float2 f = __half22float2(h);
        v[2 * i] -= f.x;
        v[2 * i + 1] -= f.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *piece(buf + p * PLANE_BYTES, row, half * 4 + i) =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    if (MODE == MODE_GRAM || MODE == MODE_POLY) {
      if (STAGED && mirror) {
        // the mirrored tile: 64 of its rows (this chunk's columns) in two
        // boxes of 64 columns; two lanes exchange a column pair, so that each
        // stores two neighbouring rows' values of one column
        const int odd = lane & 1, rr = row & ~1;
        uint8_t* box = buf + (a.out_planes + p) * PLANE_BYTES + (rr >> 6) * BOX_MN;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, w[i], 1);
          const uint32_t st = odd ? __byte_perm(other, w[i], 0x7632)
                                  : __byte_perm(w[i], other, 0x5410);
          const int y = half * 32 + 2 * i + odd;
          *reinterpret_cast<uint32_t*>(box + y * 128 + ((((rr & 63) >> 3) ^ (y & 7)) << 4) +
                                       (rr & 7) * 2) = st;
        }
      } else if (mirror) {
        // the mirrored tile, straight to memory: two lanes exchange a column
        // pair, so that each stores two neighbouring rows' values of one column
        __half* plane = (p == 0 ? a.out_hi : a.out_lo) + static_cast<size_t>(b) * a.out_bs;
        const int odd = lane & 1;
        const int rr = r - odd;              // even, and out_ld is a multiple of 64
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, w[i], 1);
          const uint32_t st = odd ? __byte_perm(other, w[i], 0x7632)
                                  : __byte_perm(w[i], other, 0x5410);
          const int c = c0 + 2 * i + odd;
          if (c < a.m && rr < a.m)
            *reinterpret_cast<uint32_t*>(plane + static_cast<size_t>(c) * a.out_ld + rr) = st;
        }
      }
    }
  }
}

// a_*, b_*: the operands' planes; add_*: the added matrix, out_*: the result,
// both in chunks of 128 rows x 64 columns.
struct NsMaps {
  CUtensorMap a[2], b[2], add[2], out[2];
  CUtensorMap mir[2];   // gram, poly: the result in boxes of 64 rows x 64 columns
};

// Bound, per launch: staging operands from L2 for large batches (about 38 bytes
// a cycle and SM), the launch gap, first loads and epilogue (5 to 6 us) for few
// tiles.  Measured, 32 of [768, 2048] bf16: gram 49 us (tensor pipe active 68 %
// of cycles, 1.06 PFLOP/s with the mirrored halves of diagonal tiles), poly 27
// us, apply 90 us (0.86 PFLOP/s, 4.5 TB/s of DRAM for the planes); 3 of [333,
// 517] fp32: 8 to 9 us each.
//
// SPLIT > 1 (128 x 64 tiles, one per cluster): the CTAs of a cluster take a part
// of the inner dimension each, hand the rows they do not finish to the CTA
// that does through distributed shared memory, and finish 128 / SPLIT rows of
// the tile.  With few tiles this shortens both the staging, which one SM's
// share of L2 bandwidth bounds, and the epilogue.
template <int MODE, int TERMS, int CG, int TN, int SPLIT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
ns_gemm_kernel(const __grid_constant__ NsMaps maps, const NsArgs args) {
  using C = Cfg<TERMS, CG, TN>;
  static_assert(SPLIT == 1 || (CG == 1 && TN == 64), "split tiles");
  constexpr int ROWS = 128 / SPLIT;               // rows of a tile this CTA finishes
  constexpr int FINISHERS = EPI_WARPS / SPLIT;    // and its warps that do
  constexpr int STAGES = C::STAGES;
  constexpr int RATIO = C::TM / TN;
  constexpr bool BMN = MODE == MODE_APPLY || MODE == MODE_LAST;
  constexpr uint32_t IDESC = idesc_f16_f32(C::TM, TN, BMN);
  constexpr int BUFS = Chunks<MODE, TERMS, CG, TN>::BUFS;
  constexpr int BUF_BYTES = Chunks<MODE, TERMS, CG, TN>::BYTES;
  static_assert(BUFS >= 1 && BUFS <= MAX_BUFS, "chunk buffers");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sEpi = smem + STAGES * C::STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sEpi + C::EPI_BYTES);
  uint64_t* full_bar = bars;                      // CG 2: rank 0's copy is used
  uint64_t* empty_bar = bars + STAGES;            // both copies
  uint64_t* tfull_bar = bars + 2 * STAGES;        // both copies
  uint64_t* tempty_bar = bars + 2 * STAGES + 2;   // rank 0's copy
  uint64_t* ready_bar = bars + 2 * STAGES + 4;    // a chunk buffer may be used
  uint64_t* done_bar = ready_bar + MAX_BUFS;      // and has been
  uint64_t* drain_bar = done_bar + MAX_BUFS;
  uint64_t* parts_bar = drain_bar + 1;            // SPLIT: the other CTAs' sums are here
  // their place, in planes a launch of one unmirrored tile a CTA does not use
  float* parts = reinterpret_cast<float*>(sEpi + 2 * PLANE_BYTES);
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  pdl_trigger();   // the grid is resident at once: the next kernel may set up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const int part = SPLIT > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / (CG * SPLIT), units = gridDim.x / (CG * SPLIT);
  const int k_first = args.kblocks * part / SPLIT, k_last = args.kblocks * (part + 1) / SPLIT;
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
      mbar_init(&tempty_bar[i], CG * EPI_WARPS);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(&ready_bar[i], 1);
      mbar_init(&done_bar[i], FINISHERS);
    }
    mbar_init(drain_bar, 1);
    if (SPLIT > 1) mbar_init(parts_bar, (SPLIT - 1) * FINISHERS);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    for (int p = 0; p < C::PLANES; ++p) {
      tma_prefetch_desc(&maps.a[p]);
      tma_prefetch_desc(&maps.b[p]);
    }
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(&s_tmem_base, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&s_tmem_base, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  pdl_wait();   // everything above touches no global memory
  tc_fence_before();
  __syncthreads();
  if constexpr (CG * SPLIT > 1) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  volatile int* abort_flag = &s_abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
      bool ok = true;
      for (long long t = unit; t < total && ok; t += units) {
        const int b = static_cast<int>(t / args.tiles);
        int ti, tj;
        tile_of<MODE, RATIO>(args, static_cast<int>(t - static_cast<long long>(b) * args.tiles),
                             ti, tj);
        const int arow = ti * C::TM + static_cast<int>(rank) * 128;
        const int bcol = tj * TN + static_cast<int>(rank) * (TN / CG);
        for (int kb = k_first; kb < k_last; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], CG * C::STAGE_BYTES);
          uint8_t* sA = smem + stage * C::STAGE_BYTES;
          uint8_t* sB = sA + C::PLANES * C::A_BYTES;
          const int k = kb * BK;
#pragma unroll
          for (int p = 0; p < C::PLANES; ++p) {
            tma_load_3d<CG>(sA + p * C::A_BYTES, &maps.a[p], &full_bar[stage], k, arow, b);
            if (BMN) {
#pragma unroll
              for (int x = 0; x < TN / CG; x += 64)
                tma_load_3d<CG>(sB + p * C::B_BYTES + (x / 64) * BOX_MN, &maps.b[p],
                                &full_bar[stage], bcol + x, k, b);
            } else {
              tma_load_3d<CG>(sB + p * C::B_BYTES, &maps.b[p], &full_bar[stage], k, bcol, b);
            }
          }
          issued_mask |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && rank == 0) {
        // (CG 2: rank 0's stage barriers count both CTAs' copies) let them land
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
      for (long long t = unit; t < total && ok; t += units) {
        for (int k0 = k_first; k0 < k_last && ok; k0 += chunk_kb, ++it) {
          const int k1 = min(k0 + chunk_kb, k_last);
          const int acc = it & 1;
          if (!mbar_wait(&tempty_bar[acc], ((it >> 1) & 1) ^ 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * TN;
          for (int kb = k0; kb < k1; ++kb) {
            if (!mbar_wait(&full_bar[stage], phase, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a_addr = smem_u32(smem + stage * C::STAGE_BYTES);
            const uint32_t b_addr = a_addr + C::PLANES * C::A_BYTES;
            // TERMS 3: hi lo, lo hi, hi hi (the small products first)
#pragma unroll
            for (int term = 3 - TERMS; term < 3; ++term) {
              const uint32_t at = a_addr + (TERMS == 3 && term == 1 ? C::A_BYTES : 0);
              const uint32_t bt = b_addr + (TERMS == 3 && term == 0 ? C::B_BYTES : 0);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk) {
                const uint64_t bd = BMN ? smem_desc_sw128_mn(bt + kk * 16 * 128, BOX_MN)
                                        : smem_desc_sw128(bt + kk * 32);
                mma<CG>(d_tmem, smem_desc_sw128(at + kk * 32), bd, IDESC,
                        (kb != k0 || kk != 0 || term != 3 - TERMS) ? 1u : 0u);
              }
            }
            issued_any = true;
            commit<CG>(&empty_bar[stage]);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          commit<CG>(&tfull_bar[acc]);
        }
      }
      if (!ok && issued_any) {
        commit<CG>(drain_bar);
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0))
          if (globaltimer_ns() - t0 > kWaitLimitNs) break;
      }
    }
  } else if (warp == 2) {
    // ------------- mover: the added matrix's chunks in, the result's chunks out
    if (lane == 0) {
      long long in_t = unit;       // the next chunk to make ready
      int in_c = 0;
      auto make_ready = [&](int buf) {
        if (in_t >= total) return;
        const int b = static_cast<int>(in_t / args.tiles);
        int ti, tj;
        tile_of<MODE, RATIO>(
            args, static_cast<int>(in_t - static_cast<long long>(b) * args.tiles), ti, tj);
        if (MODE == MODE_GRAM) {
          mbar_arrive(&ready_bar[buf]);
        } else {
          mbar_arrive_expect_tx(&ready_bar[buf], args.add_planes * ROWS * 128);
          for (int p = 0; p < args.add_planes; ++p)
            tma_load_3d<1>(sEpi + buf * BUF_BYTES + p * PLANE_BYTES + part * ROWS * 128,
                           &maps.add[p], &ready_bar[buf], tj * TN + in_c * 64,
                           ti * C::TM + static_cast<int>(rank) * 128 + part * ROWS, b);
        }
        if (++in_c == TN / 64) {
          in_c = 0;
          in_t += units;
        }
      };
      for (int i = 0; i < BUFS; ++i) make_ready(i);
      int held = -1;   // the buffer whose store may still be reading it
      bool ok = true;
      int s = 0;
      for (long long t = unit; t < total && ok; t += units) {
        const int b = static_cast<int>(t / args.tiles);
        int ti, tj;
        tile_of<MODE, RATIO>(args, static_cast<int>(t - static_cast<long long>(b) * args.tiles),
                             ti, tj);
        const int ncols = BMN ? args.n : args.m;
        for (int c = 0; c < TN / 64; ++c, ++s) {
          const int buf = s % BUFS;
          if (!mbar_wait(&done_bar[buf], (s / BUFS) & 1, abort_flag)) { ok = false; break; }
          const int row = ti * C::TM + static_cast<int>(rank) * 128 + part * ROWS;
          const int col = tj * TN + c * 64;
          const bool store = MODE != MODE_LAST && row < args.m && col < ncols;
          if (store) {
            for (int p = 0; p < args.out_planes; ++p)
              tma_store_3d(&maps.out[p],
                           sEpi + buf * BUF_BYTES + p * PLANE_BYTES + part * ROWS * 128, col, row, b);
            if (Chunks<MODE, TERMS, CG, TN>::STAGED && !args.full && tj >= RATIO * (ti + 1)) {
              for (int p = 0; p < args.out_planes; ++p)
                for (int x = 0; x < 128 && row + x < args.m; x += 64)
                  tma_store_3d(&maps.mir[p],
                               sEpi + buf * BUF_BYTES + (args.out_planes + p) * PLANE_BYTES +
                                   (x / 64) * BOX_MN,
                               row + x, col, b);
            }
            bulk_commit();
          }
          // a buffer is handed on one chunk late, while its successor's store
          // is in flight
          if (held >= 0) {
            if (store) bulk_wait_read<1>(); else bulk_wait_read<0>();
            make_ready(held);
            held = -1;
          }
          if (!store) {
            make_ready(buf);
          } else if (BUFS == 1) {
            bulk_wait_read<0>();
            make_ready(buf);
          } else {
            held = buf;
          }
        }
      }
      bulk_wait_all();
      if (!ok && MODE != MODE_GRAM) {
        // let the chunk loads in flight land
        for (int i = 0; i < BUFS; ++i) {
          const unsigned long long t0 = globaltimer_ns();
          const uint32_t par = ((s + ((i - s % BUFS) + BUFS) % BUFS) / BUFS) & 1;
          while (!mbar_try_wait(&ready_bar[i], par))
            if (globaltimer_ns() - t0 > kWaitLimitNs) break;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;              // the TMEM lanes this warp may read
    const int half = (warp - 3) >> 2;    // and its 32 columns of every 64
    const int row = q * 32 + lane;
    const uint32_t lane_addr = (static_cast<uint32_t>(q * 32) << 16) + half * 32;
    int it = 0, s = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag));
    };
    auto release = [&](uint64_t* bar) {   // an accumulator, to rank 0's issuer
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_rank0(bar); else mbar_arrive(bar);
      }
    };
    for (long long t = unit; t < total && ok; t += units) {
      const int b = static_cast<int>(t / args.tiles);
      int ti, tj;
      tile_of<MODE, RATIO>(args, static_cast<int>(t - static_cast<long long>(b) * args.tiles), ti,
                           tj);
      const int r = ti * C::TM + static_cast<int>(rank) * 128 + row;
      const bool mirror = !args.full && tj >= RATIO * (ti + 1);
      // one chunk: its buffer, the 32 sums, and the hand-over to the mover
      auto chunk = [&](int c, float (&f)[32]) {
        if constexpr (SPLIT > 1) {
          const int owner = q * SPLIT / 4, rr = row % ROWS;   // who finishes these rows
          if (owner != part) {
            const uint32_t dst = map_rank(
                smem_u32(parts + (part * 64 + half * 32) * ROWS + rr), owner);
#pragma unroll
            for (int i = 0; i < 32; ++i) st_cluster_f32(dst + i * ROWS * 4, f[i]);
            fence_cluster();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(parts_bar), owner));
            return true;
          }
          if (!__all_sync(0xffffffffu, mbar_wait_cluster(parts_bar, 0, abort_flag))) return false;
          float own[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            own[i] = f[i];
            f[i] = 0.f;
          }
#pragma unroll
          for (int p = 0; p < SPLIT; ++p)      // in the order of the inner dimension
#pragma unroll
            for (int i = 0; i < 32; ++i)
              f[i] += p == part ? own[i] : parts[(p * 64 + half * 32 + i) * ROWS + rr];
        }
        const int buf = s % BUFS;
        if (!wait(&ready_bar[buf], (s / BUFS) & 1)) return false;
        finish32<MODE, Chunks<MODE, TERMS, CG, TN>::STAGED>(args, f, sEpi + buf * BUF_BYTES, b, row, r, tj * TN + c * 64 + half * 32,
                       half, mirror, lane);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&done_bar[buf]);
        ++s;
        return true;
      };
      if constexpr (TERMS == 1) {
        const int acc = it & 1;
        ok = wait(&tfull_bar[acc], (it >> 1) & 1);
        if (!ok) break;
        ++it;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < TN / 64 && ok; ++c) {
          uint32_t v[32];
          const uint32_t t_addr = tmem_base + acc * TN + lane_addr + c * 64;
          tmem_ld16(t_addr, *reinterpret_cast<uint32_t(*)[16]>(&v[0]));
          tmem_ld16(t_addr + 16, *reinterpret_cast<uint32_t(*)[16]>(&v[16]));
          tmem_ld_wait();
          if (c + 1 == TN / 64) release(&tempty_bar[acc]);
          float f[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
          ok = chunk(c, f);
        }
      } else {
        // the accumulators of CHUNK_KB k-blocks, added in fp32
        float sum[TN / 64][32];
#pragma unroll
        for (int c = 0; c < TN / 64; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
        for (int k0 = k_first; k0 < k_last; k0 += chunk_kb, ++it) {
          const int acc = it & 1;
          ok = wait(&tfull_bar[acc], (it >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < TN / 64; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[16];
              tmem_ld16(tmem_base + acc * TN + lane_addr + c * 64 + 16 * h, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[c][16 * h + i] += __uint_as_float(v[i]);
            }
          release(&tempty_bar[acc]);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < TN / 64; ++c)
          if (ok) ok = chunk(c, sum[c]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (CG * SPLIT > 1) cluster_sync_all();   // no CTA leaves the others early
  if (threadIdx.x == 0 && s_abort) atomicOr(args.status, kDevTimeout);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else
      tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ------------------------------------------- up to 128 rows: one launch in all
// A matrix with m <= 128 and n <= 2048 (one or two of them: n <= 4096) stays in
// the shared memory of one cluster for the whole iteration: CTA `rank` of CL holds the columns
// [64 nbx rank, 64 nbx (rank + 1)) of X, and every CTA all of A and B, as pairs of
// planes in boxes of 128 rows x 64 columns (one layout serves as the
// K-major operands of the gram and poly products and as the MN-major one of
// the apply product).  Per step:
//   gram    each CTA multiplies its columns (K = 64 nbx); the CL partial
//           products meet in their rows' owners through distributed shared
//           memory, are added there in rank order in fp32, and A's planes go
//           to every CTA
//   poly    B = b A + c A A, by every CTA for itself, in A's place
//   apply   X = a X + B X on its own columns, in place
// What bounds it is latency: the products of one tile (24 with three terms, 8
// with one, at 90 cycles), their epilogues' conversions, four block barriers a step,
// and two cluster barriers with their exchanges (four where rows are received in
// A's place; [128, 128] fp32 39.5 us;
// [100, 192] 46.7 us, bf16 31.1); 17 launches of the tiled kernel, 4 us each with
// all their loads and stores, become one.
constexpr int CL_ROWS = 128;
constexpr int CL_BOX = CL_ROWS * 128;            // bytes of a box's plane
constexpr int CL_MAX_BOXES = 4;                  // of X per CTA
constexpr int CL_THREADS = 512;
constexpr int CL_RECV_BYTES = CL_ROWS * CL_ROWS * 4;

struct ClArgs {
  int batch, m, n, nbx, steps;
  float a, b, c, scale;
  double eps;
  const void* g;
  long long g_ld, g_bs;
  void* out;
  int out_bf16;
  long long o_ld, o_bs;
  int recv_apart;     // the receive buffer has its own place, else A's
  uint32_t* status;
};

template <int N>
__device__ __forceinline__ void st_cluster(uint32_t addr, const uint32_t (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "words of a store");
  if constexpr (N == 4)
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
  else if constexpr (N == 2)
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};"
                 ::"r"(addr), "r"(v[0]), "r"(v[1]) : "memory");
  else
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v[0]) : "memory");
}
__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// Splits 2 values into words of the two planes.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = half2_bits(h);
  lo = half2_bits(__floats2half2_rn(x - f.x, y - f.y));
}

// Splits 8 values into 16-byte pieces of the two planes.
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
  uint32_t* wh = reinterpret_cast<uint32_t*>(&hi);
  uint32_t* wl = reinterpret_cast<uint32_t*>(&lo);
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(v[2 * i], v[2 * i + 1], wh[i], wl[i]);
}

// v = beta (hi + lo) + v over 8 elements of a row (PAIR; else of hi alone).
template <bool PAIR>
__device__ __forceinline__ void add8(const uint4& hi, const uint4& lo, float beta, float* v) {
  const __half2* h = reinterpret_cast<const __half2*>(&hi);
  const __half2* l = reinterpret_cast<const __half2*>(&lo);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = __half22float2(h[i]);
    if (PAIR) {
      const float2 g = __half22float2(l[i]);
      f.x += g.x;
      f.y += g.y;
    }
    v[2 * i] = fmaf(beta, f.x, v[2 * i]);
    v[2 * i + 1] = fmaf(beta, f.y, v[2 * i + 1]);
  }
}

template <typename T, bool TRANS, int CL, int TERMS>
__global__ void __launch_bounds__(CL_THREADS, 1)
ns_cluster_kernel(const ClArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int nbx = args.nbx;
  uint8_t* xh = smem;                              // X: nbx boxes of each plane
  uint8_t* xl = xh + nbx * CL_BOX;
  uint8_t* ah = xl + nbx * CL_BOX;                 // A, then B: two boxes of each plane
  uint8_t* al = ah + 2 * CL_BOX;                   // (TERMS 3)
  float* recv =
      reinterpret_cast<float*>(args.recv_apart ? ah + (TERMS == 3 ? 4 : 2) * CL_BOX : ah);
  __shared__ uint64_t s_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ double s_part[CL_THREADS / 32];
  __shared__ double s_norm[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CL > 1 ? cluster_ctarank() : 0u;
  const int b = blockIdx.x / CL;
  const int m = args.m;
  const int c_first = 64 * nbx * static_cast<int>(rank);   // first column of this CTA
  const T* g = static_cast<const T*>(args.g) + static_cast<size_t>(b) * args.g_bs;

  pdl_trigger();
  if (tid == 0) {
    s_abort = 0;
    mbar_init(&s_bar, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  __syncwarp();
  // a CTA's shared memory may be stored to from its start on: waited for below
  if constexpr (CL > 1) cluster_arrive();
  pdl_wait();
  if (blockIdx.x == 0 && tid == 0) *args.status = 0u;   // the call's status starts clear
  // ------------------------------------------------------------- the norm
  // G is read once; until the norm is known its fp32 bits wait in the planes,
  // the upper half in the first, the lower in the second.
  double acc = 0.0;
  if (!TRANS) {
    // a warp per row of a box, two columns per lane
#pragma unroll 8
    for (int i = warp; i < nbx * CL_ROWS; i += CL_THREADS / 32) {
      const int bx = i / CL_ROWS, r = i % CL_ROWS;
      const int c = c_first + 64 * bx + 2 * lane;
      const T* p = g + static_cast<size_t>(r) * args.g_ld + c;
      const float v0 = r < m && c < args.n ? to_f32<T>(p[0]) : 0.f;
      const float v1 = r < m && c + 1 < args.n ? to_f32<T>(p[1]) : 0.f;
      acc = fma(static_cast<double>(v0), static_cast<double>(v0), acc);
      acc = fma(static_cast<double>(v1), static_cast<double>(v1), acc);
      const int off = bx * CL_BOX + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
      const uint32_t b0 = __float_as_uint(v0), b1 = __float_as_uint(v1);
      *reinterpret_cast<uint32_t*>(xh + off) = __byte_perm(b0, b1, 0x7632);
      *reinterpret_cast<uint32_t*>(xl + off) = __byte_perm(b0, b1, 0x5410);
    }
  } else {
    // a warp per 32 rows of a column
#pragma unroll 8
    for (int i = warp; i < 64 * nbx * 4; i += CL_THREADS / 32) {
      const int cc = i >> 2, r = (i & 3) * 32 + lane, c = c_first + cc;
      const float v = r < m && c < args.n
                          ? to_f32<T>(g[static_cast<size_t>(c) * args.g_ld + r])
                          : 0.f;
      acc = fma(static_cast<double>(v), static_cast<double>(v), acc);
      const int off = (cc >> 6) * CL_BOX + r * 128 + ((((cc & 63) >> 3) ^ (r & 7)) << 4) +
                      (cc & 7) * 2;
      *reinterpret_cast<uint16_t*>(xh + off) = static_cast<uint16_t>(__float_as_uint(v) >> 16);
      *reinterpret_cast<uint16_t*>(xl + off) = static_cast<uint16_t>(__float_as_uint(v));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) s_part[warp] = acc;
  __syncthreads();
  if constexpr (CL > 1) cluster_wait();   // every CTA of the cluster has started
  if (tid == 0) {
    double t = 0.0;
    for (int w = 0; w < CL_THREADS / 32; ++w) t += s_part[w];
    if (CL == 1) s_norm[0] = t;
    else
      for (uint32_t q = 0; q < CL; ++q) st_cluster_f64(map_rank(smem_u32(&s_norm[rank]), q), t);
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (CL > 1) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  double norm2 = 0.0;
#pragma unroll
  for (int q = 0; q < CL; ++q) norm2 += s_norm[q];
  const float inv = static_cast<float>(static_cast<double>(kScaleX) / (sqrt(norm2) + args.eps));
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  // --------------------------------------------------------- first iterate
  // (the barrier above is the block's too)
  for (int i = tid; i < nbx * CL_BOX / 16; i += CL_THREADS) {
    uint4* ph = reinterpret_cast<uint4*>(xh) + i;
    uint4* pl = reinterpret_cast<uint4*>(xl) + i;
    const uint4 vh = *ph, vl = *pl;
    const uint32_t* wh = reinterpret_cast<const uint32_t*>(&vh);
    const uint32_t* wl = reinterpret_cast<const uint32_t*>(&vl);
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(__byte_perm(wl[e], wh[e], 0x5410)) * inv;
      f[2 * e + 1] = __uint_as_float(__byte_perm(wl[e], wh[e], 0x7632)) * inv;
    }
    uint4 hi, lo;
    split8(f, hi, lo);
    *ph = hi;
    *pl = lo;
  }
  // ----------------------------------------------------------------- steps
  const int q = warp & 3, quarter = warp >> 2;     // rows, and 32 of 128 columns
  const int row = q * 32 + lane;
  const int sq_col = quarter * 32;                 // of A and B
  uint8_t* sq_h = ah + (quarter >> 1) * CL_BOX;    // their box, and the piece in it
  uint8_t* sq_l = al + (quarter >> 1) * CL_BOX;
  const int sq_piece = (quarter & 1) * 4;
  const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
  const uint32_t d_sq = tmem, d_x = tmem + 128;    // accumulators: A or A A, B X
  const int mp = (m + 15) & ~15;                   // rows that are not all zero
  const uint32_t id_sq = idesc_f16_f32(128, mp, false);
  const uint32_t id_x = idesc_f16_f32(128, 64 * nbx, true);
  uint32_t phase = 0;
  auto load32 = [&](uint32_t taddr, float factor, float (&f)[32]) {
    uint32_t v[32];
    tmem_ld16(taddr + lane_addr, *reinterpret_cast<uint32_t(*)[16]>(&v[0]));
    tmem_ld16(taddr + lane_addr + 16, *reinterpret_cast<uint32_t(*)[16]>(&v[16]));
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = factor * __uint_as_float(v[i]);
  };
  auto mma_done = [&]() {   // every thread waits for the issued products
    mbar_wait(&s_bar, phase, abort_flag);
    phase ^= 1u;
    tc_fence_after();
  };
  for (int step = 0; step < args.steps; ++step) {
    const bool last = step + 1 == args.steps;
    fence_proxy_async_all();
    tc_fence_before();
    __syncthreads();
    // ----------------------------------------------------------------- gram
    if (tid == 0) {
      tc_fence_after();
      uint32_t first = 0;
      for (int term = 3 - TERMS; term < 3; ++term)   // hi lo, lo hi, hi hi
        for (int bx = 0; bx < nbx; ++bx) {
          const uint32_t pa = smem_u32(term == 1 ? xl : xh) + bx * CL_BOX;
          const uint32_t pb = smem_u32(term == 0 ? xl : xh) + bx * CL_BOX;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            tc_mma_f16(d_sq, smem_desc_sw128(pa + kk * 32), smem_desc_sw128(pb + kk * 32), id_sq,
                       first);
            first = 1u;
          }
        }
      tc_commit(&s_bar);
    }
    mma_done();
    const float alpha = kScaleA / (kScaleX * kScaleX);
    if constexpr (CL == 1) {
      if (sq_col < mp) {                           // warp-uniform
        float f[32];
        load32(d_sq + sq_col, alpha, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 hi, lo;
          split8(f + 8 * i, hi, lo);
          *piece(sq_h, row, sq_piece + i) = hi;
          if (TERMS == 3) *piece(sq_l, row, sq_piece + i) = lo;
        }
      }
    } else {
      constexpr int R = CL_ROWS / CL;              // rows a CTA owns
      // where rows are received in A's place, no CTA may still be multiplying
      // by what the last step left there
      if (!args.recv_apart) cluster_sync_all();
      // Partial rows to their owners: [source rank][row of the owner][128].
      // The partial product is symmetric, so a lane's 32 values of row r are
      // sent as column r of 32 rows: a warp stores 32 neighbours at a time.
      if (sq_col < mp && q * 32 < mp) {
        float f[32];
        load32(d_sq + sq_col, 1.f, f);
        const uint32_t mine =
            smem_u32(recv + static_cast<int>(rank) * R * CL_ROWS + row);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int c = sq_col + i;
          st_cluster_f32(map_rank(mine + (c % R) * CL_ROWS * 4, c / R), f[i]);
        }
      }
      tc_fence_before();
      cluster_sync_all();
      // Every thread adds up a piece of the CTA's rows: 8 columns, or fewer so
      // that all threads have one.
      constexpr int PW = CL >= 4 ? 32 / CL : 8, PIECES = CL_ROWS / PW;
      constexpr int PER = R * PIECES / CL_THREADS;
      float f[PER][PW];
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int item = u * CL_THREADS + tid, rr = item / PIECES, cc = item % PIECES * PW;
#pragma unroll
        for (int i = 0; i < PW; ++i) f[u][i] = 0.f;
        if (static_cast<int>(rank) * R + rr < mp && cc < mp)
#pragma unroll
          for (int s = 0; s < CL; ++s) {
            const float2* p =
                reinterpret_cast<const float2*>(recv + (s * R + rr) * CL_ROWS + cc);
#pragma unroll
            for (int i = 0; i < PW / 2; ++i) {
              const float2 x = p[i];
              f[u][2 * i] += x.x;
              f[u][2 * i + 1] += x.y;
            }
          }
      }
      if (!args.recv_apart) cluster_sync_all();    // the sums are out of A's place
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int item = u * CL_THREADS + tid, rr = item / PIECES, cc = item % PIECES * PW;
        const int r = static_cast<int>(rank) * R + rr;
        // the rows and columns the products read
        if (cc >= mp && r >= mp) continue;
        uint32_t hi[PW / 2], lo[PW / 2];
#pragma unroll
        for (int i = 0; i < PW / 2; ++i)
          split2(alpha * f[u][2 * i], alpha * f[u][2 * i + 1], hi[i], lo[i]);
        const uint32_t off = (cc & 7) * 2;
        const uint32_t ph = smem_u32(piece(ah + (cc >> 6) * CL_BOX, r, (cc & 63) >> 3)) + off;
        const uint32_t pl = smem_u32(piece(al + (cc >> 6) * CL_BOX, r, (cc & 63) >> 3)) + off;
#pragma unroll
        for (uint32_t i = 0; i < CL; ++i) {
          const uint32_t t = (rank + i) % CL;      // not all to one CTA at a time
          st_cluster(map_rank(ph, t), hi);
          if (TERMS == 3) st_cluster(map_rank(pl, t), lo);
        }
      }
      fence_proxy_async_all();
      cluster_sync_all();
    }
    fence_proxy_async_all();
    tc_fence_before();
    __syncthreads();
    // ----------------------------------------------------------------- poly
    if (tid == 0) {
      tc_fence_after();
      uint32_t first = 0;
      for (int term = 3 - TERMS; term < 3; ++term)
        for (int k = 0; k < mp; k += 16) {
          const uint32_t off = (k >> 6) * CL_BOX + (k & 63) * 2;
          tc_mma_f16(d_sq, smem_desc_sw128(smem_u32(term == 1 ? al : ah) + off),
                     smem_desc_sw128(smem_u32(term == 0 ? al : ah) + off), id_sq, first);
          first = 1u;
        }
      tc_commit(&s_bar);
    }
    mma_done();
    if (sq_col < mp) {
      float f[32];
      load32(d_sq + sq_col, args.c / kScaleA, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4* ph = piece(sq_h, row, sq_piece + i);
        uint4* pl = piece(sq_l, row, sq_piece + i);
        add8<TERMS == 3>(*ph, TERMS == 3 ? *pl : *ph, args.b, f + 8 * i);
        uint4 hi, lo;
        split8(f + 8 * i, hi, lo);
        *ph = hi;
        if (TERMS == 3) *pl = lo;
      }
    }
    fence_proxy_async_all();
    tc_fence_before();
    __syncthreads();
    // ---------------------------------------------------------------- apply
    if (tid == 0) {
      tc_fence_after();
      uint32_t first = 0;
      for (int term = 3 - TERMS; term < 3; ++term)
        for (int k = 0; k < mp; k += 16) {
          const uint32_t off = (k >> 6) * CL_BOX + (k & 63) * 2;
          tc_mma_f16(d_x, smem_desc_sw128(smem_u32(term == 1 ? al : ah) + off),
                     smem_desc_sw128_mn(smem_u32(term == 0 ? xl : xh) + k * 128, CL_BOX), id_x,
                     first);
          first = 1u;
        }
      tc_commit(&s_bar);
    }
    mma_done();
    const float xs = last ? args.scale / kScaleX : 1.f;
    const int half = quarter & 1;                  // of a box's columns
    // the warp's boxes: every other one
    for (int b0 = 0; b0 < nbx; b0 += 2) {
      const int bx = b0 + (quarter >> 1);
      const bool have = bx < nbx;
      float f[32];
      if (have) {
        load32(d_x + bx * 64 + half * 32, xs / kScaleA, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4* ph = piece(xh + bx * CL_BOX, row, half * 4 + i);
          uint4* pl = piece(xl + bx * CL_BOX, row, half * 4 + i);
          if (TERMS == 3 || !last)   // one term: the last step adds the high plane alone
            add8<true>(*ph, *pl, xs * args.a, f + 8 * i);
          else
            add8<false>(*ph, *ph, xs * args.a, f + 8 * i);
          if (!last) {
            uint4 hi, lo;
            split8(f + 8 * i, hi, lo);
            *ph = hi;
            *pl = lo;
          }
        }
      }
      if (!last) continue;
      const int c0 = c_first + bx * 64;            // of the box
      if (TRANS) {
        // X[r][c] is out[c][r]: neighbouring lanes store neighbouring elements
        const size_t base = static_cast<size_t>(b) * args.o_bs + row;
        if (have && row < m)
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int c = c0 + half * 32 + i;
            if (c >= args.n) continue;
            const size_t o = base + static_cast<size_t>(c) * args.o_ld;
            if (args.out_bf16)
              static_cast<__nv_bfloat16*>(args.out)[o] = __float2bfloat16_rn(f[i]);
            else
              static_cast<float*>(args.out)[o] = f[i];
          }
      } else {
        // through the box's planes (fp32: columns 0-31 in the first, 32-63 in
        // the second), then along the rows
        __syncthreads();
        if (have) {
          uint8_t* place = half == 0 ? xh + bx * CL_BOX : xl + bx * CL_BOX;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *piece(place, row, i) =
                make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                           __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
        }
        __syncthreads();
#pragma unroll 4
        for (int i = warp; i < 2 * CL_ROWS; i += CL_THREADS / 32) {
          const int by = b0 + i / CL_ROWS, r = i % CL_ROWS;
          if (by >= nbx || r >= m) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = c_first + by * 64 + h * 32 + lane;
            if (c >= args.n) continue;
            const float v = reinterpret_cast<const float*>(
                piece(h == 0 ? xh + by * CL_BOX : xl + by * CL_BOX, r, lane >> 2))[lane & 3];
            const size_t o = static_cast<size_t>(b) * args.o_bs +
                             static_cast<size_t>(r) * args.o_ld + c;
            if (args.out_bf16)
              static_cast<__nv_bfloat16*>(args.out)[o] = __float2bfloat16_rn(v);
            else
              static_cast<float*>(args.out)[o] = v;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s_abort) atomicOr(args.status, kDevTimeout);
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------- norm and first iterate
constexpr int kSumThreads = 256;

// Partial sums of squares in fp64 (squares of large or tiny gradients leave
// fp32's range): block (chunk, matrix) takes every nchunk-th row.  Memory bound:
// 128 of [768, 2048] bf16 73 us, 5.5 TB/s; 4 of [5120, 4352] fp32 55 us, 6.4.
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

// kScaleX / (|G|_F + eps) of matrix b from its partial sums, to the block.
__device__ __forceinline__ float scale_of(const double* __restrict__ partial, int nchunk, int b,
                                          double eps) {
  __shared__ float s_inv;
  if (threadIdx.x < 32) {
    double t = 0.0;
    for (int i = threadIdx.x; i < nchunk; i += 32) t += partial[static_cast<size_t>(b) * nchunk + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (threadIdx.x == 0)
      s_inv = static_cast<float>(static_cast<double>(kScaleX) / (sqrt(t) + eps));
  }
  __syncthreads();
  return s_inv;
}

// X0 = G / (|G|_F + eps), scaled, as two fp16 planes [m, n] with rows of ld_o
// elements: pieces of 8 along the rows, four in flight a thread.  Memory
// bound: 128 of [768, 2048] bf16 226 us, 1.2 GB at 5.4 TB/s.
template <typename T>
__global__ void __launch_bounds__(256)
ortho_scale_kernel(const T* __restrict__ g, long long ld, long long bs,
                   const double* __restrict__ partial, int nchunk, double eps, int m, int n,
                   __half* __restrict__ hi, __half* __restrict__ lo, int ld_o) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const float inv = scale_of(partial, nchunk, b, eps);
  const T* base = g + static_cast<size_t>(b) * bs;
  const size_t obase = static_cast<size_t>(b) * m * ld_o;
  constexpr int V = 16 / sizeof(T);
  const bool vec = ld % V == 0 && (reinterpret_cast<uintptr_t>(base) & 15) == 0;
  const int per_row = ld_o / 8;
  const long long pieces = static_cast<long long>(m) * per_row;
  constexpr int U = 4;
  for (long long p0 = blockIdx.x * 256ll * U; p0 < pieces; p0 += gridDim.x * 256ll * U) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long p = p0 + u * 256 + threadIdx.x;
      const int r = static_cast<int>(p / per_row), c = static_cast<int>(p % per_row) * 8;
      const T* src = base + static_cast<size_t>(r) * ld + c;
      if (p < pieces && vec && c + 8 <= n) {
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) {
          const uint4 q = __ldcs(reinterpret_cast<const uint4*>(src) + h);
          const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
          for (int k = 0; k < V; ++k) v[u][h * V + k] = to_f32<T>(e[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][k] = p < pieces && c + k < n ? to_f32<T>(src[k]) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long p = p0 + u * 256 + threadIdx.x;
      if (p >= pieces) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][k] *= inv;
      uint4 h, l;
      split8(v[u], h, l);
      *reinterpret_cast<uint4*>(hi + obase + p * 8) = h;
      *reinterpret_cast<uint4*>(lo + obase + p * 8) = l;
    }
  }
}

// The same of G^T, by tiles of 64 x 64.  4 of [5120, 4352] fp32: 118 us, 6.0 TB/s.
template <typename T>
__global__ void __launch_bounds__(256)
ortho_transpose_kernel(const T* __restrict__ g, long long ld, long long bs,
                       const double* __restrict__ partial, int nchunk, double eps, int m, int n,
                       __half* __restrict__ hi, __half* __restrict__ lo, int ld_o) {
  pdl_trigger();
  pdl_wait();
  __shared__ float tile[64][65];
  const int b = blockIdx.z;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of X0
  const T* base = g + static_cast<size_t>(b) * bs;
  constexpr int V = 16 / sizeof(T);
  if (ld % V == 0 && (reinterpret_cast<uintptr_t>(base) & 15) == 0 && r0 + 64 <= m) {
#pragma unroll
    for (int i = 0; i < 64 * 64 / V / 256; ++i) {
      const int item = i * 256 + threadIdx.x, y = item / (64 / V), x = item % (64 / V) * V;
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (c0 + y < n)
        q = __ldcs(reinterpret_cast<const uint4*>(base + static_cast<size_t>(c0 + y) * ld + r0 + x));
      const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
      for (int k = 0; k < V; ++k) tile[x + k][y] = to_f32<T>(e[k]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int y = (threadIdx.x >> 6) + 4 * i, x = threadIdx.x & 63;
      tile[x][y] = c0 + y < n && r0 + x < m
                       ? to_f32<T>(base[static_cast<size_t>(c0 + y) * ld + r0 + x])
                       : 0.f;
    }
  }
  const float inv = scale_of(partial, nchunk, b, eps);   // and the tile is complete
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int y = (threadIdx.x >> 3) + 32 * i, x = (threadIdx.x & 7) * 8;
    const int r = r0 + y, c = c0 + x;
    if (r >= m || c >= ld_o) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[y][x + e] * inv;
    uint4 h, l;
    split8(v, h, l);
    const size_t at = (static_cast<size_t>(b) * m + r) * ld_o + c;
    *reinterpret_cast<uint4*>(hi + at) = h;
    *reinterpret_cast<uint4*>(lo + at) = l;
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

// SMs of the current device, asked for once per device.
int num_sms() {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::atomic<int>& k = known[dev & 63];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = 148;
    k.store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int MODE, int TERMS, int CG, int TN, int SPLIT = 1>
cudaError_t launch_ns(const NsMaps& maps, NsArgs args, cudaStream_t stream) {
  using C = Cfg<TERMS, CG, TN>;
  auto kern = ns_gemm_kernel<MODE, TERMS, CG, TN, SPLIT>;
  static std::atomic<unsigned long long> attr_done{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  constexpr bool SYM = MODE == MODE_GRAM || MODE == MODE_POLY;
  args.tm = (args.m + C::TM - 1) / C::TM;
  args.tn = ((SYM ? args.m : args.n) + TN - 1) / TN;
  const int max_units = num_sms() / CG;
  args.tiles = 0;
  args.full = SYM && (SPLIT > 1 || static_cast<long long>(args.batch) * args.tm * args.tn <= max_units);
  if (SYM && !args.full)
    for (int i = 0; i < args.tm; ++i) args.tiles += args.tn - C::TM / TN * i;
  else
    args.tiles = args.tm * args.tn;
  const long long total = static_cast<long long>(args.batch) * args.tiles;
  const int units = static_cast<int>(total < max_units ? total : max_units);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CG * SPLIT * units);
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG * SPLIT;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, args);
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
inline long long pad64(int v) { return (static_cast<long long>(v) + 63) / 64 * 64; }

// Do products of one term keep the directions' errors bounded?  A singular
// value x becomes x' = x (a + q) with q = b y + c y^2, y = x^2.  In a step its
// relative error e grows by |x p'(x) / p(x)|, and the roundings of X's hi plane,
// of A and of B, 2^-12 each in the mean of their range, add 2 |b y + 2 c y^2| + |q|
// of it, by x / x'.  The largest sum over values from 2^-8 (smaller ones are still
// in the polynomial's linear part) to 1 is compared with 100, 2.4e-2: Muon's
// polynomial has 92 after five steps and 138 after six, (3, -3.2, 1.2) never more than
// 9, (2, -1.5, 0.5) 2.  A simulation of 1 x 1 matrices finds 98, 141, 13.7 and 2.
// About 1 us on the host for five steps.
bool one_term_holds(float a, float b, float c, int steps) {
  constexpr int N = 128;
  float x[N], e[N];
  for (int i = 0; i < N; ++i) {
    x[i] = i == 0 ? 1.f : x[i - 1] * 0.95760328f;   // 2^(-8 / N)
    e[i] = 0.f;
  }
  for (int s = 0; s < steps; ++s)
    for (int i = 0; i < N; ++i) {
      const float y = x[i] * x[i], q = b * y + c * y * y;
      const float grow = a + 3.f * b * y + 5.f * c * y * y;
      const float add = 2.f * std::fabs(b * y + 2.f * c * y * y) + std::fabs(q);
      e[i] = (std::fabs(grow) * e[i] + add) / std::fabs(a + q);
      x[i] = std::fabs(x[i] * (a + q));
    }
  for (int i = 0; i < N; ++i)
    if (!(e[i] <= 100.f)) return false;   // a value that became 0 as well
  return true;
}

struct OrthoLayout {
  size_t status, partial, xh[2], xl[2], ah, al, bh, bl, total;
};

int sum_chunks(int rows, int batch) {
  const int c = (rows + 8 - 1) / 8;   // eight rows (one per warp) at least
  const int most = 2048 / batch > 32 ? 2048 / batch : 32;
  return c < most ? c : most;
}

OrthoLayout ortho_layout(const OrthoShape& s) {
  const int m = s.rows < s.cols ? s.rows : s.cols, n = s.rows < s.cols ? s.cols : s.rows;
  const size_t x = static_cast<size_t>(s.batch) * m * pad64(n) * 2;
  const size_t a = static_cast<size_t>(s.batch) * m * pad64(m) * 2;
  OrthoLayout L{};
  size_t o = 0;
  L.status = o;  o += 256;
  L.partial = o; o += up256(static_cast<size_t>(s.batch) * sum_chunks(s.rows, s.batch) * 8);
  for (int i = 0; i < 2; ++i) {
    L.xh[i] = o; o += up256(x);
    L.xl[i] = o; o += up256(x);
  }
  L.ah = o; o += up256(a);
  L.al = o; o += s.three_terms ? up256(a) : 0;
  L.bh = o; o += up256(a);
  L.bl = o; o += s.three_terms ? up256(a) : 0;
  L.total = o;
  return L;
}

// CTAs per cluster of the one-launch kernel, 0 where it does not apply.  Up to
// four boxes stay in one CTA, which needs no exchange ([100, 192] bf16 31.1 us,
// on two CTAs 38.8), fp32 results as well, although one matrix of 256 columns would
// gain a little (54.3 us, on four CTAs 51.2): it leaves the other SMs to a batch.
// Above, two boxes a
// CTA while every matrix has its cluster at once ([100, 512] bf16 41 us on four
// CTAs, 51 on two; [100, 1024] 45 on eight, 52 on four), else four: the 16th
// cluster of eight waits for another to end (16 of [100, 1024] bf16: 91 us on
// eight CTAs each, 53 on four).  16 CTAs, more than a cluster is sure to get,
// only for single matrices wider than 8 of them take so ([128, 2048] fp32: 85 us
// on 8 CTAs, 71 us on 16; [128, 4096], which needs 16, 91 us and 137 by the tiled
// kernel).
int cluster_size(int batch, int m, int n) {
  if (m > CL_ROWS) return 0;
  const int boxes = (n + 63) / 64;
  if (boxes <= CL_MAX_BOXES) return 1;
  if (boxes <= 8) return batch <= 32 ? 4 : 2;
  if (boxes <= 16) return batch <= 12 ? 8 : 4;
  if (batch <= 2 && boxes <= 16 * CL_MAX_BOXES) return 16;
  return boxes <= 8 * CL_MAX_BOXES ? 8 : 0;
}

// Can eight CTAs take the matrix where a cluster of 16 is not to be had?
bool fits_eight(int n) { return n <= 8 * CL_MAX_BOXES * 64; }

template <typename T, bool TRANS, int CL, int TERMS>
cudaError_t launch_cluster(const ClArgs& args, int smem, cudaStream_t stream) {
  auto kern = ns_cluster_kernel<T, TRANS, CL, TERMS>;
  static std::atomic<unsigned long long> attr_done{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448 - 512);
    if (e == cudaSuccess && CL > 8)
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL * args.batch);
  cfg.blockDim = dim3(CL_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (CL > 8) {
    // whether this device has a place for such a cluster (asked for once; the
    // caller falls back to 8 CTAs)
    static std::atomic<unsigned long long> asked{0}, fits{0};
    if (!(asked.load(std::memory_order_acquire) & bit)) {
      int n = 0;
      cfg.dynamicSmemBytes = 232448 - 512;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n >= 1)
        fits.fetch_or(bit, std::memory_order_acq_rel);
      else
        cudaGetLastError();
      asked.fetch_or(bit, std::memory_order_acq_rel);
      cfg.dynamicSmemBytes = smem;
    }
    if (!(fits.load(std::memory_order_acquire) & bit)) return cudaErrorInvalidConfiguration;
  }
  return cudaLaunchKernelEx(&cfg, kern, args);
}

template <typename T, int TERMS>
cudaError_t run_cluster(const OrthoShape& s, int cl, const void* g, void* out, void* ws,
                        cudaStream_t stream) {
  const bool trans = s.rows > s.cols;
  ClArgs a{};
  a.batch = s.batch;
  a.m = trans ? s.cols : s.rows;
  a.n = trans ? s.rows : s.cols;
  a.nbx = ((a.n + 63) / 64 + cl - 1) / cl;
  a.steps = s.steps;
  a.a = s.a;
  a.b = s.b;
  a.c = s.c;
  a.scale = s.scale;
  a.eps = static_cast<double>(s.eps);
  a.g = g;
  a.g_ld = s.g_ld;
  a.g_bs = s.g_bs;
  a.out = out;
  a.out_bf16 = s.out_bf16;
  a.o_ld = s.out_ld;
  a.o_bs = s.out_bs;
  a.status = static_cast<uint32_t*>(ws);
  // X's and A's planes; the received rows apart while that fits, else in the
  // place of A's two planes, which is as large
  static_assert(CL_RECV_BYTES == 4 * CL_BOX, "A's planes");
  static_assert((2 * CL_MAX_BOXES + 2) * CL_BOX + 1024 + CL_RECV_BYTES <= 232448 - 512,
                "one term: always apart");
  int smem = (2 * a.nbx + (TERMS == 3 ? 4 : 2)) * CL_BOX + 1024;
  if (cl > 1) {
    a.recv_apart = smem + CL_RECV_BYTES <= 232448 - 512;
    if (a.recv_apart) smem += CL_RECV_BYTES;
  }
  if (cl == 16) {
    const cudaError_t e = trans ? launch_cluster<T, true, 16, TERMS>(a, smem, stream)
                                : launch_cluster<T, false, 16, TERMS>(a, smem, stream);
    if (e == cudaSuccess) return e;
    cudaGetLastError();   // not left for the caller's next check: 8 CTAs, or tiles, do as well
    return fits_eight(a.n) ? run_cluster<T, TERMS>(s, 8, g, out, ws, stream) : e;
  }
  auto go = [&](auto one, auto two, auto four, auto eight) {
    return cl == 1 ? one(a, smem, stream)
                   : cl == 2 ? two(a, smem, stream)
                             : cl == 4 ? four(a, smem, stream) : eight(a, smem, stream);
  };
  return trans ? go(launch_cluster<T, true, 1, TERMS>, launch_cluster<T, true, 2, TERMS>,
                    launch_cluster<T, true, 4, TERMS>, launch_cluster<T, true, 8, TERMS>)
               : go(launch_cluster<T, false, 1, TERMS>, launch_cluster<T, false, 2, TERMS>,
                    launch_cluster<T, false, 4, TERMS>, launch_cluster<T, false, 8, TERMS>);
}

// Tile shapes of the tiled kernel: 256 x 256 and 256 x 128 on CTA pairs, 128 x 64
// on single CTAs.
enum TileShape { TILE_256, TILE_128, TILE_64 };

// The shape with the least estimated time for one launch: rounds of tiles
// over the SMs times k-blocks.  The cycles of a k-block are measured with all SMs
// busy: staging an SM's operands from L2 (38 bytes a cycle) bounds them, so
// the large tile moves the least per product, and the smaller ones win where
// they fill the last round better.  epi: a tile's epilogue, hidden behind
// the next tile's products but for the last; it is what a short inner
// dimension leaves visible, and long where chunks wait for their buffer (the
// large tile's stages of four planes leave room for one).
template <int MODE, int TERMS>
TileShape choose_tiles(int batch, int m, int n, int kblocks) {
  constexpr bool SYM = MODE == MODE_GRAM || MODE == MODE_POLY;
  const int sms = num_sms();
  const struct { int tm, tn, units, kb, epi; } shapes[3] = {
      {256, 256, sms / 2, TERMS == 3 ? 1750 : 860,
       TERMS == 3 ? (SYM ? 20000 : 16000) : SYM ? 4500 : 7500},
      {256, 128, sms / 2, TERMS == 3 ? 1260 : 650,
       TERMS == 3 ? (SYM ? 4500 : 6000) : SYM ? 2500 : 4200},
      {128, 64, sms, TERMS == 3 ? 1050 : 560,
       TERMS == 3 ? (SYM ? 2500 : 2800) : SYM ? 1500 : 2000}};
  TileShape best = TILE_256;
  long long least = -1;
  for (int i = 0; i < 3; ++i) {
    const auto& t = shapes[i];
    const int tm = (m + t.tm - 1) / t.tm, tn = ((SYM ? m : n) + t.tn - 1) / t.tn;
    long long tiles = static_cast<long long>(tm) * tn;
    if (SYM && tiles * batch > t.units) {
      tiles = 0;
      for (int r = 0; r < tm; ++r) tiles += tn - t.tm / t.tn * r;
    }
    const long long rounds = (tiles * batch + t.units - 1) / t.units;
    const long long work = static_cast<long long>(kblocks) * t.kb;
    const long long cost = (rounds - 1) * (work > t.epi ? work : t.epi) + work + t.epi;
    if (least < 0 || cost < least) {
      least = cost;
      best = static_cast<TileShape>(i);
    }
  }
  return best;
}

// The added matrix and the result in chunks of 128, 64 and 32 rows (32: gram's
// result only).
struct ChunkMaps {
  const CUtensorMap *add[3], *out[3];   // [rows][plane]
};

template <int MODE, int TERMS>
cudaError_t launch_best(NsMaps& maps, const CUtensorMap (&b_op)[3][2], const ChunkMaps& chunks,
                        const NsArgs& args, cudaStream_t stream) {
  const TileShape t = choose_tiles<MODE, TERMS>(args.batch, args.m, args.n, args.kblocks);
  // (an inner dimension of m that long has too many tiles, but for two CTAs
  // with three terms)
  constexpr bool FOUR = MODE == MODE_GRAM, TWO = MODE == MODE_GRAM || TERMS == 3;
  int split = 1;
  if (t == TILE_64) {
    // Few tiles and a long inner dimension: split it over the SMs that would
    // idle.  What the shorter loop saves against what a cluster and the
    // exchange of the sums cost, in cycles (measured: [512, 512] fp32, 8
    // k-blocks, gains nothing from four CTAs, [512, 2048] 206 -> 157 us).
    constexpr bool SYM = MODE == MODE_GRAM || MODE == MODE_POLY;
    const long long tiles = static_cast<long long>(args.batch) * ((args.m + 127) / 128) *
                            (((SYM ? args.m : args.n) + 63) / 64);
    const int sms = num_sms(), work = args.kblocks * (TERMS == 3 ? 1050 : 560);
    int gain = 1500;
    if (TWO && tiles * 2 <= sms && work / 2 - 3000 > gain) {
      split = 2;
      gain = work / 2 - 3000;
    }
    if (FOUR && tiles * 4 <= sms && work * 3 / 4 - 6000 > gain) split = 4;
  }
  const int rows = split == 4 ? 2 : split - 1;
  for (int p = 0; p < 2; ++p) {
    maps.b[p] = b_op[t][p];
    maps.add[p] = chunks.add[rows][p];
    maps.out[p] = chunks.out[rows][p];
  }
  if constexpr (FOUR)
    if (split == 4) return launch_ns<MODE, TERMS, 1, 64, 4>(maps, args, stream);
  if constexpr (TWO)
    if (split == 2) return launch_ns<MODE, TERMS, 1, 64, 2>(maps, args, stream);
  return t == TILE_256   ? launch_ns<MODE, TERMS, 2, 256>(maps, args, stream)
         : t == TILE_128 ? launch_ns<MODE, TERMS, 2, 128>(maps, args, stream)
                         : launch_ns<MODE, TERMS, 1, 64>(maps, args, stream);
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
  // Maps by box rows: 128 (A operand, chunks), 64 and 32 (chunks of split tiles),
  // 64 (mirrored tiles; X as the B operand of the apply product, MN-major).  The K-major B operand takes
  // 128 rows a CTA of the 256 x 256 tile, 64 of the others.
  CUtensorMap x128[2][2], x64[2][2];               // [buffer][plane]
  CUtensorMap a128[2], a64[2], a32[2], b128[2], b64[2];
  for (int i = 0; i < 2; ++i)
    for (int p = 0; p < 2; ++p) {
      const void* base = w + (p ? L.xl[i] : L.xh[i]);
      if (!make_map3(&x128[i][p], base, m, n, ldx, s.batch, bsx, 128) ||
          !make_map3(&x64[i][p], base, m, n, ldx, s.batch, bsx, 64))
        return cudaErrorInvalidValue;
    }
  for (int p = 0; p < 2; ++p) {
    const void* ap = p && al ? al : ah;
    const void* bp = p && bl ? bl : bh;
    if (!make_map3(&a128[p], ap, m, m, lda, s.batch, bsa, 128) ||
        !make_map3(&a64[p], ap, m, m, lda, s.batch, bsa, 64) ||
        !make_map3(&a32[p], ap, m, m, lda, s.batch, bsa, 32) ||
        !make_map3(&b128[p], bp, m, m, lda, s.batch, bsa, 128) ||
        !make_map3(&b64[p], bp, m, m, lda, s.batch, bsa, 64))
      return cudaErrorInvalidValue;
  }
  static_assert(BK == 64, "boxes of X in the apply product");
  NsArgs base{};
  base.batch = s.batch;
  base.m = m;
  base.n = n;
  base.status = reinterpret_cast<uint32_t*>(w + L.status);
  for (int step = 0; step < s.steps; ++step) {
    const int cur = step & 1;
    const bool last = step + 1 == s.steps;
    cudaError_t e;
    NsMaps maps;
    // A = X X^T
    NsArgs g = base;
    g.kblocks = (n + BK - 1) / BK;
    g.alpha = kScaleA / (kScaleX * kScaleX);
    g.out_planes = TERMS == 3 ? 2 : 1;
    g.out_hi = ah;
    g.out_lo = al;
    g.out_ld = lda;
    g.out_bs = bsa;
    CUtensorMap b_op[3][2];
    for (int p = 0; p < 2; ++p) {
      maps.a[p] = x128[cur][p];
      b_op[TILE_256][p] = x128[cur][p];
      b_op[TILE_128][p] = b_op[TILE_64][p] = x64[cur][p];
      maps.mir[p] = a64[p];
    }
    e = launch_best<MODE_GRAM, TERMS>(maps, b_op, {{a128, a64, a32}, {a128, a64, a32}}, g, stream);
    if (e != cudaSuccess) return e;
    // B = b A + c A A
    NsArgs p = g;
    p.kblocks = (m + BK - 1) / BK;
    p.alpha = s.c / kScaleA;
    p.beta = s.b;
    p.add_planes = g.out_planes;
    p.out_hi = bh;
    p.out_lo = bl;
    for (int q = 0; q < 2; ++q) {
      maps.a[q] = a128[q];
      b_op[TILE_256][q] = a128[q];
      b_op[TILE_128][q] = b_op[TILE_64][q] = a64[q];
      maps.mir[q] = b64[q];
    }
    e = launch_best<MODE_POLY, TERMS>(maps, b_op, {{a128, a64, a64}, {b128, b64, b64}}, p, stream);
    if (e != cudaSuccess) return e;
    // X = a X + B X; the last step of one-term products adds X's high plane
    // alone, so the step before it writes no other
    NsArgs x = base;
    x.kblocks = (m + BK - 1) / BK;
    x.alpha = 1.f / kScaleA;
    x.beta = s.a;
    x.add_planes = TERMS == 3 || !last ? 2 : 1;
    x.out_planes = TERMS == 3 || step + 2 < s.steps ? 2 : 1;
    for (int q = 0; q < 2; ++q) {
      maps.a[q] = b128[q];
      for (int t = 0; t < 3; ++t) b_op[t][q] = x64[cur][q];
    }
    const ChunkMaps chunks{{x128[cur], x64[cur], x64[cur]},
                           {x128[cur ^ 1], x64[cur ^ 1], x64[cur ^ 1]}};
    if (last) {
      x.alpha *= s.scale / kScaleX;
      x.beta *= s.scale / kScaleX;
      x.out = out;
      x.out_bf16 = s.out_bf16;
      x.out_trans = trans;
      x.o_ld = s.out_ld;
      x.o_bs = s.out_bs;
      e = launch_best<MODE_LAST, TERMS>(maps, b_op, chunks, x, stream);
    } else {
      e = launch_best<MODE_APPLY, TERMS>(maps, b_op, chunks, x, stream);
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
  const int nchunk = sum_chunks(s.rows, s.batch);
  double* partial = reinterpret_cast<double*>(w + L.partial);
  cudaError_t e =
      launch_pdl(ortho_sumsq_kernel<T>, dim3(nchunk, s.batch), dim3(kSumThreads), 0, stream, g,
                 s.rows, s.cols, s.g_ld, s.g_bs, partial,
                 reinterpret_cast<uint32_t*>(w + L.status));
  if (e != cudaSuccess) return e;
  __half* hi = reinterpret_cast<__half*>(w + L.xh[0]);
  __half* lo = reinterpret_cast<__half*>(w + L.xl[0]);
  const int ldx = static_cast<int>(pad64(n));
  const double* sums = partial;
  const double eps = static_cast<double>(s.eps);
  if (trans)
    return launch_pdl(ortho_transpose_kernel<T>,
                      dim3(static_cast<unsigned>(ldx / 64), static_cast<unsigned>(pad64(m) / 64),
                           s.batch),
                      dim3(256), 0, stream, g, s.g_ld, s.g_bs, sums, nchunk, eps, m, n, hi, lo, ldx);
  const long long blocks = (static_cast<long long>(m) * (ldx / 8) + 1023) / 1024;
  const int most = num_sms() * 16 / s.batch > 8 ? num_sms() * 16 / s.batch : 8;
  return launch_pdl(ortho_scale_kernel<T>,
                    dim3(static_cast<unsigned>(blocks < most ? blocks : most), s.batch), dim3(256),
                    0, stream, g, s.g_ld, s.g_bs, sums, nchunk, eps, m, n, hi, lo, ldx);
}

}  // namespace

bool ortho_three_terms(const OrthoShape& s) {
  return !s.out_bf16 || (s.rows < s.cols ? s.rows : s.cols) < 64 ||
         !one_term_holds(s.a, s.b, s.c, s.steps);
}

size_t ortho_workspace(const OrthoShape& s) {
  if (s.batch == 0) return 256;   // the call does nothing; no layout of no matrices
  const int m = s.rows < s.cols ? s.rows : s.cols, n = s.rows < s.cols ? s.cols : s.rows;
  return cluster_size(s.batch, m, n) > 0 && fits_eight(n) ? 256   // the status
                                                          : ortho_layout(s).total;
}

cudaError_t orthogonalize(const OrthoShape& s, const void* g, void* out, void* ws,
                          cudaStream_t stream) {
  const int m = s.rows < s.cols ? s.rows : s.cols, n = s.rows < s.cols ? s.cols : s.rows;
  const int cl = cluster_size(s.batch, m, n);
  if (cl > 0) {
    const cudaError_t ec =
        s.three_terms
            ? (s.in_bf16 ? run_cluster<__nv_bfloat16, 3>(s, cl, g, out, ws, stream)
                         : run_cluster<float, 3>(s, cl, g, out, ws, stream))
            : (s.in_bf16 ? run_cluster<__nv_bfloat16, 1>(s, cl, g, out, ws, stream)
                         : run_cluster<float, 1>(s, cl, g, out, ws, stream));
    if (ec == cudaSuccess || fits_eight(n)) return ec;
  }
  cudaError_t e = s.in_bf16 ? run_init(s, static_cast<const __nv_bfloat16*>(g), ws, stream)
                            : run_init(s, static_cast<const float*>(g), ws, stream);
  if (e != cudaSuccess) return e;
  return s.three_terms ? run_steps<3>(s, out, ws, stream) : run_steps<1>(s, out, ws, stream);
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
