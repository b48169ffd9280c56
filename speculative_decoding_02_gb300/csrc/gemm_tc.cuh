// A persistent matrix product on the tensor cores whose tiles, operands and
// epilogue come from a policy: the frame of the products in linear_ce.cu and
// newton_schulz.cu.  fp16 or bf16 operands (the same type in one product),
// products exact in fp32, sums in fp32.
//
// A unit works on tiles of kM x kN: a pair of CTAs (cta_group::2) on 256 x kN,
// 128 rows of it in each CTA's tensor memory, or a single CTA on 128 x kN.
// K goes by steps of 64, a stage of the ring each; a CTA copies its 128 rows of
// A and its share of B (kN / 2 columns of a pair's, kN of a single CTA's):
//
//   warp 0      TMA producer of its CTA; a pair's copies of a stage count on the
//               first CTA's barrier;
//   warp 1      (of the first CTA) MMA issuer;
//   warps 2-17  epilogue: a thread owns a row and kN / 4 columns, sums them in
//               registers and hands them to the policy.
//
// Either operand is K-major ([128 or fewer rows][64 of K] boxes) or not (boxes of
// [64 of K][64 rows]), tile by tile.  The tensor cores truncate when they add
// to an accumulator, so an accumulator takes p.chunk() steps of K only and the
// epilogue adds it, rounded, to its sums while the next one fills (two of them).
//
// A policy P (a kernel parameter, so its tensor maps are too) has
//   kPair, kN, kSelf (a product of one matrix with itself, from halves: a() and
//     b() are its high and low half, the sum is that of a a^T, a b^T and b a^T),
//     kBoxBytes (shared memory of an epilogue warp, a multiple of
//     1024), kExtraBytes (of the CTA); status, bf16;
//   Counts counts()                     read once a thread, behind pdl_wait
//   int chunk(counts)                   steps of K that an accumulator takes
//   bool used(counts, tile, row)        whether any of the 32 rows from `row` (of the tile) is
//   bool tile(counts, unit, units, i, Tile&)  the i-th tile of a unit, same
//     for all its threads; false when there is none
//   int segments(tile), Segment segment(tile, i)  where the operands' steps of K are
//   void epilogue(Epi&, tile, acc)      every epilogue thread, converged
//   void finish(counts, Epi)            every epilogue thread, behind its last tile
//   void prefetch()                     of the tensor maps
//   void early(unit, rank)              a warp, before pdl_wait
#pragma once

#include <algorithm>

#include "kernels.h"
#include "tc_common.cuh"

namespace dspark {
namespace gemm {

using namespace tc;

constexpr int kEpiWarps = 16;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxSmem = 232448;
constexpr int kRows = 128;      // rows of a CTA (TMEM lanes)
constexpr int kStep = 64;       // of K in a stage
constexpr int kBarBytes = 512;
constexpr int kMaxStages = 8;

struct Tile {
  int m0, n0;          // first row and column
  int steps;           // of K; with 0 the sums are zeros
  bool a_mn, b_mn;     // operand not K-major
  int kind, part, k0;  // the policy's own
};

// Steps of K that follow one another in both operands: of either the map and the
// coordinates of the tile's first row (column) and of the first k.
struct Segment {
  const CUtensorMap *a, *b;
  int am, ak, bn, bk;
  int steps;
};

struct Epi {
  int row;             // of the tile
  int row0;            // the row of this warp's lane 0
  int col;             // of the tile: the thread's columns are col .. col + kN / 4 - 1
  bool used;           // else the sums are zeros
  int q, h, lane;      // the warp's quarter of the CTA's rows and of the columns
  int n;               // tiles before this one
  unsigned char* box;    // this warp's
  unsigned char* extra;  // the CTA's
};

template <class P>
struct Shape {
  static constexpr int kM = P::kPair ? 2 * kRows : kRows;
  static constexpr int kBRows = P::kPair ? P::kN / 2 : P::kN;
  static constexpr int kABytes = kRows * 128;
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kFixed = 1024 + kEpiWarps * P::kBoxBytes + P::kExtraBytes + kBarBytes;
  static constexpr int kStages = (kMaxSmem - kFixed) / kStageBytes < kMaxStages ? (kMaxSmem - kFixed) / kStageBytes
                                                                                : kMaxStages;
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
  static constexpr int kCols = P::kN / 4;       // of an epilogue thread
  static constexpr uint32_t kTmemCols = 2 * P::kN;
  static_assert(kStages >= 3 && kSmem <= kMaxSmem, "shared memory");
  static_assert(P::kN == 64 || P::kN == 128 || P::kN == 256, "columns of a tile");
  static_assert(!P::kSelf || kBRows == kRows, "the halves' tiles are alike");
  static_assert(!P::kPair || P::kN >= 128, "a CTA's share of B is 64 columns or more");
  static_assert(P::kBoxBytes % 1024 == 0, "128-byte swizzled boxes");
};

struct __align__(8) Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

template <bool kPair>
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  if constexpr (kPair) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  }
}

// A box of a matrix into L2; nothing waits for it.
__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1)
               : "memory");
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// mbar_wait of a converged warp, which reads the clock now and then only (a tile's
// accumulators change hands several times).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  uint64_t t0 = 0;
  while (!ok) {
#pragma unroll 1
    for (int i = 0; i < 1024 && !ok; ++i) ok = mbar_try_wait(bar, parity);
    if (ok || *abort) break;
    const uint64_t now = globaltimer();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > kWaitLimitNs) {
      *abort = 1;
      record_status(status, DSPARK_ERR_TIMEOUT);
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

template <bool kPair>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kPair) umma_pair(d, a, b, idesc, accumulate);
  else umma_bf16(d, a, b, idesc, accumulate);
}
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (kPair) umma_pair_commit(bar);
  else umma_commit(bar);
}

template <class P>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ P p) {
  using S = Shape<P>;
  constexpr bool kPair = P::kPair;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* boxes = smem + S::kStages * S::kStageBytes;
  unsigned char* extra = boxes + kEpiWarps * P::kBoxBytes;
  Bars* bars = reinterpret_cast<Bars*>(extra + P::kExtraBytes);
  // (the same in a warp, which the compiler sees in a shuffle's result: the loops
  // of the producer and the issuer are the whole warp's, on uniform registers, and
  // one lane's the copies and MMAs.  A loop of one lane alone takes 600 cycles a
  // step, more than the 512 of a pair's 256 x 256 x 64)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = kPair ? (int)cluster_rank() : 0;
  const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x, units = kPair ? gridDim.x >> 1 : gridDim.x;
  volatile int* abort = &bars->abort;

  if (threadIdx.x == 0) {
    p.prefetch();
    for (int s = 0; s < S::kStages; ++s) { mbar_init(&bars->full[s], 1); mbar_init(&bars->empty[s], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->acc_full[s], 1);
      mbar_init(&bars->acc_empty[s], (kPair ? 2 : 1) * kEpiWarps);
    }
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)),
                   "r"(S::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(&bars->tmem_base, S::kTmemCols);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_meet();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  pdl_trigger();
  if (warp == 0) p.early(unit, rank);
  pdl_wait();
  const typename P::Counts counts = p.counts();
  const int chunk = p.chunk(counts);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t stages = smem_u32(smem);
    uint32_t i = 0, s = 0, phase = 1;
    bool ok = true;
    Tile t;
    for (int n = 0; ok && p.tile(counts, unit, units, n, t); ++n) {
      const int segments = p.segments(t);
      for (int q = 0; q < segments && ok; ++q) {
        Segment g = p.segment(t, q);
        g.am += rank * kRows;
        g.bn += rank * S::kBRows;
        for (int k = 0; k < g.steps; ++k, ++i, g.ak += kStep, g.bk += kStep) {
          ok = warp_wait(&bars->empty[s], phase, abort, p.status);
          if (!ok) break;
          if (elect_one()) {
            uint32_t dst = stages + s * S::kStageBytes;
            const uint32_t full = kPair ? in_cta(&bars->full[s], 0) : smem_u32(&bars->full[s]);
            if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], (kPair ? 2 : 1) * S::kStageBytes);
            if (t.a_mn) {
#pragma unroll
              for (int j = 0; j < kRows / 64; ++j) copy_box<kPair>(dst + j * 8192, g.a, g.am + j * 64, g.ak, full);
            } else {
              copy_box<kPair>(dst, g.a, g.ak, g.am, full);
            }
            dst += S::kABytes;
            if (t.b_mn) {
#pragma unroll
              for (int j = 0; j < S::kBRows / 64; ++j) copy_box<kPair>(dst + j * 8192, g.b, g.bn + j * 64, g.bk, full);
            } else {
              copy_box<kPair>(dst, g.b, g.bk, g.bn, full);
            }
          }
          __syncwarp();
          if (++s == S::kStages) s = 0, phase ^= 1;
        }
      }
    }
    // every stage is consumed before the CTA leaves (on a timeout: as far as
    // the wait's limit goes, which is longer than any copy takes)
    if (lane == 0) {
      for (int s = 0; s < S::kStages; ++s) {
        const uint32_t n = (i + S::kStages - 1 - s) / S::kStages;
        if (n > 0) mbar_drain(&bars->empty[s], (n - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      const uint32_t type = p.bf16 ? (1u << 7) | (1u << 10) : 0u;
      const uint32_t base = (1u << 4) | type | ((uint32_t)(P::kN >> 3) << 17) | ((uint32_t)(S::kM >> 4) << 24);
      const uint32_t stages = smem_u32(smem);
      uint32_t c = 0, s = 0, phase = 0;
      bool ok = true;
      Tile t;
      for (int n = 0; ok && p.tile(counts, unit, units, n, t); ++n) {
        const uint32_t idesc = base | (t.a_mn ? kAMajorM : 0u) | (t.b_mn ? kBMajorN : 0u);
        // 16 of K: 32 bytes of a K-major row, else two 1024-byte groups
        const uint32_t da = t.a_mn ? 128 : 2, db = t.b_mn ? 128 : 2;
        const uint64_t ad0 = t.a_mn ? sw128_mnmajor_desc(stages, 8192) : sw128_kmajor_desc(stages);
        const uint64_t bd0 = t.b_mn ? sw128_mnmajor_desc(stages + S::kABytes, 8192) : sw128_kmajor_desc(stages + S::kABytes);
        for (int k = 0; k < t.steps && ok; ++c) {
          const int buf = c & 1, kend = min(k + chunk, t.steps);
          ok = warp_wait(&bars->acc_empty[buf], ((c >> 1) & 1) ^ 1, abort, p.status);
          if (!ok) break;
          tc_fence_after();
          for (int kf = k; k < kend; ++k) {
            ok = warp_wait(&bars->full[s], phase, abort, p.status);
            if (!ok) break;
            tc_fence_after();
            // (shared memory addresses are below 2^18: no carry out of a descriptor's address field)
            const uint64_t ad = ad0 + s * (S::kStageBytes / 16), bd = bd0 + s * (S::kStageBytes / 16);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if constexpr (P::kSelf) {
                  mma<kPair>(tmem + buf * P::kN, ad + kk * da, ad + kk * da, idesc, k != kf || kk != 0);
                  mma<kPair>(tmem + buf * P::kN, ad + kk * da, bd + kk * db, idesc, 1);
                  mma<kPair>(tmem + buf * P::kN, bd + kk * db, ad + kk * da, idesc, 1);
                } else {
                  mma<kPair>(tmem + buf * P::kN, ad + kk * da, bd + kk * db, idesc, k != kf || kk != 0);
                }
              }
              commit<kPair>(&bars->empty[s]);
            }
            __syncwarp();
            if (++s == S::kStages) s = 0, phase ^= 1;
          }
          if (ok && elect_one()) commit<kPair>(&bars->acc_full[buf]);
          __syncwarp();
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    Epi e;
    e.lane = lane;
    // (a warp reaches the TMEM lanes of its number's low two bits)
    e.q = warp & 3;
    e.h = (warp - 2) >> 2;
    e.row0 = rank * kRows + e.q * 32;
    e.row = e.row0 + lane;
    e.col = e.h * S::kCols;
    e.box = boxes + (warp - 2) * P::kBoxBytes;
    e.extra = extra;
    const uint32_t lanes = tmem + ((uint32_t)(e.q * 32) << 16) + e.col;
    uint32_t c = 0;
    bool ok = true;
    Tile t;
    for (int n = 0; p.tile(counts, unit, units, n, t); ++n) {
      float acc[S::kCols];
      e.used = p.used(counts, t, e.row0);
#pragma unroll
      for (int j = 0; j < S::kCols; ++j) acc[j] = 0.f;
      const int chunks = (t.steps + chunk - 1) / chunk;
      for (int j = 0; j < chunks && ok; ++j, ++c) {
        const int buf = c & 1;
        ok = warp_wait(&bars->acc_full[buf], (c >> 1) & 1, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        if (e.used) {
#pragma unroll
          for (int g = 0; g < S::kCols / 16; ++g) {
            float v[16];
            tmem_load_cols<16>(lanes + buf * P::kN + g * 16, v);
#pragma unroll
            for (int x = 0; x < 16; ++x) acc[g * 16 + x] += v[x];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // (an arrival of CTA scope, for no memory but the tensor core's goes with it:
          // a release to the cluster waits 2000 cycles for this thread's stores)
          if constexpr (kPair)
            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_cta(&bars->acc_empty[buf], 0)) : "memory");
          else
            mbar_arrive(&bars->acc_empty[buf]);
        }
      }
      // (a policy's epilogue may hold barriers of the epilogue warps: a warp
      // whose wait gave up goes on through its tiles with what it has, without
      // waiting, and the status tells)
      e.n = n;
      p.epilogue(e, t, acc);
    }
    p.finish(counts, e);
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_meet();   // neither CTA's memory is used past here
  tc_fence_after();
  if (warp == 1) {
    if constexpr (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmemCols) : "memory");
    else
      tmem_dealloc(tmem, S::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// stores of an epilogue warp's 32 rows through its box, 128-byte swizzled
// (chunk j of line r at j ^ (r & 7)); `row` is the tile's row of its lane 0
// ---------------------------------------------------------------------------
constexpr int kBoxRows = 16;                  // of a store
constexpr int kStoreBox = kBoxRows * 128;

// 64 values a thread, 16-bit each (packed two a word): boxes of 16 rows x 64
// columns of a map's [rows][cols]; nothing past either end.
__device__ __forceinline__ void store_16bit(const Epi& e, const CUtensorMap* map, const uint32_t (&w)[32], int col, int cols,
                                            int row, int rows) {
#pragma unroll
  for (int g = 0; g < 32 / kBoxRows; ++g) {
    if (e.lane == 0) bulk_wait_read<0>();   // the box before is out
    __syncwarp();
    if (e.lane / kBoxRows == g) {
      const int r = e.lane % kBoxRows;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(e.box + r * 128 + ((j ^ (r & 7)) << 4)) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (e.lane == 0 && row + g * kBoxRows < rows && col < cols) {
      tma_s2g_2d(map, e.box, col, row + g * kBoxRows);
      bulk_commit();
    }
  }
}

// 64 fp32 values a thread, into or added to a map's [parts][rows][cols] in boxes
// of 16 rows x 32 columns.
__device__ __forceinline__ void store_fp32(const Epi& e, const CUtensorMap* map, const float (&v)[64], int col, int cols,
                                           int row, int rows, int part, bool add) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int g = 0; g < 32 / kBoxRows; ++g) {
      if (e.lane == 0) bulk_wait_read<0>();
      __syncwarp();
      if (e.lane / kBoxRows == g) {
        const int r = e.lane % kBoxRows;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          *reinterpret_cast<float4*>(e.box + r * 128 + ((x ^ (r & 7)) << 4)) =
              make_float4(v[j * 32 + 4 * x], v[j * 32 + 4 * x + 1], v[j * 32 + 4 * x + 2], v[j * 32 + 4 * x + 3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (e.lane == 0 && row + g * kBoxRows < rows && col + j * 32 < cols) {
        if (add)
          asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                           reinterpret_cast<uint64_t>(map)),
                       "r"(smem_u32(e.box)), "r"(col + j * 32), "r"(row + g * kBoxRows), "r"(part)
                       : "memory");
        else
          tma_s2g_3d(map, e.box, col + j * 32, row + g * kBoxRows, part);
        bulk_commit();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// A [rows, cols] matrix of 16-bit values, rows `stride` values apart, in boxes
// of box_rows x 64, 128-byte swizzled.
inline cudaError_t map_16bit(const void* base, bool bf16, long long rows, long long cols, long long stride, int box_rows,
                             CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A [parts, rows, cols] fp32 array, dense, in boxes of 16 rows x 32.
inline cudaError_t map_fp32(float* base, long long parts, long long rows, long long cols, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 4, (cuuint64_t)cols * 4 * rows};
  cuuint32_t box[3] = {32, kBoxRows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Units that run at the same time: one CTA an SM.
template <class P>
inline int max_units() {
  const int sms = sm_count();
  return P::kPair ? sms / 2 : sms;
}

// `units` of the kernel, which may start while the kernel before it ends.
template <class P>
inline cudaError_t launch(const P& p, int units, cudaStream_t stream) {
  auto kern = gemm_kernel<P>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<P>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(P::kPair ? 2 * units : units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<P>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = P::kPair ? 2 : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace gemm
}  // namespace dspark
