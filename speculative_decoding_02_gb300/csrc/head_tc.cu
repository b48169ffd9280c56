// The Markov head outside the sampling kernel, for training it ("[DeepSeek-6]
// DSpark" blog, section 4): its logits for given tokens, and the gradients of
// its two weights.  bf16 weights of rank 256, on the tensor cores.  Rows n =
// b * G + k - 1 are the positions of all requests, E[n] = W1[x_{k-1}] (x_0 the
// anchor), N = B * G of them:
//
//   markov_logits:  l = U + E W2^T                       [N, V]
//   head backward:  dW2 = D^T E                          [V, 256]
//                   dE = D W2,  dW1[t] = sum over n with x_{k-1} = t of dE[n]
//
// with D [N, V] bf16 the gradient of l.  All products are exact in fp32 and
// summed in fp32.  Both are bound by HBM when N is large: the logits by one read
// of U and one write of l (W2 stays in L2), the gradients by two reads of D and
// the writes of dW1 and dW2.
//
// Measured (GB300, N = 2048, V = 151936): the logits 392 us (6.5 TB/s, 97 % of
// the copy rate); the gradients 309 us, of which dW2 165 (1.0 GB, 6.1 TB/s; its
// flops' floor is 82) and dE 134 (0.7 GB, 5.2 TB/s), the rest the sums of the
// parts and of each token's rows.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "kernels.h"
#include "tc_common.cuh"

namespace dspark {
namespace {

using namespace tc;

constexpr int HM = 128;            // rows of a tile (TMEM lanes)
constexpr int HK = 256;            // Markov rank
constexpr int kMaxSmem = 232448;   // dynamic shared memory one CTA may use

// E[m, 64a .. 64a+63] = W1[tok] into this warp's TMEM lanes (zeros without a token).
__device__ __forceinline__ void gather_e(const __nv_bfloat16* W1, int tok, int a, uint32_t taddr) {
  const uint4* wrow = reinterpret_cast<const uint4*>(W1 + (size_t)max(tok, 0) * HK);
  uint32_t ev[32];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 val = tok >= 0 ? __ldg(wrow + a * 8 + c) : make_uint4(0, 0, 0, 0);
    ev[4 * c] = val.x; ev[4 * c + 1] = val.y; ev[4 * c + 2] = val.z; ev[4 * c + 3] = val.w;
  }
  tmem_store_32cols(taddr, ev);
}

// The token before row n's position; -1 (and DSPARK_ERR_INVALID recorded) when
// it is outside [0, V).
__device__ __forceinline__ int previous_token(const int32_t* anchor, const int32_t* x, long long n, int G, int V,
                                              int* status) {
  const long long b = n / G;
  const int k = (int)(n - b * G);
  const int t = k == 0 ? anchor[b] : x[n - 1];
  if (t >= 0 && t < V) return t;
  record_status(status, DSPARK_ERR_INVALID);
  return -1;
}

// ---------------------------------------------------------------------------
// Logits.  Persistent CTAs, each a contiguous range of tiles of 128 rows x 64
// columns, row tile by row tile:
//   warp 0     TMA producer: the W2 rows of a tile (evict_last: every row tile
//              reads them again from L2) and its U box (256 contiguous bytes a row);
//   warp 1     MMA issuer: E (tensor memory) times the W2 rows into one of two
//              accumulators;
//   warps 2-9  a thread owns a row and 32 columns: adds the accumulator to U in
//              place and one of them stores the tile by TMA; at a row tile's end
//              they gather the next E.
// ---------------------------------------------------------------------------
constexpr int GN = 64;             // columns of a tile
constexpr int GUStages = 5, GWStages = 2;
constexpr int GEpiWarps = 8;
constexpr int GThreads = 64 + 32 * GEpiWarps;
constexpr int GUBytes = HM * GN * 4;     // 32768
constexpr int GWBytes = GN * HK * 2;     // 32768
constexpr uint32_t GTmemCols = 256;      // two accumulators, then E
constexpr uint32_t GTmemE = 2 * GN;
constexpr int GSmemBytes = 1024 + GUStages * GUBytes + GWStages * GWBytes + 512;
static_assert(GSmemBytes <= kMaxSmem, "shared memory");

struct __align__(8) GBars {
  uint64_t full_u[GUStages], empty_u[GUStages];
  uint64_t full_w[GWStages], empty_w[GWStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t e_full, drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(GBars) <= 512, "barrier block");

struct LogitParams {
  const __nv_bfloat16* W1;
  const int32_t* anchor;
  const int32_t* x;
  int* status;
  int N, G, V;
  int ntiles;        // column tiles
  int tail_tile;     // the column tile that comes and goes as [rows x 32] boxes (V % 32 != 0), else -1
  long long units;
  int per;           // CTAs of a row tile, or 0
};

__device__ __forceinline__ void tma_s2g_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void tma_s2g_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void tma_s2g_4d(const CUtensorMap* map, const void* src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All bulk stores of this thread but the newest kLeft have read their shared memory.
template <int kLeft>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}

// kOut: DSPARK_F32 or DSPARK_BF16 logits.
template <int kOut>
__global__ void __launch_bounds__(GThreads, 1)
markov_logits_tc(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap u_map,
                 const __grid_constant__ CUtensorMap u4_map, const __grid_constant__ CUtensorMap o_map,
                 const __grid_constant__ CUtensorMap o4_map, const LogitParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* U_s = smem;
  unsigned char* W_s = U_s + GUStages * GUBytes;
  GBars* bars = reinterpret_cast<GBars*>(W_s + GWStages * GWBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's tiles u = row tile * ntiles + column tile: with per > 0 every
  // per-th of one row tile, else a contiguous range
  const int step = max(p.per, 1);
  const long long row0 = p.per > 0 ? (long long)(blockIdx.x / p.per) * p.ntiles : 0;
  const long long u0 = p.per > 0 ? row0 + blockIdx.x % p.per : p.units * blockIdx.x / gridDim.x;
  const long long u1 = p.per > 0 ? row0 + p.ntiles : p.units * (blockIdx.x + 1) / gridDim.x;
  volatile int* abort = &bars->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < GUStages; ++s) { mbar_init(&bars->full_u[s], 1); mbar_init(&bars->empty_u[s], 1); }
    for (int s = 0; s < GWStages; ++s) { mbar_init(&bars->full_w[s], 1); mbar_init(&bars->empty_w[s], 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(&bars->acc_full[s], 1); mbar_init(&bars->acc_empty[s], GEpiWarps); }
    mbar_init(&bars->e_full, GEpiWarps);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&w_map);
    prefetch_tensormap(&u_map);
    prefetch_tensormap(&u4_map);
    prefetch_tensormap(&o_map);
    prefetch_tensormap(&o4_map);
  }
  if (warp == 1) tmem_alloc(&bars->tmem_base, GTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol_w = policy_evict_last(), pol_u = policy_evict_normal();
      uint32_t i = 0;
      bool ok = true;
      for (long long u = u0; u < u1; u += step, ++i) {
        const int m0 = (int)(u / p.ntiles) * HM, t = (int)(u % p.ntiles), v0 = t * GN;
        const int sw = i % GWStages, su = i % GUStages;
        ok = mbar_wait(&bars->empty_w[sw], ((i / GWStages) & 1) ^ 1, abort, p.status);
        if (!ok) break;
        mbar_arrive_expect_tx(&bars->full_w[sw], GWBytes);
        for (int a = 0; a < HK / 64; ++a)
          tma_g2s_2d(W_s + sw * GWBytes + a * GN * 128, &w_map, a * 64, v0, &bars->full_w[sw], pol_w);
        ok = mbar_wait(&bars->empty_u[su], ((i / GUStages) & 1) ^ 1, abort, p.status);
        if (!ok) break;
        unsigned char* dst = U_s + su * GUBytes;
        mbar_arrive_expect_tx(&bars->full_u[su], GUBytes);
        if (t != p.tail_tile) {
          tma_g2s_4d(dst, &u4_map, 0, v0 / 32, 0, m0, &bars->full_u[su], pol_u);
        } else {
          tma_g2s_3d(dst, &u_map, v0, 0, m0, &bars->full_u[su], pol_u);
          tma_g2s_3d(dst + HM * 128, &u_map, v0 + 32, 0, m0, &bars->full_u[su], pol_u);
        }
      }
      if (*abort) {
        // what was issued lands before the CTA leaves (a wait for a phase
        // that is over returns at once)
        for (int s = 0; s < GWStages; ++s) {
          const uint32_t n = (i + GWStages - 1 - s) / GWStages + (i % GWStages == (uint32_t)s && !ok ? 1 : 0);
          if (n > 0) mbar_drain(&bars->full_w[s], (n - 1) & 1);
        }
        for (int s = 0; s < GUStages; ++s) {
          const uint32_t n = (i + GUStages - 1 - s) / GUStages;
          if (n > 0) mbar_drain(&bars->full_u[s], (n - 1) & 1);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(HM, GN);
      uint32_t i = 0, em = 0;
      int m = -1;
      bool ok = true;
      for (long long u = u0; u < u1 && ok; u += step, ++i) {
        if ((int)(u / p.ntiles) != m) {
          m = (int)(u / p.ntiles);
          if (!(ok = mbar_wait(&bars->e_full, em++ & 1, abort, p.status))) break;
        }
        const int acc = i & 1, sw = i % GWStages;
        if (!(ok = mbar_wait(&bars->acc_empty[acc], ((i >> 1) & 1) ^ 1, abort, p.status))) break;
        if (!(ok = mbar_wait(&bars->full_w[sw], (i / GWStages) & 1, abort, p.status))) break;
        tc_fence_after();
#pragma unroll
        for (int a = 0; a < HK / 64; ++a) {
          const uint64_t bd = sw128_kmajor_desc(smem_u32(W_s + sw * GWBytes + a * GN * 128));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_tmem_a(tmem + acc * GN, tmem + GTmemE + a * 32 + kk * 8, bd + (uint64_t)(kk * 2), idesc,
                             (a | kk) != 0);
        }
        umma_commit(&bars->empty_w[sw]);
        umma_commit(&bars->acc_full[acc]);
      }
      umma_commit(&bars->drain);
      mbar_drain(&bars->drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, h = (warp - 2) >> 2;
    const int r = q * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    uint32_t i = 0;
    int m = -1;
    bool ok = true;
    // (a warp whose wait gave up goes on through the tiles' barriers, which the
    // others may be at, and does nothing else)
    for (long long u = u0; u < u1; u += step, ++i) {
      const int t = (int)(u % p.ntiles);
      const int acc = i & 1, su = i % GUStages;
      unsigned char* tile = U_s + su * GUBytes;
      const int line = t != p.tail_tile ? 2 * r + h : h * HM + r;
      float v[32];
      if (ok && (int)(u / p.ntiles) != m) {
        // (this warp has seen the last accumulator of the row tile before
        // complete, so no MMA reads the old E)
        m = (int)(u / p.ntiles);
        const long long n = (long long)m * HM + r;
        const int tok = n < p.N ? previous_token(p.anchor, p.x, n, p.G, p.V, p.status) : -1;
        gather_e(p.W1, tok, 2 * h, lanes + GTmemE + 2 * h * 32);
        gather_e(p.W1, tok, 2 * h + 1, lanes + GTmemE + (2 * h + 1) * 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->e_full);
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_full[acc], (i >> 1) & 1, abort, p.status));
      if (ok) {
        tc_fence_after();
        tmem_load_cols<32>(lanes + acc * GN + h * 32, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->acc_empty[acc]);
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->full_u[su], (i / GUStages) & 1, abort, p.status));
      }
      if (ok) {
        // this thread's 32 columns of U: the 128-byte line 2r + h of a tile box
        // (h * 128 + r of a tail tile's two boxes), its 16-byte chunk j at j ^ (line & 7)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float4* c = reinterpret_cast<float4*>(tile + line * 128 + ((j ^ (line & 7)) << 4));
          float4 f = *c;
          f.x += v[4 * j]; f.y += v[4 * j + 1]; f.z += v[4 * j + 2]; f.w += v[4 * j + 3];
          if (kOut == DSPARK_F32) *c = f;
          else { v[4 * j] = f.x; v[4 * j + 1] = f.y; v[4 * j + 2] = f.z; v[4 * j + 3] = f.w; }
        }
      }
      if (kOut == DSPARK_BF16) {
        // the tile's first half becomes [128 rows][64 columns] bf16, once
        // every thread has read its U
        named_bar_sync(1, GEpiWarps * 32);
        if (ok) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            __nv_bfloat162 o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = __floats2bfloat162_rn(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
            *reinterpret_cast<uint4*>(tile + r * 128 + (((4 * h + j) ^ (r & 7)) << 4)) = *reinterpret_cast<uint4*>(o);
          }
        }
      }
      fence_proxy_async_smem();
      named_bar_sync(1, GEpiWarps * 32);
      if (ok && warp == 2 && lane == 0) {
        const int v0 = t * GN, m0 = m * HM;
        if (kOut == DSPARK_BF16) {
          tma_s2g_2d(&o_map, tile, v0, m0);
        } else if (t != p.tail_tile) {
          tma_s2g_4d(&o4_map, tile, 0, v0 / 32, 0, m0);
        } else {
          tma_s2g_3d(&o_map, tile, v0, 0, m0);
          if (v0 + 32 < p.V) tma_s2g_3d(&o_map, tile + HM * 128, v0 + 32, 0, m0);
        }
        bulk_commit();
        // the tile before is out of its stage
        bulk_wait_read<1>();
        if (i > 0) mbar_arrive(&bars->empty_u[(i - 1) % GUStages]);
      }
    }
    if (warp == 2 && lane == 0) bulk_wait_read<0>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, GTmemCols);
}

// ---------------------------------------------------------------------------
// Weight gradients.  One kernel for both products, on pairs of CTAs
// (cta_group::2): a tile of 256 x 256, 128 rows of it in each CTA's tensor
// memory, accumulated over K in stages of 64.  Each CTA copies its 128 rows of
// A and one half of B (128 of the 256 columns):
//   kW2:  dW2 tile [256 v, 256] over K = rows n:  A = D^T (the stage holds
//         [64 n][64 v] boxes, M-major), B = E [64 n][256] (N-major)
//   else: part of dE [256 n, 256] over a range of K = v:  A = D ([128 n][64 v]
//         boxes, K-major), B = W2 [64 v][256] (N-major)
//
//   warp 0     TMA producer of its CTA; all copies of a stage count on the
//              first CTA's barrier;
//   warp 1     of the first CTA: MMA issuer for both;
//   warps 2-17 a thread owns a row and 64 columns; at a tile's end they go to
//              shared memory by boxes of 16 rows x 32 columns and out by TMA.
//
// The tensor cores truncate when they add to an accumulator, which over the
// 128 additions of 2048 rows came to a relative error of 1e-5 (2-norm), an order
// more than fp32 products have.  So an accumulator takes kChunk stages only (32
// additions) and the epilogue adds it, rounded, to sums in registers, while
// the next one fills (two of them): errors of 6.6e-7 (dW1) and 6.5e-7 (dW2),
// where plain fp32 products have 1.4e-6 and 7e-7.  Longer chunks are faster and
// less exact (dW2: 156 us and 1.3e-6 by 16 stages, 165 us by 8), in shorter ones
// the epilogue's latency shows (209 us by 3, 3.3e-7).
// ---------------------------------------------------------------------------
constexpr int BEpiWarps = 16;
constexpr int BThreads = 64 + 32 * BEpiWarps;
constexpr int BStages = 5;
constexpr int kChunk = 8;
constexpr int BABytes = HM * 64 * 2;           // 16384: 128 rows of A
constexpr int BBBytes = HK / 2 * 64 * 2;       // 16384: 128 columns of B
constexpr int BStageBytes = BABytes + BBBytes;
constexpr int BBoxRows = 16;
constexpr int BBoxBytes = BBoxRows * 32 * 4;   // of an epilogue warp's output
constexpr int BZeroBytes = 4096;
constexpr int BSmemBytes = 1024 + BStages * BStageBytes + BEpiWarps * BBoxBytes + BZeroBytes + 256;
constexpr uint32_t BTmemCols = 512;            // two accumulators of 256 columns
static_assert(BSmemBytes <= kMaxSmem, "shared memory");

struct __align__(8) BBars {
  uint64_t full[BStages], empty[BStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(BBars) <= 256, "barrier block");
static_assert(BZeroBytes == 4 * HK * 4, "four rows of dW1");

struct GradParams {
  float* zero;       // kW2: dW1 [V][256], which is cleared along
  int* status;
  int rows;          // kW2: V; else the rows of this chunk of D
  int row0;          // else: the chunk's first row of D
  int ksteps;        // 64-wide steps of K
  int tiles;         // kW2: tiles of 256 v; else groups of 256 rows
  int splits;        // else: parts of K (tiles * splits pairs)
  bool wait_last;    // nothing here depends on the kernel before, but a kernel ends after it
};

// A matrix in 128-byte swizzled boxes of [K rows][64 of M or N]: 8 rows of K
// make a 1024-byte group, boxes of 64 are `box_bytes` apart.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t box_bytes) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(box_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
constexpr uint32_t kAMajorM = 1u << 15, kBMajorN = 1u << 16;   // instruction descriptor: not K-major

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address, in the cluster's window, of the same place in CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// tma_g2s_2d of a CTA pair: the bytes count on a barrier of either CTA.
__device__ __forceinline__ void tma_pair_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` of both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void umma_pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
template <bool kW2>
__global__ void __launch_bounds__(BThreads, 1) __cluster_dims__(2, 1, 1)
head_grad_tc(const __grid_constant__ CUtensorMap d_map, const __grid_constant__ CUtensorMap b_map,
             const __grid_constant__ CUtensorMap o_map, const GradParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* boxes = smem + BStages * BStageBytes;
  unsigned char* zeros = boxes + BEpiWarps * BBoxBytes;
  BBars* bars = reinterpret_cast<BBars*>(zeros + BZeroBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int* abort = &bars->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < BStages; ++s) { mbar_init(&bars->full[s], 1); mbar_init(&bars->empty[s], 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(&bars->acc_full[s], 1); mbar_init(&bars->acc_empty[s], 2 * BEpiWarps); }
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&d_map);
    prefetch_tensormap(&b_map);
    prefetch_tensormap(&o_map);
  }
  for (int i = threadIdx.x; i < BZeroBytes / 4; i += BThreads) reinterpret_cast<float*>(zeros)[i] = 0.f;
  fence_proxy_async_smem();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)),
                 "r"(BTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_meet();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  pdl_trigger();
  if (!p.wait_last) pdl_wait();

  // this pair's tiles and, of each, its steps of K: split, split + kstep, ...
  const int tile0 = kW2 ? pair : pair / p.splits;
  const int tile_step = kW2 ? pairs : p.tiles;
  const int split = kW2 ? 0 : pair % p.splits;
  // (the parts of K are interleaved, so that the pairs read neighbouring 128-byte
  // pieces of a row of D at about the same time)
  const int kstep = kW2 ? 1 : p.splits;
  const int nk = (p.ksteps - split + kstep - 1) / kstep;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      // (a copy of 128-byte pieces brings its neighbours into L2 as well, which
      // evict_first would drop before the pair next to this one reads them)
      const uint64_t pol_d = policy_evict_normal(), pol_b = policy_evict_last();
      uint32_t i = 0;
      bool ok = true;
      for (int tile = tile0; tile < p.tiles && ok; tile += tile_step) {
        const int m0 = (tile * 2 + rank) * HM;
        for (int k = split; k < p.ksteps; k += kstep, ++i) {
          const int s = i % BStages;
          ok = mbar_wait(&bars->empty[s], ((i / BStages) & 1) ^ 1, abort, p.status);
          if (!ok) break;
          unsigned char* a = smem + s * BStageBytes;
          const uint32_t full = in_cta(&bars->full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2 * BStageBytes);
          if (kW2) {
            for (int j = 0; j < 2; ++j) tma_pair_2d(a + j * 8192, &d_map, m0 + j * 64, k * 64, full, pol_d);
          } else {
            tma_pair_2d(a, &d_map, k * 64, p.row0 + m0, full, pol_d);
          }
          for (int j = 0; j < 2; ++j)
            tma_pair_2d(a + BABytes + j * 8192, &b_map, (rank * 2 + j) * 64, k * 64, full, pol_b);
        }
      }
      // every stage is consumed before the CTA leaves (on a timeout: as far as
      // the wait's limit goes, which is longer than any copy takes)
      for (int s = 0; s < BStages; ++s) {
        const uint32_t n = (i + BStages - 1 - s) / BStages;
        if (n > 0) mbar_drain(&bars->empty[s], (n - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(2 * HM, HK) | kBMajorN | (kW2 ? kAMajorM : 0u);
      uint32_t i = 0, chunk = 0;
      bool ok = true;
      for (int tile = tile0; tile < p.tiles && ok; tile += tile_step) {
        for (int k = 0; k < nk && ok; ++chunk) {
          const int buf = chunk & 1, kend = min(k + kChunk, nk);
          ok = mbar_wait(&bars->acc_empty[buf], ((chunk >> 1) & 1) ^ 1, abort, p.status);
          if (!ok) break;
          tc_fence_after();
          for (int kf = k; k < kend; ++k, ++i) {
            const int s = i % BStages;
            ok = mbar_wait(&bars->full[s], (i / BStages) & 1, abort, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = smem_u32(smem + s * BStageBytes);
            const uint64_t ad = kW2 ? sw128_mnmajor_desc(a, 8192) : sw128_kmajor_desc(a);
            const uint64_t bd = sw128_mnmajor_desc(a + BABytes, 8192);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)   // 16 of K: two 1024-byte groups, or 32 bytes of a K-major row
              umma_pair(tmem + buf * HK, ad + (uint64_t)(kk * (kW2 ? 128 : 2)), bd + (uint64_t)(kk * 128), idesc,
                        k != kf || kk != 0);
            umma_pair_commit(&bars->empty[s]);
          }
          if (ok) umma_pair_commit(&bars->acc_full[buf]);
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, h = (warp - 2) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + h * 64;
    unsigned char* box = boxes + (warp - 2) * BBoxBytes;
    const int nchunks = (nk + kChunk - 1) / kChunk;
    uint32_t chunk = 0;
    bool ok = true;
    for (int tile = tile0; tile < p.tiles && ok; tile += tile_step) {
      float acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0.f;
      for (int n = 0; n < nchunks && ok; ++n, ++chunk) {
        const int buf = chunk & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_full[buf], (chunk >> 1) & 1, abort, p.status));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[16];
          tmem_load_cols<16>(lanes + buf * HK + j * 16, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[j * 16 + e] += v[e];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_in_cluster(in_cta(&bars->acc_empty[buf], 0));
      }
      if (!ok) break;
      // this warp's 32 rows and 64 columns by boxes, 128-byte swizzled (chunk j
      // of row r at j ^ (r & 7)); rows past the output's end are clipped
      const int row = (tile * 2 + rank) * HM + q * 32;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int g = 0; g < 32 / BBoxRows; ++g) {
          if (lane == 0) bulk_wait_read<0>();   // the box before is out
          __syncwarp();
          if (lane / BBoxRows == g) {
            const int r = lane % BBoxRows;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(box + r * 128 + ((e ^ (r & 7)) << 4)) =
                  make_float4(acc[j * 32 + 4 * e], acc[j * 32 + 4 * e + 1], acc[j * 32 + 4 * e + 2],
                              acc[j * 32 + 4 * e + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row + g * BBoxRows < p.rows) {
            tma_s2g_3d(&o_map, box, h * 64 + j * 32, row + g * BBoxRows, split);
            bulk_commit();
          }
        }
      }
      if (kW2 && lane == 0) {
        // zeros into 8 of the 32 rows of dW1
        for (int i = 0; i < 2; ++i) {
          const int z = row + h * 8 + i * 4, n = min(4, p.rows - z);
          if (n > 0)
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p.zero + (size_t)z * HK),
                         "r"(smem_u32(zeros)), "r"(n * HK * 4)
                         : "memory");
        }
        bulk_commit();
      }
    }
    if (lane == 0) bulk_wait_read<0>();
  }
  if (p.wait_last) pdl_wait();
  tc_fence_before();
  __syncthreads();
  cluster_meet();   // neither CTA's memory is used past here
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(BTmemCols) : "memory");
}

// E [N][256] and the previous tokens [N] (-1: none), a warp per row.
__global__ void __launch_bounds__(256) gather_rows(const __nv_bfloat16* __restrict__ W1, const int32_t* __restrict__ anchor,
                                                   const int32_t* __restrict__ x, int N, int G, int V,
                                                   uint4* __restrict__ E, int32_t* __restrict__ prev, int* status) {
  const int n = (int)((blockIdx.x * (long long)blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  pdl_trigger();
  if (n >= N) return;
  const int tok = previous_token(anchor, x, n, G, V, status);
  E[(size_t)n * 32 + lane] =
      tok >= 0 ? __ldg(reinterpret_cast<const uint4*>(W1 + (size_t)tok * HK) + lane) : make_uint4(0, 0, 0, 0);
  if (lane == 0) prev[n] = tok;
}

// dE of a chunk of rows: the sum of its parts, into the first.
__global__ void __launch_bounds__(256) sum_parts(float4* part, int rows, int splits) {
  pdl_trigger();
  pdl_wait();
  const size_t n = (size_t)rows * (HK / 4), i = blockIdx.x * (size_t)256 + threadIdx.x;
  if (i >= n) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    const float4 v = part[s * n + i];
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  }
  part[i] = a;
}

// dW1 of a chunk of rows: the block of a token's first row in the chunk adds
// dE of every row of that token, in order of the rows, to dW1[token].
__global__ void __launch_bounds__(HK) scatter_rows(const float* dE, const int32_t* prev,
                                                   int rows, float* dW1) {
  pdl_trigger();
  pdl_wait();
  const int n = blockIdx.x, tok = prev[n];
  if (tok < 0) return;
  // bit i: row i * HK + threadIdx.x has this token
  unsigned mine = 0;
#pragma unroll 8
  for (int i = 0; i < div_up(rows, HK); ++i) {
    const int j = i * HK + threadIdx.x;
    if ((j < rows ? prev[j] : -1) == tok) mine |= 1u << i;
  }
  __shared__ unsigned some[HK / 32], hits[HK / 32];
  __shared__ int list[HK];
  const int warp = threadIdx.x >> 5;
  const unsigned warp_has = __reduce_or_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0) some[warp] = warp_has;
  if (__syncthreads_or(mine != 0 && (__ffs(mine) - 1) * HK + (int)threadIdx.x < n)) return;   // not the first
  unsigned all = 0;
  for (int w = 0; w < HK / 32; ++w) all |= some[w];
  float acc = 0.f;
  for (unsigned left = all; left != 0; left &= left - 1) {
    const int i0 = __ffs(left) - 1, j = i0 * HK + threadIdx.x;
    const bool same = mine >> i0 & 1u;
    if (left != all) __syncthreads();   // (the list before has been read)
    const unsigned h = __ballot_sync(0xffffffffu, same);
    if ((threadIdx.x & 31) == 0) hits[warp] = h;
    __syncthreads();
    int before = 0, count = 0;
    for (int w = 0; w < HK / 32; ++w) {
      if (w < warp) before += __popc(hits[w]);
      count += __popc(hits[w]);
    }
    if (same) list[before + __popc(h & ((1u << (threadIdx.x & 31)) - 1u))] = j;
    __syncthreads();
    for (int i = 0; i < count; i += 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = i + u < count ? dE[(size_t)list[i + u] * HK + threadIdx.x] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) acc += v[u];
    }
  }
  dW1[(size_t)tok * HK + threadIdx.x] += acc;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A [rows, cols] bf16 matrix in boxes of `box_rows` x 64, 128-byte swizzled.
cudaError_t make_bf16_map(const void* base, int rows, int cols, int box_rows, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

template <bool kW2>
cudaError_t launch_grad(int pairs, const CUtensorMap& d, const CUtensorMap& b, float* out, const GradParams& p,
                        cudaStream_t stream) {
  // the output [splits][rows][256] in boxes of 16 x 32, 128-byte swizzled
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap o;
  cuuint64_t dims[3] = {(cuuint64_t)HK, (cuuint64_t)p.rows, (cuuint64_t)p.splits};
  cuuint64_t strides[2] = {(cuuint64_t)HK * 4, (cuuint64_t)HK * 4 * p.rows};
  cuuint32_t box[3] = {32, BBoxRows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  if (enc(&o, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  auto kern = head_grad_tc<kW2>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(2 * pairs), dim3(BThreads), BSmemBytes, stream, d, b, o, p);
}

// Rows of D whose dE parts the workspace holds at a time, and parts of K for
// them: one CTA an SM.
constexpr int kChunkRows = 4096;
static_assert(kChunkRows / HK <= 32, "scatter_rows keeps a bit for every HK rows");
constexpr int kMaxPairs = 80;

}  // namespace

// Workspace: status word, previous tokens, E, the dE parts of a chunk.
size_t head_workspace_bytes(int N, int V) {
  // rows * splits of a chunk: at most 256 rows for each pair, and at most
  // kMaxPairs or V / (64 kChunk) parts of the rows there are
  const size_t splits = std::min(kMaxPairs, div_up(div_up(V, 64), kChunk));
  const size_t parts = std::min<size_t>((size_t)kMaxPairs * 2 * HM, splits * std::min(N, kChunkRows));
  return 256 + align256(4ull * N) + align256(512ull * N) + align256(1024ull * parts);
}

cudaError_t launch_markov_logits(const MarkovLogitArgs& a, cudaStream_t stream) {
  const int N = a.B * a.G;
  CUtensorMap w, u, u4, o, o4;
  cudaError_t e;
  if ((e = make_w2_tensor_map(a.W2, a.V, &w, GN)) != cudaSuccess) return e;
  if ((e = make_u_tensor_map(a.U, N, 1, a.V, HM, &u)) != cudaSuccess) return e;
  if ((e = make_u_tile_map(a.U, N, 1, a.V, HM, &u4)) != cudaSuccess) return e;
  if (a.odtype == DSPARK_F32) {
    if ((e = make_u_tensor_map(static_cast<const float*>(a.out), N, 1, a.V, HM, &o)) != cudaSuccess) return e;
    if ((e = make_u_tile_map(static_cast<const float*>(a.out), N, 1, a.V, HM, &o4)) != cudaSuccess) return e;
  } else {
    if ((e = make_bf16_map(a.out, N, a.V, HM, &o)) != cudaSuccess) return e;
    o4 = o;
  }
  LogitParams p{};
  p.W1 = static_cast<const __nv_bfloat16*>(a.W1);
  p.anchor = a.anchor;
  p.x = a.x;
  p.status = a.status;
  p.N = N; p.G = a.G; p.V = a.V;
  p.ntiles = div_up(a.V, GN);
  p.tail_tile = a.V % 32 != 0 ? p.ntiles - 1 : -1;
  p.units = (long long)div_up(N, HM) * p.ntiles;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  // CTAs side by side on one row tile read neighbouring columns at about the
  // same time, which DRAM serves faster than one range a CTA: 393 against 449 us
  // at 16 row tiles of 151936 columns, 163 against 181 at 60 of 16384 although
  // that leaves a fifth of the SMs idle.  With one CTA a row tile there are no
  // neighbours (297 against 301 at 100 row tiles): ranges, on every SM.
  const int mtiles = div_up(N, HM);
  p.per = std::min(sms / mtiles, p.ntiles);
  if (p.per == 1 && p.ntiles > 1) p.per = 0;
  const int grid = p.per > 0 ? mtiles * p.per : (int)std::min<long long>(p.units, sms);
  auto kern = a.odtype == DSPARK_F32 ? markov_logits_tc<DSPARK_F32> : markov_logits_tc<DSPARK_BF16>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GSmemBytes)) != cudaSuccess) return e;
  kern<<<grid, GThreads, GSmemBytes, stream>>>(w, u, u4, o, o4, p);
  return cudaGetLastError();
}

cudaError_t launch_markov_head_backward(const HeadBackwardArgs& a, cudaStream_t stream) {
  const int N = a.B * a.G;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  char* ws = static_cast<char*>(a.ws);
  int* status = a.status;
  int32_t* prev = reinterpret_cast<int32_t*>(ws + 256);
  char* E = ws + 256 + align256(4ull * N);
  float* part = reinterpret_cast<float*>(E + align256(512ull * N));
  cudaError_t e;
  gather_rows<<<(unsigned)div_up(N, 8), 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(a.W1), a.anchor, a.x, N,
                                                         a.G, a.V, reinterpret_cast<uint4*>(E), prev, status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  // dW2 (and zeros into dW1)
  const int pairs = std::min(sms / 2, kMaxPairs);
  CUtensorMap dm, bm;
  if ((e = make_bf16_map(a.dlogits, N, a.V, 64, &dm)) != cudaSuccess) return e;
  if ((e = make_bf16_map(E, N, HK, 64, &bm)) != cudaSuccess) return e;
  GradParams p{};
  p.zero = a.dW1;
  p.status = status;
  p.rows = a.V;
  p.ksteps = div_up(N, 64);
  p.tiles = div_up(a.V, 2 * HM);
  p.splits = 1;
  if ((e = launch_grad<true>(std::min(p.tiles, pairs), dm, bm, a.dW2, p, stream)) != cudaSuccess) return e;

  // dE and dW1, a chunk of rows at a time
  if ((e = make_bf16_map(a.dlogits, N, a.V, HM, &dm)) != cudaSuccess) return e;
  if ((e = make_bf16_map(a.W2, a.V, HK, 64, &bm)) != cudaSuccess) return e;
  for (int r0 = 0; r0 < N; r0 += kChunkRows) {
    const int rows = std::min(N - r0, kChunkRows);
    p.rows = rows;
    p.row0 = r0;
    p.ksteps = div_up(a.V, 64);
    p.tiles = div_up(rows, 2 * HM);
    // (a part of K shorter than one chunk costs more in sum_parts than it gives:
    // 64 rows of 8192 take 21 us by 16 parts, 41 by 76)
    p.splits = std::max(1, std::min(pairs / p.tiles, div_up(p.ksteps, kChunk)));
    p.wait_last = r0 == 0;   // (a later chunk's parts replace those of the one before)
    if ((e = launch_grad<false>(p.tiles * p.splits, dm, bm, part, p, stream)) != cudaSuccess) return e;
    if (p.splits > 1) {
      e = launch_pdl(sum_parts, dim3((unsigned)div_up(rows * (HK / 4), 256)), dim3(256), 0, stream,
                     reinterpret_cast<float4*>(part), rows, p.splits);
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(scatter_rows, dim3((unsigned)rows), dim3(HK), 0, stream, (const float*)part, (const int32_t*)(prev + r0),
                   rows, a.dW1);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dspark
