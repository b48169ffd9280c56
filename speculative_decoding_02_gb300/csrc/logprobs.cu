// Log probabilities of given tokens with the row's entropy and its K most
// probable entries, and the gradient of the first two.
//
//   lse = log sum_v exp x_v,   logp = x_t - lse,   H = -sum_v p_v log p_v
//   dx_v = g_logp (1[v = t] - p_v) - g_H p_v (log p_v + H)
//
// Forward: one pass over the row (logits_row.cuh); HBM bounds it.  A cluster
// of 1 to 8 CTAs takes a row; their states and top lists meet in CTA 0 through
// distributed shared memory.  The top entries cost the pass one maximum per
// lane and one stored maximum per block:
//   1. the K-th largest of the CTA's 256 lane maxima is a lower bound of the row
//      part's K-th largest entry (K distinct entries are at least that large);
//   2. only the blocks whose maximum reaches it are read again (from L2), and
//      their entries that reach it become candidates, about K (1 + K / 512)
//      of them in a row of no particular order;
//   3. a candidate's rank is the number of larger ones (64-bit keys of value,
//      then lower index, so no two are equal and ties go to the lowest index).
// Rows whose candidates overflow the buffer (thousands of equal or ascending
// entries) find the K-th largest key by bisection over its 64 bits instead.
#include "logits_row.cuh"

namespace dspark {
namespace {

using namespace lrow;

constexpr int kMaxBlocks = 1024;     // blocks of one CTA's part of a row
constexpr int kCandidates = 4096;
constexpr int kRankDirect = 512;     // candidates ranked by counting; more are bisected first
// the order key (see argmax_key) of -inf, which is never an alternative
constexpr uint32_t kNegInfOrder = 0x007FFFFFu;

struct Shared {
  Stat part[kWarps];
  Stat cta;
  int ncand, nlist, count;
  float bmax[kMaxBlocks];
  unsigned long long cand[kCandidates];
  unsigned long long list[kMaxTop];
  unsigned long long sorted[kMaxTop];
};
static_assert(sizeof(Shared) <= 48 * 1024, "static shared memory");
static_assert(kMaxCluster * kMaxTop <= kCandidates, "CTA 0 gathers every list in its candidate buffer");

__device__ __forceinline__ uint32_t order32(float x) { return (uint32_t)(argmax_key(x + 0.0f, 0) >> 32); }
__device__ __forceinline__ unsigned long long entry_key(float x, int v) { return argmax_key(x + 0.0f, v); }

// The token of a row and whether the row is scored.
__device__ __forceinline__ bool row_token(const LogprobArgs& p, int row, int* tok) {
  const int b = row / p.R, j = row - b * p.R;
  if (p.n != nullptr) {
    const int n = min(p.n[b], p.R - 1);
    if (j > n) return false;
    *tok = j < n ? p.x[(size_t)b * (p.R - 1) + j] : p.tok[b];
    return true;
  }
  if (p.lens != nullptr && j >= p.lens[b]) return false;
  *tok = p.tokens[row];
  return true;
}

// Adds up `mine` over the CTA (every thread gets the sum).
__device__ __forceinline__ int cta_sum(int mine, int* slot) {
  const int w = __reduce_add_sync(0xffffffffu, mine);
  __syncthreads();
  if (threadIdx.x == 0) *slot = 0;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) atomicAdd(slot, w);
  __syncthreads();
  return *slot;
}

// The K-th largest key: the largest 64-bit value that at least K keys reach,
// bit by bit.  count(t) gives this thread's share of the keys >= t.
template <typename Count>
__device__ unsigned long long kth_largest(int K, int* slot, Count count) {
  unsigned long long t = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const unsigned long long c = t | (1ull << bit);
    if (cta_sum(count(c), slot) >= K) t = c;
  }
  return t;
}

__device__ __forceinline__ void append(Shared& sh, unsigned long long key) {
  const int i = atomicAdd(&sh.nlist, 1);
  if (i < kMaxTop) sh.list[i] = key;
}

__device__ __forceinline__ float order_value(uint32_t o) { return argmax_key_value((unsigned long long)o << 32); }

// Calls f(key) for every entry that reaches the order t0, block by block of
// this warp's.
template <typename T, typename F>
__device__ __forceinline__ void for_candidates(const Row<T>& R, const BlockRange& br, const float* bmax, uint32_t t0,
                                               int warp, int lane, F f) {
  const float least = order_value(t0);
  const int mine = br.begin + warp;   // this warp's blocks: mine, mine + kWarps, ...
  for (int b0 = mine; b0 < br.end; b0 += 32 * kWarps) {
    const int bl = b0 + lane * kWarps;
    unsigned hit = __ballot_sync(0xffffffffu, bl < br.end && !(bmax[bl < br.end ? bl - br.begin : 0] < least));
    for (; hit != 0; hit &= hit - 1) {
      const int b = b0 + (__ffs(hit) - 1) * kWarps;
      uint4 r[kVecPerLane];
      R.load_block(b, lane, r);
      if (lane_max(r, (const T*)nullptr) < least) continue;
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) {
        float v[Elem<T>::VEC];
        Elem<T>::unpack(r[j], v);
        const int e0 = R.first_entry(b * kBlockVecs + j * 32 + lane);
#pragma unroll
        for (int e = 0; e < Elem<T>::VEC; ++e)
          if (v[e] >= least) f(entry_key(v[e], e0 + e));
      }
    }
    __syncwarp();
  }
}

// The CTA's K largest entries, in no order, into sh.list; their count into
// sh.nlist.  tmax: the largest entry this thread has read.
template <typename T>
__device__ void cta_top(Shared& sh, const Row<T>& R, const BlockRange& br, float tmax, int K, int warp, int lane) {
  const int tid = threadIdx.x;
  const uint32_t mine = order32(tmax);
  uint32_t t0 = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = t0 | (1u << bit);
    const int n = __syncthreads_count(mine >= c);
    if (n >= K) t0 = c;
    if (n >= K && n <= K + K / 8) break;   // (any lower bound will do)
  }
  t0 = max(t0, kNegInfOrder + 1);
  if (tid == 0) sh.ncand = sh.nlist = 0;
  __syncthreads();
  for_candidates(R, br, sh.bmax, t0, warp, lane, [&](unsigned long long key) {
    const int i = atomicAdd(&sh.ncand, 1);
    if (i < kCandidates) sh.cand[i] = key;
  });
  __syncthreads();
  const int n = sh.ncand;
  if (n <= kRankDirect) {
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long key = sh.cand[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += sh.cand[j] > key;
      if (rank < K) sh.list[rank] = key;
    }
    if (tid == 0) sh.nlist = min(n, K);
    __syncthreads();
    return;
  }
  // (more than kRankDirect >= K candidates: exactly K keys reach the K-th)
  if (n <= kCandidates) {
    const unsigned long long kth = kth_largest(K, &sh.count, [&](unsigned long long t) {
      int c = 0;
      for (int i = tid; i < n; i += kThreads) c += sh.cand[i] >= t;
      return c;
    });
    for (int i = tid; i < n; i += kThreads)
      if (sh.cand[i] >= kth) append(sh, sh.cand[i]);
  } else {
    const unsigned long long kth = kth_largest(K, &sh.count, [&](unsigned long long t) {
      int c = 0;
      for_candidates(R, br, sh.bmax, max(t0, (uint32_t)(t >> 32)), warp, lane,
                     [&](unsigned long long key) { c += key >= t; });
      return c;
    });
    for_candidates(R, br, sh.bmax, max(t0, (uint32_t)(kth >> 32)), warp, lane, [&](unsigned long long key) {
      if (key >= kth) append(sh, key);
    });
  }
  __syncthreads();
}
static_assert(kRankDirect >= kMaxTop, "the bisection needs at least K candidates");

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobArgs p) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int c = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = (int)(blockIdx.x / c);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int tok = -1;
  if (!row_token(p, row, &tok)) {
    // not scored: zeros, and no alternatives
    if (rank == 0) {
      if (tid == 0) p.logp[row] = p.entropy[row] = p.lse[row] = 0.f;
      if (kTop && tid < p.K) {
        p.top_idx[(size_t)row * p.K + tid] = -1;
        p.top_logp[(size_t)row * p.K + tid] = -INFINITY;
      }
    }
    return;
  }
  const T* rp = static_cast<const T*>(p.logits) + (size_t)row * p.row_stride;
  float xt = 0.f;
  if (rank == 0 && tid == 0 && tok >= 0 && tok < p.V) xt = Elem<T>::to_float(rp[tok]);
  const Row<T> R(rp, p.V);
  const BlockRange br = block_range(R.nvec, rank, c);

  float tmax = -INFINITY;
  stat_row<T, true>(R, br, kLog2e, 1.f, sh.part, &sh.cta, Nothing(), Nothing(), [&](int b, float lm, float bm) {
    if (kTop) {
      tmax = fmaxf(tmax, lm);
      if (lane == 0) sh.bmax[b - br.begin] = bm;
    }
  });
  if (kTop) cta_top<T>(sh, R, br, tmax, p.K, warp, lane);

  cluster.sync();
  if (rank == 0) {
    const Stat v = stat_cluster(cluster, &sh.cta, c, 1.f);
    const bool bad = stat_bad(v);
    const bool none = v.m == -INFINITY;   // every entry is -inf
    const float ls = none ? 0.f : logf(v.s);
    const float nan = __int_as_float(0x7FC00000);
    if (tid == 0) {
      float logp = none ? -INFINITY : (xt - v.m) - ls;
      if (tok == -1) logp = 0.f;
      else if (tok < 0 || tok >= p.V) logp = nan;
      p.logp[row] = bad ? nan : logp;
      p.entropy[row] = bad ? nan : (none ? 0.f : fmaxf(ls + v.t / v.s, 0.f));
      p.lse[row] = bad ? nan : v.m + ls;
    }
    if (kTop) {
      // the c lists as one, then each key's rank
      const unsigned long long* keys = sh.list;
      int n = min(sh.nlist, p.K);
      if (c > 1) {
        for (int i = tid; i < c * p.K; i += kThreads) {
          const int r = i / p.K, j = i - r * p.K;
          const bool has = j < min(*cluster.map_shared_rank(&sh.nlist, r), p.K);
          sh.cand[i] = has ? cluster.map_shared_rank(sh.list, r)[j] : 0ull;
        }
        keys = sh.cand;
        n = c * p.K;
      }
      if (tid < p.K) sh.sorted[tid] = 0ull;
      __syncthreads();
      for (int i = tid; i < n; i += kThreads) {
        const unsigned long long key = keys[i];
        int at = 0;
        for (int j = 0; j < n; ++j) at += keys[j] > key;
        if (key != 0ull && at < p.K) sh.sorted[at] = key;
      }
      __syncthreads();
      if (tid < p.K) {
        const unsigned long long key = sh.sorted[tid];
        const bool has = key != 0ull && !bad;
        p.top_idx[(size_t)row * p.K + tid] = has ? argmax_key_index(key) : -1;
        p.top_logp[(size_t)row * p.K + tid] = bad ? nan : (has ? (argmax_key_value(key) - v.m) - ls : -INFINITY);
      }
    }
  }
  cluster.sync();   // the other CTAs' shared memory is read until here
}

// The gradient, one warp a block at a time: HBM bounds it (one read, one
// write).  An output row whose vectors start where the logits' do is stored by
// vectors, any other entry by entry.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) logprobs_backward_kernel(const LogprobBackwardArgs p) {
  constexpr int VEC = Elem<T>::VEC;
  __shared__ Stat part[kWarps], cta;
  cg::cluster_group cluster = cg::this_cluster();
  const int c = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = (int)(blockIdx.x / c);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Row<T> R(static_cast<const T*>(p.logits) + (size_t)row * p.row_stride, p.V);
  const BlockRange br = block_range(R.nvec, rank, c);
  T* out = static_cast<T*>(p.dlogits) + (size_t)row * p.V;
  const int b0 = row / p.R, j0 = row - b0 * p.R;
  const bool on = p.lens == nullptr || j0 < p.lens[b0];
  const int tok = on ? p.tokens[row] : -1;
  const float nan = __int_as_float(0x7FC00000);
  float gl = on && p.g_logp != nullptr && tok != -1 ? p.g_logp[row] : 0.f;
  if (tok < -1 || tok >= p.V) gl = nan;
  const float gh = on && p.g_entropy != nullptr ? p.g_entropy[row] : 0.f;
  // p_v = exp(x_v - ref - ls)
  float ref = on ? p.lse[row] : -INFINITY, ls = 0.f;
  if (ref != ref) gl = nan;
  if (fabsf(ref) > kLargeLse && ref != -INFINITY) {
    stat_row<T, false>(R, br, kLog2e, 1.f, part, &cta, Nothing(), Nothing(), Nothing());
    cluster.sync();
    const Stat v = stat_cluster(cluster, &cta, c, 1.f);
    cluster.sync();
    if (stat_bad(v)) gl = nan;
    ref = v.m;
    ls = logf(v.s);
  }
  const bool zero = ref == -INFINITY;   // not scored, or no entry above -inf
  const float a = gh != 0.f ? fmaf(gh, p.entropy[row], gl) : gl;
  const bool aligned = ((reinterpret_cast<uintptr_t>(out) - R.shift * sizeof(T)) & 15) == 0;
  for (int b = br.begin + warp; b < br.end; b += kWarps) {
    uint4 r[kVecPerLane];
    if (!zero) R.load_block(b, lane, r);
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) {
      const int i = b * kBlockVecs + j * 32 + lane, e0 = R.first_entry(i);
      alignas(16) T g[VEC];
      if (zero) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[e] = Elem<T>::from_float(0.f);
      } else {
        float x[VEC];
        Elem<T>::unpack(r[j], x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = fmaxf((x[e] - ref) - ls, -1000.f);   // (an entry of -inf: p = 0, gradient 0)
          const float pr = ex2(d * kLog2e);
          float v = -pr * fmaf(gh, d, a);
          if (e0 + e == tok) v += gl;
          g[e] = Elem<T>::from_float(v);
        }
      }
      if (aligned && R.whole(i)) {
        __stcs(reinterpret_cast<uint4*>(out + e0), *reinterpret_cast<const uint4*>(g));
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (e0 + e >= 0 && e0 + e < p.V) out[e0 + e] = g[e];
      }
    }
  }
}

template <typename T>
cudaError_t forward(const LogprobArgs& a, int c, cudaStream_t stream) {
  return a.K > 0 ? launch_rows(logprobs_kernel<T, true>, a.N, c, 0, stream, a)
                 : launch_rows(logprobs_kernel<T, false>, a.N, c, 0, stream, a);
}

template <typename T>
cudaError_t backward(const LogprobBackwardArgs& a, cudaStream_t stream) {
  const int nblk = div_up(div_up(a.V, Elem<T>::VEC) + 1, kBlockVecs);
  int c = 1;
  while (c < 8 && nblk > 2 * kWarps * c) c *= 2;   // two blocks a warp and more
  return launch_rows(logprobs_backward_kernel<T>, a.N, c, 0, stream, a);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int per_block = kBlockVecs * (a.dtype == DSPARK_F32 ? 4 : 8);
  const int nblk = div_up(a.V, per_block) + 1;
  const int c = cluster_for(a.N, nblk, div_up(nblk, kMaxBlocks), sms);
  if (a.dtype == DSPARK_F32) return forward<float>(a, c, stream);
  if (a.dtype == DSPARK_BF16) return forward<__nv_bfloat16>(a, c, stream);
  return forward<__half>(a, c, stream);
}

cudaError_t launch_token_logprobs_backward(const LogprobBackwardArgs& a, cudaStream_t stream) {
  if (a.dtype == DSPARK_F32) return backward<float>(a, stream);
  if (a.dtype == DSPARK_BF16) return backward<__nv_bfloat16>(a, stream);
  return backward<__half>(a, stream);
}

}  // namespace dspark
