// Log probabilities of given tokens with the row's entropy and its K most
// probable entries, and the gradient of the first two.
//
//   lse = log sum_v exp x_v,   logp = x_t - lse,   H = -sum_v p_v log p_v
//   dx_v = g_logp (1[v = t] - p_v) - g_H p_v (log p_v + H)
//
// Forward: one pass over the row (logits_row.cuh); HBM bounds it.  A cluster
// of 1 to 16 CTAs takes a row; their states and candidates meet in CTA 0 through
// distributed shared memory.  The top entries cost the pass one maximum per
// lane and one stored maximum per quarter of a block:
//   1. the K-th largest of the lanes' maxima (256 of each CTA), or a little less
//      by a histogram, is a lower bound of the row's K-th largest entry (K
//      distinct entries are at least that large);
//   2. only the quarters whose maximum reaches it are read again, and their
//      entries that reach it become candidates: hardly more than K in a row of no
//      particular order.  A list of the quarters deals them out evenly to the
//      warps, four at a time, so that few loads' latencies follow each other (64
//      alternatives: 147 us by each warp's own, one ahead; 138 by four of its
//      own, 133 by the list);
//   3. a candidate's rank is the number of larger ones (64-bit keys of value,
//      then lower index, so no two are equal and ties go to the lowest index);
//      more than 512 of them are sorted instead.
// Where the candidates overflow their buffer (thousands of equal or ascending
// entries) each CTA finds its own K largest by bisection over the keys' bits.
//
// Measured (GB300, the kernel alone): 2048 rows of 151936 take 179 us in fp32
// (7.0 TB/s) and 102 us in bf16 (6.1 TB/s), with 20 alternatives 192 and 117 us,
// with 64 205 and 131 us (about 100 instructions a candidate and 8000 a row of
// the 40000 of its sums, in phases that no load overlaps); one row takes 5 us, with 20 alternatives 8.5, with 128 10.5 us (latency: two cluster
// barriers, the histogram's four, one read of L2).  The gradients of those rows
// take 366 us in fp32 (6.8 TB/s) and 205 us in bf16 (6.1 TB/s).
#include <float.h>

#include "logits_row.cuh"

namespace dspark {
namespace {

using namespace lrow;

constexpr int kMaxBlocks = 512;      // blocks of one CTA's part of a row
constexpr int kCandidates = 4096;
constexpr int kHits = 4;             // quarters that a warp reads again at a time (2: 139 us, 4: 133, 6: 136, 8: 138)
constexpr int kRankDirect = 512;     // candidates ranked by counting; more are sorted
struct Shared {
  Stat part[kWarps];
  Stat cta;
  int count[2][kWarps];
  int ncand, nhits;
  float lane_max[kThreads];                   // each lane's largest entry
  float2 range[kWarps];
  int bins[256];
  int cut;
  float4 quarter[kMaxBlocks];                 // maxima of each block's quarters
  unsigned short hits[4 * kMaxBlocks];        // quarters that are read again
  unsigned long long cand[kCandidates];       // (CTA 0's)
  unsigned long long sorted[kMaxTop];
};
static_assert(sizeof(Shared) <= 48 * 1024, "static shared memory");
static_assert(kMaxCluster * kMaxTop <= kCandidates, "the lists of all CTAs");

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

// Places behind *n, counted on, for the lanes that want one.
__device__ __forceinline__ int warp_slots(int* n, bool want) {
  const int lane = threadIdx.x & 31;
  const unsigned b = __ballot_sync(0xffffffffu, want);
  int at = 0;
  if (lane == 0 && b != 0) at = atomicAdd(n, __popc(b));
  return __shfl_sync(0xffffffffu, at, 0) + __popc(b & ((1u << lane) - 1u));
}

// Adds up `mine` over the CTA (every thread gets the sum) with one barrier;
// calls alternate `which`.
__device__ __forceinline__ int cta_sum(Shared& sh, int which, int mine) {
  const int w = __reduce_add_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0) sh.count[which][threadIdx.x >> 5] = w;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) s += sh.count[which][i];
  return s;
}

// The quarters of this CTA's blocks whose maximum reaches `least`, into sh.hits
// (in any order; behind a barrier).
__device__ __forceinline__ void find_quarters(Shared& sh, const BlockRange& br, float least) {
  const int lane = threadIdx.x & 31, n = 4 * (br.end - br.begin);
  const float* q = reinterpret_cast<const float*>(sh.quarter);
  for (int i0 = threadIdx.x - lane; i0 < n; i0 += kThreads) {
    const bool hit = i0 + lane < n && !(q[i0 + lane] < least);
    const int at = warp_slots(&sh.nhits, hit);
    if (hit) sh.hits[at] = (unsigned short)(i0 + lane);
  }
  __syncthreads();
}

// Calls f(has, key), with the whole warp, until every entry of this warp's share
// of the quarters that reaches `least` has been a lane's key with has.
template <typename T, typename F>
__device__ __forceinline__ void for_candidates(const Shared& sh, const Row<T>& R, const BlockRange& br, float least, F f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = sh.nhits;
  for (int h = warp; h < n; h += kHits * kWarps) {
    // (their loads are under way together)
    uint4 r[kHits];
    int i[kHits];
#pragma unroll
    for (int u = 0; u < kHits; ++u) {
      i[u] = 0;
      r[u] = make_uint4(Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf);
      if (h + u * kWarps < n) {
        i[u] = br.begin * kBlockVecs + sh.hits[h + u * kWarps] * 32 + lane;
        r[u] = R.load(i[u], NoPolicy());
      }
    }
    unsigned mine = 0;   // those of this lane's vectors that reach `least`
#pragma unroll
    for (int u = 0; u < kHits; ++u) mine |= (!(vec_max(r[u], (const T*)nullptr) < least) ? 1u : 0u) << u;
    while (__any_sync(0xffffffffu, mine != 0)) {
      // one vector of each lane, then one entry of each lane at a time
      uint4 q = r[0];
      int at = i[0];
#pragma unroll
      for (int u = 1; u < kHits; ++u)
        if (!(mine & ((1u << u) - 1u))) {
          q = r[u];
          at = i[u];
        }
      unsigned es = 0;
      float v[Elem<T>::VEC];
      Elem<T>::unpack(q, v);
#pragma unroll
      for (int e = 0; e < Elem<T>::VEC; ++e) es |= (mine != 0 && v[e] >= least ? 1u : 0u) << e;
      mine &= mine - 1;
      while (__any_sync(0xffffffffu, es != 0)) {
        const int e = max(__ffs(es) - 1, 0);
        f(es != 0, entry_key(Elem<T>::entry(q, e), R.first_entry(at) + e));
        es &= es - 1;
      }
    }
  }
}

// A lower bound of the row's K-th largest entry: about the K-th largest of the
// cluster's lane maxima.  They are counted in 256 bins of equal width between
// the smallest and the largest; the bound is the smallest one in the bins down
// to that of the K-th.  Fewer than K maxima above -inf: the lowest number.
__device__ __forceinline__ float lower_bound(Shared& sh, cg::cluster_group& cluster, int c, int K) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  static_assert(kThreads == 256, "a bin for every thread");
  float v[kMaxCluster];
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) {
    v[r] = -INFINITY;
    if (r < c) v[r] = c == 1 ? sh.lane_max[tid] : cluster.map_shared_rank(sh.lane_max, r)[tid];
    if (v[r] > -INFINITY) lo = fminf(lo, v[r]);
    hi = fmaxf(hi, v[r]);
  }
  sh.bins[tid] = 0;
  asm volatile("redux.sync.min.f32 %0, %0, 0xffffffff;" : "+f"(lo));
  asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(hi));
  if (lane == 0) sh.range[warp] = make_float2(lo, hi);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    lo = fminf(lo, sh.range[w].x);
    hi = fmaxf(hi, sh.range[w].y);
  }
  const float scale = 255.f / (hi - lo);   // (0 * inf below where they are equal: bin 0)
  int bin[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) {
    if (r >= c) break;
    bin[r] = v[r] > -INFINITY ? min(max((int)((v[r] - lo) * scale), 0), 255) : -1;
    if (bin[r] >= 0) atomicAdd(&sh.bins[bin[r]], 1);
  }
  __syncthreads();
  if (warp == 0) {
    // lane l: bins 255 - 8 l and the seven below; their sum and that of all above
    int n[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += n[i] = sh.bins[255 - 8 * lane - i];
    int upto = sum;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += o;
    }
    int above = upto - sum;
    if (above < K && upto >= K) {
      int i = 0;
      while (above + n[i] < K) above += n[i++];
      sh.cut = 255 - 8 * lane - i;
    }
    if (lane == 31 && upto < K) sh.cut = -1;
  }
  __syncthreads();
  const int cut = sh.cut;
  float least = INFINITY;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) {
    if (r >= c) break;
    if (bin[r] >= cut && bin[r] >= 0) least = fminf(least, v[r]);
  }
  asm volatile("redux.sync.min.f32 %0, %0, 0xffffffff;" : "+f"(least));
  if (lane == 0) sh.range[warp].x = least;   // (everyone has read the range)
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) least = fminf(least, sh.range[w].x);
  return cut < 0 ? -FLT_MAX : least;
}

// This CTA's K largest entries into to[0 .. K - 1], in no order, zeros behind
// them; for rows whose candidates overflow.  The K-th largest key is the largest
// 64-bit value that at least K keys reach, bit by bit.
template <typename T>
__device__ __noinline__ void top_by_bisection(Shared& sh, const Row<T>& R, const BlockRange& br, float least, int K,
                                              unsigned long long* to) {
  unsigned long long kth = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const unsigned long long t = kth | (1ull << bit);
    int mine = 0;
    for_candidates(sh, R, br, least, [&](bool has, unsigned long long key) { mine += has && key >= t; });
    if (cta_sum(sh, bit & 1, mine) >= K) kth = t;
  }
  int* n = sh.count[0];
  __syncthreads();
  if (threadIdx.x == 0) *n = 0;
  for (int i = threadIdx.x; i < K; i += kThreads) to[i] = 0ull;
  __syncthreads();
  for_candidates(sh, R, br, least, [&](bool has, unsigned long long key) {
    if (!has || key < kth) return;
    const int i = atomicAdd(n, 1);
    if (i < K) to[i] = key;
  });
}

// The K largest of sh.cand[0 .. n - 1] into sh.sorted, largest first, zeros
// behind them.
__device__ __forceinline__ void rank_candidates(Shared& sh, int n, int K) {
  const int tid = threadIdx.x;
  if (n <= kRankDirect) {
    if (tid < K) sh.sorted[tid] = 0ull;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long key = sh.cand[i];
      int at = 0;
      for (int j = 0; j < n; ++j) at += sh.cand[j] > key;
      if (key != 0ull && at < K) sh.sorted[at] = key;
    }
    __syncthreads();
    return;
  }
  // a bitonic network over the next power of two
  int m = 2 * kRankDirect;
  while (m < n) m *= 2;
  for (int i = n + tid; i < m; i += kThreads) sh.cand[i] = 0ull;
  for (int k = 2; k <= m; k *= 2) {
    for (int j = k / 2; j > 0; j /= 2) {
      __syncthreads();
      for (int i = tid; i < m / 2; i += kThreads) {
        const int lo = 2 * j * (i / j) + i % j, hi = lo + j;
        const unsigned long long a = sh.cand[lo], b = sh.cand[hi];
        if ((a < b) == ((lo & k) == 0)) {
          sh.cand[lo] = b;
          sh.cand[hi] = a;
        }
      }
    }
  }
  __syncthreads();
  if (tid < K) sh.sorted[tid] = sh.cand[tid];
  __syncthreads();
}
static_assert(kCandidates >= 2 * kRankDirect && (kCandidates & (kCandidates - 1)) == 0 && kRankDirect >= kMaxTop,
              "the sorted lengths are powers of two up to the buffer's");

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logprobs_kernel(const LogprobArgs p, int ahead) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int c = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = (int)(blockIdx.x / c);
  const int tid = threadIdx.x, lane = tid & 31;
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
  if (kTop && tid == 0) sh.ncand = sh.nhits = 0;
  auto seen = [&](int b, float lm, float4 q) {
    tmax = fmaxf(tmax, lm);
    if (lane == 0) sh.quarter[b - br.begin] = q;
  };
  // (the row that takes this CTA's place)
  auto next = [&]() {
    if (tid == 0 && row + ahead < p.N && ahead > 0) prefetch_row(rp + (size_t)ahead * p.row_stride, p.V, 4);
  };
  if constexpr (kTop)   // (some of the row is read again, so L2 is not asked to drop it)
    stat_row<T, true, true>(R, br, kLog2e, 1.f, NoPolicy(), sh.part, &sh.cta, Nothing(), Nothing(), seen, next);
  else
    stat_row<T, true, false>(R, br, kLog2e, 1.f, tc::policy_evict_first(), sh.part, &sh.cta, Nothing(), Nothing(), Nothing(), next);
  if (kTop) sh.lane_max[tid] = tmax;
  cluster_meet(c);
  const Stat v = stat_cluster(cluster, &sh.cta, c, 1.f);
  if (kTop) {
    const float least = lower_bound(sh, cluster, c, p.K);
    int* ncand = c == 1 ? &sh.ncand : cluster.map_shared_rank(&sh.ncand, 0);
    unsigned long long* cand = c == 1 ? sh.cand : cluster.map_shared_rank(sh.cand, 0);
    find_quarters(sh, br, least);
    for_candidates(sh, R, br, least, [&](bool has, unsigned long long key) {
      const int i = warp_slots(ncand, has);
      if (has && i < kCandidates) cand[i] = key;
    });
    cluster_meet(c);
    int n = *ncand;
    if (n > kCandidates) {
      cluster_meet(c);   // (every CTA has read the count)
      top_by_bisection(sh, R, br, least, p.K, cand + rank * p.K);
      cluster_meet(c);
      n = c * p.K;
    }
    if (rank == 0) rank_candidates(sh, n, p.K);
  }
  if (rank == 0) {
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
    if (kTop && tid < p.K) {
      const unsigned long long key = sh.sorted[tid];
      const bool has = key != 0ull && !bad;
      p.top_idx[(size_t)row * p.K + tid] = has ? argmax_key_index(key) : -1;
      p.top_logp[(size_t)row * p.K + tid] = bad ? nan : (has ? (argmax_key_value(key) - v.m) - ls : -INFINITY);
    }
  }
  if (c > 1) cluster_meet(c);   // a CTA's shared memory is read until here
}

// The gradient, one warp a block at a time: HBM bounds it (one read, one
// write).  An output row whose vectors start where the logits' do is stored by
// vectors, any other entry by entry.
template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logprobs_backward_kernel(const LogprobBackwardArgs p) {
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
  const bool bad_tok = tok < -1 || tok >= p.V;
  if (bad_tok) gl = nan;
  const float gh = on && p.g_entropy != nullptr ? p.g_entropy[row] : 0.f;
  // p_v = exp(x_v - ref - ls)
  float ref = on ? p.lse[row] : -INFINITY, ls = 0.f;
  if (ref != ref) gl = nan;
  if (lse_is_large(ref)) {
    stat_row<T, false, false>(R, br, kLog2e, 1.f, NoPolicy(), part, &cta, Nothing(), Nothing(), Nothing(), Nothing());
    cluster_meet(c);
    const Stat v = stat_cluster(cluster, &cta, c, 1.f);
    cluster_meet(c);
    if (stat_bad(v)) gl = nan;
    ref = v.m;
    ls = logf(v.s);
  }
  const bool zero = ref == -INFINITY && !bad_tok;   // not scored, or no entry above -inf
  const float a = gh != 0.f ? fmaf(gh, p.entropy[row], gl) : gl;
  const bool aligned = ((reinterpret_cast<uintptr_t>(out) - R.shift * sizeof(T)) & 15) == 0;
  // the token's own entry is stored last, over what the loop leaves there; its
  // logit is read first, for out may be the logits
  const int place0 = br.begin * kBlockVecs * VEC - R.shift;
  const bool last = threadIdx.x == 0 && !zero && tok >= place0 && tok < place0 + (br.end - br.begin) * kBlockVecs * VEC;
  const float xt = last && tok < p.V ? Elem<T>::to_float(R.row[max(tok, 0)]) : 0.f;
  __syncthreads();
  auto store = [&](int b, int j, bool inside, const T(&g)[VEC]) {
    const int i = b * kBlockVecs + j * 32 + lane, e0 = R.first_entry(i);
    if (inside || (aligned && R.whole(i))) {
      __stcs(reinterpret_cast<uint4*>(out + e0), *reinterpret_cast<const uint4*>(g));
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e0 + e >= 0 && e0 + e < p.V) out[e0 + e] = g[e];
    }
  };
  if (zero) {
    alignas(16) T none[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e += 2) put2(none + e, 0.f, 0.f);
    for (int b = br.begin + warp; b < br.end; b += kWarps) {
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) store(b, j, aligned && R.inside(b), none);
    }
    return;
  }
  // with d = x - ref and f = exp(-ls): -p (a + g_H (d - ls)) = exp(d) (-f (a - g_H ls) - f g_H d)
  const float f = expf(-ls), c0 = -f * fmaf(-gh, ls, a), c1 = -f * gh;
  const uint64_t ref2 = pack2(-ref, -ref), scale2 = pack2(kLog2e, kLog2e), c02 = pack2(c0, c0), c12 = pack2(c1, c1);
  auto gradient = [&](int b, const uint4(&r)[kVecPerLane]) {
    const bool inside = aligned && R.inside(b);
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) {
      alignas(16) T g[VEC];
      float x[VEC];
      Elem<T>::unpack(r[j], x);
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        float u, v;
        unpack2(add2(pack2(x[e], x[e + 1]), ref2), u, v);
        const uint64_t d = pack2(fmaxf(u, -1000.f), fmaxf(v, -1000.f));   // (an entry of -inf: p = 0, gradient 0)
        unpack2(mul2(d, scale2), u, v);
        unpack2(mul2(pack2(ex2(u), ex2(v)), fma2(c12, d, c02)), u, v);
        put2(g + e, u, v);
      }
      store(b, j, inside, g);
    }
  };
  for (int b = br.begin + warp; b < br.end; b += kWarps) {
    uint4 r[kVecPerLane];
    R.load_block(b, lane, r, NoPolicy());
    gradient(b, r);
  }
  __syncthreads();
  if (last && tok >= 0 && tok < p.V) {
    const float d = fmaxf(xt - ref, -1000.f);
    out[tok] = Elem<T>::from_float(fmaf(ex2(d * kLog2e), fmaf(c1, d, c0), gl));
  }
}

template <typename T>
cudaError_t forward(const LogprobArgs& a, int c, int ahead, cudaStream_t stream) {
  return a.K > 0 ? launch_rows(logprobs_kernel<T, true>, a.N, c, 0, stream, a, ahead)
                 : launch_rows(logprobs_kernel<T, false>, a.N, c, 0, stream, a, ahead);
}

template <typename T>
cudaError_t backward(const LogprobBackwardArgs& a, cudaStream_t stream) {
  const int nblk = div_up(div_up(a.V, Elem<T>::VEC) + 1, kBlockVecs);
  int c = 1;
  while (c < 8 && nblk > 2 * kWarps * c) c *= 2;
  // (two blocks a warp and more: 640 rows of 151936 take 145 us by one CTA each,
  // 124, 119 and 115 by 2, 4 and 8)
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
  // the CTAs that run at a time, where they are rows that all count
  const int ahead = c == 1 && a.lens == nullptr && a.n == nullptr ? kCtasPerSm * sms : 0;
  if (a.dtype == DSPARK_F32) return forward<float>(a, c, ahead, stream);
  if (a.dtype == DSPARK_BF16) return forward<__nv_bfloat16>(a, c, ahead, stream);
  return forward<__half>(a, c, ahead, stream);
}

cudaError_t launch_token_logprobs_backward(const LogprobBackwardArgs& a, cudaStream_t stream) {
  if (a.dtype == DSPARK_F32) return backward<float>(a, stream);
  if (a.dtype == DSPARK_BF16) return backward<__nv_bfloat16>(a, stream);
  return backward<__half>(a, stream);
}

}  // namespace dspark
