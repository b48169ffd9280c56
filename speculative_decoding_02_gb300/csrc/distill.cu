// Distillation of a student's logits S from a teacher's K kept logits, forward
// and backward.  With z = S / tau, q = softmax(z) and the teacher's entries
// (i_k, t_k), t'_k = t_k / tau:
//
//   without the teacher's lse:  p = softmax(t') over the kept entries,
//     L = sum_k p_k (log p_k - log q_{i_k}),      dL/dS_v = (q_v - p(v)) / tau
//   with it:  p_k = exp(t'_k - lse_t), the rest p_r = 1 - sum_k p_k is one
//     bucket, matched with the student's mass q_r outside the kept entries:
//     L = (the sum above) + p_r (log p_r - log q_r),
//     dL/dS_v = (q_v - p(v)) / tau on a kept entry,
//               q_v (1 - p_r / q_r) / tau = r_v (q_r - p_r) / tau elsewhere
//   where p(v) is the sum of p_k over the k with i_k = v and r = q / q_r.
//
// q_r is not taken as 1 - sum q (which loses it when the kept entries hold
// almost everything): the kept entries, which a bitmap of the segment in shared
// memory marks, leave the row's sum, and their exponentials are added afterwards.
//
// Two kernels, each bound by HBM.  The first sums a row by a cluster of 1 to 16
// CTAs (logits_row.cuh), whose CTA 0 finishes the row: its loss and, into the
// workspace, the coefficients of its gradient and the gradients of its kept
// entries.  The second streams the gradient; it starts while the first one
// ends (programmatic dependent launch), with its first loads under way.
#include <algorithm>

#include "logits_row.cuh"

namespace dspark {
namespace {

using namespace lrow;

constexpr int kMarkedPlaces = 262144;   // of a CTA's part of a row: a bitmap of 32 KB

// What the first kernel leaves for the second.
struct WsView {
  float4* coef;      // [N] ref, cw, whether the row has a gradient
  int* kept_at;      // [N][K] entry whose gradient is kept_g (-1: none)
  float* kept_g;
  size_t total;
};
__host__ __device__ inline WsView ws_view(void* ws, int N, int K) {
  WsView v;
  v.coef = ws_ptr<float4>(ws, 0);
  size_t off = align256(16ull * N);
  v.kept_at = ws_ptr<int>(ws, off);       off = align256(off + 4ull * N * K);
  v.kept_g = ws_ptr<float>(ws, off);      off = align256(off + 4ull * N * K);
  v.total = off;
  return v;
}

__device__ __forceinline__ bool scored(const DistillArgs& p, int row) {
  if (p.lens == nullptr) return true;
  const int g = row / p.R;
  return row - g * p.R < p.lens[g];
}

struct Shared {
  Stat part[kWarps];
  Stat cta;               // of this CTA's part, outside the kept entries with a tail
  int idx[kMaxTop];       // the row's kept entries, -1: absent
  float p[kMaxTop];       // the teacher's probability
  float red[3][kWarps];
};

// Sums over the CTA (every thread gets them): slot `which` of sh.red.
__device__ __forceinline__ float cta_add(Shared& sh, int which, float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) sh.red[which][threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += sh.red[which][w];
  return s;
}
__device__ __forceinline__ float cta_max(Shared& sh, int which, float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, off));
  if ((threadIdx.x & 31) == 0) sh.red[which][threadIdx.x >> 5] = v;
  __syncthreads();
  float s = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s = max_nan(s, sh.red[which][w]);
  return s;
}

// A row's loss and statistics and its gradient's coefficients, by one whole
// CTA, from the row's state (`pass`; outside the kept entries with a tail) or
// from the statistics of the forward call.
template <typename T, bool kTail>
__device__ void finish_row(Shared& sh, const DistillArgs& p, int row, bool pass, const Stat rest, float lse_in,
                           float lse_rest_in) {
  const int tid = threadIdx.x, lane = tid & 31;
  const T* rp = static_cast<const T*>(p.logits) + (size_t)row * p.row_stride;
  const float nan = __int_as_float(0x7FC00000);
  // entry k of the teacher, a thread each
  int idx = -1;
  float val = -INFINITY, z = 0.f;
  bool bad = false;
  if (tid < p.K) {
    idx = p.top_idx[(size_t)row * p.K + tid];
    val = p.top_val[(size_t)row * p.K + tid];
    bad = idx < -1 || idx >= p.V;
    if (idx < 0 || bad) {
      idx = -1;
      val = -INFINITY;
    } else {
      z = Elem<T>::to_float(rp[idx]);
    }
  }
  if (tid < kMaxTop) sh.idx[tid] = idx;
  const bool any = __syncthreads_or(val != -INFINITY);
  bad = __syncthreads_or(bad);

  // log p_k and p_k (products and differences rounded once)
  float t = -INFINITY, base = 0.f;
  if (kTail) {
    if (val != -INFINITY) t = fmaf(val, p.inv_tau, -p.teacher_lse[row]);
  } else {
    const float m = cta_max(sh, 0, val);
    if (val != -INFINITY) t = (val - m) * p.inv_tau;
    base = logf(cta_add(sh, 1, t == -INFINITY ? 0.f : expf(t)));
  }
  const float logp = t == -INFINITY ? -INFINITY : t - base;
  const float pk = t == -INFINITY ? 0.f : expf(logp);
  if (tid < kMaxTop) sh.p[tid] = pk;
  const float total = cta_add(sh, 2, pk);
  const float p_rest = kTail ? (total > 1.f ? 0.f : 1.f - total) : 0.f;   // (a NaN total stays one)
  // p(v): equal indices add up in the first of them
  float pv = 0.f;
  bool first = idx >= 0;
  if (first) {
    for (int k = 0; k < p.K; ++k) {
      if (sh.idx[k] != idx) continue;
      if (k < tid) {
        first = false;
        break;
      }
      pv += sh.p[k];
    }
  }

  // the student's side
  bool none = false;
  float ref = 0.f, coef = 0.f, q_ref = 0.f, q_scale = 0.f, ls = 0.f, lse = 0.f, lse_rest = 0.f;
  if (pass) {
    Stat all = rest;
    if (kTail) {
      const float m = cta_max(sh, 0, first ? z : -INFINITY);
      const float s = cta_add(sh, 1, first && m != -INFINITY ? expf((z - m) * p.inv_tau) : 0.f);
      all = stat_reduce<2>(lane & 1 ? Stat{m, s, 0.f} : rest, p.inv_tau);
    }
    none = all.m == -INFINITY;
    ls = none ? 0.f : logf(all.s);
    lse = fmaf(all.m, p.inv_tau, ls);
    lse_rest = rest.m == -INFINITY ? -INFINITY : fmaf(rest.m, p.inv_tau, logf(rest.s));
    q_ref = all.m;
    q_scale = 1.f / all.s;
    ref = all.m;
    coef = q_scale;
    if (kTail) {
      ref = rest.m == -INFINITY ? 0.f : rest.m;
      const float q_rest = rest.m == -INFINITY ? 0.f : expf((rest.m - all.m) * p.inv_tau) * rest.s / all.s;
      coef = rest.m == -INFINITY ? 0.f : (q_rest - p_rest) / rest.s;
    }
    if (any && stat_bad(all)) {
      bad = true;
      lse = lse_rest = nan;
    }
  } else {
    none = lse_in == -INFINITY;
    // the references in units of the logits, with what their rounding lost
    q_ref = none ? 0.f : lse_in * p.tau;
    q_scale = expf(-fmaf(lse_in, p.tau, -q_ref) * p.inv_tau);
    ref = q_ref;
    coef = q_scale;
    if (kTail) {
      ref = lse_rest_in == -INFINITY ? 0.f : lse_rest_in * p.tau;
      coef = lse_rest_in == -INFINITY
                 ? 0.f
                 : (expf(lse_rest_in - lse_in) - p_rest) * expf(-fmaf(lse_rest_in, p.tau, -ref) * p.inv_tau);
    }
  }
  const bool on = (any || bad) && !none;
  if (p.stats_in == nullptr) {
    float L = !(pk == 0.f) ? pk * (logp - ((z - q_ref) * p.inv_tau - ls)) : 0.f;
    L = cta_add(sh, 0, L);
    if (kTail && !(p_rest == 0.f)) L += p_rest * (logf(p_rest) - (lse_rest - lse));
    if (tid == 0) {
      const bool counts = any || bad;
      p.loss[row] = bad ? nan : (on ? L : 0.f);
      p.stats[2 * (size_t)row] = bad ? nan : (counts ? lse : 0.f);
      p.stats[2 * (size_t)row + 1] = bad ? nan : (counts ? (kTail ? lse_rest : lse) : 0.f);
    }
  }
  if (bad) coef = q_scale = nan;
  if (p.dlogits != nullptr) {
    const WsView ws = ws_view(p.ws, p.N, p.K);
    const float w = (p.weight != nullptr ? p.weight[row] : 1.f) * p.inv_tau;
    if (tid == 0) ws.coef[row] = make_float4(ref, coef * w, on ? 1.f : 0.f, 0.f);
    if (tid < p.K) {
      ws.kept_at[(size_t)row * p.K + tid] = on && first ? idx : -1;
      ws.kept_g[(size_t)row * p.K + tid] = w * (q_scale * ex2((z - q_ref) * p.inv_tau * kLog2e) - pv);
    }
  }
}

// The first kernel.  kTail: the teacher's lse is given.  With p.stats_in (the
// backward pass alone) only rows whose lse is too large to be used are summed.
template <typename T, bool kTail>
__global__ void __launch_bounds__(kThreads, 4) distill_sum_kernel(const DistillArgs p) {
  constexpr int VEC = Elem<T>::VEC;
  constexpr int kBlockPlaces = kBlockVecs * VEC;
  __shared__ Shared sh;
  extern __shared__ uint32_t marked[];   // kTail: one bit per place of the part, then a byte per block
  cg::cluster_group cluster = cg::this_cluster();
  const int c = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = (int)(blockIdx.x / c);
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_trigger();
  const bool backward = p.stats_in != nullptr;
  if (!scored(p, row)) {
    if (rank == 0 && tid == 0) {
      if (!backward) p.loss[row] = p.stats[2 * (size_t)row] = p.stats[2 * (size_t)row + 1] = 0.f;
      if (p.dlogits != nullptr) ws_view(p.ws, p.N, p.K).coef[row] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  float lse_in = 0.f, lse_rest_in = 0.f;
  if (backward) {
    lse_in = p.stats_in[2 * (size_t)row];
    lse_rest_in = p.stats_in[2 * (size_t)row + 1];
  }
  const bool pass = !backward || (lse_in != -INFINITY && fabsf(lse_in) > kLargeLse);
  if (!pass) {
    if (rank == 0) finish_row<T, kTail>(sh, p, row, false, stat_empty(), lse_in, lse_rest_in);
    return;
  }
  const Row<T> R(static_cast<const T*>(p.logits) + (size_t)row * p.row_stride, p.V);
  const BlockRange br = block_range(R.nvec, rank, c);
  const int place0 = br.begin * kBlockPlaces - R.shift;   // entry at the part's first place
  const int nblk = br.end - br.begin, words = nblk * (kBlockPlaces / 32);
  unsigned char* block_marked = reinterpret_cast<unsigned char*>(marked + words);
  auto mark = [&]() {
    if constexpr (kTail) {
      const int i = tid < p.K ? p.top_idx[(size_t)row * p.K + tid] : -1;
      for (int k = tid; k < words; k += kThreads) marked[k] = 0;
      for (int k = tid; k < nblk; k += kThreads) block_marked[k] = 0;
      __syncthreads();
      const int place = i - place0;
      if (i >= 0 && i < p.V && place >= 0 && place < nblk * kBlockPlaces) {
        atomicOr(&marked[place >> 5], 1u << (place & 31));
        block_marked[place / kBlockPlaces] = 1;
      }
      __syncthreads();
    }
  };
  auto leave_out = [&](int b, uint4(&cur)[kVecPerLane]) {
    if constexpr (kTail) {
      if (!block_marked[b - br.begin]) return;
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) {
        const int place = ((b - br.begin) * kBlockVecs + j * 32 + lane) * VEC;
        const uint32_t m = (marked[place >> 5] >> (place & 31)) & ((1u << VEC) - 1u);
        if (m == 0) continue;
        T* e = reinterpret_cast<T*>(&cur[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (m >> i & 1u) e[i] = Elem<T>::from_float(-INFINITY);
      }
    }
  };
  stat_row<T, false>(R, br, p.inv_tau * kLog2e, p.inv_tau, sh.part, &sh.cta, mark, leave_out, Nothing());
  cluster.sync();
  Stat v = stat_empty();
  if (rank == 0) v = stat_cluster(cluster, &sh.cta, c, p.inv_tau);
  cluster.sync();   // the other CTAs' shared memory is read until here
  if (rank == 0) finish_row<T, kTail>(sh, p, row, true, v, 0.f, 0.f);
}

// The second kernel: c CTAs a row, one warp a block at a time.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads, 4) distill_gradient_kernel(const DistillArgs p, int c) {
  constexpr int VEC = Elem<T>::VEC;
  constexpr int kBlockPlaces = kBlockVecs * VEC;
  const int row = (int)(blockIdx.x / c), rank = (int)(blockIdx.x % c);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const WsView ws = ws_view(p.ws, p.N, p.K);
  const Row<T> R(static_cast<const T*>(p.logits) + (size_t)row * p.row_stride, p.V);
  const BlockRange br = block_range(R.nvec, rank, c);
  const int lo = max(br.begin * kBlockPlaces - R.shift, 0), hi = min(br.end * kBlockPlaces - R.shift, p.V);
  const float scale = p.inv_tau * kLog2e;
  const bool on = scored(p, row);
  uint4 cur[kVecPerLane], nxt[kVecPerLane];
  int b = br.begin + warp;
  if (on && b < br.end) R.load_block(b, lane, cur);
  pdl_wait();
  const float4 k = __ldcg(ws.coef + row);
  const bool live = k.z != 0.f;
  const float ref = k.x, cw = k.y;
  int kept = -1;
  float kept_g = 0.f;
  if (live && tid < p.K) {
    kept = __ldcg(ws.kept_at + (size_t)row * p.K + tid);
    kept_g = __ldcg(ws.kept_g + (size_t)row * p.K + tid);
  }
  G* out = static_cast<G*>(p.dlogits) + (size_t)row * p.V;
  // an output row whose vectors start where the logits' do is stored by vectors
  const bool aligned = ((reinterpret_cast<uintptr_t>(out) - R.shift * sizeof(G)) & (VEC * sizeof(G) - 1)) == 0;
  for (; b < br.end; b += kWarps) {
    if (live && b + kWarps < br.end) R.load_block(b + kWarps, lane, nxt);
    const bool inside = aligned && R.inside(b);
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) {
      const int i = b * kBlockVecs + j * 32 + lane, e0 = R.first_entry(i);
      alignas(16) G g[VEC];
      float x[VEC];
      if (live) Elem<T>::unpack(cur[j], x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[e] = Elem<G>::from_float(live ? ex2((x[e] - ref) * scale) * cw : 0.f);
      if (inside || (aligned && R.whole(i))) {
        if constexpr (sizeof(G) * VEC == 16) __stcs(reinterpret_cast<uint4*>(out + e0), *reinterpret_cast<const uint4*>(g));
        else __stcs(reinterpret_cast<uint2*>(out + e0), *reinterpret_cast<const uint2*>(g));
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (e0 + e >= 0 && e0 + e < p.V) out[e0 + e] = g[e];
      }
    }
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) cur[j] = nxt[j];
  }
  if (live) {
    __syncthreads();   // the kept entries' gradients replace what the loop stored there
    if (kept >= lo && kept < hi) out[kept] = Elem<G>::from_float(kept_g);
  }
}

template <typename T>
cudaError_t launch_sum(const DistillArgs& a, int sms, cudaStream_t stream) {
  constexpr int kBlockPlaces = kBlockVecs * Elem<T>::VEC;
  const int nblk = div_up(a.V, kBlockPlaces) + 1;
  // (a backward pass seldom sums a row)
  const int least = div_up(nblk, kMarkedPlaces / kBlockPlaces);
  int c = 1;
  if (a.stats_in == nullptr) c = cluster_for(a.N, nblk, least, sms);
  else while (c < least) c *= 2;
  const bool tail = a.teacher_lse != nullptr;
  const int smem = tail ? div_up(nblk, c) * (kBlockPlaces / 8 + 1) : 0;
  auto kern = tail ? distill_sum_kernel<T, true> : distill_sum_kernel<T, false>;
  return launch_rows(kern, a.N, c, smem, stream, a);
}

template <typename T, typename G>
cudaError_t launch(const DistillArgs& a, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if ((e = launch_sum<T>(a, sms, stream)) != cudaSuccess || a.dlogits == nullptr) return e;
  const int nblk = div_up(a.V, kBlockVecs * Elem<T>::VEC) + 1;
  const int c = div_up(nblk, 8 * kWarps);   // at most eight blocks a warp
  if ((long long)a.N * c > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_pdl(distill_gradient_kernel<T, G>, dim3((unsigned)a.N * c), dim3(kThreads), 0, stream, a, c);
}

}  // namespace

size_t distill_workspace_bytes(int N, int V, int K) {
  (void)V;
  return ws_view(nullptr, N, K).total;
}

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
  if (a.dtype == DSPARK_F32)
    return a.gdtype == DSPARK_BF16 ? launch<float, __nv_bfloat16>(a, stream) : launch<float, float>(a, stream);
  if (a.dtype == DSPARK_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
  return launch<__half, __half>(a, stream);
}

}  // namespace dspark
