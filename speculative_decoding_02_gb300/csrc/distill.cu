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
//               q_v (1 - p_r / q_r) / tau elsewhere
//   where p(v) is the sum of p_k over the k with i_k = v.
//
// q_r is not taken as 1 - sum q (which loses it when the kept entries hold
// almost everything): the pass sums the entries outside the kept ones, which a
// bitmap of the row in shared memory marks and a flag per block makes cheap,
// and adds the kept entries' exponentials afterwards.
//
// A cluster of CTAs takes a row (logits_row.cuh).  The loss needs one pass; its
// gradient a second one over the same row, which then comes from L2 when the
// rows in flight fit there, so that HBM sees one read and one write.  The
// gradient of the kept entries is stored after the others', behind a barrier.
#include <algorithm>

#include "logits_row.cuh"

namespace dspark {
namespace {

using namespace lrow;

struct Shared {
  Stat part[kWarps];
  Stat cta;               // of this CTA's part, outside the kept entries with a tail
  float z[kMaxTop];       // the student's kept logits, unscaled
  float p[kMaxTop];       // the teacher's probability of entry k
  float psum[kMaxTop];    // p(i_k); -1 where entry k is absent or an earlier one has its index
  int idx[kMaxTop];       // -1: absent
  double logp[kMaxTop];   // log p_k
  float p_rest;
  int bad, any;           // an index outside [-1, V); an entry with mass
};

// The teacher's side of one row and the student's logits there, in shared
// memory (each CTA of a cluster for itself).  Entries of the row outside the
// places [lo, hi) are not read from the student.
template <typename T, bool kTail>
__device__ void load_teacher(Shared& sh, const DistillArgs& p, int row, const T* rp, int lo, int hi) {
  const int tid = threadIdx.x;
  if (tid == 0) sh.bad = 0;
  __syncthreads();
  if (tid < kMaxTop) {
    int i = tid < p.K ? p.top_idx[(size_t)row * p.K + tid] : -1;
    if (i < -1 || i >= p.V) {
      sh.bad = 1;
      i = -1;
    }
    sh.idx[tid] = i;
    sh.z[tid] = i >= lo && i < hi ? Elem<T>::to_float(rp[i]) : 0.f;
    sh.logp[tid] = i >= 0 ? (double)p.top_val[(size_t)row * p.K + tid] * (double)p.inv_tau : -INFINITY;
  }
  __syncthreads();
  if (tid < 32) {
    constexpr int PER = kMaxTop / 32;
    double base;
    if (kTail) {
      base = (double)p.teacher_lse[row];
    } else {
      double m = -INFINITY, s = 0.0;
#pragma unroll
      for (int j = 0; j < PER; ++j) m = fmax(m, sh.logp[tid + 32 * j]);
      for (int off = 16; off > 0; off >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, off));
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const double t = sh.logp[tid + 32 * j];
        if (t != -INFINITY) s += (double)expf((float)(t - m));
      }
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      base = m + (double)logf((float)s);
    }
    double total = 0.0;
    bool any = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int k = tid + 32 * j;
      double lp = sh.logp[k];
      float pk = 0.f;
      if (lp != -INFINITY) {   // (-inf: no mass)
        lp -= base;
        pk = expf((float)lp);
        sh.logp[k] = lp;
        any = true;
      }
      sh.p[k] = pk;
      total += (double)pk;
    }
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    any = __any_sync(0xffffffffu, any);
    if (tid == 0) {
      sh.p_rest = kTail ? (total <= 1.0 ? (float)(1.0 - total) : (total > 1.0 ? 0.f : (float)total)) : 0.f;
      sh.any = any;
    }
  }
  __syncthreads();
  if (tid < p.K) {
    const int i = sh.idx[tid];
    float s = i < 0 ? -1.f : 0.f;
    for (int k = 0; i >= 0 && k < p.K; ++k) {
      if (sh.idx[k] != i) continue;
      if (k < tid) {
        s = -1.f;
        break;
      }
      s += sh.p[k];
    }
    sh.psum[tid] = s;
  }
  __syncthreads();
}

// kTail: the teacher's lse is given.  With p.stats_in the backward pass alone.
template <typename T, typename G, bool kTail>
__global__ void __launch_bounds__(kThreads, 2) distill_kernel(const DistillArgs p) {
  constexpr int VEC = Elem<T>::VEC;
  constexpr int kBlockPlaces = kBlockVecs * VEC;
  __shared__ Shared sh;
  extern __shared__ __align__(16) uint32_t bits[];   // kTail: one bit per place of this CTA's part, then a byte per block
  cg::cluster_group cluster = cg::this_cluster();
  const int c = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = (int)(blockIdx.x / c);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool backward = p.stats_in != nullptr;
  const bool grad = p.dlogits != nullptr;
  const T* rp = static_cast<const T*>(p.logits) + (size_t)row * p.row_stride;
  const Row<T> R(rp, p.V);
  const BlockRange br = block_range(R.nvec, rank, c);
  const int lo = max(br.begin * kBlockPlaces - R.shift, 0), hi = min(br.end * kBlockPlaces - R.shift, p.V);
  const int b0 = row / p.R;
  bool on = p.lens == nullptr || row - b0 * p.R < p.lens[b0];
  float lse_in = 0.f, lse_rest_in = 0.f;
  if (backward && on) {
    lse_in = p.stats_in[2 * (size_t)row];
    lse_rest_in = p.stats_in[2 * (size_t)row + 1];
  }
  const bool pass = !backward || (lse_in != -INFINITY && fabsf(lse_in) > kLargeLse);
  if (on) {
    // (a pass over the row reads every kept logit; a backward pass, whose CTAs
    // do not wait for each other and may overwrite the logits, only its own part's)
    load_teacher<T, kTail>(sh, p, row, rp, pass ? 0 : lo, pass ? p.V : hi);
    on = sh.any != 0 || sh.bad != 0;
  }

  // q_v outside the kept entries is coef0 * exp((x - ref) / tau), the gradient
  // coef * that; a kept entry's is q_scale * exp((x - q_ref) / tau) - p(v), times w
  float ref = 0.f, coef = 0.f, q_ref = 0.f, q_scale = 0.f;
  float w = 0.f;
  if (grad && on) w = (p.weight != nullptr ? p.weight[row] : 1.f) * p.inv_tau;
  const float nan = __int_as_float(0x7FC00000);
  const float scale = p.inv_tau * kLog2e;

  if (on && pass) {
    if (kTail) {
      const int nblk = br.end - br.begin;
      const int words = nblk * (kBlockPlaces / 32);
      unsigned char* flag = reinterpret_cast<unsigned char*>(bits + words);
      for (int i = tid; i < words; i += kThreads) bits[i] = 0;
      for (int i = tid; i < nblk; i += kThreads) flag[i] = 0;
      __syncthreads();
      if (tid < p.K && sh.idx[tid] >= lo && sh.idx[tid] < hi) {
        const int place = sh.idx[tid] + R.shift - br.begin * kBlockPlaces;
        atomicOr(&bits[place >> 5], 1u << (place & 31));
        flag[place / kBlockPlaces] = 1;
      }
      __syncthreads();
    }
    const unsigned char* flag = reinterpret_cast<const unsigned char*>(bits + (br.end - br.begin) * (kBlockPlaces / 32));
    stat_row<T, false>(
        R, br, scale, p.inv_tau, sh.part, &sh.cta,
        [&](int b, uint4(&cur)[kVecPerLane]) {
          if constexpr (kTail) {
            if (!flag[b - br.begin]) return;
            // kept entries leave the sum of the rest
#pragma unroll
            for (int j = 0; j < kVecPerLane; ++j) {
              const int place = ((b - br.begin) * kBlockVecs + j * 32 + lane) * VEC;
              const uint32_t m = (bits[place >> 5] >> (place & 31)) & ((1u << VEC) - 1u);
              if (m == 0) continue;
              T* e = reinterpret_cast<T*>(&cur[j]);
#pragma unroll
              for (int i = 0; i < VEC; ++i)
                if (m >> i & 1u) e[i] = Elem<T>::from_float(-INFINITY);
            }
          }
        },
        [](int, float, float) {});
    cluster.sync();
    // every CTA: the states of all parts, then the kept entries' with a tail
    const Stat rest = stat_cluster(cluster, &sh.cta, c, p.inv_tau);
    Stat all = rest;
    if (kTail) {
      Stat kept = stat_empty();
#pragma unroll
      for (int j = 0; j < kMaxTop / 32; ++j) {
        const int k = lane + 32 * j;
        if (k < p.K && sh.psum[k] != -1.f) kept = stat_merge(kept, Stat{sh.z[k], 1.f, 0.f}, p.inv_tau);
      }
      all = stat_merge(stat_reduce<32>(kept, p.inv_tau), rest, p.inv_tau);
    }
    const bool bad = stat_bad(all) || sh.bad != 0;
    const bool none = all.m == -INFINITY;
    const float ls = none ? 0.f : logf(all.s);
    const float lse = fmaf(all.m, p.inv_tau, ls);
    const float lse_rest = rest.m == -INFINITY ? -INFINITY : fmaf(rest.m, p.inv_tau, logf(rest.s));
    // the student's mass outside the kept entries
    const float q_rest = kTail && rest.m != -INFINITY ? expf((rest.m - all.m) * p.inv_tau) * rest.s / all.s : 0.f;
    if (!backward && rank == 0 && warp == 0) {
      float L = 0.f;
#pragma unroll
      for (int j = 0; j < kMaxTop / 32; ++j) {
        const int k = lane + 32 * j;
        if (sh.p[k] > 0.f || sh.p[k] != sh.p[k])
          L += sh.p[k] * (float)(sh.logp[k] - (((double)sh.z[k] - all.m) * p.inv_tau - ls));
      }
      for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
      if (kTail && !(sh.p_rest == 0.f)) L += sh.p_rest * (logf(sh.p_rest) - (lse_rest - lse));
      if (lane == 0) {
        p.loss[row] = bad ? nan : (none ? 0.f : L);
        p.stats[2 * (size_t)row] = bad ? nan : lse;
        p.stats[2 * (size_t)row + 1] = bad ? nan : (kTail ? lse_rest : lse);
      }
    }
    if (bad) {
      coef = q_scale = nan;
    } else if (none) {
      w = 0.f;
    } else {
      q_ref = all.m;
      q_scale = 1.f / all.s;
      ref = kTail ? (rest.m == -INFINITY ? 0.f : rest.m) : q_ref;
      coef = kTail ? (rest.m == -INFINITY ? 0.f : (q_rest - sh.p_rest) / rest.s) : q_scale;
    }
    on = on && !none;
  } else if (on) {
    const float lse = lse_in, lse_rest = lse_rest_in;
    if (lse == -INFINITY) {
      on = false;
    } else {
      // the references in units of the logits, with what their rounding lost
      q_ref = lse * p.tau;
      q_scale = expf(-fmaf(lse, p.tau, -q_ref) * p.inv_tau);
      ref = q_ref;
      coef = q_scale;
      if (kTail) {
        ref = lse_rest == -INFINITY ? 0.f : lse_rest * p.tau;
        coef = lse_rest == -INFINITY ? 0.f
                                     : (expf(lse_rest - lse) - sh.p_rest) * expf(-fmaf(lse_rest, p.tau, -ref) * p.inv_tau);
      }
      if (sh.bad) coef = q_scale = nan;
    }
  } else if (!backward && rank == 0 && tid == 0) {
    p.loss[row] = p.stats[2 * (size_t)row] = p.stats[2 * (size_t)row + 1] = 0.f;
  }

  if (grad) {
    G* out = static_cast<G*>(p.dlogits) + (size_t)row * p.V;
    const bool aligned = ((reinterpret_cast<uintptr_t>(out) - R.shift * sizeof(G)) & (VEC * sizeof(G) - 1)) == 0;
    const float cw = coef * w;
    for (int b = br.begin + warp; b < br.end; b += kWarps) {
      uint4 r[kVecPerLane];
      if (on) {
#pragma unroll
        for (int j = 0; j < kVecPerLane; ++j) r[j] = R.load(b * kBlockVecs + j * 32 + lane);
      }
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) {
        const int i = b * kBlockVecs + j * 32 + lane, e0 = R.first_entry(i);
        alignas(16) G g[VEC];
        float x[VEC];
        if (on) Elem<T>::unpack(r[j], x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[e] = Elem<G>::from_float(on ? ex2((x[e] - ref) * scale) * cw : 0.f);
        if (aligned && R.whole(i)) {
          if constexpr (sizeof(G) * VEC == 16) __stcs(reinterpret_cast<uint4*>(out + e0), *reinterpret_cast<const uint4*>(g));
          else __stcs(reinterpret_cast<uint2*>(out + e0), *reinterpret_cast<const uint2*>(g));
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (e0 + e >= 0 && e0 + e < p.V) out[e0 + e] = g[e];
        }
      }
    }
    if (on) {
      __syncthreads();   // the kept entries' gradients replace what the loop stored there
      if (tid < p.K && sh.idx[tid] >= lo && sh.idx[tid] < hi && sh.psum[tid] != -1.f)
        out[sh.idx[tid]] =
            Elem<G>::from_float(w * (q_scale * ex2((sh.z[tid] - q_ref) * scale) - sh.psum[tid]));
    }
  }
  if (pass) cluster.sync();   // a neighbour's shared memory is read until here
}

template <typename T, typename G>
cudaError_t launch(const DistillArgs& a, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  constexpr int kBlockPlaces = kBlockVecs * Elem<T>::VEC;
  const int nblk = div_up(a.V, kBlockPlaces) + 1;
  const bool backward = a.stats_in != nullptr;
  const bool tail = a.teacher_lse != nullptr;
  int c;
  if (backward) {
    c = 1;
    while (c < kMaxCluster && nblk > 2 * kWarps * c) c *= 2;   // about two blocks a warp
  } else {
    int least = div_up(nblk * (kBlockPlaces / 1024), 256);   // 256 K places: a bitmap of 32 KB
    if (a.dlogits != nullptr) {
      // the second pass finds the row in L2 while the rows in flight stay under 48 MB
      const long long row_bytes = (long long)a.V * (long long)sizeof(T);
      least = std::max(least, (int)std::min<long long>(row_bytes * 2 * sms / (48ll << 20) + 1, kMaxCluster));
    }
    c = cluster_for(a.N, least, sms);
  }
  const size_t smem = tail ? (size_t)div_up(nblk, c) * (kBlockPlaces / 8 + 1) + 16 : 0;
  auto kern = tail ? distill_kernel<T, G, true> : distill_kernel<T, G, false>;
  if (smem > 0 && (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return e;
  return launch_rows(kern, a.N, c, smem, stream, a);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
  if (a.dtype == DSPARK_F32)
    return a.gdtype == DSPARK_BF16 ? launch<float, __nv_bfloat16>(a, stream) : launch<float, float>(a, stream);
  if (a.dtype == DSPARK_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
  return launch<__half, __half>(a, stream);
}

}  // namespace dspark
