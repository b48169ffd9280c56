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
// A cluster of 1 to 16 CTAs takes a row (logits_row.cuh) and HBM bounds it.  The
// loss needs one pass; the gradient a second one over the same part by the same
// CTA, backwards: its last blocks are still in shared memory (fp32), and L2 holds
// the others when the rows in flight fit there, so that HBM sees about one read and
// one write.  What depends on the teacher alone is worked out while the first
// blocks' loads are under way.
//
// Measured (GB300, 2048 rows of 151936 and 64 kept entries with the teacher's lse,
// four calls in a graph): the loss 183 us in fp32 (6.8 TB/s) and 104 us in bf16;
// with its gradient 442 us (one read and one write at 5.6 TB/s; HBM reads 1.49 GB
// for 1.24, L2 keeping most of the 92 MB in flight), 370 us where that is bf16 and
// 245 us for bf16 logits (5.1 TB/s); the gradient alone 380 and 197 us.
// Two passes through HBM (a kernel for the sums, one for the gradients) took
// 600 us; parts held in shared memory between the passes 830 us and more, for
// their copies, barriers and passes hardly overlap; tasks in an order that
// leaves L2 a short reuse distance 730 us, for their waits.
#include <float.h>
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "logits_row.cuh"

namespace dspark {
namespace {

using namespace lrow;

// of shared memory a CTA, so that four leave L1 the room that their loads in flight
// take: the step takes 456 us with nothing held between the passes, 450 with 23
// KB, 444 with 31, 445 with 39 and 488 with 55.  fp32 alone: in bf16, where each
// block has more entries to work on, the copy costs what it saves (253 and 258)
constexpr int kSmemPerCta = 31 * 1024;
constexpr int kMarkedPlaces = 262144;           // of a CTA's part of a row: a bitmap of 32 KB
// of the rows in flight with a gradient: the step above takes 453 to 456 us for
// 75 to 96 MB, 471 for 130 to 160 (L2 keeps less) and took 590 for one CTA a row
constexpr long long kFlightBytes = 96ll << 20;

struct Shared {
  Stat part[kWarps];
  Stat cta;               // of this CTA's part, outside the kept entries with a tail
  // the row's kept entries
  alignas(16) int idx[kMaxTop];   // -1: absent
  float p[kMaxTop];       // the teacher's probability
  float logp[kMaxTop];
  float pv[kMaxTop];      // p(v) at the first entry of its index, -1 elsewhere
  float z[kMaxTop];       // the student's logit
  float red[4][kWarps];
  int2 mass[kMaxTop / 32];   // sums of the teacher's probabilities (rest_mass)
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

// A state's log-sum-exp, held in fp32's finite range unless the state is empty: a
// row of the lowest value at a temperature below 1 is none.
__device__ __forceinline__ float finite_lse(float m, float inv_tau, float ls) {
  return m == -INFINITY ? m : fminf(fmaxf(fmaf(m, inv_tau, ls), -FLT_MAX), FLT_MAX);
}

// A number as the sum of two floats, l below half a step of h (T. J. Dekker, "A
// floating-point technique for extending the available precision", 1971; the exact
// sum of any two numbers is D. E. Knuth's).  The _rn forms are never fused.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair sum_of(float a, float b) {
  const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ Pair sum_of_ordered(float a, float b) {   // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return Pair{s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair product_of(Pair a, Pair b) {
  const float h = __fmul_rn(a.h, b.h);
  return Pair{h, fmaf(a.h, b.l, fmaf(a.l, b.h, fmaf(a.h, b.h, -h)))};
}
constexpr __device__ Pair pair_of(double v) { return Pair{(float)v, (float)(v - (double)(float)v)}; }

// t / tau - lse.
__device__ __forceinline__ Pair teacher_log(float t, const DistillArgs& p, float lse) {
  // (a difference that cancels may be smaller than what the product's rounding left)
  const float u = __fmul_rn(t, p.inv_tau);
  const Pair s = sum_of(u, -lse);
  const float l = __fadd_rn(s.l, fmaf(t, p.inv_tau, -u) + t * p.inv_tau_low);
  return fabsf(s.h) <= FLT_MAX ? sum_of(s.h, l) : Pair{s.h, 0.f};
}

// e^t for -80 <= t <= 0: t = n ln 2 + r with |r| <= 0.35 and the Taylor series of
// e^r, its terms from r^7 in single floats.  Off by 1e-14 at most, of 1 (and by
// 3e-13 of its value), over 2e7 arguments.
__device__ __forceinline__ Pair exp_of(Pair t) {
  constexpr double kLn2 = 0.693147180559945309417;
  constexpr float kLn2a = 0.693145751953125f;   // 15 bits: its products with n are exact
  constexpr float kLn2b = (float)(kLn2 - kLn2a), kLn2c = (float)(kLn2 - kLn2a - kLn2b);
  const float n = rintf(t.h * kLog2e);
  const float m = __fmul_rn(n, kLn2b);
  const Pair d = sum_of(fmaf(-n, kLn2a, t.h), -m);
  const Pair r = sum_of_ordered(d.h, d.l - fmaf(n, kLn2b, -m) + t.l - n * kLn2c);
  float f = 1.f / 479001600.f;
  f = fmaf(f, r.h, 1.f / 39916800.f);
  f = fmaf(f, r.h, 1.f / 3628800.f);
  f = fmaf(f, r.h, 1.f / 362880.f);
  f = fmaf(f, r.h, 1.f / 40320.f);
  f = fmaf(f, r.h, 1.f / 5040.f);
  Pair q{f, 0.f};
  constexpr Pair kTerms[5] = {pair_of(1. / 720), pair_of(1. / 120), pair_of(1. / 24), pair_of(1. / 6), pair_of(0.5)};
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const Pair x = product_of(q, r), y = sum_of_ordered(kTerms[i].h, x.h);
    q = Pair{y.h, __fadd_rn(y.l, __fadd_rn(x.l, kTerms[i].l))};
  }
  q = product_of(product_of(r, r), q);
  const Pair e = sum_of_ordered(r.h, q.h);
  const Pair y = sum_of_ordered(1.f, e.h);
  const float scale = __int_as_float(((int)n + 127) << 23);
  return Pair{y.h * scale, __fadd_rn(y.l, __fadd_rn(e.l, __fadd_rn(q.l, r.l))) * scale};
}

// What a teacher's probabilities leave of 1.  It is all of the gradient outside the kept
// entries, and 1 - sum p in 32 bits is off by 2^-24 of 1, however little it is:
// 3e-4 of it where they hold 99.98 %, all of it past 99.99999 %.  So each is
// taken in two floats and the sums in whole numbers, p = (i + j 2^-26) 2^-25.
// (With double exponentials the step of 2048 rows of 151936 took 448 us, so 443 as
// with sums in 32 bits; the gradient alone of 1400 fp16 rows of 50257 61, so 58.)
constexpr int kMassNan = INT_MIN;
__device__ __forceinline__ int2 warp_mass(bool has, Pair t) {
  int i = 0, j = 0;
  if (has && t.h >= -80.f) {
    const Pair p = t.h < 0.f ? exp_of(t) : Pair{1.f, 0.f};   // (one of 1 or more leaves nothing)
    i = __float2int_rn(p.h * 0x1p25f);
    j = __float2int_rn(fmaf(p.l, 0x1p25f, fmaf(p.h, 0x1p25f, -(float)i)) * 0x1p26f);
  }
  i = __reduce_add_sync(0xffffffffu, i);
  j = __reduce_add_sync(0xffffffffu, j);
  return make_int2(__any_sync(0xffffffffu, has && t.h != t.h) ? kMassNan : i, j);
}
__device__ __forceinline__ float rest_mass(const int2* mass) {
  long long left = 1ll << 51;
  bool nan = false;
#pragma unroll
  for (int w = 0; w < kMaxTop / 32; ++w) {
    left -= mass[w].x * (1ll << 26) + mass[w].y;
    nan |= mass[w].x == kMassNan;
  }
  return nan ? __int_as_float(0x7FC00000) : (left > 0 ? (float)left * 0x1p-51f : 0.f);
}

// The teacher's side of a row and the student's logits there, by the CTA, into
// sh; returns the state of the kept entries (with a tail, if `state`), the
// rest's mass, whether an index is out of range and whether an entry has mass.
struct Kept {
  Stat stat;
  float p_rest;
  bool bad, any;
};
template <typename T, bool kTail>
__device__ __forceinline__ Kept load_kept(Shared& sh, const DistillArgs& p, int row, const T* rp, bool state) {
  const int tid = threadIdx.x;
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
  // the teacher's probabilities once more for their sum, by the warps that hold
  // no entry, beside the search for equal indices
  static_assert(kThreads >= 2 * kMaxTop, "a second thread for every entry");
  const int k2 = tid - (kThreads - kMaxTop);
  Pair t2{-INFINITY, 0.f};
  if (kTail && k2 >= 0 && k2 < p.K) t2 = teacher_log(p.top_val[(size_t)row * p.K + k2], p, p.teacher_lse[row]);
  Kept r;
  // log p_k and p_k (products and differences rounded once)
  float t = -INFINITY, base = 0.f;
  if (kTail) {
    if (val != -INFINITY) t = teacher_log(val, p, p.teacher_lse[row]).h;
  } else {
    const float m = cta_max(sh, 0, val);
    if (val != -INFINITY) t = (val - m) * p.inv_tau;
    base = logf(cta_add(sh, 1, t == -INFINITY ? 0.f : expf(t)));
  }
  const float logp = t == -INFINITY ? -INFINITY : t - base;
  if (tid < kMaxTop) {
    sh.p[tid] = t == -INFINITY ? 0.f : expf(logp);
    sh.logp[tid] = logp;
    sh.z[tid] = z;
  }
  __syncthreads();
  const float pk = tid < kMaxTop ? sh.p[tid] : 0.f;
  // p(v): equal indices add up in the first of them
  float pv = pk;
  bool first = idx >= 0;
  if (first) {
    int equal = 0;
#pragma unroll 4
    for (int k = 0; k < p.K; k += 4) {
      const int4 i = *reinterpret_cast<const int4*>(sh.idx + k);
      equal += (i.x == idx) + (i.y == idx) + (i.z == idx) + (i.w == idx);
    }
    if (equal > 1) {
      pv = 0.f;
      for (int k = 0; first && k < p.K; ++k) {
        if (sh.idx[k] != idx) continue;
        first = k >= tid;
        pv += sh.p[k];
      }
    }
  }
  if (tid < kMaxTop) sh.pv[tid] = first ? pv : -1.f;
  if (kTail && k2 >= 0) {
    const int2 m = warp_mass(k2 < p.K && sh.idx[k2] >= 0, t2);
    if ((tid & 31) == 0) sh.mass[k2 >> 5] = m;
  }
  r.stat = stat_empty();
  if (kTail && state) {
    r.stat.m = cta_max(sh, 3, first ? z : -INFINITY);
    r.stat.s = cta_add(sh, 0, first && r.stat.m != -INFINITY ? expf((z - r.stat.m) * p.inv_tau) : 0.f);
  }
  r.any = __syncthreads_or(val != -INFINITY);
  r.bad = __syncthreads_or(bad);
  r.p_rest = kTail ? rest_mass(sh.mass) : 0.f;
  return r;
}

// kTail: the teacher's lse is given.  With p.stats_in the backward pass alone,
// which takes the row's state anew only where one of its stats is too large to be used.
// kStash: the part's last `stash` blocks stay in shared memory between the passes.
template <typename T, typename G, bool kTail, bool kStash>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) distill_kernel(const DistillArgs p, int ahead, int stash) {
  constexpr int VEC = Elem<T>::VEC;
  constexpr int kBlockPlaces = kBlockVecs * VEC;
  __shared__ Shared sh;
  extern __shared__ uint4 dynamic[];   // `stash` blocks; kTail: one bit per place of the part, then a byte per block
  cg::cluster_group cluster = cg::this_cluster();
  const int c = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = (int)(blockIdx.x / c);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool backward = p.stats_in != nullptr, grad = p.dlogits != nullptr;
  const float nan = __int_as_float(0x7FC00000);
  const float scale = p.inv_tau * kLog2e;
  const uint64_t drop = tc::policy_evict_first();   // of what is read for the last time
  const T* rp = static_cast<const T*>(p.logits) + (size_t)row * p.row_stride;
  const Row<T> R(rp, p.V);
  const BlockRange br = block_range(R.nvec, rank, c);
  const int place0 = br.begin * kBlockPlaces - R.shift;   // entry at the part's first place
  const int nblk = br.end - br.begin;
  const int stash_from = br.end - (kStash ? stash : 0);
  uint32_t* marked = reinterpret_cast<uint32_t*>(dynamic + (kStash ? stash : 0) * kBlockVecs);
  const int group = row / p.R;
  bool on = p.lens == nullptr || row - group * p.R < p.lens[group];
  float lse_in = 0.f, lse_rest_in = 0.f;
  if (backward && on) {
    lse_in = p.stats_in[2 * (size_t)row];
    lse_rest_in = p.stats_in[2 * (size_t)row + 1];
  }
  // (the second one is the tail's reference: masks of finite values outside the
  // kept entries leave it far from zero beside an ordinary lse)
  const bool pass = on && (!backward || lse_is_large(lse_in) || (kTail && lse_is_large(lse_rest_in)));

  Kept kept;
  kept.any = kept.bad = false;
  // outside the kept entries the gradient is cw exp((x - ref) / tau), on one
  // w (q_scale exp((x - q_ref) / tau) - p(v))
  float ref = 0.f, cw = 0.f, q_ref = 0.f, q_scale = 0.f;
  const float w = grad && on ? (p.weight != nullptr ? p.weight[row] : 1.f) * p.inv_tau : 0.f;

  // The gradient goes through the part backwards: what was read last is surest
  // to be in L2.  Its first block is under way while the CTAs meet.
  uint4 cur[kVecPerLane], nxt[kVecPerLane];
  int b = nblk > warp ? br.begin + warp + (nblk - 1 - warp) / kWarps * kWarps : -1;
  auto load_again = [&](int k, uint4(&r)[kVecPerLane]) {
    if (!kStash || k < stash_from) {
      R.load_block(k, lane, r, drop);
    } else {
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) r[j] = dynamic[(k - stash_from) * kBlockVecs + j * 32 + lane];
    }
  };
  auto first_block = [&]() {
    if (grad && b >= 0) load_again(b, cur);
  };

  // the row that takes this CTA's place (without a second pass, which needs L2 for
  // the rows in flight)
  auto next = [&]() {
    if (tid == 0 && row + ahead < p.N && ahead > 0) prefetch_row(rp + (size_t)ahead * p.row_stride, p.V, backward ? 2 : 4);
  };
  if (pass) {
    const int words = nblk * (kBlockPlaces / 32);
    unsigned char* block_marked = reinterpret_cast<unsigned char*>(marked + words);
    auto before = [&]() {
      if constexpr (kTail) {
        for (int k = tid; k < words; k += kThreads) marked[k] = 0;
        for (int k = tid; k < nblk; k += kThreads) block_marked[k] = 0;
      }
      kept = load_kept<T, kTail>(sh, p, row, rp, true);
      if constexpr (kTail) {
        const int place = tid < p.K && sh.idx[tid] >= 0 ? sh.idx[tid] - place0 : -1;
        if (place >= 0 && place < nblk * kBlockPlaces) {
          atomicOr(&marked[place >> 5], 1u << (place & 31));
          block_marked[place / kBlockPlaces] = 1;
        }
        __syncthreads();
      }
    };
    auto leave_out = [&](int b, uint4(&cur)[kVecPerLane]) {
      if (kStash && b >= stash_from) {
#pragma unroll
        for (int j = 0; j < kVecPerLane; ++j) dynamic[(b - stash_from) * kBlockVecs + j * 32 + lane] = cur[j];
      }
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
    // (with a gradient to come L2 is asked to keep the row for it)
    const uint64_t keep = grad ? tc::policy_evict_last() : drop;
    std::conditional_t<kStash, SplitPolicy, uint64_t> policy;
    if constexpr (kStash) policy = SplitPolicy{keep, drop, stash_from};
    else policy = keep;
    stat_row<T, false, false>(R, br, scale, p.inv_tau, policy, sh.part, &sh.cta, before,
                              leave_out, Nothing(), next);
    cluster_arrive(c);
    first_block();
    cluster_wait(c);
    const Stat rest = stat_cluster(cluster, &sh.cta, c, p.inv_tau);
    cluster_arrive(c);   // (this CTA has read the others' shared memory)
    const Stat all = kTail ? stat_reduce<2>(lane & 1 ? kept.stat : rest, p.inv_tau) : rest;
    const bool bad = kept.bad || (kept.any && stat_bad(all));
    const bool none = all.m == -INFINITY;
    const float ls = none ? 0.f : logf(all.s);
    q_ref = none ? 0.f : all.m;
    q_scale = 1.f / all.s;
    ref = q_ref;
    cw = w * q_scale;
    if (kTail) {
      ref = rest.m == -INFINITY ? 0.f : rest.m;
      const float q_rest = expf((rest.m - all.m) * p.inv_tau) * rest.s / all.s;
      cw = rest.m == -INFINITY ? 0.f : w * ((q_rest - kept.p_rest) / rest.s);
    }
    on = bad || (kept.any && !none);
    if (bad) cw = q_scale = nan;
    if (!backward && rank == 0) {
      const float pk = tid < p.K ? sh.p[tid] : 0.f;
      // p (log p - log q) with -log q = distance / tau + ls; the distance is taken
      // down by p first, for over tau alone it may pass fp32's range
      float L = cta_add(sh, 1, !(pk == 0.f) ? fmaf(pk * (q_ref - sh.z[tid]), p.inv_tau, pk * (sh.logp[tid] + ls)) : 0.f);
      const float ls_rest = logf(rest.s);
      const float lse = finite_lse(all.m, p.inv_tau, ls), lse_rest = finite_lse(rest.m, p.inv_tau, ls_rest);
      if (kTail && !(kept.p_rest == 0.f)) {
        // (log q_r not as lse_rest - lse: of rows far from zero the two keep no fraction)
        const float below = rest.m == -INFINITY ? INFINITY : kept.p_rest * (all.m - rest.m);
        L += fmaf(below, p.inv_tau, kept.p_rest * (logf(kept.p_rest) + (ls - ls_rest)));
      }
      if (tid == 0) {
        const bool counts = kept.any || bad;
        p.loss[row] = bad ? nan : (on ? L : 0.f);
        p.stats[2 * (size_t)row] = bad ? nan : (counts ? lse : 0.f);
        p.stats[2 * (size_t)row + 1] = bad ? nan : (counts ? (kTail ? lse_rest : lse) : 0.f);
      }
    }
  } else if (on) {
    first_block();
    kept = load_kept<T, kTail>(sh, p, row, rp, false);
    // the references in units of the logits, with what their rounding lost
    on = (kept.any || kept.bad) && lse_in != -INFINITY;
    q_ref = on ? lse_in * p.tau : 0.f;
    q_scale = expf(-fmaf(lse_in, p.tau, -q_ref) * p.inv_tau);
    ref = q_ref;
    cw = w * q_scale;
    if (kTail) {
      ref = lse_rest_in == -INFINITY ? 0.f : lse_rest_in * p.tau;
      cw = lse_rest_in == -INFINITY ? 0.f
                                    : w * ((expf(lse_rest_in - lse_in) - kept.p_rest) *
                                           expf(-fmaf(lse_rest_in, p.tau, -ref) * p.inv_tau));
    }
    if (kept.bad) cw = q_scale = nan;
  } else if (!backward && rank == 0 && tid == 0) {
    p.loss[row] = p.stats[2 * (size_t)row] = p.stats[2 * (size_t)row + 1] = 0.f;
  }

  if (grad) {
    G* out = static_cast<G*>(p.dlogits) + (size_t)row * p.V;
    // an output row whose vectors start where the logits' do is stored by vectors
    const bool aligned = ((reinterpret_cast<uintptr_t>(out) - R.shift * sizeof(G)) & (VEC * sizeof(G) - 1)) == 0;
    auto store = [&](int k, int j, bool inside, const G(&g)[VEC]) {
      const int i = k * kBlockVecs + j * 32 + lane, e0 = R.first_entry(i);
      if (inside || (aligned && R.whole(i))) {
        if constexpr (sizeof(G) * VEC == 16) __stcs(reinterpret_cast<uint4*>(out + e0), *reinterpret_cast<const uint4*>(g));
        else __stcs(reinterpret_cast<uint2*>(out + e0), *reinterpret_cast<const uint2*>(g));
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (e0 + e >= 0 && e0 + e < p.V) out[e0 + e] = g[e];
      }
    };
    if (!on) {
      alignas(16) G none[VEC];
#pragma unroll
      for (int e = 0; e < VEC; e += 2) put2(none + e, 0.f, 0.f);
      for (; b >= br.begin + warp; b -= kWarps) {
#pragma unroll
        for (int j = 0; j < kVecPerLane; ++j) store(b, j, aligned && R.inside(b), none);
      }
    }
    const uint64_t ref2 = pack2(-ref, -ref), scale2 = pack2(scale, scale), cw2 = pack2(cw, cw);
    auto gradient = [&](int k, const uint4(&r)[kVecPerLane]) {
      const bool inside = aligned && R.inside(k);
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) {
        alignas(16) G g[VEC];
        float x[VEC];
        Elem<T>::unpack(r[j], x);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          float u, v;
          unpack2(mul2(add2(pack2(x[e], x[e + 1]), ref2), scale2), u, v);
          unpack2(mul2(pack2(ex2(u), ex2(v)), cw2), u, v);
          put2(g + e, u, v);
        }
        store(k, j, inside, g);
      }
    };
    for (; b >= br.begin + warp; b -= kWarps) {
      if (b - kWarps >= br.begin + warp) load_again(b - kWarps, nxt);
      gradient(b, cur);
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) cur[j] = nxt[j];
    }
    if (backward) next();
    if (on) {
      __syncthreads();   // the kept entries' gradients replace what the loop stored there
      if (tid < p.K && sh.pv[tid] != -1.f) {
        const int place = sh.idx[tid] - place0;
        if (place >= 0 && place < nblk * kBlockPlaces)
          out[sh.idx[tid]] = Elem<G>::from_float(w * (q_scale * ex2((sh.z[tid] - q_ref) * scale) - sh.pv[tid]));
      }
    }
  }
  if (pass && c > 1) cluster_wait(c);   // the others have read this one's
}

template <typename T, typename G>
cudaError_t launch(const DistillArgs& a, cudaStream_t stream) {
  constexpr int kBlockPlaces = kBlockVecs * Elem<T>::VEC;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int nblk = div_up(a.V, kBlockPlaces) + 1;
  int least = div_up(nblk, kMarkedPlaces / kBlockPlaces);
  if (a.stats_in != nullptr) {
    least = std::max(least, std::min(div_up(nblk, 8 * kWarps), 8));   // eight blocks a warp, or more
    // (1400 rows of 50257 fp16 entries: 71 us so, 73 and 94 with four and two)
  } else if (a.dlogits != nullptr) {
    const long long flight = (long long)a.V * (long long)sizeof(T) * std::min(a.N, kCtasPerSm * sms);
    least = std::max(least, (int)std::min<long long>((flight + kFlightBytes - 1) / kFlightBytes, kMaxCluster));
  }
  const int c = cluster_for(a.N, nblk, least, sms);
  const bool two_passes = a.dlogits != nullptr && a.stats_in == nullptr;
  const int ahead = c == 1 && a.lens == nullptr && !two_passes ? kCtasPerSm * sms : 0;
  const bool tail = a.teacher_lse != nullptr;
  const int marks = tail ? (div_up(nblk, c) * (kBlockPlaces / 8 + 1) + 15) & ~15 : 0;
  if constexpr (sizeof(T) == 4) {
    if (two_passes) {
      const int room = std::max(0, kSmemPerCta - (int)sizeof(Shared) - marks);
      const int stash = std::min(room / (kBlockVecs * 16), nblk / c);
      const int smem = stash * kBlockVecs * 16 + marks;
      return launch_rows(tail ? distill_kernel<T, G, true, true> : distill_kernel<T, G, false, true>, a.N, c, smem,
                         stream, a, ahead, stash);
    }
  }
  return launch_rows(tail ? distill_kernel<T, G, true, false> : distill_kernel<T, G, false, false>, a.N, c, marks,
                     stream, a, ahead, 0);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
  if (a.dtype == DSPARK_F32)
    return a.gdtype == DSPARK_BF16 ? launch<float, __nv_bfloat16>(a, stream) : launch<float, float>(a, stream);
  if (a.dtype == DSPARK_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
  return launch<__half, __half>(a, stream);
}

}  // namespace dspark
