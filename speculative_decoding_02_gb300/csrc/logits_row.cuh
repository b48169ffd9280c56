// Streaming one row of logits: what the log-probability and distillation
// kernels share.  A row of V entries (fp32, bf16 or fp16) starts at any
// element, so its 16-byte vectors are counted from the row's address rounded
// down to 16 bytes: vector i holds entries i * VEC - shift + e, and only the
// first and last vector of a row can hold places outside it, which are read
// as -inf.  128 consecutive vectors (2 KB; four per lane, 32 apart) are a
// block, the unit one warp reads at a time; a cluster of c CTAs splits a row's
// blocks evenly.
//
// The softmax of a row is taken in one pass: each warp keeps a maximum m that
// is the same on its 32 lanes, and per lane s = sum exp(x - m) and
// t = sum exp(x - m) (m - x) over what it has read (from which the entropy is
// log s + t / s); a block whose maximum is above m rescales both first.  Two
// entries share each packed fp32 addition, product and fused product.
//
// CTAs of 256 threads, four to an SM, rather than two of 512: a row's
// barriers and short serial phases (merging states, choosing alternatives, the
// teacher's side) then overlap with the other rows' streams (2048 bf16 rows of
// 129280 with 64 alternatives, as the kernel was when both sizes were timed: 171 us
// against 210; it takes 116 now).
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "tc_common.cuh"

namespace dspark {
namespace lrow {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecPerLane = 4;
constexpr int kBlockVecs = 32 * kVecPerLane;
constexpr int kMaxCluster = 16;
constexpr int kCtasPerSm = 4;
constexpr float kLog2e = 1.4426950408889634f;

// Word i of a vector.
__device__ __forceinline__ uint32_t word(uint4 r, int i) {
  const uint32_t lo = i & 1 ? r.y : r.x, hi = i & 1 ? r.w : r.z;
  return i & 2 ? hi : lo;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int VEC = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static __device__ __forceinline__ float to_float(float v) { return v; }
  static __device__ __forceinline__ float from_float(float v) { return v; }
  static __device__ __forceinline__ void unpack(uint4 r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
  // Entry e of a vector.
  static __device__ __forceinline__ float entry(uint4 r, int e) { return __uint_as_float(word(r, e)); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void unpack(uint4 r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  // Entry e of a vector.
  static __device__ __forceinline__ float entry(uint4 r, int e) { return __uint_as_float(word(r, e >> 1) >> 16 * (e & 1) << 16); }
};
template <>
struct Elem<__half> {
  static constexpr int VEC = 8;
  static constexpr uint32_t kNegInf = 0xFC00FC00u;
  static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ void unpack(uint4 r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  // Entry e of a vector.
  static __device__ __forceinline__ float entry(uint4 r, int e) { return __half2float(__ushort_as_half((unsigned short)(word(r, e >> 1) >> 16 * (e & 1)))); }
};

// A 16-byte load past L1; a policy (createpolicy) says how long L2 holds it, and
// none costs no register.
struct NoPolicy {};
__device__ __forceinline__ uint4 ld_stream(const uint4* p, NoPolicy) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_stream(const uint4* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy)
               : "memory");
  return v;
}

// Asks L2 for the start of a row that a CTA will take soon: 1 / part of it, 64 KB
// at most.  The CTAs of a launch take in rows of one length in step, and so come
// to the end of one together, where nothing is asked of HBM until they have
// begun the next (3 of 30 us at 151936 bf16 entries).  2048 rows of those take 101
// us so and 109 without (fp32: 179 and 190; 105 by 128 KB, 106 by 16 KB); 10000
// rows of 32000 128 us by a quarter of a row, 132 without, 145 by the whole.
constexpr uint64_t kAheadBytes = 65536;
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* row, int V, int part) {
  const uint64_t a = ((uint64_t)__cvta_generic_to_global(row) + 15) & ~15ull;
  const uint64_t n = min((uint64_t)V * sizeof(T) / part, kAheadBytes) & ~15ull;   // (a - row < 16 bytes: inside the row)
  if (n > 16)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"((uint32_t)n - 16) : "memory");
}

// One policy for the blocks before `from`, another from there on.
struct SplitPolicy {
  uint64_t before, behind;
  int from;
};
__device__ __forceinline__ NoPolicy policy_of(NoPolicy p, int) { return p; }
__device__ __forceinline__ uint64_t policy_of(uint64_t p, int) { return p; }
__device__ __forceinline__ uint64_t policy_of(const SplitPolicy& p, int b) { return b < p.from ? p.before : p.behind; }

// A row as its vectors: `base` is the row's address rounded down to 16 bytes.
template <typename T>
struct Row {
  const T* row;
  const uint4* base;
  int shift;     // places of vector 0 before the row
  int V;
  int nvec;
  __device__ __forceinline__ Row(const T* r, int V_) : row(r), V(V_) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(r);
    shift = (int)((a & 15) / sizeof(T));
    base = reinterpret_cast<const uint4*>(a & ~(uintptr_t)15);
    nvec = (shift + V + Elem<T>::VEC - 1) / Elem<T>::VEC;
  }
  __device__ __forceinline__ int first_entry(int i) const { return i * Elem<T>::VEC - shift; }
  __device__ __forceinline__ bool whole(int i) const {
    const int e0 = first_entry(i);
    return e0 >= 0 && e0 + Elem<T>::VEC <= V;
  }
  // Vector i with -inf in the places outside the row (i >= nvec: all of them).
  template <typename P>
  __device__ __forceinline__ uint4 load(int i, P policy) const {
    return whole(i) ? ld_stream(base + i, policy) : load_edge(i);
  }
  __device__ __noinline__ uint4 load_edge(int i) const {
    uint4 v = make_uint4(Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf);
    T* p = reinterpret_cast<T*>(&v);
    const int e0 = first_entry(i);
    for (int e = 0; e < Elem<T>::VEC; ++e)
      if (e0 + e >= 0 && e0 + e < V) p[e] = row[e0 + e];
    return v;
  }
  // Every vector of block b is whole.
  __device__ __forceinline__ bool inside(int b) const {
    return first_entry(b * kBlockVecs) >= 0 && first_entry((b + 1) * kBlockVecs) <= V;
  }
  // This lane's vectors of block b.
  template <typename P>
  __device__ __forceinline__ void load_block(int b, int lane, uint4 (&r)[kVecPerLane], P policy) const {
    const int i0 = b * kBlockVecs + lane;
    if (inside(b)) {
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) r[j] = ld_stream(base + i0 + j * 32, policy);
    } else {
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) r[j] = load(i0 + j * 32, policy);
    }
  }
};

// The blocks [begin, end) of a row that CTA `rank` of `c` reads.
struct BlockRange {
  int begin, end;
};
__device__ __forceinline__ BlockRange block_range(int nvec, int rank, int c) {
  const int nblk = (nvec + kBlockVecs - 1) / kBlockVecs;
  const int per = (nblk + c - 1) / c;
  BlockRange r;
  r.begin = min(rank * per, nblk);
  r.end = min(r.begin + per, nblk);
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest of a vector's entries (NaN if one is).
__device__ __forceinline__ float vec_max(uint4 r, const float*) {
  float f[4];
  Elem<float>::unpack(r, f);
  return max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3]));
}
template <typename T2>
__device__ __forceinline__ T2 vec_max2(const uint4& r) {
  const T2* q = reinterpret_cast<const T2*>(&r);
  return __hmax2_nan(__hmax2_nan(q[0], q[1]), __hmax2_nan(q[2], q[3]));
}
__device__ __forceinline__ float vec_max(uint4 r, const __nv_bfloat16*) {
  const __nv_bfloat162 m = vec_max2<__nv_bfloat162>(r);
  return max_nan(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float vec_max(uint4 r, const __half*) {
  const __half2 m = vec_max2<__half2>(r);
  return max_nan(__low2float(m), __high2float(m));
}
// The largest of a lane's four vectors of a block.
__device__ __forceinline__ float lane_max(const uint4 (&r)[kVecPerLane], const float* t) {
  return max_nan(max_nan(vec_max(r[0], t), vec_max(r[1], t)), max_nan(vec_max(r[2], t), vec_max(r[3], t)));
}
template <typename T2>
__device__ __forceinline__ float lane_max2(const uint4 (&r)[kVecPerLane]) {
  const T2 m = __hmax2_nan(__hmax2_nan(vec_max2<T2>(r[0]), vec_max2<T2>(r[1])),
                           __hmax2_nan(vec_max2<T2>(r[2]), vec_max2<T2>(r[3])));
  return max_nan(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float lane_max(const uint4 (&r)[kVecPerLane], const __nv_bfloat16*) {
  return lane_max2<__nv_bfloat162>(r);
}
__device__ __forceinline__ float lane_max(const uint4 (&r)[kVecPerLane], const __half*) { return lane_max2<__half2>(r); }

// Softmax state: maximum, sum exp(x - m), sum exp(x - m) (m - x).
struct Stat {
  float m, s, t;
};
__device__ __forceinline__ Stat stat_empty() { return Stat{-INFINITY, 0.f, 0.f}; }

// The states of W lanes of one row (exponents scaled by `inv`; t: for inv = 1)
// as one, on each of the W.  A NaN or +inf maximum gives a NaN sum.
template <int W>
__device__ __forceinline__ Stat stat_reduce(const Stat& v, float inv = 1.f) {
  float M = v.m;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  // (a state so far below M that its factor is 0 adds nothing: M - m may be inf)
  const float f = v.m == -INFINITY && M == M ? 0.f : expf((v.m - M) * inv);
  float s = v.s * f;
  float t = f > 0.f ? f * fmaf(v.s, M - v.m, v.t) : f;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, off);
    t += __shfl_xor_sync(0xffffffffu, t, off);
  }
  return Stat{M, s, t};
}

// Packed fp32 arithmetic on the pairs of a 64-bit register.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two results, rounded, next to each other.
__device__ __forceinline__ void put2(float* g, float a, float b) { g[0] = a; g[1] = b; }
__device__ __forceinline__ void put2(__nv_bfloat16* g, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(g) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void put2(__half* g, float a, float b) {
  *reinterpret_cast<__half2*>(g) = __floats2half2_rn(a, b);
}

// A lane's running state: the warp's maximum, and the sums of its even and odd
// entries (t with the opposite sign).
struct LaneStat {
  float m;
  uint64_t s, t;
};
__device__ __forceinline__ LaneStat lane_stat_empty() { return LaneStat{-INFINITY, 0, 0}; }

// Takes a lane's vectors of one block into its state; bmax is the block's
// maximum (the same on every lane, as the state's is).
// With kEntropy d = x - m is held at -1000 and above so that an entry of -inf
// adds 0 to t (0 * -1000) and not NaN.
template <typename T, bool kEntropy>
__device__ __forceinline__ void stat_block(LaneStat& st, const uint4 (&r)[kVecPerLane], float bmax, float scale) {
  if (!(bmax <= st.m)) {
    if (st.m != -INFINITY) {
      const float up = bmax - st.m, f = ex2(-up * scale);
      const uint64_t f2 = pack2(f, f);
      if (kEntropy) st.t = f > 0.f ? mul2(f2, fma2(st.s, pack2(-up, -up), st.t)) : f2;
      st.s = mul2(st.s, f2);
    }
    st.m = bmax;
  }
  const float m = st.m == -INFINITY ? 0.f : st.m;
  const uint64_t nm = pack2(-m, -m), sc = pack2(scale, scale);
#pragma unroll
  for (int j = 0; j < kVecPerLane; ++j) {
    float f[Elem<T>::VEC];
    Elem<T>::unpack(r[j], f);
#pragma unroll
    for (int e = 0; e < Elem<T>::VEC; e += 2) {
      uint64_t d = add2(pack2(f[e], f[e + 1]), nm);
      float a, b;
      if (kEntropy) {
        unpack2(d, a, b);
        d = pack2(fmaxf(a, -1000.f), fmaxf(b, -1000.f));
      }
      unpack2(mul2(d, sc), a, b);
      const uint64_t p = pack2(ex2(a), ex2(b));
      st.s = add2(st.s, p);
      if (kEntropy) st.t = fma2(p, d, st.t);
    }
  }
}

// The warp's state from its lanes'.
__device__ __forceinline__ Stat lanes_sum(const LaneStat& v) {
  float s, s1, t, t1;
  unpack2(v.s, s, s1);
  unpack2(v.t, t, t1);
  s += s1;
  t += t1;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, off);
    t += __shfl_xor_sync(0xffffffffu, t, off);
  }
  return Stat{v.m, s, -t};
}

// The states of the CTA's warps as one in *out, which is read behind a barrier.
__device__ __forceinline__ void cta_stat(const LaneStat& st, float inv, Stat* part, Stat* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Stat v = lanes_sum(st);
  if (lane == 0) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const Stat w = stat_reduce<kWarps>(lane < kWarps ? part[lane] : stat_empty(), inv);
    if (lane == 0) *out = w;
  }
}

// The state of this CTA's blocks of a row, read from global memory, in *out
// (behind a barrier).  before() runs once the first two blocks' loads are in flight
// and last() behind the last block;
// each(b, vectors) may change a block's vectors before they are taken in.  With
// kSeen seen(b, lane maximum, float4) sees a block's maxima: those of its four
// quarters (one vector of every lane).  The next blocks' loads are in flight
// while one is taken in.
template <typename T, bool kEntropy, bool kSeen, typename P, typename Before, typename Each, typename Seen, typename Last>
__device__ __forceinline__ void stat_row(const Row<T>& R, const BlockRange& br, float scale, float inv, P policy, Stat* part,
                                         Stat* out, Before before, Each each, Seen seen, Last last) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  LaneStat st = lane_stat_empty();
  uint4 cur[kVecPerLane], nxt[kVecPerLane];
  int b = br.begin + warp;
  if (b < br.end) R.load_block(b, lane, cur, policy_of(policy, b));
  if (b + kWarps < br.end) R.load_block(b + kWarps, lane, nxt, policy_of(policy, b + kWarps));
  before();
  auto take = [&](int k, uint4(&v)[kVecPerLane]) {
    each(k, v);
    float bm;
    if constexpr (kSeen) {
      static_assert(kVecPerLane == 4, "four quarters");
      float m[4], q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = vec_max(v[j], (const T*)nullptr);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = warp_max_nan(m[j]);
      bm = max_nan(max_nan(q[0], q[1]), max_nan(q[2], q[3]));
      seen(k, max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3])), make_float4(q[0], q[1], q[2], q[3]));
    } else {
      bm = warp_max_nan(lane_max(v, (const T*)nullptr));
    }
    stat_block<T, kEntropy>(st, v, bm, scale);
    if (k + 2 * kWarps < br.end) R.load_block(k + 2 * kWarps, lane, v, policy_of(policy, k + 2 * kWarps));
  };
  // (two blocks a turn, each in registers of its own)
  for (; b < br.end; b += 2 * kWarps) {
    take(b, cur);
    if (b + kWarps < br.end) take(b + kWarps, nxt);
  }
  last();
  cta_stat(st, inv, part, out);
}

// The state of a whole row from the `cta` of each of the cluster's c CTAs, the
// same on every lane; behind a cluster barrier, and another one has to follow
// before a CTA leaves.
__device__ __forceinline__ Stat stat_cluster(cg::cluster_group& cluster, Stat* cta, int c, float inv) {
  if (c == 1) return *cta;
  const int lane = threadIdx.x & 31;
  Stat v = stat_reduce<kMaxCluster>(lane < c ? *cluster.map_shared_rank(cta, lane) : stat_empty(), inv);
  v.m = __shfl_sync(0xffffffffu, v.m, 0);
  v.s = __shfl_sync(0xffffffffu, v.s, 0);
  v.t = __shfl_sync(0xffffffffu, v.t, 0);
  return v;
}

// The cluster's barrier, whole and in its two halves (one CTA: the CTA's).
__device__ __forceinline__ void cluster_arrive(int c) {
  if (c > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait(int c) {
  if (c > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else __syncthreads();
}
__device__ __forceinline__ void cluster_meet(int c) {
  cluster_arrive(c);
  cluster_wait(c);
}

// A hook of stat_row that does nothing.
struct Nothing {
  __device__ __forceinline__ void operator()() const {}
  __device__ __forceinline__ void operator()(int, uint4 (&)[kVecPerLane]) const {}
  __device__ __forceinline__ void operator()(int, float, float4) const {}
};

// A NaN or +inf was in the row.
__device__ __forceinline__ bool stat_bad(const Stat& v) { return !(v.m < INFINITY) || !(v.s >= 0.f); }

// The backward passes take p_v = exp(x_v - lse) from an lse rounded to fp32,
// which is off by |lse| 2^-24 of its value: past this size (rows far from
// zero, and rows that a mask of the type's lowest value fills, whose log V is
// lost beside it) they take the row's state anew.  An empty row's -inf is exact.
constexpr float kLargeLse = 1024.f;
__device__ __forceinline__ bool lse_is_large(float lse) { return lse != -INFINITY && fabsf(lse) > kLargeLse; }

// CTAs a row: at least `least` (1 to 16), and for few rows up to 8 as long as
// every warp keeps a block and the SMs have about two each.  Rows of 151936
// fp32 entries with 20 alternatives: one row takes 21 us by one CTA, 9.5 by 8 and
// 9.7 by 16; 16 rows 21, 10.6 and 15.7; 152 rows 31 by one each, 24 by 2 and 30
// by 4; 304 rows 38, 36 and 51.
inline int cluster_for(int rows, int nblk, int least, int sms) {
  int c = least;
  while (2 * c <= 8 && (long long)rows * c <= sms && nblk > kWarps * c) c *= 2;
  return c;
}

// Launches kern with clusters of c CTAs, c * rows of them.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_rows(void (*kern)(KArgs...), int rows, int c, size_t smem, cudaStream_t stream,
                               Args&&... args) {
  if (c > 8) {
    // (8 is the largest size that needs no opt-in)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)rows * c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

inline cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace lrow
}  // namespace dspark
