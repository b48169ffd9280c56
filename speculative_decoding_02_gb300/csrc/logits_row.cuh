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
// log s + t / s); a block whose maximum is above m rescales both first.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"

namespace dspark {
namespace lrow {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVecPerLane = 4;
constexpr int kBlockVecs = 32 * kVecPerLane;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

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
};

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
  __device__ __forceinline__ uint4 load(int i) const {
    if (whole(i)) {
      uint4 v;
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "l"(base + i)
                   : "memory");
      return v;
    }
    return load_edge(i);
  }
  __device__ __noinline__ uint4 load_edge(int i) const {
    uint4 v = make_uint4(Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf);
    T* p = reinterpret_cast<T*>(&v);
    const int e0 = first_entry(i);
    for (int e = 0; e < Elem<T>::VEC; ++e)
      if (e0 + e >= 0 && e0 + e < V) p[e] = row[e0 + e];
    return v;
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

// The largest of a lane's four vectors of a block (NaN if one is).
__device__ __forceinline__ float lane_max(const uint4 (&r)[kVecPerLane], const float*) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kVecPerLane; ++j) {
    float f[4];
    Elem<float>::unpack(r[j], f);
    m = max_nan(m, max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3])));
  }
  return m;
}
template <typename T2>
__device__ __forceinline__ T2 lane_max2(const uint4 (&r)[kVecPerLane]) {
  T2 m = *reinterpret_cast<const T2*>(&r[0].x);
#pragma unroll
  for (int j = 0; j < kVecPerLane; ++j) {
    const T2* q = reinterpret_cast<const T2*>(&r[j]);
    m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(q[0], q[1]), __hmax2_nan(q[2], q[3])));
  }
  return m;
}
__device__ __forceinline__ float lane_max(const uint4 (&r)[kVecPerLane], const __nv_bfloat16*) {
  const __nv_bfloat162 m = lane_max2<__nv_bfloat162>(r);
  return max_nan(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float lane_max(const uint4 (&r)[kVecPerLane], const __half*) {
  const __half2 m = lane_max2<__half2>(r);
  return max_nan(__low2float(m), __high2float(m));
}

// Softmax state: maximum, sum exp(x - m), sum exp(x - m) (m - x).
struct Stat {
  float m, s, t;
};
__device__ __forceinline__ Stat stat_empty() { return Stat{-INFINITY, 0.f, 0.f}; }

// Two states of one row whose exponents are scaled by `inv` (t: for inv = 1).
__device__ __forceinline__ Stat stat_merge(const Stat& a, const Stat& b, float inv = 1.f) {
  // (a NaN maximum or sum stays one: such a row is reported by NaN outputs)
  if (b.m == -INFINITY) return a;
  if (a.m == -INFINITY) return b;
  const float M = max_nan(a.m, b.m);
  const float fa = expf((a.m - M) * inv), fb = expf((b.m - M) * inv);
  // a state so far below M that its factor is 0 adds nothing (M - m may be inf)
  const float ta = fa > 0.f ? fa * fmaf(a.s, M - a.m, a.t) : fa;
  const float tb = fb > 0.f ? fb * fmaf(b.s, M - b.m, b.t) : fb;
  return Stat{M, a.s * fa + b.s * fb, ta + tb};
}
template <int W>
__device__ __forceinline__ Stat stat_reduce(Stat v, float inv = 1.f) {
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) {
    Stat o;
    o.m = __shfl_xor_sync(0xffffffffu, v.m, off);
    o.s = __shfl_xor_sync(0xffffffffu, v.s, off);
    o.t = __shfl_xor_sync(0xffffffffu, v.t, off);
    v = stat_merge(v, o, inv);
  }
  return v;
}

// Takes a lane's vectors of one block into its state; bmax is the block's
// maximum (the same on every lane), the state's maximum is too.
// d = x - m is held at -1000 / scale and above so that an entry of -inf adds 0
// to t (0 * -1000) and not NaN.
template <typename T, bool kEntropy>
__device__ __forceinline__ void stat_block(Stat& st, const uint4 (&r)[kVecPerLane], float bmax, float scale) {
  if (!(bmax <= st.m)) {
    const float m = bmax;
    if (st.m == -INFINITY) {
      st.m = m;
    } else {
      const float f = ex2((st.m - m) * scale);
      if (kEntropy) st.t = f > 0.f ? f * fmaf(st.s, m - st.m, st.t) : f;
      st.s *= f;
      st.m = m;
    }
  }
  const float m = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
  for (int j = 0; j < kVecPerLane; ++j) {
    float f[Elem<T>::VEC];
    Elem<T>::unpack(r[j], f);
#pragma unroll
    for (int e = 0; e < Elem<T>::VEC; ++e) {
      float d = f[e] - m;
      if (kEntropy) d = fmaxf(d, -1000.f);
      const float p = ex2(d * scale);
      st.s += p;
      if (kEntropy) st.t = fmaf(-p, d, st.t);
    }
  }
}

// The state of this CTA's blocks of a row, the same on warp 0's lanes (left in
// *out, which the caller reads behind a barrier).  `each(b, cur)` may change a
// block's vectors before they are taken in; `seen(b, lane maximum, block
// maximum)` sees what a block holds.  The next block's loads are in flight
// while one is taken in.
template <typename T, bool kEntropy, typename Each, typename Seen>
__device__ __forceinline__ void stat_row(const Row<T>& R, const BlockRange& br, float scale, float inv, Stat* part,
                                         Stat* out, Each each, Seen seen) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Stat st = stat_empty();
  uint4 cur[kVecPerLane], nxt[kVecPerLane];
  int b = br.begin + warp;
  if (b < br.end) {
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) cur[j] = R.load(b * kBlockVecs + j * 32 + lane);
  }
  for (; b < br.end; b += kWarps) {
    if (b + kWarps < br.end) {
#pragma unroll
      for (int j = 0; j < kVecPerLane; ++j) nxt[j] = R.load((b + kWarps) * kBlockVecs + j * 32 + lane);
    }
    each(b, cur);
    const float lm = lane_max(cur, (const T*)nullptr);
    const float bm = warp_max_nan(lm);
    seen(b, lm, bm);
    stat_block<T, kEntropy>(st, cur, bm, scale);
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) cur[j] = nxt[j];
  }
  st = stat_reduce<32>(st, inv);
  if (lane == 0) part[warp] = st;
  __syncthreads();
  if (warp == 0) {
    st = stat_reduce<kWarps>(lane < kWarps ? part[lane] : stat_empty(), inv);
    if (lane == 0) *out = st;
  }
}

// The state of a whole row from the `cta` of each of the cluster's c CTAs, the
// same on every lane; behind a cluster barrier, and another one has to follow
// before a CTA leaves.
__device__ __forceinline__ Stat stat_cluster(cg::cluster_group& cluster, Stat* cta, int c, float inv) {
  const int lane = threadIdx.x & 31;
  Stat v = lane < c ? *cluster.map_shared_rank(cta, lane) : stat_empty();
  v = stat_reduce<kMaxCluster>(v, inv);
  v.m = __shfl_sync(0xffffffffu, v.m, 0);
  v.s = __shfl_sync(0xffffffffu, v.s, 0);
  v.t = __shfl_sync(0xffffffffu, v.t, 0);
  return v;
}

// A NaN or +inf was in the row.
__device__ __forceinline__ bool stat_bad(const Stat& v) { return !(v.m < INFINITY) || !(v.s >= 0.f); }

// The backward passes take p_v = exp(x_v - lse) from an lse rounded to fp32,
// which is off by |lse| 2^-24 of its value: past this size (rows far from
// zero, and rows that a mask of the type's lowest value fills, whose log V is
// lost beside it) they take the row's state anew.
constexpr float kLargeLse = 1024.f;

// c CTAs a row so that a call with few rows still fills the card (about two
// CTAs on each SM); `least` from what one CTA can hold.
inline int cluster_for(int rows, int least, int sms) {
  int c = 1;
  while (c < kMaxCluster && (c < least || (long long)rows * c * 2 <= 2ll * sms)) c *= 2;
  return c;
}

// Launches kern with clusters of c CTAs, c * rows of them.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_rows(void (*kern)(KArgs...), int rows, int c, size_t smem, cudaStream_t stream,
                               Args&&... args) {
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
