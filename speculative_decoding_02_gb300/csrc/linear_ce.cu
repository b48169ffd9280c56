// Softmax cross entropy of hidden states under an output head, in pieces of the
// vocabulary, without keeping the logits, and its gradients: the loss a draft's
// hidden states are trained with ("[DeepSeek-6] DSpark" blog, section 9).  For
// the rows n that count, z = h W^T [N, V], t the row's token:
//
//   loss:      lse = log sum_v exp z_v,  loss = lse - z_t
//   gradients: s_v = (g_loss + g_lse) exp(z_v - lse) - g_loss 1[v = t]
//              dh = s W,  dW = s^T h
//
// Four products of 2 N V D operations (the gradients form z again), bound by the
// tensor cores as soon as there are a few hundred rows and by the read of W below.
// The rows that count are gathered first, so the others cost nothing.
//
// Measured (GB300, bf16): 2048 rows under a head of 151936 x 2560, the loss 803 us
// (1.98 PFLOP/s, tensor pipe 97 %; 921 us for seconds on end, under the power
// cap), dh 1678 us (1.90 PFLOP/s; 1949); one row 131 us (5.9 TB/s of W).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_tc.cuh"

namespace dspark {
namespace {

using namespace gemm;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kMaxSplits = 32;   // parts of dh

struct Counts {
  int n;            // rows that count
  int all;          // and, of few rows with dW wanted, as many that hold what a rounding takes
  int full;         // tiles of dh taken whole, the first ones
  int splits;       // parts of K of the others
  float scale;      // of the slopes, a power of two
  float inv_scale;
  int done;         // CTAs of the loss' tiles that are done
};

// A row, for its slopes.
struct __align__(16) RowInfo {
  float lse2;       // lse log2 e
  float up, down;   // scale (g_loss + g_lse), scale g_loss
  int token;        // or -2 - token: the row holds what the rounding of that slope took; -1: zeros
};

// What the rounding of a token's slope takes shows in dW, where a token that comes
// once has that slope alone, and the slopes of a token that comes often are near one
// another (-g, where g_loss is a mean's) and so are their remainders: up to 2^-8 of
// the token's row in bf16 and 2^-11 in fp16, as much as dW's own rounding.  Up to
// kRestRows rows are repeated, from the next multiple of 32 on, with those
// remainders alone as slopes: they fill the step of 64 rows that one row takes
// anyway, and cost up to two steps more.  With more rows, which would be formed and
// multiplied twice, the remainders stay out: dW of 1340 rows under 129280 x 4096
// (bf16) is off by 2.2e-3 of its 2-norm, where its own rounding takes 1.6e-3.  (Added
// in dW's epilogue, with the rows in order of tokens, they cost 1 % where a token
// comes once or twice, but 36 -> 150 us of 2048 rows under 1000 x 512 with frequent
// tokens, and 256 -> 610 of 2048 rows of one token under 32000 x 1024.)
constexpr int kRestRows = 128;
__host__ __device__ constexpr int rest_at(int n) { return (n + 31) / 32 * 32; }

__host__ __device__ constexpr long long ceil_to(long long x, long long m) { return (x + m - 1) / m * m; }

// ---------------------------------------------------------------------------
// which rows count, and the rows themselves
// ---------------------------------------------------------------------------
struct ScanParams {
  const int32_t* tokens;
  const int32_t* lens;
  int N, R, V;
  float* loss;              // forward: written where a row does not count
  float* lse;
  const float* g_loss;      // backward
  const float* g_lse;
  bool common;              // the slopes have one scale
  int D, dt, kx, wt, units, max_splits;   // dt: column tiles of dh, wt: row tiles of a piece of dW (0: not wanted)
  Counts* counts;
  int32_t* list;            // [N]: the rows that count, in order
  int32_t* slot;            // [N]: a row's place there; -1 none, -2 none and its token is out of range
  int* status;
};

// The parts of K that give tx tiles of dh and dW's the earliest end: a tile takes
// its steps of K and, where few follow one another in a unit, some 20 steps' time
// for its first copies and its epilogue (64 rows under a head of 8192 x 512: 33.5 us,
// with 4 steps' time and so twice the parts 35.9).  A warp, a choice a lane.
constexpr int kTileSteps = 20;
__device__ int choose_splits(int tx, int tw, int kx, int kw, int units, int most) {
  static_assert(kMaxSplits <= 32, "a lane each");
  const int s = (threadIdx.x & 31) + 1;
  const long long cx = div_up(kx, s) + kTileSteps;
  const long long waves = div_up(tx * s, units) * cx;
  const long long all = ((long long)tx * s * cx + (long long)tw * (kw + kTileSteps)) / units;
  long long cost = s <= most ? (waves > all ? waves : all) : 1ll << 56;
  cost = cost << 6 | s;   // (of equal ones the fewest parts)
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    const long long other = __shfl_xor_sync(0xffffffffu, cost, d);
    cost = other < cost ? other : cost;
  }
  return (int)(cost & 63);
}

// With dh alone, as many tiles as fill all units go whole and the others in
// parts: 80 tiles of 792 steps on 76 pairs by 76 whole and 4 in 19 parts end
// after 834 steps (all 80 in 14 parts: 855, and 14 times the sums to keep).
// Beside dW, whose tiles fill what is left, by parts only.  A whole warp.
__device__ Counts counts_of(const ScanParams& p, int n, int exponent) {
  Counts c{n, p.wt > 0 && n <= kRestRows ? rest_at(n) + n : n, 0, 1, ldexpf(1.f, exponent), ldexpf(1.f, -exponent), 0};
  if (p.dt > 0) {
    const int tiles = div_up(n, 256) * p.dt;
    c.full = p.wt == 0 ? tiles / p.units * p.units : 0;
    if (c.full < tiles)
      c.splits = choose_splits(tiles - c.full, p.wt * div_up(p.D, 256), p.kx, div_up(c.all, kStep), p.units,
                               p.max_splits);
  }
  return c;
}
// The scale of fp16 slopes, 2 to this, when g is the largest |g_loss| or |g_loss +
// g_lse|: of the row for dh alone, whose rows are sums of their own, of all rows when dW
// sums over them.  fp16 has all its digits from 2^-14 to 65504 (and its last
// one at 2^-24): the slopes, at most 2 g, go up to 2^15, so that g times a probability
// of 2^-27 keeps its digits.  (bf16 has fp32's range.)
__device__ int slope_exponent(float g) {
  int e = 0;
  if (!(g > 0.f && g < INFINITY)) return 0;
  frexpf(g, &e);   // g < 2^e
  return max(-100, min(100, 14 - e));
}
__device__ __forceinline__ bool in_group(const ScanParams& p, int n) {
  return p.lens == nullptr || n % p.R < p.lens[n / p.R];
}
// Of a row that counts, what its slopes are scaled by.
__device__ __forceinline__ float upstream(const float* g_loss, const float* g_lse, long long n) {
  const float a = g_loss[n], b = g_lse ? a + g_lse[n] : a;
  return fmaxf(fabsf(a), fabsf(b));
}
// The outputs of a row that does not count.
__device__ __forceinline__ void leave_out(const ScanParams& p, long long n, bool in, int token) {
  const bool bad = in && token != -1;
  if (bad) record_status(p.status, DSPARK_ERR_INVALID);
  if (p.loss) {
    p.loss[n] = bad ? __int_as_float(0x7fc00000) : 0.f;
    p.lse[n] = 0.f;
  }
  if (p.slot) p.slot[n] = bad ? -2 : -1;
}

constexpr int kScanThreads = 1024, kScanEach = 8;

// One block: the rows that count, in order (27 us of 32768 rows, 770 of 2^20).
__global__ void __launch_bounds__(kScanThreads) ce_scan(const ScanParams p) {
  __shared__ int sums[32], before[32];
  __shared__ float most[32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  float g = 0.f;
  for (long long n0 = 0; n0 < p.N; n0 += kScanThreads * kScanEach) {
    const long long first = n0 + (long long)threadIdx.x * kScanEach;
    unsigned on = 0;
#pragma unroll
    for (int j = 0; j < kScanEach; ++j) {
      const long long n = first + j;
      if (n >= p.N) break;
      const int t = p.tokens[n];
      const bool in = in_group(p, (int)n);
      if (in && t >= 0 && t < p.V) {
        on |= 1u << j;
        if (p.common) g = fmaxf(g, upstream(p.g_loss, p.g_lse, n));
      } else {
        leave_out(p, n, in, t);
      }
    }
    const int mine = __popc(on);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      int v = sums[lane];
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
      }
      before[lane] = v;
    }
    __syncthreads();
    int at = base + incl - mine + (warp > 0 ? before[warp - 1] : 0);
    for (; on != 0; on &= on - 1, ++at) {
      const long long n = first + __ffs(on) - 1;
      p.list[at] = (int)n;
      if (p.slot) p.slot[n] = at;
    }
    base += before[31];
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
  if (lane == 0) most[warp] = g;
  __syncthreads();
  if (warp == 0) {
    for (int w = 0; w < 32; ++w) g = fmaxf(g, most[w]);
    const Counts c = counts_of(p, base, slope_exponent(g));
    if (lane == 0) *p.counts = c;
  }
}

struct GatherParams {
  const unsigned short* h;
  const unsigned short* W;
  long long h_stride, W_stride;
  const int32_t* tokens;
  const int32_t* list;
  const Counts* counts;
  int D;
  bool vec;                 // rows of h start on 16 bytes
  unsigned short* rows;     // [..][ld]
  int ld;
  float* logit;             // forward: the token's logit
  const float* lse;         // backward
  const float* g_loss;
  const float* g_lse;
  bool own_scale;           // the row's slopes are scaled by itself
  RowInfo* info;
};

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<__half2*>(&w));
}

template <bool kBf16>
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 u = unpack2<kBf16>(x[j]), v = unpack2<kBf16>(y[j]);
    s = fmaf(u.x, v.x, s);
    s = fmaf(u.y, v.y, s);
  }
  return s;
}

// Gathered row j, a block of 128 threads: `row` of h, dense, and its token's logit
// (in fp32 from the row itself: a loss is the difference of two logits that may be
// near each other) or what its slopes need; zeros without a row.
template <bool kBf16>
__device__ __forceinline__ void gather_row(const GatherParams& p, int j, int row, float scale, float* sums,
                                           bool rest = false) {
  uint4* out = reinterpret_cast<uint4*>(p.rows + (size_t)j * p.ld);
  const int chunks = p.D / 8;
  if (row < 0) {
    for (int c = threadIdx.x; c < chunks; c += 128) out[c] = make_uint4(0, 0, 0, 0);
    if (p.info && threadIdx.x == 0) p.info[j] = RowInfo{0.f, 0.f, 0.f, -1};
    return;
  }
  const int t = p.tokens[row];
  const unsigned short* src = p.h + (size_t)row * p.h_stride;
  const uint4* w = reinterpret_cast<const uint4*>(p.W + (size_t)t * p.W_stride);
  float s = 0.f;
  for (int c = threadIdx.x; c < chunks; c += 128) {
    uint4 v;
    if (p.vec) {
      v = reinterpret_cast<const uint4*>(src)[c];
    } else {
      uint32_t x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = src[8 * c + 2 * e] | (uint32_t)src[8 * c + 2 * e + 1] << 16;
      v = make_uint4(x[0], x[1], x[2], x[3]);
    }
    out[c] = v;
    if (p.logit) s = dot8<kBf16>(v, __ldg(w + c), s);
  }
  if (p.logit) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) p.logit[j] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  } else if (threadIdx.x == 0) {
    const float g = p.g_loss[row];
    if (!kBf16 && p.own_scale) scale = ldexpf(1.f, slope_exponent(upstream(p.g_loss, p.g_lse, row)));
    p.info[j] = RowInfo{p.lse[row] * kLog2e, scale * (p.g_lse ? g + p.g_lse[row] : g), scale * g,
                        rest ? -2 - t : t};
  }
}

// A block per gathered row; the rows up to the next multiple of 256 are zeros.
template <bool kBf16>
__global__ void __launch_bounds__(128) ce_gather(const GatherParams p) {
  __shared__ float sums[4];
  pdl_trigger();
  pdl_wait();
  const int j = blockIdx.x, n = p.counts->n, rest = rest_at(n);
  if (j >= ceil_to(n, 256)) return;
  const bool again = p.counts->all > n && j >= rest && j < rest + n;
  gather_row<kBf16>(p, j, again ? p.list[j - rest] : j < n ? p.list[j] : -1, p.counts->scale, sums, again);
}

// Both for few rows, without a kernel in between: every block counts the rows
// before its own and all of them (2048 blocks read 16 MB of tokens from L2), then
// copies its row to its place and, beyond the last place, clears one.
constexpr int kFewRows = 2048;

template <bool kBf16>
__global__ void __launch_bounds__(128) ce_scan_gather(const ScanParams p, const GatherParams q) {
  __shared__ int counted[2][4];
  __shared__ float most[4], sums[4];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x;
  int before = 0, all = 0;
  float g = 0.f;
  for (int n = threadIdx.x; n < p.N; n += 128) {
    const int t = p.tokens[n];
    if (t < 0 || t >= p.V || !in_group(p, n)) continue;
    ++all;
    if (n < b) ++before;
    if (p.common) g = fmaxf(g, upstream(p.g_loss, p.g_lse, n));
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
#pragma unroll
  for (int d = 16; d > 0; d /= 2) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    counted[0][warp] = before;
    counted[1][warp] = all;
    most[warp] = g;
  }
  __syncthreads();
  before = counted[0][0] + counted[0][1] + counted[0][2] + counted[0][3];
  all = counted[1][0] + counted[1][1] + counted[1][2] + counted[1][3];
  g = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
  const int e = slope_exponent(g), rest = rest_at(all);
  const bool again = p.wt > 0 && all <= kRestRows;
  if (b == 0 && warp == 0) {
    const Counts c = counts_of(p, all, e);
    if (threadIdx.x == 0) *p.counts = c;
  }
  if (b < p.N) {
    const int t = p.tokens[b];
    const bool in = in_group(p, b);
    if (in && t >= 0 && t < p.V) {
      if (threadIdx.x == 0) {
        p.list[before] = b;
        if (p.slot) p.slot[b] = before;
      }
      gather_row<kBf16>(q, before, b, ldexpf(1.f, e), sums);
      if (again) gather_row<kBf16>(q, rest + before, b, ldexpf(1.f, e), sums, true);
    } else if (threadIdx.x == 0) {
      leave_out(p, b, in, t);
    }
  }
  if (b >= all && b < ceil_to(all, 256) && !(again && b >= rest && b < rest + all)) gather_row<kBf16>(q, b, -1, 0.f, sums);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

struct CombineParams {
  const float2* part;      // [rows][vocabulary tiles]
  int vtiles;
  Counts* counts;
  const float* logit;
  const int32_t* list;
  float* loss;
  float* lse;
};

// Row j from its tiles' maxima and sums; a warp.
__device__ __forceinline__ void combine_row(const CombineParams& p, int j) {
  const int lane = threadIdx.x & 31;
  const float2* part = p.part + (size_t)j * p.vtiles;
  float m = -INFINITY, s = 0.f;
  for (int v0 = 0; v0 < p.vtiles; v0 += 32 * 8) {
    float2 x[8];
    float M = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int v = v0 + i * 32 + lane;
      x[i] = v < p.vtiles ? __ldcg(part + v) : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) M = fmaxf(M, x[i].x);
    const float top = M == -INFINITY ? 0.f : M;
    s *= exp2f(m - top);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i].y, exp2f(x[i].x - top), s);
    m = M;
  }
  float M = m;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  s *= exp2f(m - (M == -INFINITY ? 0.f : M));
#pragma unroll
  for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane != 0) return;
  const int row = p.list[j];
  const float l = log2f(s);
  p.lse[row] = (M + l) * kLn2;
  p.loss[row] = (fmaf(-p.logit[j], kLog2e, M) + l) * kLn2;
}

// z = h W^T by tiles; of a tile's rows, the maximum (in units of log 2) and the
// sum of 2^(z log2 e - maximum) of its 256 columns.
template <bool kPairs>
struct LossTiles {
  CUtensorMap h, w;
  static constexpr bool kPair = kPairs, kSelf = false;   // single CTAs: up to 128 rows, a tile each
  static constexpr int kM = kPairs ? 256 : 128, kN = 256, kBoxBytes = 0, kTables = 2 * 4 * kRows * 8, kExtraBytes = kTables + 128;
  using Counts = int;
  int* status;
  bool bf16;
  const dspark::Counts* live;
  bool one_row_tile;     // N <= 256
  bool last_combines;    // the last CTA to end has the rows combined; else a kernel does
  CombineParams rows;
  float2* part;          // [rows][vocabulary tiles]
  int V, steps, vtiles;

  __device__ void prefetch() const {
    prefetch_tensormap(&h);
    prefetch_tensormap(&w);
  }
  // W, which no kernel of this call writes, on its way into L2 while the rows are
  // gathered: the unit's first tile, known when there is one row tile (behind the
  // kernel before, which began when all earlier work was done)
  __device__ void early(int unit, int rank) const {
    if (!one_row_tile) return;
    for (int k = threadIdx.x; k < steps; k += 32) prefetch_box(&w, k * kStep, unit * kN + rank * 128);
  }
  __device__ int counts() const { return live->n; }
  // An accumulator loses about half a step an addition, always towards zero: by
  // 16 steps of K an lse of 14 is off by -3.4e-6 (1.3e-6 at random besides; plain
  // fp32 products: up to 9e-7 for the lse, 3e-6 to 5e-6 for the loss, at random), by 8
  // -2e-6, by 4 -1e-6, by 2 -6e-7.  N = 2048, V = 151936, D = 2560: 800, 805, 837 and
  // 899 us; one row: 135, 135, 135 and 139.
  __device__ int chunk(int n) const { return n > 256 ? 8 : n > 32 && steps > 8 ? 4 : 2; }
  __device__ bool used(int n, const Tile& t, int row) const { return t.m0 + row < n; }
  __device__ bool tile(int n, int unit, int units, int i, Tile& t) const {
    // neighbouring units take the row tiles of the same columns, so that W
    // comes once from HBM
    const int mt = div_up(n, kM);
    const long long u = (long long)i * units + unit;
    if (u >= (long long)mt * vtiles) return false;
    t.m0 = (int)(u % mt) * kM;
    t.n0 = (int)(u / mt) * kN;
    t.steps = steps;
    t.a_mn = t.b_mn = false;
    return true;
  }
  __device__ int segments(const Tile&) const { return 1; }
  __device__ Segment segment(const Tile& t, int) const { return Segment{&h, &w, t.m0, 0, t.n0, 0, t.steps}; }

  // A few rows are combined here, which saves a launch (3 us).
  __device__ void finish(int n, const Epi& e) const {
    if (!last_combines || n == 0) return;
    int* last = reinterpret_cast<int*>(e.extra + kTables);
    named_bar_sync(5, kEpiWarps * 32);
    if (threadIdx.x == 64) {
      __threadfence();   // (all of this CTA's parts, through the barrier)
      *last = atomicAdd(&rows.counts->done, 1) == (int)gridDim.x - 1;
      __threadfence();
    }
    named_bar_sync(5, kEpiWarps * 32);
    if (!*last) return;
    for (int j = (threadIdx.x >> 5) - 2; j < n; j += kEpiWarps) combine_row(rows, j);
  }

  __device__ void epilogue(const Epi& e, const Tile& t, float (&z)[64]) const {
    if (!e.used) {   // (nor are the other warps of these rows)
      named_bar_sync(1 + e.q, 128);
      return;
    }
    const int left = V - (t.n0 + e.col);
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      if (j >= left) z[j] = -INFINITY;
      m = fmaxf(m, z[j]);
    }
    // (a row of -inf, or a quarter past the vocabulary's end: a sum of zeros)
    m = m == -INFINITY ? m : m * kLog2e;
    const float at = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 64; ++j) s += ex2_approx(fmaf(z[j], kLog2e, -at));
    // the four warps of these rows; two tables in turn, so that one barrier a tile is
    // enough: behind tile n's reads its readers meet the others at tile n + 1's
    // (whether that one is used or not) before any of these writes tile n + 2's
    float2* table = reinterpret_cast<float2*>(e.extra) + (e.n & 1) * 4 * kRows;
    const int r = e.q * 32 + e.lane;
    table[e.h * kRows + r] = make_float2(m, s);
    named_bar_sync(1 + e.q, 128);
    if (e.h == 0) {
      float2 v[4];
      float M = -INFINITY, S = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = table[i * kRows + r];
        M = fmaxf(M, v[i].x);
      }
      const float top = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int i = 0; i < 4; ++i) S += v[i].y * ex2_approx(v[i].x - top);
      part[(size_t)(t.m0 + e.row) * vtiles + t.n0 / 256] = make_float2(M, S);
    }
  }
};

// A warp a row.
__global__ void __launch_bounds__(128) ce_combine(const CombineParams p) {
  pdl_trigger();
  pdl_wait();
  const int j = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (j < p.counts->n) combine_row(p, j);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// The slopes of a piece of the vocabulary, rounded to the operands' type for the
// products that follow: by up to 2^-8 of each in bf16 and 2^-11 in fp16.  The many small
// ones' roundings average out over a sum.  That of the token's own, which is most
// of a row's dh, is kept apart and added to dh; for dW see kRestRows.
struct SlopeTiles {
  CUtensorMap h, w, out;
  static constexpr bool kPair = true, kSelf = false;
  static constexpr int kN = 256, kBoxBytes = kStoreBox, kExtraBytes = 0;
  using Counts = int;
  int* status;
  bool bf16;
  const dspark::Counts* live;
  const RowInfo* info;
  float* corr;           // what the rounding of the token's slope took
  int rows;              // of the slopes' matrix
  int v0, V, steps, vtiles;

  __device__ void prefetch() const {
    prefetch_tensormap(&h);
    prefetch_tensormap(&w);
    prefetch_tensormap(&out);
  }
  __device__ void early(int, int) const {}
  template <class C>
  __device__ void finish(const C&, const Epi&) const {}
  __device__ int counts() const { return live->all; }
  __device__ int chunk(int) const { return 64; }   // (far below the slopes' rounding)
  __device__ bool used(int n, const Tile& t, int row) const { return t.m0 + row < n; }
  __device__ bool tile(int n, int unit, int units, int i, Tile& t) const {
    const int mt = div_up(n, 256);
    const long long u = (long long)i * units + unit;
    if (u >= (long long)mt * vtiles) return false;
    t.m0 = (int)(u % mt) * 256;
    t.n0 = (int)(u / mt) * 256;
    t.steps = steps;
    t.a_mn = t.b_mn = false;
    return true;
  }
  __device__ int segments(const Tile&) const { return 1; }
  __device__ Segment segment(const Tile& t, int) const { return Segment{&h, &w, t.m0, 0, v0 + t.n0, 0, t.steps}; }

  __device__ float rounded(float x) const {
    return bf16 ? __bfloat162float(__float2bfloat16_rn(x)) : __half2float(__float2half_rn(x));
  }
  __device__ void epilogue(const Epi& e, const Tile& t, float (&z)[64]) const {
    const RowInfo r = info[t.m0 + e.row];
    const bool rest = r.token < -1;
    const int first = v0 + t.n0 + e.col, left = rest ? 0 : V - first, at = (rest ? -2 - r.token : r.token) - first;
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 64; j += 2) {
      float x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = j + i < left || j + i == at ? ex2_approx(fmaf(z[j + i], kLog2e, -r.lse2)) * r.up : 0.f;
        if (j + i == at) {
          x[i] -= r.down;
          if (rest) x[i] -= rounded(x[i]);
        }
      }
      float2 back;
      if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[0], x[1]);
        w[j / 2] = *reinterpret_cast<const uint32_t*>(&v);
        back = unpack2<true>(w[j / 2]);
      } else {
        const __half2 v = __floats2half2_rn(x[0], x[1]);
        w[j / 2] = *reinterpret_cast<const uint32_t*>(&v);
        back = unpack2<false>(w[j / 2]);
      }
      if (j == at) corr[t.m0 + e.row] = x[0] - back.x;
      if (j + 1 == at) corr[t.m0 + e.row] = x[1] - back.y;
    }
    if (r.token == -1) {   // (zeros by choice, not by up = 0: the head may hold infinities)
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = 0;
    }
    store_16bit(e, &out, w, t.n0 + e.col, vtiles * 256, t.m0 + e.row0, rows);
  }
};

// dh += s W and dW = s^T h of a piece, in one launch: first dh's tiles, in parts
// of K, which are long, then dW's, dealt so that all units end at about the
// same time.
struct GradTiles {
  CUtensorMap s_k, s_mn, w, h, dh, dW;
  static constexpr bool kPair = true, kSelf = false;
  static constexpr int kN = 256, kBoxBytes = kStoreBox, kExtraBytes = 0;
  struct Counts {
    int n, mt, full, splits, kw, tx, tw, shared;   // tx: work items of dh
    float inv_scale;
  };
  int* status;
  bool bf16;
  const dspark::Counts* live;
  int rows;              // of the slopes' matrix
  int v0, V, kx, wt;     // the piece: first column, of V; steps of K and (for dW) tiles of 256
  int D, dt;             // tiles of D
  bool want_dh, add;     // add: a piece came before

  __device__ void prefetch() const {
    for (const CUtensorMap* m : {&s_k, &s_mn, &w, &h, &dh, &dW}) prefetch_tensormap(m);
  }
  __device__ void early(int, int) const {}
  template <class C>
  __device__ void finish(const C&, const Epi&) const {}
  __device__ Counts counts() const {
    const dspark::Counts l = *live;
    Counts c;
    c.n = l.n;
    c.mt = div_up(l.n, 256);
    c.full = l.full;
    c.splits = l.splits;
    c.kw = div_up(l.all, kStep);
    c.tx = want_dh ? c.full + (c.mt * dt - c.full) * c.splits : 0;
    c.tw = wt * dt;
    c.inv_scale = l.inv_scale;
    // dW tiles that every unit takes: those with one more of dh's take no
    // more than these (see tile)
    const int units = gridDim.x >> 1;
    const float cx = (float)(div_up(kx, c.splits) + 4), cw = (float)(c.kw + 4);
    const float all = (c.tx * cx + c.tw * cw) / units;
    const int most = div_up(c.tx, units);
    c.shared = min(max((int)((all - most * cx) / cw + 0.5f), 0), c.tw / units);
    return c;
  }
  __device__ int chunk(const Counts&) const { return 64; }
  __device__ bool used(const Counts& c, const Tile& t, int row) const {
    return t.kind == 0 ? t.m0 + row < c.n : v0 + t.m0 + row < V;
  }
  __device__ bool tile(const Counts& c, int unit, int units, int i, Tile& t) const {
    const int more = c.tx % units;                      // the first `more` units take one more of dh's
    const int own = c.tx / units + (unit < more ? 1 : 0);
    if (i < own) {
      const int u = i * units + unit, rest = c.mt * dt - c.full;
      t.kind = 0;
      t.part = u < c.full ? 0 : (u - c.full) / rest;
      const int v = u < c.full ? u : c.full + (u - c.full) % rest;
      const int each = u < c.full ? kx : div_up(kx, c.splits);
      t.m0 = v % c.mt * 256;
      t.n0 = v / c.mt * 256;
      t.k0 = t.part * each;
      t.steps = max(0, min(each, kx - t.k0));
      t.a_mn = false;
      t.b_mn = true;
      return true;
    }
    i -= own;
    int u;
    if (i < c.shared) {
      u = i * units + unit;
    } else {
      if (unit < more) return false;
      u = c.shared * units + (i - c.shared) * (units - more) + unit - more;
    }
    if (u >= c.tw) return false;
    t.kind = 1;
    t.part = 0;
    t.m0 = u / dt * 256;
    t.n0 = u % dt * 256;
    t.steps = c.kw;
    t.a_mn = t.b_mn = true;
    return true;
  }
  __device__ int segments(const Tile&) const { return 1; }
  __device__ Segment segment(const Tile& t, int) const {
    if (t.kind == 1) return Segment{&s_mn, &h, t.m0, 0, t.n0, 0, t.steps};
    return Segment{&s_k, &w, t.m0, t.k0 * kStep, t.n0, v0 + t.k0 * kStep, t.steps};
  }

  __device__ void epilogue(const Epi& e, const Tile& t, float (&v)[64]) const {
    if (!e.used) return;
    if (t.kind == 0) {
      store_fp32(e, &dh, v, t.n0 + e.col, D, t.m0 + e.row0, rows, t.part, add);
      return;
    }
    const float scale = live->inv_scale;
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 64; j += 2) {
      if (bf16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[j] * scale, v[j + 1] * scale);
        w[j / 2] = *reinterpret_cast<const uint32_t*>(&x);
      } else {
        const __half2 x = __floats2half2_rn(v[j] * scale, v[j + 1] * scale);
        w[j / 2] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    store_16bit(e, &dW, w, t.n0 + e.col, D, v0 + t.m0 + e.row0, V);
  }
};

struct FinishParams {
  const float* part;        // [splits][rows][D]
  long long rows;
  const Counts* counts;
  const int32_t* slot;
  const float* corr;
  const RowInfo* info;
  const unsigned short* W;
  long long W_stride;
  int D;
  unsigned short* dh;       // [N][D]
  const float* g_loss;      // where slopes were scaled by the row, else null
  const float* g_lse;
};

// What a remainder of a slope adds of x: nothing where x is infinite, for the slope's
// own product is infinite there (and the remainder may be 0 or of the other sign).
__device__ __forceinline__ float remainder_times(float corr, float x) {
  return fabsf(x) < INFINITY ? corr * x : 0.f;
}

// dh of a row: the sum of its parts and what the rounding of its token's slope took.
template <bool kBf16>
__global__ void __launch_bounds__(128) ce_finish(const FinishParams p) {
  pdl_trigger();
  pdl_wait();
  const int j = p.slot[blockIdx.x];
  uint4* out = reinterpret_cast<uint4*>(p.dh + (size_t)blockIdx.x * p.D);
  const int chunks = p.D / 8;
  if (j < 0) {
    const uint32_t v = j == -2 ? 0x7fff7fffu : 0u;   // NaN in either type
    for (int c = threadIdx.x; c < chunks; c += 128) out[c] = make_uint4(v, v, v, v);
    return;
  }
  const Counts counts = *p.counts;
  const float corr = p.corr[j];
  float inv_scale = counts.inv_scale;
  if (!kBf16 && p.g_loss) inv_scale = ldexpf(1.f, -slope_exponent(upstream(p.g_loss, p.g_lse, blockIdx.x)));
  const int mt = div_up(counts.n, 256);
  const uint4* w = reinterpret_cast<const uint4*>(p.W + (size_t)p.info[j].token * p.W_stride);
  for (int c = threadIdx.x; c < chunks; c += 128) {
    float a[8];
    const uint4 x = __ldg(w + c);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = unpack2<kBf16>(xs[e]);
      a[2 * e] = remainder_times(corr, u.x);
      a[2 * e + 1] = remainder_times(corr, u.y);
    }
    const int parts = (c * 8 / 256) * mt + j / 256 < counts.full ? 1 : counts.splits;
    for (int s = 0; s < parts; ++s) {
      const float4* q = reinterpret_cast<const float4*>(p.part + ((size_t)s * p.rows + j) * p.D + 8 * c);
      const float4 u = q[0], v = q[1];
      a[0] += u.x; a[1] += u.y; a[2] += u.z; a[3] += u.w;
      a[4] += v.x; a[5] += v.y; a[6] += v.z; a[7] += v.w;
    }
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = a[2 * e] * inv_scale, hi = a[2 * e + 1] * inv_scale;
      if constexpr (kBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        o[e] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        o[e] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    out[c] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ---------------------------------------------------------------------------
// workspace
// ---------------------------------------------------------------------------
constexpr long long kPieceBytes = 256ll << 20;   // of the slopes
constexpr long long kPartBytes = 256ll << 20;    // of dh's parts

struct Layout {
  long long rows;                  // N, in whole row tiles
  int ld;                          // of the gathered rows: on 128 bytes (copies of rows that straddle such lines take longer)
  size_t counts, list, slot, info, logit, corr, h, part, slopes, dh, total;
  int vtiles;                      // of the vocabulary
  int piece;                       // columns of a piece (a multiple of 256)
  int splits;                      // parts of dh at most
};

Layout layout(int N, int V, int D, bool backward, bool want_dh) {
  Layout l{};
  l.rows = ceil_to(N, 256);
  l.ld = (int)ceil_to(D, 64);
  l.vtiles = div_up(V, 256);
  size_t at = 256;                 // the status word
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align256(bytes);
    return a;
  };
  l.counts = take(sizeof(Counts));
  l.list = take(4ull * N);
  l.h = take(2ull * l.rows * l.ld);
  if (!backward) {
    l.logit = take(4ull * N);
    l.part = take(8ull * l.rows * l.vtiles);
  } else {
    l.slot = take(4ull * N);
    l.info = take(16ull * l.rows);
    l.corr = take(4ull * l.rows);
    const long long most = std::max<long long>(256, kPieceBytes / (2 * l.rows) / 256 * 256);
    const int pieces = (int)((V + most - 1) / most);
    l.piece = (int)ceil_to((V + pieces - 1) / pieces, 256);
    l.slopes = take(2ull * l.rows * l.piece);
    if (want_dh) {
      l.splits = (int)std::max<long long>(1, std::min<long long>(kMaxSplits, kPartBytes / (4 * l.rows * D)));
      l.dh = take(4ull * l.splits * l.rows * D);
    }
  }
  l.total = at;
  return l;
}

}  // namespace

size_t linear_ce_workspace_bytes(int N, int V, int D, bool backward, bool want_dh) {
  return layout(N, V, D, backward, want_dh).total;
}

namespace {

template <class K, class... A>
cudaError_t small(K kern, long long grid, int block, cudaStream_t stream, const A&... args) {
  return launch_pdl(kern, dim3((unsigned)grid), dim3((unsigned)block), 0, stream, args...);
}

#define CE_TRY(expr)                            \
  do {                                          \
    const cudaError_t _e = (expr);              \
    if (_e != cudaSuccess) return _e;           \
  } while (0)

cudaError_t scan_and_gather(const LinearCeArgs& a, const Layout& l, char* ws, const ScanParams& s, GatherParams& g,
                            cudaStream_t stream) {
  g.h = static_cast<const unsigned short*>(a.h);
  g.W = static_cast<const unsigned short*>(a.W);
  g.h_stride = a.h_stride;
  g.W_stride = a.W_stride;
  g.tokens = a.tokens;
  g.list = s.list;
  g.counts = s.counts;
  g.D = a.D;
  g.vec = reinterpret_cast<uintptr_t>(a.h) % 16 == 0 && (a.N == 1 || a.h_stride % 8 == 0);
  g.ld = l.ld;
  g.rows = reinterpret_cast<unsigned short*>(ws + l.h);
  const bool bf16 = a.dtype == DSPARK_BF16;
  if (a.N <= kFewRows) {
    auto kern = bf16 ? ce_scan_gather<true> : ce_scan_gather<false>;
    kern<<<(unsigned)l.rows, 128, 0, stream>>>(s, g);
    return cudaGetLastError();
  }
  ce_scan<<<1, kScanThreads, 0, stream>>>(s);
  CE_TRY(cudaGetLastError());
  return small(bf16 ? ce_gather<true> : ce_gather<false>, l.rows, 128, stream, g);
}

ScanParams scan_params(const LinearCeArgs& a, const Layout& l, char* ws) {
  ScanParams s{};
  s.tokens = a.tokens;
  s.lens = a.lens;
  s.N = a.N; s.R = a.R; s.V = a.V;
  s.counts = reinterpret_cast<Counts*>(ws + l.counts);
  s.list = reinterpret_cast<int32_t*>(ws + l.list);
  s.status = a.status;
  return s;
}

// The tiles and, unless the last of them does it, the rows combined.
template <bool kPairs>
cudaError_t launch_loss(const LinearCeArgs& a, const Layout& l, char* ws, const ScanParams& s, const GatherParams& g,
                        cudaStream_t stream) {
  const bool bf16 = a.dtype == DSPARK_BF16;
  LossTiles<kPairs> t{};
  CE_TRY(map_16bit(g.rows, bf16, l.rows, a.D, l.ld, kRows, &t.h));
  CE_TRY(map_16bit(a.W, bf16, a.V, a.D, a.W_stride, Shape<LossTiles<kPairs>>::kBRows, &t.w));
  t.status = a.status;
  t.bf16 = bf16;
  t.live = s.counts;
  t.one_row_tile = l.rows == 256;
  t.part = reinterpret_cast<float2*>(ws + l.part);
  t.V = a.V;
  t.steps = div_up(a.D, kStep);
  t.vtiles = l.vtiles;
  t.rows = CombineParams{t.part, l.vtiles, s.counts, g.logit, s.list, a.loss, a.lse_out};
  // (16 warps, 256 tiles at a time: up to 5 turns of about 0.7 us)
  t.last_combines = (long long)div_up(a.N, kEpiWarps) * div_up(l.vtiles, 256) <= 5;
  const int units = max_units<LossTiles<kPairs>>();
  if (units <= 0) return cudaErrorUnknown;
  CE_TRY(launch(t, (int)std::min<long long>(units, (long long)div_up(a.N, LossTiles<kPairs>::kM) * l.vtiles), stream));
  return t.last_combines ? cudaSuccess : small(ce_combine, div_up(a.N, 4), 128, stream, t.rows);
}

}  // namespace

cudaError_t launch_linear_ce(const LinearCeArgs& a, cudaStream_t stream) {
  const Layout l = layout(a.N, a.V, a.D, false, false);
  char* ws = static_cast<char*>(a.ws);
  ScanParams s = scan_params(a, l, ws);
  s.loss = a.loss;
  s.lse = a.lse_out;
  GatherParams g{};
  g.logit = reinterpret_cast<float*>(ws + l.logit);
  CE_TRY(scan_and_gather(a, l, ws, s, g, stream));

  // (pairs would pad to 256 rows: one row under a head of 151936 x 2560 takes 132 us by
  // single CTAs, 135 by pairs; 56 rows under 32000 x 1024, 21 and 25)
  return a.N <= kRows ? launch_loss<false>(a, l, ws, s, g, stream) : launch_loss<true>(a, l, ws, s, g, stream);
}

cudaError_t launch_linear_ce_backward(const LinearCeArgs& a, cudaStream_t stream) {
  const bool want_dh = a.dh != nullptr, want_dW = a.dW != nullptr;
  const Layout l = layout(a.N, a.V, a.D, true, want_dh);
  char* ws = static_cast<char*>(a.ws);
  const bool bf16 = a.dtype == DSPARK_BF16;
  const int units = max_units<GradTiles>();
  if (units <= 0) return cudaErrorUnknown;
  ScanParams s = scan_params(a, l, ws);
  s.slot = reinterpret_cast<int32_t*>(ws + l.slot);
  s.g_loss = a.g_loss;
  s.g_lse = a.g_lse;
  s.common = !bf16 && want_dW;
  s.D = a.D;
  s.dt = want_dh ? div_up(a.D, 256) : 0;
  s.kx = l.piece / kStep;
  s.wt = want_dW ? l.piece / 256 : 0;
  s.units = units;
  s.max_splits = l.splits;
  GatherParams g{};
  g.lse = a.lse_in;
  g.g_loss = a.g_loss;
  g.g_lse = a.g_lse;
  g.own_scale = !bf16 && !want_dW;
  g.info = reinterpret_cast<RowInfo*>(ws + l.info);
  CE_TRY(scan_and_gather(a, l, ws, s, g, stream));

  unsigned short* slopes = reinterpret_cast<unsigned short*>(ws + l.slopes);
  SlopeTiles t{};
  CE_TRY(map_16bit(g.rows, bf16, l.rows, a.D, l.ld, kRows, &t.h));
  CE_TRY(map_16bit(a.W, bf16, a.V, a.D, a.W_stride, kRows, &t.w));
  CE_TRY(map_16bit(slopes, bf16, l.rows, l.piece, l.piece, kBoxRows, &t.out));
  t.status = a.status;
  t.bf16 = bf16;
  t.live = s.counts;
  t.info = g.info;
  t.corr = reinterpret_cast<float*>(ws + l.corr);
  t.rows = (int)l.rows;
  t.V = a.V;
  t.steps = div_up(a.D, kStep);

  GradTiles d{};
  CE_TRY(map_16bit(slopes, bf16, l.rows, l.piece, l.piece, kRows, &d.s_k));
  CE_TRY(map_16bit(slopes, bf16, l.rows, l.piece, l.piece, kStep, &d.s_mn));
  CE_TRY(map_16bit(a.W, bf16, a.V, a.D, a.W_stride, kStep, &d.w));
  CE_TRY(map_16bit(g.rows, bf16, l.rows, a.D, l.ld, kStep, &d.h));
  d.dh = d.dW = d.w;
  if (want_dh) CE_TRY(map_fp32(reinterpret_cast<float*>(ws + l.dh), l.splits, l.rows, a.D, &d.dh));
  if (want_dW) CE_TRY(map_16bit(a.dW, bf16, a.V, a.D, a.D, kBoxRows, &d.dW));
  d.status = a.status;
  d.bf16 = bf16;
  d.live = s.counts;
  d.rows = (int)l.rows;
  d.V = a.V;
  d.D = a.D;
  d.dt = div_up(a.D, 256);
  d.want_dh = want_dh;

  const long long mt = l.rows / 256;
  for (int v0 = 0; v0 < a.V; v0 += l.piece) {
    const int cols = std::min(l.piece, a.V - v0);
    t.v0 = d.v0 = v0;
    t.vtiles = div_up(cols, 256);
    d.kx = div_up(cols, kStep);
    d.wt = want_dW ? t.vtiles : 0;
    d.add = v0 > 0;
    CE_TRY(launch(t, (int)std::min<long long>(units, mt * t.vtiles), stream));
    CE_TRY(launch(d, units, stream));
  }
  if (!want_dh) return cudaSuccess;
  FinishParams f{reinterpret_cast<const float*>(ws + l.dh), l.rows, s.counts, s.slot, t.corr, g.info, g.W, a.W_stride, a.D,
                 static_cast<unsigned short*>(a.dh), g.own_scale ? a.g_loss : nullptr, a.g_lse};
  return small(bf16 ? ce_finish<true> : ce_finish<false>, a.N, 128, stream, f);
}

}  // namespace dspark
