// An update orthogonalised by Newton-Schulz products, as the Muon optimiser (Jordan
// et al., 2024) takes its steps: X_0 = M / (|M|_F + eps), then
//
//   A = X X^T,  B = b A + c A A,  X <- a X + B X        (`steps` times)
//
// with the Gram matrix on the shorter side (A = X^T X and X B for a tall M),
// which takes X's singular values through s -> a s + b s^3 + c s^5.
//
// Numbers.  A step multiplies the weakest directions by a = 3.4 and leaves the
// strongest where they are, so what rounding adds to X among the strong ones grows
// by up to 3.4 a step against them: with every product of bf16 operands the result
// is off by 1.2e-2 (2-norm, Gaussian 512 x 512).  Here the operands are fp16, scaled
// by 2^10 (an entry of X is at most 1 at first and its singular values stay
// near 1), and a X is added from X's high and low halves, 22 bits: 1.5e-3 of such
// a matrix, 2e-4 of a nearly low-rank one, below the 1.7e-3 that rounding the result
// to bf16 takes.  The shorter the Gram matrix's side, the less of this averages out
// (16 x 16: up to 3e-3), and the less a product's time depends on its length:
// up to kHalvesSide every operand is taken in halves, high x high + high x low +
// low x high, and the result is off by 1e-6 before its rounding.  Sums are fp32.
//
// The linear terms a X and b A are products too, with a diagonal tile as an operand
// (of X's halves with ones, of A with b / c in halves), so that no epilogue
// reads anything: its loads took 5 us of a tile for A, 10 for X, against 0.3 us for
// each step of 64 of K.  B is kept as B / a (of halves with a on its diagonal, so that
// X <- B X is all of the step).
//
// Measured (GB300, 5 steps): 4096 x 4096 1181 us (1.16 PFLOP/s of the symmetric
// count), bound by whole waves of tiles and 15 launches; 1000 x 777 115 us, 256 x 256
// 86 us, bound by latency; 151936 x 256 362 us, half of it at HBM's rate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "gemm_tc.cuh"

namespace dspark {
namespace {

using namespace gemm;

constexpr int kHalvesSide = 512;
constexpr float kScale = 1024.f, kInvScale = 1.f / 1024.f;   // of X, A and B in fp16

// ---------------------------------------------------------------------------
// the norm, and X_0
// ---------------------------------------------------------------------------
template <int kType>
__device__ __forceinline__ float load_value(const void* p, size_t i) {
  if constexpr (kType == DSPARK_F32) return static_cast<const float*>(p)[i];
  else if constexpr (kType == DSPARK_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return __half2float(static_cast<const __half*>(p)[i]);
}

// 4 values of a row from column c (4 | c): one load when `vec`, zeros past the end.
template <int kType>
__device__ __forceinline__ float4 load4(const void* base, size_t row, int c, int cols, bool vec) {
  if (vec && c + 4 <= cols) {
    if constexpr (kType == DSPARK_F32) {
      return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + row + c);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(base) + row + c);
      float2 u, v;
      if constexpr (kType == DSPARK_BF16) {
        u = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
        v = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
      } else {
        u = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
        v = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
      }
      return make_float4(u.x, u.y, v.x, v.y);
    }
  }
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = c + e < cols ? load_value<kType>(base, row + c + e) : 0.f;
  return make_float4(x[0], x[1], x[2], x[3]);
}

struct InputParams {
  const void* M;
  long long stride;
  int rows, cols;
  bool vec;             // rows of M start on 4 of its values
  bool flat;            // and M and the halves are dense arrays of whole fours
  float eps;
  double* partial;      // [blocks] sums of squares
  int* counters;        // cleared for the kernels that follow
  int blocks;
  __half *hi, *lo;      // [rows][ld]
  long long ld;
  __half* units;        // [3][256][256]: ones, b / c's halves on the diagonal
  float ratio;          // b / c
};

// Where the i-th four values of M and of the halves are.
struct Place {
  size_t row, to;       // of M's row and of the halves' four
  int c;
};
__device__ __forceinline__ Place place_of(const InputParams& p, long long i, int chunks) {
  if (p.flat) return Place{(size_t)i * 4, (size_t)i * 4, 0};   // (no division: 360 against 364 us of 151936 x 256)
  const long long r = i / chunks;
  const int c = (int)(i - r * chunks) * 4;
  return Place{(size_t)r * p.stride, (size_t)r * p.ld + c, c};
}

constexpr int kNormThreads = 256;
constexpr int kPrograms = 64;   // counters of programs
constexpr int kUnit = 256;   // side of a diagonal tile

// Four times four values of a thread's, kNormThreads apart and all loads first.
template <int kType, class F>
__device__ __forceinline__ void each_four(const InputParams& p, F f) {
  const int chunks = (p.cols + 3) / 4;
  const long long all = (long long)p.rows * chunks, step = (long long)gridDim.x * kNormThreads;
  long long i = (long long)blockIdx.x * kNormThreads + threadIdx.x;
  for (; i + 3 * step < all; i += 4 * step) {
    float4 v[4];
    Place at[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      at[u] = place_of(p, i + u * step, chunks);
      v[u] = load4<kType>(p.M, at[u].row, at[u].c, p.cols, p.vec);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) f(v[u], at[u]);
  }
  for (; i < all; i += step) {
    const Place at = place_of(p, i, chunks);
    f(load4<kType>(p.M, at.row, at.c, p.cols, p.vec), at);
  }
}

__device__ __forceinline__ float block_sum(float s, float* table) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
  __syncthreads();   // (the sums before have been read)
  if ((threadIdx.x & 31) == 0) table[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (int w = 0; w < kNormThreads / 32; ++w) s += table[w];
  return s;
}

// Sums of squares of values of any size.  A block whose plain sum lies in the middle
// of fp32's range has lost nothing that counts; another (of huge or tiny values, or
// of zeros) sums again in three ranges, each scaled so that no square leaves fp32's
// range.  The blocks' sums are joined in 64 bits.
template <int kType>
__global__ void __launch_bounds__(kNormThreads) ns_norm(const InputParams p) {
  __shared__ float table[kNormThreads / 32];
  pdl_trigger();
  pdl_wait();
  for (int i = blockIdx.x * kNormThreads + threadIdx.x; i < kPrograms; i += gridDim.x * kNormThreads) p.counters[i] = 0;
  float s = 0.f;
  each_four<kType>(p, [&](float4 v, const Place&) { s = fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, s)))); });
  s = block_sum(s, table);
  if (s > 0x1p-60f && s < 0x1p100f) {
    if (threadIdx.x == 0) p.partial[blockIdx.x] = (double)s;
    return;
  }
  float small = 0.f, middle = 0.f, large = 0.f;
  each_four<kType>(p, [&](float4 v, const Place&) {
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = fabsf(x[e]);
      if (t > 0x1p40f) large = fmaf(t * 0x1p-88f, t * 0x1p-88f, large);
      else if (t < 0x1p-40f) small = fmaf(t * 0x1p88f, t * 0x1p88f, small);
      else middle = fmaf(t, t, middle);   // (and NaN)
    }
  });
  small = block_sum(small, table);
  middle = block_sum(middle, table);
  large = block_sum(large, table);
  // (64-bit arithmetic is slow here: one thread's)
  if (threadIdx.x == 0) p.partial[blockIdx.x] = (double)middle + (double)large * 0x1p176 + (double)small * 0x1p-176;
}

// X_0 in high and low halves, and the diagonal tiles.
template <int kType>
__global__ void __launch_bounds__(kNormThreads) ns_split(const InputParams p) {
  __shared__ float factors[3];
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x < 32) {
    // (64-bit arithmetic is slow here: one warp's)
    double s = 0.0;
    for (int i = threadIdx.x; i < p.blocks; i += 32) s += p.partial[i];
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (threadIdx.x == 0) {
      s = (double)kScale / (sqrt(s) + (double)p.eps);
      // as a factor of fp32's range and a power of two in two halves (M may be as
      // small as fp32 goes)
      int e = 0;
      if (isfinite(s) && s > 0.0) s = frexp(s, &e);
      factors[0] = (float)s;
      factors[1] = ldexpf(1.f, e / 2);
      factors[2] = ldexpf(1.f, e - e / 2);
    }
  }
  const __half high = __float2half_rn(p.ratio * kScale), low = __float2half_rn(p.ratio * kScale - __half2float(high));
  for (int i = blockIdx.x * kNormThreads + threadIdx.x; i < kUnit * kUnit; i += gridDim.x * kNormThreads) {
    const bool on = i / kUnit == i % kUnit;
    const __half zero = __float2half_rn(0.f);
    p.units[i] = on ? __float2half_rn(kScale) : zero;
    p.units[kUnit * kUnit + i] = on ? high : zero;
    p.units[2 * kUnit * kUnit + i] = on ? low : zero;
  }
  __syncthreads();
  const float f = factors[0], p0 = factors[1], p1 = factors[2];
  each_four<kType>(p, [&](float4 v, const Place& at) {
    const float x[4] = {v.x * p0 * p1 * f, v.y * p0 * p1 * f, v.z * p0 * p1 * f, v.w * p0 * p1 * f};
    __half2 h[2], l[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      h[j] = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
      const float2 back = __half22float2(h[j]);
      l[j] = __floats2half2_rn(x[2 * j] - back.x, x[2 * j + 1] - back.y);
    }
    *reinterpret_cast<uint2*>(p.hi + at.to) = *reinterpret_cast<uint2*>(h);
    *reinterpret_cast<uint2*>(p.lo + at.to) = *reinterpret_cast<uint2*>(l);
  });
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------
enum Kind { kGram, kGramPart, kGramSelf, kSquare, kStepX, kLastX };

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// kGram    A = X X^T (or X^T X), lower tiles and their mirrors
// kGramPart  the same over a part of K, fp32;  kGramSelf  of one tile, from halves
// kSquare  B = b A + c A A, lower tiles and their mirrors
// kStepX   X' = a X + B X (or X B) in halves;  kLastX  in bf16
template <bool kPairs, int kTileN, Kind kKind>
struct NsTiles {
  static constexpr bool kPair = kPairs, kSelf = kKind == kGramSelf;
  static constexpr int kN = kTileN, kM = kPairs ? 256 : 128, kCols = kTileN / 4;
  static constexpr int kBoxBytes = kStoreBox, kExtraBytes = 0;
  static constexpr bool kSymmetric = kKind == kGram || kKind == kGramPart || kKind == kGramSelf || kKind == kSquare;
  using Counts = int;

  CUtensorMap left, left_low, right, right_low;
  CUtensorMap unit, unit_low;   // the diagonal tile's halves (low: kSquare)
  CUtensorMap out0, out1;   // stores of 64 columns a warp
  int* status;
  bool bf16;             // false: fp16 operands
  bool left_mn, right_mn;
  int rows, cols;        // of the product
  int mt, nt, steps, parts;
  int products;          // 1, or 3: high high, high low, low high
  int extra;             // products with the diagonal tile
  bool unit_is_left;
  const __half *in0, *in1;   // without the diagonal tile: A's halves, or X's (low: may be null); else null
  __half *to0, *to1;         // halves (low: may be null)
  __nv_bfloat16* out;
  long long ld, ld_out;  // of in and to (a multiple of 8); of out
  bool vec;              // out takes stores of 16 bytes
  float ca, cb, cc;      // of X, A and the product
  float diag;            // kSquare: added on the diagonal (times 2^10)

  __device__ void prefetch() const {
    for (const CUtensorMap* m : {&left, &left_low, &right, &right_low, &unit, &unit_low, &out0, &out1}) prefetch_tensormap(m);
  }
  __device__ void early(int, int) const {}
  __device__ void finish(int, const Epi&) const {}
  __device__ int counts() const { return 0; }
  __device__ int chunk(int) const { return kSelf ? 4 : 8; }
  __device__ bool used(int, const Tile&, int) const { return true; }
  __device__ bool tile(int, int unit, int units, int i, Tile& t) const {
    const int u = i * units + unit;
    constexpr int r = kM / kN > 0 ? kM / kN : 1;   // tiles of a row tile on the diagonal
    static_assert(kN <= kM, "square tiles or narrower");
    const int tiles = kSymmetric ? r * (mt * (mt + 1) / 2) : mt * nt;
    if (u >= tiles * parts) return false;
    const int part = u / tiles, v = u - part * tiles;
    int m, n;
    if (kSymmetric) {
      const int w = v / r;
      m = (int)((sqrtf(8.f * w + 1.f) - 1.f) * 0.5f);
      while (m * (m + 1) / 2 > w) --m;
      while ((m + 1) * (m + 2) / 2 <= w) ++m;
      n = v - r * (m * (m + 1) / 2);
    } else {
      m = v % mt;
      n = v / mt;
    }
    t.m0 = m * kM;
    t.n0 = n * kN;
    const int each = div_up(steps, parts);
    t.part = part;
    t.kind = max(0, min(each, steps - part * each));   // steps of one product
    t.k0 = part * each;
    t.steps = t.kind * products + extra * unit_steps();
    t.a_mn = left_mn;
    t.b_mn = right_mn;
    return true;
  }
  __device__ int unit_steps() const { return (unit_is_left ? kM : kN) / kStep; }
  __device__ int segments(const Tile&) const { return products + extra; }
  __device__ Segment segment(const Tile& t, int i) const {
    const int k = t.k0 * kStep;
    if (kSelf) return Segment{&left, &left_low, t.m0, k, t.n0, k, t.kind};
    if (i < products) return Segment{i == 2 ? &left_low : &left, i == 1 ? &right_low : &right, t.m0, k, t.n0, k, t.kind};
    const int u = i - products;
    if (unit_is_left) return Segment{&unit, u == 1 ? &right_low : &right, 0, 0, t.n0, t.m0, unit_steps()};
    // A with b / c, with its low half, A's low half with b / c; X's halves
    return Segment{(kKind == kSquare ? u == 2 : u == 1) ? &left_low : &left, kKind == kSquare && u == 1 ? &unit_low : &unit,
                   t.m0, t.n0, 0, 0, unit_steps()};
  }

  // 8 values of a row, zeros outside the matrix (whose rows are padded to 8)
  // and without one
  __device__ __forceinline__ void load8(const __half* p, int row, int col, float (&v)[8]) const {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (p != nullptr && row < rows && col < cols) w = *reinterpret_cast<const uint4*>(p + (size_t)row * ld + col);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&x[e]));
      v[2 * e] = u.x;
      v[2 * e + 1] = u.y;
    }
  }
  // v = f v, or v = f v + g in without the diagonal tile
  __device__ static __forceinline__ void scale(float (&v)[kCols], float f) {
#pragma unroll
    for (int j = 0; j < kCols; ++j) v[j] *= f;
  }
  __device__ __forceinline__ void add_linear(float (&v)[kCols], int row, int col, float f, float g) const {
#pragma unroll
    for (int j = 0; j < kCols; j += 8) {
      float hi[8], lo[8];
      load8(in0, row, col + j, hi);
      load8(in1, row, col + j, lo);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j + i] = fmaf(v[j + i], f, g * (hi[i] + lo[i]));
    }
  }
  __device__ static __forceinline__ void pack_high(const float (&v)[kCols], uint32_t (&w)[kCols / 2]) {
#pragma unroll
    for (int j = 0; j < kCols; j += 2) w[j / 2] = pack_half(v[j], v[j + 1]);
  }
  // what pack_high's rounding took (w: its result)
  __device__ static __forceinline__ void pack_low(const float (&v)[kCols], uint32_t (&w)[kCols / 2]) {
#pragma unroll
    for (int j = 0; j < kCols; j += 2) {
      const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&w[j / 2]));
      w[j / 2] = pack_half(v[j] - back.x, v[j + 1] - back.y);
    }
  }
  __device__ __forceinline__ void store_mirror(__half* p, const uint32_t (&w)[kCols / 2], int row, int col) const {
#pragma unroll
    for (int j = 0; j < kCols; j += 2) {
      const __half2 x = *reinterpret_cast<const __half2*>(&w[j / 2]);
      if (col + j < cols) p[(size_t)(col + j) * ld + row] = __low2half(x);
      if (col + j + 1 < cols) p[(size_t)(col + j + 1) * ld + row] = __high2half(x);
    }
  }
  // a thread's packed values into a matrix of 16-bit values, rows padded to 8
  template <class T>
  __device__ __forceinline__ void store_direct(T* p, long long stride, const uint32_t (&w)[kCols / 2], int row, int col) const {
    if (row >= rows) return;
#pragma unroll
    for (int j = 0; j < kCols / 8; ++j)
      if (col + 8 * j < cols)
        *reinterpret_cast<uint4*>(p + (size_t)row * stride + col + 8 * j) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
  __device__ __forceinline__ void store_half(const Epi& e, const Tile& t, const CUtensorMap* map, __half* p,
                                             const uint32_t (&w)[kCols / 2]) const {
    if constexpr (kCols == 64) store_16bit(e, map, w, t.n0 + e.col, cols, t.m0 + e.row0, rows);
    else store_direct(p, ld, w, t.m0 + e.row, t.n0 + e.col);
  }

  __device__ void epilogue(const Epi& e, const Tile& t, float (&v)[kCols]) const {
    const int row = t.m0 + e.row, col = t.n0 + e.col;
    uint32_t w[kCols / 2];
    if constexpr (kKind == kGramPart || kKind == kGramSelf) {
      static_assert(kCols == 64, "parts go out by boxes");
      store_fp32(e, &out0, v, col, cols, t.m0 + e.row0, rows, t.part, false);
      return;
    }
    if constexpr (kKind == kGram || kKind == kSquare) {
      if (kKind == kSquare && in0 != nullptr) add_linear(v, row, col, cc * kInvScale, cb);
      else scale(v, cc * kInvScale);
      if (kKind == kSquare && diag != 0.f) {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          if (col + j == row) v[j] += diag;
      }
      const bool mirror = t.n0 + kN <= t.m0 && row < rows;   // above the diagonal
      pack_high(v, w);
      store_half(e, t, &out0, to0, w);
      if (mirror) store_mirror(to0, w, row, col);
      if (to1 != nullptr) {
        pack_low(v, w);
        store_half(e, t, &out1, to1, w);
        if (mirror) store_mirror(to1, w, row, col);
      }
      return;
    }
    if constexpr (kKind == kStepX || kKind == kLastX) {
      if (in0 != nullptr) add_linear(v, row, col, kInvScale, ca);
      else scale(v, ca * kInvScale);
      if constexpr (kKind == kStepX) {
        pack_high(v, w);
        store_half(e, t, &out0, to0, w);
        pack_low(v, w);
        store_half(e, t, &out1, to1, w);
      } else {
#pragma unroll
        for (int j = 0; j < kCols; j += 2) w[j / 2] = pack_bf16(v[j] * kInvScale, v[j + 1] * kInvScale);
        if (vec) {
          if constexpr (kCols == 64) store_16bit(e, &out0, w, col, cols, t.m0 + e.row0, rows);
          else store_direct(out, ld_out, w, row, col);
        } else if (row < rows) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[j / 2]);
            if (col + j < cols) out[(size_t)row * ld_out + col + j] = j % 2 ? __high2bfloat16(x) : __low2bfloat16(x);
          }
        }
      }
    }
  }
};

// A from its parts (lower tiles of 256), whole.
struct JoinParams {
  const float* part;     // [parts][n][cols]
  int parts, n;
  long long cols, ld;
  __half *A, *low;       // halves (low: may be null)
};
// A row a block: 64 threads take 4 columns each, four groups of them every fourth part.
__global__ void __launch_bounds__(256) ns_join(const JoinParams p) {
  __shared__ float4 sums[3][64];
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x, g = threadIdx.x / 64, x = threadIdx.x % 64;
  const size_t plane = (size_t)p.n * p.cols;
  for (int c0 = 0; c0 < p.n && c0 / 256 <= r / 256; c0 += 256) {
    const int c = c0 + 4 * x;
    const bool on = c < p.n;   // (rows of the parts are padded to 8)
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* from = p.part + (size_t)r * p.cols + c;
    if (on) {
#pragma unroll 10
      for (int i = g; i < p.parts; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(from + i * plane);
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
    }
    __syncthreads();   // (the sums before have been read)
    if (g > 0) sums[g - 1][x] = s;
    __syncthreads();
    if (g > 0 || !on) continue;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const float4 v = sums[i][x];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    const float v[4] = {s.x * kInvScale, s.y * kInvScale, s.z * kInvScale, s.w * kInvScale};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c + j >= p.n) break;
      const __half h = __float2half_rn(v[j]), l = __float2half_rn(v[j] - __half2float(h));
      const size_t at = (size_t)r * p.ld + c + j, mirror = (size_t)(c + j) * p.ld + r;
      p.A[at] = h;
      if (p.low != nullptr) p.low[at] = l;
      if ((c + j) / 256 < r / 256) {
        p.A[mirror] = h;
        if (p.low != nullptr) p.low[mirror] = l;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// several products in one launch
//
// Products of a few hundred rows take 8 to 10 us each as kernels of their own,
// of which 2 are spent on K: the rest is the next kernel's start behind the last
// store, its first copies and its parameters.  Here persistent CTAs (a cooperative
// launch) go from product to product: a tile's stores are followed by an increment
// of a counter in global memory, and a product's copies wait until the counter
// shows all tiles that it reads (bounded, as every wait).  Tiles are 128 x 64, a
// CTA each.
// ---------------------------------------------------------------------------
constexpr int kMaxOps = 24, kMaxMaps = 32;   // of a launch
constexpr int kOpM = 128, kOpN = 64, kOpCols = kOpN / 4;
constexpr int kOpLeftBytes = kOpM * 128, kOpRightBytes = kOpN * 128, kOpStepBytes = kOpLeftBytes + kOpRightBytes;

// A stage of the ring holds a bundle, whose wait and commit its steps share.  Of
// halves: both operands' for one step of K, which three products use (or two steps
// of a product with a diagonal tile); else four steps.  Taken side by side, 256 x 256
// (halves) had 86 us by the first form and 92 by the second, 1000 x 777 112 and 105
// (on rows and tiles before the present ones, with which it has 115).
template <bool kHalves>
struct OpShape {
  static constexpr int kSlots = kHalves ? 2 : 4, kStages = kHalves ? 3 : 2;
  static constexpr int kStageBytes = kSlots * kOpStepBytes;
  // where the right operand's and the next slot's tiles are
  static constexpr int kRight = kHalves ? 2 * kOpLeftBytes : kOpLeftBytes;
  static constexpr int kLeftSlot = kHalves ? kOpLeftBytes : kOpStepBytes, kRightSlot = kHalves ? kOpRightBytes : kOpStepBytes;
  static constexpr int kRowsBytes = (kHalves ? 2 : 1) * kOpM * 128;
  static constexpr int kChunk = kHalves ? 3 : 2;   // bundles that an accumulator takes: 24 to 36 additions
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kRowsBytes + kBarBytes;
  static_assert(kSmem + 1024 + 24 * 160 <= kMaxSmem, "shared memory (and the static part)");
};

// One product of a program.  Its sum over K is that of segments, each a pair of
// maps and a number of steps: up to three products of halves, then up to three with
// a diagonal tile.
struct Op {
  short left, left_low, right, right_low;   // maps (low: of three products)
  short unit[3], of[3];        // maps of the diagonal tiles and of their other factors
  short products, extra, steps, unit_steps;   // steps: of a product's K
  bool left_mn, right_mn, unit_is_left, symmetric, vec;
  int rows, cols, mt, nt;
  int tiles;
  int base;                    // what the counter has to show first
  int first;                   // the CTA that takes its first item
  float scale, diag;           // result = scale sum + diag on the diagonal
  long long ld, ld_out;
  __half *to0, *to1;           // halves (low: may be null)
  __nv_bfloat16* out;          // or the last X
};

struct Program {
  CUtensorMap maps[kMaxMaps];
  Op ops[kMaxOps];
  int map_count, count;
  int* counter;                // tiles done
  int* status;
};

struct Item {
  int m0, n0;
};

__device__ __forceinline__ bool item_of(const Op& op, int unit, int units, int i, Item& t) {
  const int u = (unit >= op.first ? unit - op.first : unit + units - op.first) + i * units;
  if (u >= op.tiles) return false;
  int m, n;
  if (op.symmetric) {   // tiles on or below the diagonal: two more for each row tile
    const int w = u / 2;
    m = (int)((sqrtf(8.f * w + 1.f) - 1.f) * 0.5f);
    while (m * (m + 1) / 2 > w) --m;
    while ((m + 1) * (m + 2) / 2 <= w) ++m;
    n = u - m * (m + 1);
  } else {
    n = u / op.mt;
    m = u - n * op.mt;
  }
  t.m0 = m * kOpM;
  t.n0 = n * kOpN;
  return true;
}
// Bundles of a tile: of the operands' products, and of those with a diagonal tile
// (which follow the product's steps in its bundles when there are no halves).
struct Bundles {
  int main, more;
};
template <bool kHalves>
__device__ __forceinline__ Bundles bundles_of(const Op& op) {
  constexpr int kSlots = OpShape<kHalves>::kSlots;
  const int more = op.extra * op.unit_steps;
  return kHalves ? Bundles{op.steps, div_up(more, kSlots)} : Bundles{div_up(op.steps + more, kSlots), 0};
}

// Until `counter` shows `least`; a converged warp.  What other CTAs stored before
// they counted is seen by this warp's loads and its copies (the async proxy).
__device__ __forceinline__ bool wait_count(const int* counter, int least, volatile int* abort, int* status) {
  bool ok = true;
  uint64_t t0 = 0;
  for (unsigned polls = 0;; ++polls) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
    if (v >= least) break;
    if (polls % 256 != 255) continue;
    if (*abort) { ok = false; break; }
    const uint64_t now = globaltimer();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > kWaitLimitNs) {
      *abort = 1;
      record_status(status, DSPARK_ERR_TIMEOUT);
      ok = false;
      break;
    }
  }
  ok = __all_sync(0xffffffffu, ok);
  asm volatile("fence.proxy.async;" ::: "memory");
  return ok;
}

template <bool kHalves>
__global__ void __launch_bounds__(kThreads, 1) ns_program(const __grid_constant__ Program p) {
  using S = OpShape<kHalves>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* rows_s = smem + S::kStages * S::kStageBytes;   // a tile's rows on their way out
  Bars* bars = reinterpret_cast<Bars*>(rows_s + S::kRowsBytes);
  // (in shared memory: a read of the parameters that misses their small cache takes 200 cycles)
  __shared__ Op ops[kMaxOps];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int unit = blockIdx.x, units = gridDim.x;
  volatile int* abort = &bars->abort;
  for (int i = threadIdx.x; i < p.count * (int)(sizeof(Op) / 4); i += kThreads)
    reinterpret_cast<int*>(ops)[i] = reinterpret_cast<const int*>(p.ops)[i];
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) { mbar_init(&bars->full[s], 1); mbar_init(&bars->empty[s], 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(&bars->acc_full[s], 1); mbar_init(&bars->acc_empty[s], kEpiWarps); }
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bars->tmem_base, 2 * kOpN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    static_assert(kMaxMaps <= 32, "a lane each");
    if (lane < p.map_count) prefetch_tensormap(&p.maps[lane]);
    const uint32_t stages = smem_u32(smem);
    uint32_t i = 0, s = 0, phase = 1;
    bool ok = true;
    Item t;
    for (int o = 0; o < p.count && ok; ++o) {
      const Op& op = ops[o];
      const bool left_mn = op.left_mn, right_mn = op.right_mn;
      const CUtensorMap *l0 = &p.maps[op.left], *l1 = &p.maps[op.left_low], *r0 = &p.maps[op.right], *r1 = &p.maps[op.right_low];
      for (int n = 0; ok && item_of(op, unit, units, n, t); ++n) {
        if (n == 0 && op.base > 0 && !(ok = wait_count(p.counter, op.base, abort, p.status))) break;
        const Bundles all = bundles_of<kHalves>(op);
        // steps one by one: those left; segment, its steps left, maps and coordinates
        int left = (kHalves ? 0 : op.steps) + op.extra * op.unit_steps, q = kHalves ? 3 : 0, in = 0;
        const CUtensorMap *lm = nullptr, *rm = nullptr;
        int lr = 0, lk = 0, rr = 0, rk = 0;
        for (int k = 0; k < all.main + all.more; ++k, ++i) {
          ok = warp_wait(&bars->empty[s], phase, abort, p.status);
          if (!ok) break;
          uint32_t l = stages + s * S::kStageBytes, r = l + S::kRight;
          const uint32_t full = smem_u32(&bars->full[s]);
          // (one lane's are the copies alone, and a step needs no division: an issuing
          // loop that is longer shows in every product)
          if (kHalves && k < all.main) {
            const int at = k * kStep;
            if (elect_one()) {
              mbar_arrive_expect_tx(&bars->full[s], 2 * kOpStepBytes);
              const int lx = left_mn ? t.m0 : at, ly = left_mn ? at : t.m0, rx = right_mn ? t.n0 : at, ry = right_mn ? at : t.n0;
              copy_box<false>(l, l0, lx, ly, full);
              if (left_mn) copy_box<false>(l + 8192, l0, lx + 64, ly, full);
              copy_box<false>(r, r0, rx, ry, full);
              copy_box<false>(r + kOpRightBytes, r1, rx, ry, full);   // the low halves in the second slot
              copy_box<false>(l + kOpLeftBytes, l1, lx, ly, full);
              if (left_mn) copy_box<false>(l + kOpLeftBytes + 8192, l1, lx + 64, ly, full);
            }
            __syncwarp();
          } else {
            const int group = min(left, S::kSlots);
            left -= group;
            if (elect_one()) mbar_arrive_expect_tx(&bars->full[s], group * kOpStepBytes);
            __syncwarp();
            for (int g = 0; g < group; ++g, l += S::kLeftSlot, r += S::kRightSlot) {
              if (in == 0) {   // the next segment
                lr = t.m0;
                rr = t.n0;
                lk = rk = 0;
                if (q < op.products) {
                  in = op.steps;
                  lm = l0;
                  rm = r0;
                } else {
                  const int x = q - op.products;
                  in = op.unit_steps;
                  lm = &p.maps[op.unit_is_left ? op.unit[x] : op.of[x]];
                  rm = &p.maps[op.unit_is_left ? op.of[x] : op.unit[x]];
                  if (op.unit_is_left) lr = 0, lk = 0, rk = t.m0;
                  else lk = t.n0, rr = 0, rk = 0;
                }
                ++q;
              }
              // (the coordinate along K is the second one of an operand that is not K-major)
              if (elect_one()) {
                copy_box<false>(l, lm, left_mn ? lr : lk, left_mn ? lk : lr, full);
                if (left_mn) copy_box<false>(l + 8192, lm, lr + 64, lk, full);
                copy_box<false>(r, rm, right_mn ? rr : rk, right_mn ? rk : rr, full);
              }
              __syncwarp();
              --in;
              lk += kStep;
              rk += kStep;
            }
          }
          if (++s == S::kStages) s = 0, phase ^= 1;
        }
      }
    }
    if (lane == 0) {
      for (int s = 0; s < S::kStages; ++s) {
        const uint32_t n = (i + S::kStages - 1 - s) / S::kStages;
        if (n > 0) mbar_drain(&bars->empty[s], (n - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t base = (1u << 4) | ((uint32_t)(kOpN >> 3) << 17) | ((uint32_t)(kOpM >> 4) << 24);   // fp16
    const uint32_t stages = smem_u32(smem);
    uint32_t c = 0, s = 0, phase = 0;
    bool ok = true;
    Item t;
    for (int o = 0; o < p.count && ok; ++o) {
      const Op& op = ops[o];
      const uint32_t idesc = base | (op.left_mn ? kAMajorM : 0u) | (op.right_mn ? kBMajorN : 0u);
      const uint32_t da = op.left_mn ? 128 : 2, db = op.right_mn ? 128 : 2;
      const uint64_t ad0 = op.left_mn ? sw128_mnmajor_desc(stages, 8192) : sw128_kmajor_desc(stages);
      const uint64_t bd0 = op.right_mn ? sw128_mnmajor_desc(stages + S::kRight, 8192) : sw128_kmajor_desc(stages + S::kRight);
      const Bundles bundles = bundles_of<kHalves>(op);
      const int all = bundles.main + bundles.more;
      for (int n = 0; ok && item_of(op, unit, units, n, t); ++n) {
        for (int k = 0; k < all && ok; ++c) {
          const int buf = c & 1, kend = min(k + S::kChunk, all);
          ok = warp_wait(&bars->acc_empty[buf], ((c >> 1) & 1) ^ 1, abort, p.status);
          if (!ok) break;
          tc_fence_after();
          for (int kf = k; k < kend; ++k) {
            ok = warp_wait(&bars->full[s], phase, abort, p.status);
            if (!ok) break;
            tc_fence_after();
            uint64_t ad = ad0 + s * (S::kStageBytes / 16), bd = bd0 + s * (S::kStageBytes / 16);
            constexpr uint64_t a1 = S::kLeftSlot / 16, b1 = S::kRightSlot / 16;
            const uint32_t d = tmem + buf * kOpN;
            const int n = (kHalves ? S::kSlots * bundles.main : op.steps) + op.extra * op.unit_steps - S::kSlots * k;   // (of halves: behind the products)
            if (elect_one()) {
              if (kHalves) {
                const bool three = k < bundles.main;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_bf16(d, ad + kk * da, bd + kk * db, idesc, k != kf || kk != 0);
                if (three) {
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) {
                    umma_bf16(d, ad + kk * da, bd + b1 + kk * db, idesc, 1);
                    umma_bf16(d, ad + a1 + kk * da, bd + kk * db, idesc, 1);
                  }
                } else if (n > 1) {
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) umma_bf16(d, ad + a1 + kk * da, bd + b1 + kk * db, idesc, 1);
                }
              } else if (n >= S::kSlots) {
#pragma unroll
                for (int g = 0; g < S::kSlots; ++g) {
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    umma_bf16(d, ad + g * a1 + kk * da, bd + g * b1 + kk * db, idesc, g > 0 || kk > 0 || k != kf);
                }
              } else {
                for (int g = 0; g < n; ++g, ad += a1, bd += b1) {
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) umma_bf16(d, ad + kk * da, bd + kk * db, idesc, k != kf || g != 0 || kk != 0);
                }
              }
              umma_commit(&bars->empty[s]);
            }
            __syncwarp();
            if (++s == S::kStages) s = 0, phase ^= 1;
          }
          if (ok && elect_one()) umma_commit(&bars->acc_full[buf]);
          __syncwarp();
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, h = (warp - 2) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + h * kOpCols;
    uint32_t c = 0;
    bool ok = true;
    Item t;
    for (int o = 0; o < p.count; ++o) {
      const Op& op = ops[o];
      for (int n = 0; item_of(op, unit, units, n, t); ++n) {
        const Bundles bundles = bundles_of<kHalves>(op);
        const int chunks = div_up(bundles.main + bundles.more, S::kChunk);
        float v[kOpCols];
#pragma unroll
        for (int j = 0; j < kOpCols; ++j) v[j] = 0.f;
        for (int j = 0; j < chunks && ok; ++j, ++c) {
          const int buf = c & 1;
          ok = warp_wait(&bars->acc_full[buf], (c >> 1) & 1, abort, p.status);
          if (!ok) break;
          tc_fence_after();
          float x[kOpCols];
          tmem_load_cols<kOpCols>(lanes + buf * kOpN, x);
#pragma unroll
          for (int e = 0; e < kOpCols; ++e) v[e] += x[e];
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->acc_empty[buf]);
        }
        // (a warp whose wait gave up goes on through the barriers)
        const int row = t.m0 + q * 32 + lane, col = t.n0 + h * kOpCols;
#pragma unroll
        for (int j = 0; j < kOpCols; ++j) {
          v[j] *= op.scale;
          if (op.diag != 0.f && col + j == row) v[j] += op.diag;
        }
        uint32_t w[kOpCols / 2];
        unsigned char* mine = rows_s + q * 4096;   // (and 16 KB on for low halves)
        // this warp's 16 columns of 32 rows beside those of the other three, then
        // whole rows of 128 bytes: a store of a row a thread takes 32 turns, of 4 rows
        // a warp 4
        auto place = [&](unsigned char* at) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            *reinterpret_cast<uint4*>(at + lane * 128 + (((h * 2 + j) ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        };
        auto store_rows = [&](const unsigned char* at, void* to, long long ld) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = h * 8 + j * 4 + lane / 8, x = lane % 8, gr = t.m0 + q * 32 + r, gc = t.n0 + x * 8;
            const uint4 y = *reinterpret_cast<const uint4*>(at + r * 128 + ((x ^ (r & 7)) << 4));
            if (gr < op.rows && gc < op.cols)
              *reinterpret_cast<uint4*>(static_cast<unsigned short*>(to) + (size_t)gr * ld + gc) = y;
          }
        };
        if (op.out != nullptr) {
#pragma unroll
          for (int j = 0; j < kOpCols; j += 2) w[j / 2] = pack_bf16(v[j], v[j + 1]);
          if (op.vec) {
            place(mine);
            named_bar_sync(2 + q, 128);
            store_rows(mine, op.out, op.ld_out);
            named_bar_sync(2 + q, 128);   // (the next tile's rows take their place)
          } else if (row < op.rows) {
            unsigned short* dst = reinterpret_cast<unsigned short*>(op.out) + (size_t)row * op.ld_out + col;
#pragma unroll
            for (int j = 0; j < kOpCols; ++j)
              if (col + j < op.cols) dst[j] = (unsigned short)(j % 2 ? w[j / 2] >> 16 : w[j / 2]);
          }
          continue;
        }
        const bool mirror = !kHalves && op.symmetric && t.n0 + kOpN <= t.m0 && row < op.rows;
        auto store_mirror = [&](__half* to) {
#pragma unroll
          for (int j = 0; j < kOpCols; ++j)
            if (col + j < op.cols)
              reinterpret_cast<unsigned short*>(to)[(size_t)(col + j) * op.ld + row] =
                  (unsigned short)(j % 2 ? w[j / 2] >> 16 : w[j / 2]);
        };
        auto make_low = [&] {
#pragma unroll
          for (int j = 0; j < kOpCols; j += 2) {
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&w[j / 2]));
            w[j / 2] = pack_half(v[j] - back.x, v[j + 1] - back.y);
          }
        };
#pragma unroll
        for (int j = 0; j < kOpCols; j += 2) w[j / 2] = pack_half(v[j], v[j + 1]);
        place(mine);
        if (mirror) store_mirror(op.to0);
        if (kHalves && op.to1 != nullptr) {
          make_low();
          place(mine + kOpM * 128);
        }
        named_bar_sync(2 + q, 128);
        store_rows(mine, op.to0, op.ld);
        if (kHalves) {
          if (op.to1 != nullptr) store_rows(mine + kOpM * 128, op.to1, op.ld);
        } else if (op.to1 != nullptr) {   // (X's, in the place of the high ones)
          make_low();
          named_bar_sync(2 + q, 128);
          place(mine);
          if (mirror) store_mirror(op.to1);
          named_bar_sync(2 + q, 128);
          store_rows(mine, op.to1, op.ld);
        }
        // the tile is done: its stores are seen by who sees the counter (and, behind
        // the fence there, by copies, the async proxy)
        named_bar_sync(1, kEpiWarps * 32);
        if (threadIdx.x == 64) {
          asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p.counter) : "memory");
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * kOpN);
}

// ---------------------------------------------------------------------------
// workspace and launches
// ---------------------------------------------------------------------------
constexpr long long kPartBytes = 64ll << 20;
constexpr int kNormBlocks = 1216;    // 8 an SM

struct Layout {
  long long ld, lda, ldp;   // of X, of A and B, of the parts
  int small;                // the shorter side
  int parts;                // of the Gram matrix's K at most
  size_t partial, counters, units, x[2][2], A[2], B[2], more[4][2], part, total;
  bool halves;
};

// Rows start on 128 bytes: copies of rows that straddle such lines take half as long again.
long long pad_row(long long x) { return (x + 63) / 64 * 64; }

Layout layout(int rows, int cols) {
  Layout l{};
  l.small = std::min(rows, cols);
  l.ld = pad_row(cols);
  l.lda = l.ldp = pad_row(l.small);
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align256(bytes);
    return a;
  };
  l.partial = take(8ull * kNormBlocks);
  l.counters = take(4ull * (kPrograms));
  l.units = take(3 * 2ull * kUnit * kUnit);
  for (auto& half : l.x)
    for (auto& x : half) x = take(2ull * rows * l.ld);
  l.halves = l.small <= kHalvesSide;
  for (int i = 0; i <= (int)l.halves; ++i) {
    l.A[i] = take(2ull * l.small * l.lda);
    l.B[i] = take(2ull * l.small * l.lda);
    if (l.halves)
      for (auto& m : l.more) m[i] = take(2ull * l.small * l.lda);
  }
  l.parts = (int)std::min<long long>(76, kPartBytes / (4ll * l.small * l.ldp));
  if (l.parts > 1) l.part = take(4ull * l.parts * l.small * l.ldp);
  l.total = at;
  return l;
}

// Everything one product needs but the tile's shape.
struct Product {
  Kind kind;
  const __half *left, *left_low, *right, *right_low;   // operands (both low halves: three products)
  long long left_rows, left_cols, left_ld, right_rows, right_cols, right_ld;
  bool left_mn, right_mn;
  int rows, cols, K;
  const __half *unit, *unit_low;       // the diagonal tile's halves, or null
  int extra;
  bool unit_is_left;
  const __half *in0, *in1;
  __half *to0, *to1;
  long long ld;
  __nv_bfloat16* out;
  long long ld_out;
  float* part;
  long long ld_part;
  int parts;
  float a, b, c, diag;
  int* status;
};

#define NS_TRY(expr)                   \
  do {                                 \
    const cudaError_t _e = (expr);     \
    if (_e != cudaSuccess) return _e;  \
  } while (0)

template <bool kPairs, int kTileN, Kind kKind>
cudaError_t launch_product(const Product& q, cudaStream_t stream) {
  using P = NsTiles<kPairs, kTileN, kKind>;
  P p{};
  NS_TRY(map_16bit(q.left, false, q.left_rows, q.left_cols, q.left_ld, q.left_mn ? kStep : kRows, &p.left));
  NS_TRY(map_16bit(q.right, false, q.right_rows, q.right_cols, q.right_ld, q.right_mn ? kStep : Shape<P>::kBRows, &p.right));
  p.left_low = p.left;
  p.right_low = p.right;
  p.products = 1;
  if (q.left_low && q.right_low && kKind != kGramSelf) p.products = 3;
  if (q.left_low)
    NS_TRY(map_16bit(q.left_low, false, q.left_rows, q.left_cols, q.left_ld, q.left_mn ? kStep : kRows, &p.left_low));
  if (q.right_low)
    NS_TRY(map_16bit(q.right_low, false, q.right_rows, q.right_cols, q.right_ld, q.right_mn ? kStep : Shape<P>::kBRows,
                     &p.right_low));
  p.unit = p.unit_low = p.left;
  p.extra = q.unit ? q.extra : 0;
  p.unit_is_left = q.unit_is_left;
  if (p.extra) {
    const int box = q.unit_is_left ? kRows : Shape<P>::kBRows;
    NS_TRY(map_16bit(q.unit, false, kUnit, kUnit, kUnit, box, &p.unit));
    if (q.unit_low) NS_TRY(map_16bit(q.unit_low, false, kUnit, kUnit, kUnit, box, &p.unit_low));
  }
  p.status = q.status;
  p.bf16 = false;
  p.left_mn = q.left_mn;
  p.right_mn = q.right_mn;
  p.rows = q.rows;
  p.cols = q.cols;
  p.mt = div_up(q.rows, P::kM);
  p.nt = div_up(q.cols, P::kN);
  p.steps = div_up(q.K, kStep);
  constexpr bool kParts = kKind == kGramPart || kKind == kGramSelf;
  p.parts = kParts ? q.parts : 1;
  p.in0 = q.in0; p.in1 = q.in1;
  p.to0 = q.to0; p.to1 = q.to1;
  p.out = q.out;
  p.ld = q.ld;
  p.ld_out = q.ld_out;
  p.vec = kKind == kLastX && q.ld_out % 8 == 0 && q.cols % 8 == 0 && reinterpret_cast<uintptr_t>(q.out) % 16 == 0;
  p.ca = q.a; p.cb = q.b; p.cc = q.c;
  p.diag = q.diag;
  p.out0 = p.out1 = p.left;
  if (P::kCols == 64) {
    if (kParts) {
      NS_TRY(map_fp32(q.part, q.parts, q.rows, q.ld_part, &p.out0));
    } else if (kKind == kLastX) {
      if (p.vec) NS_TRY(map_16bit(q.out, true, q.rows, q.cols, q.ld_out, kBoxRows, &p.out0));
    } else {
      NS_TRY(map_16bit(q.to0, false, q.rows, q.cols, q.ld, kBoxRows, &p.out0));
      if (q.to1) NS_TRY(map_16bit(q.to1, false, q.rows, q.cols, q.ld, kBoxRows, &p.out1));
    }
  }
  const int units = max_units<P>();
  if (units <= 0) return cudaErrorUnknown;
  const long long tiles = (P::kSymmetric ? (long long)(P::kM / P::kN) * p.mt * (p.mt + 1) / 2 : (long long)p.mt * p.nt) * p.parts;
  return launch(p, (int)std::min<long long>(units, tiles), stream);
}

template <Kind kKind>
cudaError_t choose_product(const Product& q, int sms, cudaStream_t stream) {
  // Time of a product by tiles of a shape (us): the waves' steps of K, and the
  // launch, its first copies and last epilogue.  Measured, fp16: the Gram matrix of
  // 4096 x 4096 by tiles of 256 x 256, 128 x 128, 128 x 64: 56, 77 and 118; of
  // 1024 x 1024: 16, 11 and 9.
  constexpr bool sym = kKind == kGram || kKind == kSquare;
  auto cost = [&](int tm, int tn, int units, double step, double more) {
    const double mt = div_up(q.rows, tm), nt = div_up(q.cols, tn);
    const double tiles = sym ? (double)tm / tn * mt * (mt + 1) / 2 : mt * nt;
    return std::max(1.0, std::ceil(tiles / units)) * div_up(q.K, kStep) * (q.left_low && q.right_low ? 3 : 1) * step + more;
  };
  const double big = cost(256, 256, sms / 2, 0.36, 9.0), mid = cost(128, 128, sms, 0.28, 6.5),
               low = cost(128, 64, sms, 0.25, 5.0);
  if (big <= mid && big <= low) return launch_product<true, 256, kKind>(q, stream);
  if (mid <= low) return launch_product<false, 128, kKind>(q, stream);
  return launch_product<false, 64, kKind>(q, stream);
}

// A matrix in fp16 halves (low: may be null).
struct Halves {
  __half *hi, *lo;
  long long rows, cols, ld;
};

// Builds programs and launches them when they are full or done.
struct Builder {
  Program p{};
  int tiles = 0, items = 0, programs = 0;
  int* counters;
  int* status;
  int sms;
  cudaStream_t stream;
  cudaError_t error = cudaSuccess;

  bool halves;   // of every op's operands

  Builder(bool halves, int* counters, int* status, int sms, cudaStream_t stream)
      : counters(counters), status(status), sms(sms), stream(stream), halves(halves) {}

  void start() {
    p.map_count = p.count = 0;
    tiles = items = 0;
  }
  short map(const __half* base, long long rows, long long cols, long long ld, int box) {
    for (int i = 0; i < p.map_count; ++i)
      if (base_[i] == base && box_[i] == box) return (short)i;
    if (p.map_count == kMaxMaps) {
      error = cudaErrorInvalidValue;
      return 0;
    }
    const cudaError_t e = map_16bit(base, false, rows, cols, ld, box, &p.maps[p.map_count]);
    if (e != cudaSuccess) error = e;
    base_[p.map_count] = base;
    box_[p.map_count] = box;
    return (short)p.map_count++;
  }
  short left(const __half* base, const Halves& m, bool mn) { return map(base, m.rows, m.cols, m.ld, mn ? kStep : kOpM); }
  short right(const __half* base, const Halves& m) { return map(base, m.rows, m.cols, m.ld, kOpN); }

  // The product of two matrices (three products where both have low halves).
  Op& add(const Halves& l, bool l_mn, const Halves& r, bool r_mn, int rows, int cols, int K, bool symmetric) {
    Op& op = p.ops[p.count++];
    op = Op{};
    op.products = l.lo && r.lo ? 3 : 1;
    op.left = left(l.hi, l, l_mn);
    op.right = right(r.hi, r);
    if (op.products == 3) {
      op.left_low = left(l.lo, l, l_mn);
      op.right_low = right(r.lo, r);
    }
    op.left_mn = l_mn;
    op.right_mn = r_mn;
    op.rows = rows;
    op.cols = cols;
    op.steps = (short)div_up(K, kStep);
    op.mt = div_up(rows, kOpM);
    op.nt = div_up(cols, kOpN);
    // (the tiles above the diagonal where there are SMs for them, as for all operands in
    // halves, at most 512 x 512: mirroring takes longer)
    op.symmetric = symmetric && !halves && op.mt * op.nt > sms;
    op.tiles = op.symmetric ? op.mt * (op.mt + 1) : op.mt * op.nt;
    op.base = tiles;
    op.scale = kInvScale;
    return op;
  }
  // After everything about the op but its place is known.
  void place(Op& op) {
    tiles += op.tiles;
    items = std::max(items, op.tiles);
  }
  void into(Op& op, const Halves& to) {
    op.to0 = to.hi;
    op.to1 = to.lo;
    op.ld = to.ld;
    place(op);
  }
  bool room(int ops) const { return p.count + ops <= kMaxOps; }

  cudaError_t launch() {
    if (error != cudaSuccess || p.count == 0) return error;
    if (programs == kPrograms) return cudaErrorInvalidValue;
    p.counter = counters + programs++;
    p.status = status;
    auto kern = halves ? ns_program<true> : ns_program<false>;
    const int smem = halves ? OpShape<true>::kSmem : OpShape<false>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min(sms, items));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // its CTAs wait for one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    start();
    return e;
  }

 private:
  const __half* base_[kMaxMaps];
  int box_[kMaxMaps];
};

template <int kType>
cudaError_t launch_input(const InputParams& p, cudaStream_t stream) {
  ns_norm<kType><<<p.blocks, kNormThreads, 0, stream>>>(p);
  NS_TRY(cudaGetLastError());
  return launch_pdl(ns_split<kType>, dim3((unsigned)p.blocks), dim3(kNormThreads), 0, stream, p);
}

}  // namespace

size_t newton_schulz_workspace_bytes(int rows, int cols) { return layout(rows, cols).total; }

cudaError_t launch_newton_schulz(const NewtonSchulzArgs& a, cudaStream_t stream) {
  const Layout l = layout(a.rows, a.cols);
  char* ws = static_cast<char*>(a.ws);
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  __half* x[2][2];
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) x[i][j] = reinterpret_cast<__half*>(ws + l.x[i][j]);
  __half *A[2] = {}, *B[2] = {};
  for (int i = 0; i <= (int)l.halves; ++i) {
    A[i] = reinterpret_cast<__half*>(ws + l.A[i]);
    B[i] = reinterpret_cast<__half*>(ws + l.B[i]);
  }

  InputParams in{};
  in.M = a.M;
  in.stride = a.row_stride;
  in.rows = a.rows;
  in.cols = a.cols;
  const int size = a.dtype == DSPARK_F32 ? 4 : 2;
  in.vec = reinterpret_cast<uintptr_t>(a.M) % (4 * size) == 0 && (a.rows == 1 || a.row_stride % 4 == 0);
  in.flat = in.vec && a.cols % 4 == 0 && l.ld == a.cols && (a.rows == 1 || a.row_stride == a.cols);
  in.eps = a.eps;
  in.partial = reinterpret_cast<double*>(ws + l.partial);
  in.blocks = (int)std::min<long long>(kNormBlocks, ((long long)a.rows * ((a.cols + 3) / 4) + kNormThreads - 1) / kNormThreads);
  in.hi = x[0][0];
  in.lo = x[0][1];
  in.ld = l.ld;
  in.counters = reinterpret_cast<int*>(ws + l.counters);
  in.units = reinterpret_cast<__half*>(ws + l.units);
  // the linear terms are products with a diagonal tile as long as all its
  // values and B / a stay well within fp16, else an epilogue adds them
  const float most = 16.f;
  const bool fold = std::fabs(a.b) <= most * std::fabs(a.c) && std::fabs(a.b) <= most * std::fabs(a.a) &&
                    std::fabs(a.c) <= most * std::fabs(a.a) && a.a != 0.f && a.c != 0.f;
  in.ratio = fold ? a.b / a.c : 0.f;
  if (a.dtype == DSPARK_F32) NS_TRY(launch_input<DSPARK_F32>(in, stream));
  else if (a.dtype == DSPARK_BF16) NS_TRY(launch_input<DSPARK_BF16>(in, stream));
  else NS_TRY(launch_input<DSPARK_F16>(in, stream));

  const bool tall = a.rows > a.cols;
  const int small = l.small, large = std::max(a.rows, a.cols);
  const Halves mA{A[0], A[1], small, small, l.lda}, mB{B[0], B[1], small, small, l.lda};
  auto X = [&](int i, bool low) { return Halves{x[i & 1][0], low ? x[i & 1][1] : nullptr, a.rows, a.cols, l.ld}; };
  const Halves one{in.units, nullptr, kUnit, kUnit, kUnit}, ratio{in.units + kUnit * kUnit, in.units + 2 * kUnit * kUnit, kUnit, kUnit, kUnit};
  Builder build(l.halves, in.counters, a.status, sms, stream);
  // b A + c A A + diag: b / c A by the diagonal tile
  auto square = [&](const Halves& from, const Halves& to, float c, float diag) {
    Op& op = build.add(from, false, from, false, small, small, small, true);
    op.extra = l.halves ? 3 : 2;
    op.unit_steps = kOpN / kStep;
    op.of[0] = op.of[1] = op.left;
    op.unit[0] = op.unit[2] = build.right(ratio.hi, ratio);
    op.unit[1] = build.right(ratio.lo, ratio);
    op.of[2] = op.left_low;
    op.scale = c * kInvScale;
    op.diag = diag * kScale;
    build.into(op, to);
  };
  // Everything in one launch, or by groups of steps, or product by product.
  // Measured side by side (us; the first form before its bundles), in that order:
  // 256 x 256: 92, 114, 123; 256 x 512: 103, 119, 137; 512 x 1000: 195, 167, 197; 64 x 4000: 175, 119, 164; 16000 x 256: 466,
  // 169, 240; without halves 1000 x 777: 109, -, 129; 2048 x 2048: 359, -, 411;
  // 1536 x 1536: 234, -, 222; 3000 x 3000 product by product 603.
  const long long x_tiles = (long long)div_up(a.rows, kOpM) * div_up(a.cols, kOpN);
  const bool in_order = fold && (l.halves ? large <= 2 * small && x_tiles < 64 : x_tiles <= 4 * sms);

  if (in_order) {
    // everything in one launch (of 8 steps each)
    for (int i = 0; i < a.steps; ++i) {
      if (!build.room(3)) NS_TRY(build.launch());
      // A
      Op& gram = build.add(X(i, l.halves), tall, X(i, l.halves), tall, small, small, large, true);
      build.into(gram, mA);
      // B: with a on its diagonal, or divided by a
      square(mA, mB, l.halves ? a.c : a.c / a.a, l.halves ? a.a : 0.f);
      // X
      Op& op = tall ? build.add(X(i, l.halves), false, mB, false, a.rows, a.cols, small, false)
                    : build.add(mB, false, X(i, l.halves), true, a.rows, a.cols, small, false);
      if (!l.halves) {
        const Halves from = X(i, true);
        op.extra = 2;
        op.unit_is_left = !tall;
        op.unit_steps = (tall ? kOpN : kOpM) / kStep;
        op.unit[0] = op.unit[1] = tall ? build.right(one.hi, one) : build.left(one.hi, one, false);
        op.of[0] = tall ? build.left(from.hi, from, false) : build.right(from.hi, from);
        op.of[1] = tall ? build.left(from.lo, from, false) : build.right(from.lo, from);
        op.scale *= a.a;
      }
      if (i + 1 < a.steps) {
        build.into(op, X(i + 1, true));
      } else {
        op.out = static_cast<__nv_bfloat16*>(a.out);
        op.ld_out = a.cols;
        op.vec = a.cols % 8 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
        op.scale *= kInvScale;
        build.place(op);
      }
    }
    return build.launch();
  }

  Product q{};
  q.status = a.status;
  // A by parts of K, where the tiles of 256 leave most pairs idle and each part is still 16 steps or more
  auto gram_parts = [&] {
    const int mt = div_up(small, 256), tiles = mt * (mt + 1) / 2;
    return std::min({l.parts, sms / 2 / tiles, div_up(large, kStep) / 16});
  };
  auto gram = [&](const Halves& from) {
    q.unit = q.unit_low = q.in0 = q.in1 = nullptr;
    q.diag = 0.f;
    q.c = 1.f;
    q.left = q.right = from.hi;
    q.left_low = q.right_low = from.lo;
    q.left_rows = q.right_rows = a.rows;
    q.left_cols = q.right_cols = a.cols;
    q.left_ld = q.right_ld = l.ld;
    q.left_mn = q.right_mn = tall;
    q.rows = q.cols = small;
    q.K = large;
    q.to0 = A[0];
    q.to1 = A[1];
    q.ld = l.lda;
    q.parts = gram_parts();
    if (q.parts <= 1) return choose_product<kGram>(q, sms, stream);
    q.part = reinterpret_cast<float*>(ws + l.part);
    q.ld_part = l.ldp;
    // (of one tile's halves each is read once, not three times)
    if (from.lo && small <= 256) NS_TRY((launch_product<true, 256, kGramSelf>(q, stream)));
    else NS_TRY((launch_product<true, 256, kGramPart>(q, stream)));
    JoinParams j{q.part, q.parts, small, l.ldp, l.lda, A[0], A[1]};
    return launch_pdl(ns_join, dim3((unsigned)small), dim3(256), 0, stream, j);
  };
  // X' = X P or P X
  auto times = [&](const Halves& from, const Halves& P, int i, bool last) {
    Product s = q;
    if (tall) {
      s.left = from.hi; s.left_low = from.lo; s.left_rows = a.rows; s.left_cols = a.cols; s.left_ld = l.ld;
      s.right = P.hi; s.right_low = P.lo; s.right_rows = s.right_cols = small; s.right_ld = l.lda;
      s.right_mn = false;
    } else {
      s.left = P.hi; s.left_low = P.lo; s.left_rows = s.left_cols = small; s.left_ld = l.lda;
      s.right = from.hi; s.right_low = from.lo; s.right_rows = a.rows; s.right_cols = a.cols; s.right_ld = l.ld;
      s.right_mn = true;
    }
    s.left_mn = false;
    s.unit = s.unit_low = s.in0 = s.in1 = nullptr;
    s.rows = a.rows;
    s.cols = a.cols;
    s.K = small;
    s.a = a.a;
    if (l.halves) {
      s.a = 1.f;
    } else if (fold) {
      s.unit = in.units;
      s.extra = 2;
      s.unit_is_left = !tall;
    }
    if (!fold) {
      s.a = a.a;
      s.in0 = from.hi;
      s.in1 = from.lo;
    }
    s.ld = l.ld;
    s.to0 = x[1 - (i & 1)][0];
    s.to1 = x[1 - (i & 1)][1];
    if (!last) return choose_product<kStepX>(s, sms, stream);
    s.out = static_cast<__nv_bfloat16*>(a.out);
    s.ld_out = a.cols;
    return choose_product<kLastX>(s, sms, stream);
  };

  // A long X is read and written once for several steps: X_k = X_0 P with P a
  // polynomial in A alone, whose products are small.  By two and three steps at a
  // time A's error stays far below what matters (2e-5 of nearly singular
  // updates; by five at a time they diverge), so every group of steps starts
  // from the Gram matrix of its own X.
  const bool in_groups = fold && l.halves && std::fabs(a.a) < 3.9f;   // (P's values, up to a^3, stay within fp16)
  if (in_groups) {
    const Halves T{reinterpret_cast<__half*>(ws + l.more[0][0]), reinterpret_cast<__half*>(ws + l.more[0][1]), small, small, l.lda};
    const Halves A2{reinterpret_cast<__half*>(ws + l.more[1][0]), reinterpret_cast<__half*>(ws + l.more[1][1]), small, small, l.lda};
    const Halves P[2] = {{reinterpret_cast<__half*>(ws + l.more[2][0]), reinterpret_cast<__half*>(ws + l.more[2][1]), small, small, l.lda},
                         {reinterpret_cast<__half*>(ws + l.more[3][0]), reinterpret_cast<__half*>(ws + l.more[3][1]), small, small, l.lda}};
    auto small_product = [&](const Halves& left, const Halves& right, const Halves& to) -> Op& {
      Op& op = build.add(left, false, right, false, small, small, small, true);
      build.into(op, to);
      return op;
    };
    const int groups = (a.steps + 2) / 3;
    for (int g = 0, left = a.steps; g < groups; ++g) {
      const int n = left / (groups - g);   // (the earlier ones, where X is worst conditioned, are the shorter ones)
      left -= n;
      NS_TRY(gram(X(g, true)));
      const Halves* from = &mA;
      int at = 0;                          // P's buffer
      for (int k = 0; k < n; ++k) {
        const Halves& Q = k == 0 ? P[0] : mB;
        square(*from, Q, a.c, a.a);
        if (k + 1 < n) {
          const Halves* to = from == &mA ? &A2 : &mA;
          Op& t = small_product(*from, Q, T);
          if (k > 0) {
            // beside it, by the CTAs that it leaves idle
            Op& p = small_product(P[at], Q, P[1 - at]);
            build.items = std::max(build.items, 2 * t.tiles);
            p.base = t.base;
            p.first = t.tiles % std::min(sms, build.items);
            at = 1 - at;
          }
          small_product(T, Q, *to);
          from = to;
        } else if (k > 0) {
          small_product(P[at], Q, P[1 - at]);
          at = 1 - at;
        }
      }
      NS_TRY(build.launch());
      NS_TRY(times(X(g, true), P[at], g, g + 1 == groups));
    }
    return cudaSuccess;
  }

  for (int i = 0; i < a.steps; ++i) {
    NS_TRY(gram(X(i, l.halves)));
    // B: with a on its diagonal, or divided by a
    q.left = q.right = A[0];
    q.left_low = q.right_low = A[1];
    q.left_rows = q.right_rows = q.left_cols = q.right_cols = small;
    q.left_ld = q.right_ld = l.lda;
    q.left_mn = q.right_mn = false;
    q.K = small;
    if (fold) {
      q.unit = ratio.hi;
      q.unit_low = ratio.lo;
      q.extra = l.halves ? 3 : 2;
      q.unit_is_left = false;
      q.c = l.halves ? a.c : a.c / a.a;
      q.diag = l.halves ? a.a * kScale : 0.f;
    } else {
      q.in0 = A[0];
      q.in1 = A[1];
      q.b = a.b;
      q.c = a.c;
    }
    q.to0 = B[0];
    q.to1 = B[1];
    NS_TRY(choose_product<kSquare>(q, sms, stream));
    NS_TRY(times(X(i, true), mB, i, i + 1 == a.steps));
  }
  return cudaSuccess;
}

}  // namespace dspark
