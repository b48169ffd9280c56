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
// each step of 64 of K.  B is kept as B / a.
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
  float eps;
  double* partial;      // [blocks] sums of squares
  int blocks;
  __half *hi, *lo;      // [rows][ld]
  long long ld;
  __half* units;        // [3][256][256]: ones, b / c's halves on the diagonal
  float ratio;          // b / c
};

constexpr int kNormThreads = 256;
constexpr int kUnit = 256;   // side of a diagonal tile

__device__ __forceinline__ double block_sum(double v, double* table) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) table[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kNormThreads / 32; ++w) s += table[w];
  return s;
}

// Sums of squares of values of any size: fp32 sums of three ranges, each scaled
// so that no square leaves fp32's range, joined in 64 bits.
template <int kType>
__global__ void __launch_bounds__(kNormThreads) ns_norm(const InputParams p) {
  __shared__ double table[kNormThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int chunks = (p.cols + 3) / 4;
  const long long all = (long long)p.rows * chunks;
  float small = 0.f, middle = 0.f, large = 0.f;
#pragma unroll 4
  for (long long i = (long long)blockIdx.x * kNormThreads + threadIdx.x; i < all; i += (long long)gridDim.x * kNormThreads) {
    const long long r = i / chunks;
    const float4 v = load4<kType>(p.M, (size_t)r * p.stride, (int)(i - r * chunks) * 4, p.cols, p.vec);
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = fabsf(x[e]);
      if (t > 0x1p40f) large = fmaf(t * 0x1p-88f, t * 0x1p-88f, large);
      else if (t < 0x1p-40f) small = fmaf(t * 0x1p88f, t * 0x1p88f, small);
      else middle = fmaf(t, t, middle);   // (and NaN)
    }
  }
  const double s = block_sum((double)middle + (double)large * 0x1p176 + (double)small * 0x1p-176, table);
  if (threadIdx.x == 0) p.partial[blockIdx.x] = s;
}

// X_0 in high and low halves, and the diagonal tiles.
template <int kType>
__global__ void __launch_bounds__(kNormThreads) ns_split(const InputParams p) {
  __shared__ double table[kNormThreads / 32];
  pdl_trigger();
  pdl_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < p.blocks; i += kNormThreads) s += p.partial[i];
  s = (double)kScale / (sqrt(block_sum(s, table)) + (double)p.eps);
  const __half high = __float2half_rn(p.ratio * kScale), low = __float2half_rn(p.ratio * kScale - __half2float(high));
  for (int i = blockIdx.x * kNormThreads + threadIdx.x; i < kUnit * kUnit; i += gridDim.x * kNormThreads) {
    const bool on = i / kUnit == i % kUnit;
    const __half zero = __float2half_rn(0.f);
    p.units[i] = on ? __float2half_rn(kScale) : zero;
    p.units[kUnit * kUnit + i] = on ? high : zero;
    p.units[2 * kUnit * kUnit + i] = on ? low : zero;
  }
  // s as a factor of fp32's range and a power of two in two halves (M may be
  // as small as fp32 goes)
  int e = 0;
  if (isfinite(s) && s > 0.0) s = frexp(s, &e);
  const int e0 = e / 2;
  const float f = (float)s, p0 = ldexpf(1.f, e0), p1 = ldexpf(1.f, e - e0);
  const int chunks = (p.cols + 3) / 4;
  const long long all = (long long)p.rows * chunks;
#pragma unroll 4
  for (long long i = (long long)blockIdx.x * kNormThreads + threadIdx.x; i < all; i += (long long)gridDim.x * kNormThreads) {
    const long long r = i / chunks;
    const int c = (int)(i - r * chunks) * 4;
    const float4 v = load4<kType>(p.M, (size_t)r * p.stride, c, p.cols, p.vec);
    const float x[4] = {v.x * p0 * p1 * f, v.y * p0 * p1 * f, v.z * p0 * p1 * f, v.w * p0 * p1 * f};
    __half2 h[2], l[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      h[j] = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
      const float2 back = __half22float2(h[j]);
      l[j] = __floats2half2_rn(x[2 * j] - back.x, x[2 * j + 1] - back.y);
    }
    *reinterpret_cast<uint2*>(p.hi + (size_t)r * p.ld + c) = *reinterpret_cast<uint2*>(h);
    *reinterpret_cast<uint2*>(p.lo + (size_t)r * p.ld + c) = *reinterpret_cast<uint2*>(l);
  }
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------
enum Kind { kGram, kGramPart, kSquare, kStepX, kLastX };

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// kGram    A = X X^T (or X^T X), lower tiles and their mirrors
// kGramPart  the same over a part of K, fp32
// kSquare  B = b A + c A A, lower tiles and their mirrors
// kStepX   X' = a X + B X (or X B) in halves;  kLastX  in bf16
template <bool kPairs, int kTileN, Kind kKind>
struct NsTiles {
  static constexpr bool kPair = kPairs;
  static constexpr int kN = kTileN, kM = kPairs ? 256 : 128, kCols = kTileN / 4;
  static constexpr int kBoxBytes = kStoreBox, kExtraBytes = 0;
  static constexpr bool kSymmetric = kKind == kGram || kKind == kGramPart || kKind == kSquare;
  using Counts = int;

  CUtensorMap left, left_low, right, right_low;
  CUtensorMap unit, unit_low;   // the diagonal tile's halves (low: kSquare)
  CUtensorMap out0, out1;   // stores of 64 columns a warp
  int* status;
  bool bf16;             // false: fp16 operands
  int chunk;
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

  __device__ void prefetch() const {
    for (const CUtensorMap* m : {&left, &left_low, &right, &right_low, &unit, &unit_low, &out0, &out1}) prefetch_tensormap(m);
  }
  __device__ int counts() const { return 0; }
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
    t.kind = max(1, min(each, steps - part * each));   // steps of one product
    t.k0 = part * each;
    t.steps = max(0, min(each, steps - t.k0)) * products + extra * unit_steps();
    t.a_mn = left_mn;
    t.b_mn = right_mn;
    return true;
  }
  __device__ int unit_steps() const { return (unit_is_left ? kM : kN) / kStep; }
  __device__ Src a(const Tile& t, int k) const {
    const int q = k / t.kind;
    if (q < products) return Src{q == 2 ? &left_low : &left, t.m0, (t.k0 + k - q * t.kind) * kStep};
    k -= products * t.kind;
    const int u = k / unit_steps(), j = (k - u * unit_steps()) * kStep;
    if (unit_is_left) return Src{&unit, 0, j};
    // A with b / c, its low half, A's low half with b / c; X's halves
    return Src{(kKind == kSquare ? u == 2 : u == 1) ? &left_low : &left, t.m0, t.n0 + j};
  }
  __device__ Src b(const Tile& t, int k) const {
    const int q = k / t.kind;
    if (q < products) return Src{q == 1 ? &right_low : &right, t.n0, (t.k0 + k - q * t.kind) * kStep};
    k -= products * t.kind;
    const int u = k / unit_steps(), j = (k - u * unit_steps()) * kStep;
    if (unit_is_left) return Src{u == 1 ? &right_low : &right, t.n0, t.m0 + j};
    return Src{kKind == kSquare && u == 1 ? &unit_low : &unit, 0, j};
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
    if constexpr (kKind == kGramPart) {
      static_assert(kCols == 64, "parts go out by boxes");
      store_fp32(e, &out0, v, col, cols, t.m0 + e.row0, rows, t.part, false);
      return;
    }
    if constexpr (kKind == kGram || kKind == kSquare) {
      if (kKind == kSquare && in0 != nullptr) add_linear(v, row, col, cc * kInvScale, cb);
      else scale(v, cc * kInvScale);
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
__global__ void __launch_bounds__(256) ns_join(const JoinParams p) {
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.y * 16 + threadIdx.x / 16, c = blockIdx.x * 16 + threadIdx.x % 16;
  if (r >= p.n || c >= p.n || c / 256 > r / 256) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = 0; i < p.parts; ++i) s += p.part[((size_t)i * p.n + r) * p.cols + c];
  s *= kInvScale;
  const __half h = __float2half_rn(s), l = __float2half_rn(s - __half2float(h));
  const size_t at = (size_t)r * p.ld + c, mirror = (size_t)c * p.ld + r;
  p.A[at] = h;
  if (p.low != nullptr) p.low[at] = l;
  if (c / 256 < r / 256) {
    p.A[mirror] = h;
    if (p.low != nullptr) p.low[mirror] = l;
  }
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
  size_t partial, units, x[2][2], A[2], B[2], part, total;
  bool halves;
};

long long pad8(long long x) { return (x + 7) / 8 * 8; }

Layout layout(int rows, int cols) {
  Layout l{};
  l.small = std::min(rows, cols);
  l.ld = pad8(cols);
  l.lda = l.ldp = pad8(l.small);
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align256(bytes);
    return a;
  };
  l.partial = take(8ull * kNormBlocks);
  l.units = take(3 * 2ull * kUnit * kUnit);
  for (auto& half : l.x)
    for (auto& x : half) x = take(2ull * rows * l.ld);
  l.halves = l.small <= kHalvesSide;
  for (int i = 0; i <= (int)l.halves; ++i) {
    l.A[i] = take(2ull * l.small * l.lda);
    l.B[i] = take(2ull * l.small * l.lda);
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
  float a, b, c;
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
  if (q.left_low && q.right_low) p.products = 3;
  if (q.left_low)
    NS_TRY(map_16bit(q.left_low, false, q.left_rows, q.left_cols, q.left_ld, q.left_mn ? kStep : kRows, &p.left_low));
  if (q.right_low)
    NS_TRY(map_16bit(q.right_low, false, q.right_rows, q.right_cols, q.right_ld, q.right_mn ? kStep : Shape<P>::kBRows,
                     &p.right_low));
  p.unit = p.unit_low = p.left;
  p.extra = kKind == kGramPart || !q.unit ? 0 : q.extra;
  p.unit_is_left = q.unit_is_left;
  if (p.extra) {
    const int box = q.unit_is_left ? kRows : Shape<P>::kBRows;
    NS_TRY(map_16bit(q.unit, false, kUnit, kUnit, kUnit, box, &p.unit));
    if (q.unit_low) NS_TRY(map_16bit(q.unit_low, false, kUnit, kUnit, kUnit, box, &p.unit_low));
  }
  p.status = q.status;
  p.bf16 = false;
  p.chunk = 8;
  p.left_mn = q.left_mn;
  p.right_mn = q.right_mn;
  p.rows = q.rows;
  p.cols = q.cols;
  p.mt = div_up(q.rows, P::kM);
  p.nt = div_up(q.cols, P::kN);
  p.steps = div_up(q.K, kStep);
  p.parts = kKind == kGramPart ? q.parts : 1;
  p.in0 = q.in0; p.in1 = q.in1;
  p.to0 = q.to0; p.to1 = q.to1;
  p.out = q.out;
  p.ld = q.ld;
  p.ld_out = q.ld_out;
  p.vec = kKind == kLastX && q.ld_out % 8 == 0 && q.cols % 8 == 0 && reinterpret_cast<uintptr_t>(q.out) % 16 == 0;
  p.ca = q.a; p.cb = q.b; p.cc = q.c;
  p.out0 = p.out1 = p.left;
  if (P::kCols == 64) {
    if (kKind == kGramPart) {
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
  // time of a product by tiles of a shape: waves of a tile's steps and epilogue (us)
  constexpr bool sym = kKind == kGram || kKind == kSquare;
  auto cost = [&](int tm, int tn, int units, double step, double more) {
    const double mt = div_up(q.rows, tm), nt = div_up(q.cols, tn);
    const double tiles = sym ? (double)tm / tn * mt * (mt + 1) / 2 : mt * nt;
    return std::max(1.0, std::ceil(tiles / units)) * (div_up(q.K, kStep) * (q.left_low && q.right_low ? 3 : 1) * step + more);
  };
  const double big = cost(256, 256, sms / 2, 0.34, 2.0), mid = cost(128, 128, sms, 0.17, 1.4),
               low = cost(128, 64, sms, 0.12, 1.0);
  if (big <= mid && big <= low) return launch_product<true, 256, kKind>(q, stream);
  if (mid <= low) return launch_product<false, 128, kKind>(q, stream);
  return launch_product<false, 64, kKind>(q, stream);
}

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
  in.eps = a.eps;
  in.partial = reinterpret_cast<double*>(ws + l.partial);
  in.blocks = (int)std::min<long long>(kNormBlocks, ((long long)a.rows * ((a.cols + 3) / 4) + kNormThreads - 1) / kNormThreads);
  in.hi = x[0][0];
  in.lo = x[0][1];
  in.ld = l.ld;
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
  Product q{};
  q.status = a.status;
  for (int i = 0; i < a.steps; ++i) {
    __half *hi = x[i & 1][0], *lo = x[i & 1][1];
    // A
    q.unit = q.unit_low = q.in0 = q.in1 = nullptr;
    q.c = 1.f;
    q.left = q.right = hi;
    q.left_low = q.right_low = l.halves ? lo : nullptr;
    q.left_rows = q.right_rows = a.rows;
    q.left_cols = q.right_cols = a.cols;
    q.left_ld = q.right_ld = l.ld;
    q.left_mn = q.right_mn = tall;
    q.rows = q.cols = small;
    q.K = large;
    q.to0 = A[0];
    q.to1 = A[1];
    q.ld = l.lda;
    // K in parts where the tiles of 256 leave most pairs idle and each part is
    // still 16 steps or more
    const int mt = div_up(small, 256), tiles = mt * (mt + 1) / 2;
    const int parts = std::min({l.parts, sms / 2 / tiles, div_up(large, kStep) / 16});
    if (parts > 1) {
      q.part = reinterpret_cast<float*>(ws + l.part);
      q.ld_part = l.ldp;
      q.parts = parts;
      NS_TRY((launch_product<true, 256, kGramPart>(q, stream)));
      JoinParams j{q.part, parts, small, l.ldp, l.lda, A[0], A[1]};
      NS_TRY(launch_pdl(ns_join, dim3((unsigned)div_up(small, 16), (unsigned)div_up(small, 16)), dim3(256), 0, stream, j));
    } else {
      NS_TRY(choose_product<kGram>(q, sms, stream));
    }
    // B
    q.left = q.right = A[0];
    q.left_low = q.right_low = A[1];
    q.left_rows = q.right_rows = q.left_cols = q.right_cols = small;
    q.left_ld = q.right_ld = l.lda;
    q.left_mn = q.right_mn = false;
    q.K = small;
    if (fold) {
      q.unit = in.units + kUnit * kUnit;
      q.unit_low = in.units + 2 * kUnit * kUnit;
      q.extra = l.halves ? 3 : 2;
      q.unit_is_left = false;
      q.c = a.c / a.a;
    } else {
      q.in0 = A[0];
      q.in1 = A[1];
      q.b = a.b;
      q.c = a.c;
    }
    q.to0 = B[0];
    q.to1 = B[1];
    NS_TRY(choose_product<kSquare>(q, sms, stream));
    // X
    Product s = q;
    if (tall) {
      s.left = hi; s.left_low = lo; s.left_rows = a.rows; s.left_cols = a.cols; s.left_ld = l.ld;
      s.right = B[0]; s.right_low = B[1];
    } else {
      s.left = B[0]; s.left_low = B[1];
      s.right = hi; s.right_low = lo; s.right_rows = a.rows; s.right_cols = a.cols; s.right_ld = l.ld;
      s.right_mn = true;
    }
    s.rows = a.rows;
    s.cols = a.cols;
    s.a = a.a;
    if (fold) {
      s.unit = in.units;
      s.unit_low = nullptr;
      s.extra = 2;
      s.unit_is_left = !tall;
    } else {
      s.in0 = hi;
      s.in1 = lo;
    }
    s.ld = l.ld;
    s.to0 = x[1 - (i & 1)][0];
    s.to1 = x[1 - (i & 1)][1];
    if (i + 1 < a.steps) {
      NS_TRY(choose_product<kStepX>(s, sms, stream));
    } else {
      s.out = static_cast<__nv_bfloat16*>(a.out);
      s.ld_out = a.cols;
      NS_TRY(choose_product<kLastX>(s, sms, stream));
    }
  }
  return cudaSuccess;
}

}  // namespace dspark
