// Orthogonalised update of E matrices g [N, K] by Newton-Schulz steps:
//   X = g / (|g|_F + eps),   then for each step's (a, b, c)
//   A = X X^T,  B = a I + b A + c A^2,  X = B X,      out = scale X.
// The steps push every singular value of X towards 1 and leave its directions, so
// that out is near U V^T of g = U S V^T.
//
// X lies with its shorter side m as rows (g is transposed on the way in, and the
// last product's stores on the way out), so A and B are m x m.  A and B are
// symmetric: in square tiles (128 on one SM, 256 on a pair) only those on and below the
// diagonal are computed, each stored on both sides, m^2 M + m^3 + 2 m^2 M operations a
// step instead of 4 m^2 M + 2 m^3 (M the longer side) but for the tiles' upper halves.
// Tiles of other shapes, and those of clusters, compute all of A and B.
//
// Operands are fp16, whose 11 bits matter here: with bf16's 8 the result is 1% off
// (rms) and more.  X, A and B are scaled by powers of two into fp16's range: |X|, |A|
// and |B| are at most about 1.3, 1.6 and 4 (for the usual coefficients), and their
// typical elements are 1 / sqrt(m M) and less.
//
// The steps raise small singular values up to 3.4-fold each while large ones stay, so
// what a rounding of X loses beside a large singular value grows too (one direction
// 50 times the rest's: 1% off; and what is noise in the null space of a gradient of
// few rows grows likewise).  So X is kept as a hi and a lo part, 22 bits together, in
// all steps but the last; products take the hi part, and X = a X + (b A + c A^2) X
// adds a times both in the epilogue, where rounding the hi part only costs what is
// multiplied by b A + c A^2.  The last step folds a into B: B = a I + b A + c A^2, X =
// B X, whose smaller elements round better; with the last two steps folded the error was
// up to 0.29% where the rank is low.
//
// What remains are the roundings of A and B themselves.  They count against |b| |A| + |c|
// |A|^2, which may be ten times what a + b A + c A^2 leaves, and later steps enlarge them
// again: by the polynomial's slope where a singular value is large, a-fold where it is
// small.  Five steps of (3.4445, -4.7750, 2.0315) end at 0.19 to 0.25% (rms, with the
// rounding of the result to bf16, 0.17%), where many singular values are equal at 0.4%
// (roundings of equal numbers add up instead of averaging; at most 1.2% of a singular
// value), eight such steps at 0.35%, twenty at 0.6%, steeper schedules at 0.5 to 2.5%.
// So in two cases the operands too are the hi and the lo part, and a product is three (hi
// hi + hi lo + lo hi) over one accumulator: where the steps enlarge roundings more than
// those five do (`steep`), and, since sums over few elements average less, up to m = 128,
// where all products are short.  That leaves 0.17% for sides up to 2^14, and costs (five
// steps) 139 us instead of 86 for 8 x 512 x 256, 690 instead of 220 for 16 x 1031 x 517,
// 16.1 ms instead of 5.8 for 16 x 7168 x 2048.
//
// Forming A anew in each step, rather than carrying it along as B A B, costs the m^2
// M product but keeps small singular values: an error of A enters B X relative to
// X, while that of a carried A grows twelvefold a step.
#include <algorithm>
#include <cmath>

#include "dense_gemm.h"
#include "moe_common.cuh"
#include "moe_internal.h"
#include "ortho_cluster.h"
#include "pdl.cuh"
#include "ragged.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPrecise = 128;                 // shorter sides up to here take hi and lo parts
constexpr int kFolded = 1;                    // last steps that fold a X into B
constexpr float kGain = 400.0f, kGrowth = 160.0f;   // of schedules for 11 bits
constexpr float kScaleX = 4096.0f, kScaleA = 1024.0f, kScaleB = 1024.0f;
constexpr int kMaxChunks = 304;               // partial sums of a matrix
constexpr int kRowsPerThread = 4, kTiles = 4; // of k_ortho_scale, k_ortho_transpose

template <int TYPE>
__device__ __forceinline__ float load1(const void* p, long long i) {
  if (TYPE == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return TYPE == 0 ? Half16<__nv_bfloat16>::value(b) : Half16<__half>::value(b);
}
// The two (16-bit) values of a word.
template <int TYPE>
__device__ __forceinline__ float2 word2(uint32_t w) {
  using T = typename std::conditional<TYPE == 1, __half, __nv_bfloat16>::type;
  return make_float2(Half16<T>::value((uint16_t)(w & 0xFFFFu)),
                     Half16<T>::value((uint16_t)(w >> 16)));
}
// Eight values as they lie in memory: n (at most 8) from element i, zeros behind
// them; `wide`: i and n are whole 16-byte pieces.
template <int TYPE>
struct Raw8 {
  uint4 w[TYPE == 2 ? 2 : 1];
};
template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> load8(const void* p, long long i, int n, bool wide) {
  Raw8<TYPE> r;
  if (wide) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) +
                                                    i * (TYPE == 2 ? 4 : 2));
    r.w[0] = n > 0 ? __ldg(q) : make_uint4(0, 0, 0, 0);
    if (TYPE == 2) r.w[TYPE == 2 ? 1 : 0] = n > 4 ? __ldg(q + 1) : make_uint4(0, 0, 0, 0);
  } else if (TYPE == 2) {
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? static_cast<const uint32_t*>(p)[i + k] : 0u;
    r.w[0] = make_uint4(v[0], v[1], v[2], v[3]);
    r.w[TYPE == 2 ? 1 : 0] = make_uint4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? static_cast<const uint16_t*>(p)[i + k] : 0u;
    r.w[0] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
  return r;
}
template <int TYPE>
__device__ __forceinline__ void unpack8(const Raw8<TYPE>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
  if (TYPE == 2) {
    const uint4& b = r.w[TYPE == 2 ? 1 : 0];
    const uint32_t x[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = __uint_as_float(w[k]);
      v[4 + k] = __uint_as_float(x[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = word2<TYPE>(w[k]);
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
    }
  }
}
// Eight values as fp16, and what that leaves of them lo columns on.
__device__ __forceinline__ void store8(__half* out, long long lo, float inv, const float (&v)[8]) {
  uint32_t hi[4], rest[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x = v[2 * k] * inv, y = v[2 * k + 1] * inv;
    const __half2 h = __floats2half2_rn(x, y);
    hi[k] = *reinterpret_cast<const uint32_t*>(&h);
    rest[k] = Half16<__half>::pack(x - __low2float(h), y - __high2float(h));
  }
  *reinterpret_cast<uint4*>(out) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  if (lo != 0) *reinterpret_cast<uint4*>(out + lo) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
}

__device__ __forceinline__ double block_sum(double v, double* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += smem[w];
  return v;
}

// Squares of part blockIdx.x of matrix blockIdx.y (n elements): in fp32 over at most
// 64 values, in fp64 beyond (fp64 additions and conversions are slow enough to
// bound the pass if there is one for every few values) or where that sum overflows.
template <int TYPE>
__global__ void __launch_bounds__(kThreads) k_ortho_norm(const void* g, long long n, int chunks,
                                                         double* partial, uint32_t* done) {
  __shared__ double smem[kThreads / 32];
  griddep_launch();
  griddep_wait();
  constexpr int size = TYPE == 2 ? 4 : 2, per = 16 / size;
  const char* base = static_cast<const char*>(g) + (long long)blockIdx.y * n * size;
  double sum = 0.0;
  // 16-byte pieces from the first aligned element on, the elements beside them singly
  const long long head =
      min((long long)((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / size, n);
  const long long pieces = (n - head) / per;
  const uint4* p = reinterpret_cast<const uint4*>(base + head * size);
  const long long end = pieces * (blockIdx.x + 1) / chunks;
  for (long long i = pieces * blockIdx.x / chunks + threadIdx.x; i < end; i += 8 * kThreads) {
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = i + k * kThreads < end ? __ldg(p + i + k * kThreads) : make_uint4(0, 0, 0, 0);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (TYPE == 2) {
          const float f = __uint_as_float(w[j]);
          s[j] += f * f;
        } else {
          const float2 f = word2<TYPE>(w[j]);
          s[j] += f.x * f.x;
          s[j] += f.y * f.y;
        }
      }
    }
    const float all = (s[0] + s[1]) + (s[2] + s[3]);
    if (all <= 3.402823466e38f) {
      sum += all;
    } else {       // squares within fp32's range whose sum is not: once more, one by one
      const long long first = head + i * per;
#pragma unroll 1
      for (int k = 0; k < 8 * per; ++k) {
        const long long at = first + (long long)(k / per) * kThreads * per + k % per;
        const float f = at < head + end * per ? load1<TYPE>(base, at) : 0.0f;
        sum += f * f;
      }
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    const long long tail = head + pieces * per;
    if (threadIdx.x < head) {
      const float f = load1<TYPE>(base, threadIdx.x);
      sum += f * f;
    }
    if (threadIdx.x < n - tail) {
      const float f = load1<TYPE>(base, tail + threadIdx.x);
      sum += f * f;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) done[blockIdx.y] = 0;     // for ortho_cluster.cu
  sum = block_sum(sum, smem);
  if (threadIdx.x == 0) partial[(size_t)blockIdx.y * chunks + blockIdx.x] = sum;
}

// Factor from matrix e's values to X's.  One warp adds, one lane divides: fp64 by
// every thread took four times as long as the copy (466 against 70 us of the norm's
// own pass over the same bytes).
__device__ __forceinline__ float scale_of(const double* partial, int chunks, int e, float eps,
                                          float* smem) {
  if (threadIdx.x < 32) {
    double total = 0.0;
    for (int i = threadIdx.x; i < chunks; i += 32) total += partial[(size_t)e * chunks + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (threadIdx.x == 0) *smem = (float)((double)kScaleX / (sqrt(total) + (double)eps));
  }
  __syncthreads();
  return *smem;
}

// X of matrix blockIdx.z from g [m, M], zeros behind its M columns.  A thread takes
// eight columns of kRowsPerThread rows, 1 << log_tx threads a row.
template <int TYPE>
__global__ void __launch_bounds__(kThreads)
    k_ortho_scale(const void* g, int m, int M, int Mp, int ld, long long lo, int log_tx, bool wide,
                  int chunks, const double* partial, float eps, __half* x) {
  __shared__ float smem;
  griddep_launch();
  griddep_wait();
  const int rows = kThreads >> log_tx;
  const int c = 8 * ((blockIdx.x << log_tx) + (threadIdx.x & ((1 << log_tx) - 1)));
  const long long first = (long long)blockIdx.z * m;
  float inv = 0.0f;
  for (int i = blockIdx.y; i * rows * kRowsPerThread < m; i += gridDim.y) {
    const int r0 = i * rows * kRowsPerThread + (threadIdx.x >> log_tx);
    Raw8<TYPE> raw[kRowsPerThread];
#pragma unroll
    for (int u = 0; u < kRowsPerThread; ++u) {
      const int r = r0 + u * rows;
      raw[u] = load8<TYPE>(g, (first + r) * M + c, r < m ? min(M - c, 8) : 0, wide);
    }
    // the sums of squares while the loads are on their way
    if (i == blockIdx.y) inv = scale_of(partial, chunks, blockIdx.z, eps, &smem);
#pragma unroll
    for (int u = 0; u < kRowsPerThread; ++u) {
      const int r = r0 + u * rows;
      float v[8];
      unpack8<TYPE>(raw[u], v);
      if (r < m && c < Mp) store8(x + (first + r) * ld + c, lo, inv, v);
    }
  }
}

// The same from g [M, m]: tiles of 64 x 64 through shared memory, as fp16 pairs of
// neighbouring columns of X.  Lanes take 4 x 8 pieces when they write the tile and 8
// x 4 when they read it, so that with rows of 33 words no bank is hit twice.
template <int TYPE, bool LO>
__global__ void __launch_bounds__(kThreads, TYPE == 2 ? 5 : 6)
    k_ortho_transpose(const void* g, int m, int M, int Mp, int ld, long long lo, bool wide, int chunks,
                      const double* partial, float eps, __half* x) {
  __shared__ float smem;
  __shared__ uint32_t tile[LO ? 2 : 1][64][33];
  griddep_launch();
  griddep_wait();
  const int ra = 8 * ((threadIdx.x & 3) + 4 * (threadIdx.x >> 7)), pair = (threadIdx.x >> 2) & 31;
  const int cb = threadIdx.x & 7, rb = threadIdx.x >> 3;
  const int r0 = 64 * blockIdx.y;
  const long long first = (long long)blockIdx.z * M;
  const int c_end = min(Mp, (int)(blockIdx.x + 1) * 64 * kTiles);
  const int begin = blockIdx.x * 64 * kTiles;
  Raw8<TYPE> next[2];
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = c0 + 2 * pair + u;
      next[u] = load8<TYPE>(g, (first + c) * m + r0 + ra, c < M ? min(m - r0 - ra, 8) : 0, wide);
    }
  };
  load(begin);
  const float inv = scale_of(partial, chunks, blockIdx.z, eps, &smem);
  for (int c0 = begin; c0 < c_end; c0 += 64) {
    float v[2][8];
    unpack8<TYPE>(next[0], v[0]);
    unpack8<TYPE>(next[1], v[1]);
    if (c0 + 64 < c_end) load(c0 + 64);      // while this tile is turned
    __syncthreads();                         // the tile before has been read
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = v[0][k] * inv, b = v[1][k] * inv;
      const __half2 h = __floats2half2_rn(a, b);
      tile[0][ra + k][pair] = *reinterpret_cast<const uint32_t*>(&h);
      if (LO)
        tile[LO ? 1 : 0][ra + k][pair] =
            Half16<__half>::pack(a - __low2float(h), b - __high2float(h));
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = rb + 32 * u;
      if (r0 + row < m) {
        __half* out = x + ((long long)blockIdx.z * m + r0 + row) * ld + c0 + 8 * cb;
#pragma unroll
        for (int p = 0; p < (LO ? 2 : 1); ++p) {
          const uint32_t* w = &tile[p][row][4 * cb];
          *reinterpret_cast<uint4*>(out + p * lo) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
}

struct Layout {
  int m, M, mp, Mp, parts, chunks;
  size_t x_bytes, a_bytes, partial, done, a, b, x0, x1, lo, part, total;
};
size_t pad(size_t v) { return (v + 255) / 256 * 256; }

DenseProduct product(const Layout& l, int E) {
  DenseProduct d{};
  d.E = E;
  d.m = l.m;
  d.segs = l.parts == 2 ? 3 : 1;
  return d;
}
// A = X X^T from x, scaled
DenseProduct gram(const Layout& l, int E, const void* x, void* a) {
  DenseProduct d = product(l, E);
  d.nt = true;
  d.width = l.mp;
  d.rows = d.w = x;
  d.rows_ld = d.w_ld = l.parts * l.Mp;
  d.rows_lo = d.w_lo = l.Mp;
  d.seg_kb = l.Mp / 64;
  d.c_acc = kScaleA / (kScaleX * kScaleX);
  d.out = a;
  d.out_ld = l.parts * l.mp;
  d.out_lo = l.parts == 2 ? l.mp : 0;
  return d;
}
// B = a I + b A + c A^2
DenseProduct polynomial(const Layout& l, int E, const void* a, void* b, const float* c) {
  DenseProduct d = product(l, E);
  d.nt = true;
  d.width = l.mp;
  d.rows = d.w = d.mat = a;
  d.rows_ld = d.w_ld = d.out_ld = l.parts * l.mp;
  d.rows_lo = d.w_lo = l.mp;
  d.mat_lo = d.out_lo = l.parts == 2 ? l.mp : 0;
  d.seg_kb = l.mp / 64;
  d.c_acc = c[2] * (kScaleB / (kScaleA * kScaleA));
  d.c_mat = c[1] * (kScaleB / kScaleA);
  d.c_diag = c[0] * kScaleB;
  d.out = b;
  return d;
}
// X = B X
DenseProduct apply(const Layout& l, int E, const void* b, const void* x, void* out) {
  DenseProduct d = product(l, E);
  d.width = l.Mp;
  d.rows = b;
  d.rows_ld = l.parts * l.mp;
  d.rows_lo = l.mp;
  d.w = x;
  d.w_ld = d.out_ld = l.parts * l.Mp;
  d.w_lo = l.Mp;
  d.out_lo = l.parts == 2 ? l.Mp : 0;
  d.seg_kb = l.mp / 64;
  d.c_acc = 1.0f / kScaleB;
  d.out = out;
  return d;
}

// Sizes of workspaces do not depend on the number of steps, so plans are made for this.
constexpr int kModelSteps = 5;
OrthoClusterPlan cluster_plan(const Layout& l, int E) {
  return ortho_cluster_plan(E, l.m, l.mp, l.M, l.Mp, l.parts, kModelSteps);
}
OrthoClusterPlan grid_plan(const Layout& l, int E) {
  return ortho_grid_plan(E, l.m, l.mp, l.M, l.Mp, l.parts, kModelSteps);
}

// Where everything lies, up to the slices' sums.
Layout places(int E, int N, int K, int parts) {
  Layout l;
  l.m = std::min(N, K);
  l.M = std::max(N, K);
  l.mp = (l.m + 63) / 64 * 64;
  l.Mp = (l.M + 63) / 64 * 64;
  l.parts = parts;
  const long long n = (long long)N * K;
  l.chunks = (int)std::max<long long>(
      1, std::min<long long>({(n + 8191) / 8192, kMaxChunks, std::max(1, 1216 / E)}));
  l.x_bytes = pad((size_t)E * l.m * l.parts * l.Mp * 2);
  l.a_bytes = pad((size_t)E * l.m * l.parts * l.mp * 2);
  l.partial = 0;
  l.done = pad((size_t)E * l.chunks * sizeof(double));
  l.a = l.done + pad(E * sizeof(uint32_t));
  l.b = l.a + l.a_bytes;
  l.x0 = l.b + l.a_bytes;
  l.x1 = l.x0 + l.x_bytes;
  l.lo = l.x1 + l.x_bytes;
  l.part = l.lo + (l.parts == 1 ? l.x_bytes : 0);
  l.total = l.part;
  return l;
}
Layout layout(int E, int N, int K, int parts) {
  Layout l = places(E, N, K, parts);
  const float c[3] = {};
  DenseProduct last = apply(l, E, nullptr, nullptr, nullptr);
  last.width = l.M;
  l.total = l.part + pad(std::max({dense_part_bytes(gram(l, E, nullptr, nullptr)),
                                   dense_part_bytes(polynomial(l, E, nullptr, nullptr, c)),
                                   dense_part_bytes(apply(l, E, nullptr, nullptr, nullptr)),
                                   dense_part_bytes(last),
                                   ortho_cluster_part_bytes(cluster_plan(l, E), E)}));
  return l;
}

// Products as launches of their own, or one launch for all steps (ortho_cluster.cu): in
// clusters or over the whole grid.  By modelled cycles; against the products, clusters and
// the grid count with the factors that their models were measured to be off by (the grid
// against clusters without).  X is kept in two parts beyond kPrecise, and what the
// last product of a step moves for it (hi and lo, read and written) is counted at the
// rates that the forms' epilogues reach.  A product of its own takes some 3500 cycles
// more (its launch).  Up to kPrecise the whole grid never was the fastest, and with 22 bits
// beyond it is not considered.  us for five steps in a graph (bf16), as products / in
// clusters / over the grid:
//   8 x 64 x 64     78 /  57 /  76      8 x 1024 x 1024   313 /  519 /  238
//   8 x 256 x 512   92 /  82 /  90      16 x 768 x 2048   592 / 1003 /  475
//   8 x 512 x 512  124 / 153 / 121      64 x 512 x 1024   677 /  712 /  548
//   2 x 200 x 2000 103 / 162 / 119      1 x 1024 x 2048   174 /  766 /  215
//                                       16 x 2048 x 7168 6300 / 19084 / 7690
// It is not always right: 200 x 160 x 160 takes the products (256, the grid 203), 2 x 1024
// x 1024 the grid (174, the products 162), 8 x 256 x 2048 too (141, 137).
enum class Form { PRODUCTS, CLUSTERS, GRID };
Form form_of(const Layout& l, int E) {
  if (ortho_form() != 0)
    return ortho_form() == 4 ? Form::GRID : ortho_form() == 3 ? Form::CLUSTERS : Form::PRODUCTS;
  const float c[3] = {};
  const long long x_bytes = l.parts == 1 ? 8ll * E * l.m * l.Mp : 0;
  const long long products =
      kModelSteps * (dense_cycles(gram(l, E, nullptr, nullptr)) +
                     dense_cycles(polynomial(l, E, nullptr, nullptr, c)) +
                     std::max(dense_cycles(apply(l, E, nullptr, nullptr, nullptr)), x_bytes / 1450) +
                     3 * 3500);
  const long long clusters = cluster_plan(l, E).cycles * 6 / 5 + kModelSteps * x_bytes / 3300;
  if (l.parts == 1) {
    const long long grid = grid_plan(l, E).cycles;
    if (grid * 19 / 20 < products && grid < clusters) return Form::GRID;
  }
  return clusters < products ? Form::CLUSTERS : Form::PRODUCTS;
}

cudaError_t run(const DenseProduct& d, void* part, cudaStream_t stream) {
  return dense_on_pairs(d) ? launch_dense_2sm(d, stream) : launch_dense(d, part, stream);
}

template <int TYPE>
cudaError_t prepare(const Layout& l, int E, bool transposed, const void* g, float eps,
                    double* partial, uint32_t* done, __half* x, long long lo,
                    cudaStream_t stream) {
  const long long n = (long long)l.m * l.M;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(l.chunks, E, 1);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_ortho_norm<TYPE>, g, n, l.chunks, partial, done);
  if (e != cudaSuccess) return e;
  const int ld = l.parts * l.Mp;
  const double* sums = partial;
  // rows of g in whole 16-byte pieces
  const bool wide = reinterpret_cast<uintptr_t>(g) % 16 == 0 &&
                    (transposed ? l.m : l.M) % (TYPE == 2 ? 4 : 8) == 0;
  if (transposed) {
    cfg.gridDim = dim3((l.Mp / 64 + kTiles - 1) / kTiles, (l.m + 63) / 64, E);
    return cudaLaunchKernelEx(
        &cfg, lo != 0 ? k_ortho_transpose<TYPE, true> : k_ortho_transpose<TYPE, false>, g, l.m, l.M,
        l.Mp, ld, lo, wide, l.chunks, sums, eps, x);
  }
  int log_tx = 3;
  while (log_tx < 8 && 8 << log_tx < l.Mp) ++log_tx;
  const int rows = (kThreads >> log_tx) * kRowsPerThread;
  cfg.gridDim = dim3((l.Mp / 8 + (1 << log_tx) - 1) >> log_tx, std::min((l.m + rows - 1) / rows, 32768),
                     E);
  return cudaLaunchKernelEx(&cfg, k_ortho_scale<TYPE>, g, l.m, l.M, l.Mp, ld, lo, log_tx, wide,
                            l.chunks, sums, eps, x);
}

// Whether the steps enlarge roundings of their operands more than five steps of the usual
// triple do, which are 310 and 141 by these two figures; six are 476 and 485.
// gain: relative roundings of 1 of A, B and X in a step move a singular value s by
//   s (2 |b| s^2 + 5 |c| s^4 + |p - a| + |p|),  p = a + b s^2 + c s^4,
// (A enters b A and twice A^2, whose sum counts once; B, its product with X) and each later
// step enlarges that by its slope a + 3 b s^2 + 5 c s^4.  The largest over s from 2^-14 to
// 1 and over the steps.
// growth: of what is left in directions of (nearly) no singular value.
// Steps that raise neither, as (1.5, -0.5, 0) or (2, -1.5, 0.5), stay with 11 bits and end
// below 0.2%.
bool steep(int steps, const float* c) {
  constexpr int kValues = 64;
  const float ratio = exp2f(-14.0f / (kValues - 1));
  float s[kValues], d[kValues], growth = 1.0f;
  for (int i = 0; i < kValues; ++i) {
    s[i] = i == 0 ? 1.0f : s[i - 1] * ratio;
    d[i] = 0.0f;
  }
  for (int k = 0; k < steps; ++k, c += 3) {
    if (k > 0) growth *= fabsf(c[0]);
    bool below = growth <= kGrowth;
    for (int i = 0; i < kValues; ++i) {
      const float s2 = s[i] * s[i], b = c[1] * s2, q = c[2] * s2 * s2, p = c[0] + b + q;
      d[i] = fabsf(c[0] + 3.0f * b + 5.0f * q) * d[i] +
             s[i] * (2.0f * fabsf(b) + 5.0f * fabsf(q) + fabsf(b + q) + fabsf(p));
      s[i] = fabsf(s[i] * p);
      below &= d[i] <= kGain;
    }
    if (!below) return true;
  }
  return false;
}

// The workspace takes E matrices of 11 bits (6 bytes an element and 4 of a square).  Those
// of 22 bits (8 and 8) go through the steps in groups that fit there, or in kSlack bytes
// more: a launch of few small matrices takes as long as one of many (8 x 512 x 256, one by
// one: 482 us).
constexpr size_t kSlack = 32 << 20;
struct Groups {
  int n, last;          // matrices of each, and of the last one
  Layout l, l_last;
  size_t bytes() const { return std::max(l.total, l_last.total); }
};
Groups groups_of(int E, int N, int K, size_t bytes) {
  Groups r;
  for (int groups = 1;; ++groups) {
    r.n = (E + groups - 1) / groups;
    if (r.n > 1 && places(r.n, N, K, 2).total > bytes + kSlack) continue;
    r.last = (E - 1) % r.n + 1;
    r.l = layout(r.n, N, K, 2);
    r.l_last = r.last == r.n ? r.l : layout(r.last, N, K, 2);   // (fewer may be sliced more)
    if (r.n == 1 || r.bytes() <= bytes + kSlack) return r;
  }
}

cudaError_t launch(const Layout& l, int E, int N, int K, const void* g, int type, void* out,
                   int steps, const float* coefficients, float eps, float scale, void* workspace,
                   cudaStream_t stream) {
  const bool transposed = N > K;
  char* ws = static_cast<char*>(workspace);
  void *a = ws + l.a, *b = ws + l.b, *x = ws + l.x0, *y = ws + l.x1, *part = ws + l.part;
  double* partial = reinterpret_cast<double*>(ws + l.partial);
  uint32_t* done = reinterpret_cast<uint32_t*>(ws + l.done);
  // steps that add a X in the epilogue, from X's hi and lo parts
  const int kept = l.parts == 1 ? std::max(0, steps - kFolded) : 0;
  __half* lo = reinterpret_cast<__half*>(ws + l.lo);
  __half* x0 = static_cast<__half*>(x);
  const long long x_lo = l.parts == 2 ? l.Mp : kept > 0 ? lo - x0 : 0;
  cudaError_t e = type == 0   ? prepare<0>(l, E, transposed, g, eps, partial, done, x0, x_lo, stream)
                  : type == 1 ? prepare<1>(l, E, transposed, g, eps, partial, done, x0, x_lo, stream)
                              : prepare<2>(l, E, transposed, g, eps, partial, done, x0, x_lo, stream);
  if (e != cudaSuccess) return e;
  const Form form = form_of(l, E);
  if (form != Form::PRODUCTS) {
    OrthoClusterProblem d{form == Form::GRID ? grid_plan(l, E) : cluster_plan(l, E),
                          E, l.m, l.M, l.mp, l.Mp, l.parts, steps, transposed,
                          {x, y}, l.parts == 1 ? lo : nullptr, a, b, out, part, kept};
    d.c_gram = gram(l, E, x, a).c_acc;
    d.c_apply = apply(l, E, b, x, y).c_acc;
    d.c_last = d.c_apply * (scale / kScaleX);
    float coef[3 * MOE_MAX_ORTHOGONALIZE_STEPS];
    for (int s = 0; s < steps; ++s) {
      const DenseProduct p = polynomial(l, E, a, b, coefficients + 3 * s);
      coef[3 * s] = s < kept ? coefficients[3 * s] : p.c_diag;
      coef[3 * s + 1] = p.c_mat;
      coef[3 * s + 2] = p.c_acc;
    }
    d.coef = coef;
    d.done = done;
    e = launch_ortho_cluster(d, stream);
    // The whole grid has to be on the GPU at once.  Where the context has fewer SMs than the
    // device (a partition), that is refused, and the products need no such thing.
    if (form != Form::GRID || e != cudaErrorCooperativeLaunchTooLarge) return e;
    (void)cudaGetLastError();       // seen
    e = cudaSuccess;
  }
  for (int s = 0; s < steps && e == cudaSuccess; ++s) {
    e = run(gram(l, E, x, a), part, stream);
    if (e != cudaSuccess) return e;
    DenseProduct poly = polynomial(l, E, a, b, coefficients + 3 * s);
    DenseProduct last = apply(l, E, b, x, y);
    if (s < kept) {
      poly.c_diag = 0.0f;
      last.mat = x;
      last.c_mat = coefficients[3 * s];
      last.mat_lo = lo - static_cast<__half*>(x);
      if (s + 1 < kept) last.out_lo = lo - static_cast<__half*>(y);
    }
    e = run(poly, part, stream);
    if (e != cudaSuccess) return e;
    if (s == steps - 1) {
      last.width = l.M;
      last.c_acc *= scale / kScaleX;
      last.final_out = out;
      last.transposed = transposed;
    }
    e = run(last, part, stream);
    std::swap(x, y);
  }
  return e;
}

}  // namespace

size_t orthogonalize_bytes(int E, int N, int K) {
  if (std::min(N, K) <= kPrecise) return layout(E, N, K, 2).total;
  const size_t all = layout(E, N, K, 1).total;
  return std::max(all, groups_of(E, N, K, all).bytes());
}

cudaError_t launch_orthogonalize(int E, int N, int K, const void* g, int type, void* out,
                                 int steps, const float* coefficients, float eps, float scale,
                                 void* workspace, cudaStream_t stream) {
  if (std::min(N, K) <= kPrecise || !steep(steps, coefficients))
    return launch(layout(E, N, K, std::min(N, K) <= kPrecise ? 2 : 1), E, N, K, g, type, out, steps,
                  coefficients, eps, scale, workspace, stream);
  const Groups r = groups_of(E, N, K, layout(E, N, K, 1).total);
  const size_t each = (size_t)N * K;
  for (int at = 0; at < E; at += r.n) {
    const bool last = E - at <= r.n;
    const cudaError_t e = launch(last ? r.l_last : r.l, last ? r.last : r.n, N, K,
                                 static_cast<const char*>(g) + at * each * (type == 2 ? 4 : 2), type,
                                 static_cast<char*>(out) + at * each * 2, steps, coefficients, eps,
                                 scale, workspace, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
