// Pieces shared by the ragged grouped products (ragged_one.cuh on one SM,
// ragged_pair.cuh on SM pairs, ragged_mxfp4.cu): segments of rows given by
// expert offsets on the device, their cut into tiles, operand descriptors and
// epilogue stores.
//
// The products, with w [E, N, K] and the rows o[e] .. o[e+1]-1 of expert e:
//   forward  y[r, n]     = sum_k x[r, k]  w[e, n, k]
//   dgrad    dx[r, k]    = sum_n dy[r, n] w[e, n, k]
//   wgrad    dw[e, n, k] = sum_r dy[r, n] x[r, k]
//
// Forward and dgrad put the weights in the MMA's M (128 or 256 of them) and
// the tokens in its N: N can be any multiple of 16, so a segment's rows are
// cut evenly into tiles of at most 256 tokens and almost no MMA work falls on
// rows of other segments, whatever the segment's length.  With the tokens in
// M every segment would be rounded up to 128 or 256 rows.
#pragma once

#include <cuda_fp16.h>

#include "moe_common.cuh"

namespace moe {

enum : int { RAG_FWD = 0, RAG_DGRAD = 1, RAG_WGRAD = 2 };

constexpr int kRagMaxExperts = 1024;
// Shared memory of the segment table: header, then for each segment with rows
// the first token tile (prefix), first row, rows and expert.
constexpr int kRagSchedBytes = 16 + 4 * (4 * (kRagMaxExperts + 1));

// Division by a launch constant: q = (n * m) >> (31 + shift), exact for
// 0 <= n < 2^30 (an integer division takes some 100 cycles, and a tile's lookup
// has three on the way to its first copy).
struct FastDiv {
  uint32_t mul, shift;
  int d;
};
inline FastDiv fast_div(int d) {
  // With 2^s <= d < 2^(s + 1) and m = ceil(2^(31 + s) / d) <= 2^31:
  // m d = 2^(31 + s) + r with r < d <= 2^(s + 1), so n m / 2^(31 + s) exceeds
  // n / d by n r / (d 2^(31 + s)) < 2^30 2^(s + 1) / (d 2^(31 + s)) = 1 / d.
  FastDiv f;
  f.d = d;
  uint32_t s = 0;
  while ((2ll << s) <= d) ++s;
  f.shift = s;
  const uint64_t one = 1ull << (31 + s);
  f.mul = (uint32_t)((one + d - 1) / d);
  return f;
}
__device__ __forceinline__ int operator/(int n, const FastDiv& f) {
  return (int)(((uint64_t)(uint32_t)n * f.mul) >> (31 + f.shift));
}

// What a product's epilogue does with the sums: rounds and stores them, or one of
// the fused forms (ragged_epi.cuh).
enum : int { EPI_PLAIN = 0, EPI_GATED = 1, EPI_GATED_GRAD = 2, EPI_DENSE = 3 };

// Arguments of the gated forward and of its gradient.
struct RagGated {
  const void* h;            // gradient: the sums before the activation [R, 2 inter]
  void* h_out;              // forward: those sums, or null; gradient: dh
  void* z;                  // [R, inter]; gradient: or null
  long long ldh, ldh_out, ldz;
  int inter;
  float alpha, beta, limit; // limit: +inf clamps nothing
};
// Arguments of a batch of dense products of E matrices of m rows (ragged_epi.cuh).
struct RagDense {
  int m;                    // rows of a matrix
  int sym;                  // symmetric output of mp rows and columns, zeros from m on
  int mp;                   // sym: columns of the output, m rounded up to 64
  int tri;                  // sym: tiles on and below the diagonal, stored on both sides
  int per;                  // rows of a token tile; sym: a multiple of 32
  int tok_tiles;
  FastDiv e_tiles;          // tiles of a matrix
  int seg_kb;               // steps of each of the reduction's segments (hi and lo parts)
  int a_lo, b_lo;           // columns from the hi to the lo part of the operands
  float c_acc, c_mat, c_diag;
  const __half* mat;        // added, c_mat times: [E, m, ...] as the output, or null
  long long mat_lo, out_lo; // from mat and the output to their lo parts, or 0
  __nv_bfloat16* final_out; // the last product: [E, m, W], or [E, W, m] with `transposed`
  int transposed;
};

// Everything a ragged product kernel needs beside its tensor maps.
struct RagArgs {
  const int32_t* offsets;   // [E + 1]
  int R, E;
  int W;                    // forward, dgrad: columns of the output (N or K)
  int num_kb;               // forward, dgrad: 64-deep steps of the reduction
  FastDiv w_tiles;          // forward, dgrad: tiles of W; wgrad: tiles of N
  FastDiv k_tiles;          // wgrad: tiles of K
  FastDiv e_tiles;          // wgrad: tiles of an expert
  int N, K;                 // wgrad: the output of one expert
  int tile_rows;            // forward, dgrad: most token rows of a tile
  int group_max;            // token tiles walked together (forward, dgrad)
  int stages;
  int wide_a, wide_b;       // MN-major operand whose map has its chunks as a dimension
  void* out;
  long long ldo;            // row stride of out (forward, dgrad)
  const void* bias;         // forward: [E, N] in the operands' type, or null
  int out_f32;              // wgrad: dw is fp32
  int accumulate;           // wgrad: dw += instead of dw =
  int splits;               // one SM: CTAs (a cluster) that share a tile's reduction, and
  float* part;              //   their sums [tiles, splits, tile_rows, 128] (wgrad: 128, 256)
  uint64_t limit_ns;
  int never_arrive;
  int* err;
  RagGated gated;
  RagDense dense;
};

struct RagSched {
  const int* tile0;   // first token tile of each segment; tile0[nseg] = all
  const int* row0;
  const int* cnt;
  const int* exp;
  int nseg;
};

// Rows of each token tile of a segment of cnt rows: the fewest tiles of at
// most tile_rows rows, all of the same size rounded up to G rows.
template <int G>
__device__ __forceinline__ int rag_rows_per_tile(int cnt, int tile_rows) {
  if (cnt <= tile_rows) return (cnt + G - 1) / G * G;
  const int nt = (cnt + tile_rows - 1) / tile_rows;
  return ((cnt + nt - 1) / nt + G - 1) / G * G;
}

// Builds the segment table of this CTA from the offsets.  Every thread calls
// it (it contains __syncthreads).  Offsets are read once, clamped into
// [0, R] and made non-decreasing, so no table they can hold reaches outside
// the tensors or gives a row to two experts; offsets that needed it are
// reported in the device error word.  scratch: E + 1 ints of shared memory
// free until this returns.
template <int G>
__device__ __forceinline__ RagSched rag_sched_build(const RagArgs& a, int* mem, int* scratch) {
  int* hdr = mem;
  int* tile0 = mem + 4;
  int* row0 = tile0 + kRagMaxExperts + 1;
  int* cnt = row0 + kRagMaxExperts + 1;
  int* exp = cnt + kRagMaxExperts + 1;
  // up to 32 experts: straight into the scanning warp's registers
  const bool few = a.E <= 32;
  if (!few) {
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) scratch[e] = a.offsets[e];
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int nseg = 0, tiles = 0, top = 0;   // top: largest offset so far
    bool bad = false;
    for (int base = 0; base < a.E; base += 32) {
      const int e = base + lane;
      const int32_t* off = few ? a.offsets : scratch;
      const int b_raw = off[min(e, a.E)], e_raw = off[min(e + 1, a.E)];
      bad |= b_raw < 0 || e_raw > a.R || e_raw < b_raw;
      int mx = max(min(max(b_raw, 0), a.R), top);   // running maximum of the offsets
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, mx, o);
        if (lane >= o) mx = max(mx, v);
      }
      const int end = max(mx, min(max(e_raw, 0), a.R));
      const int n = e < a.E ? end - mx : 0;
      const int per = n > 0 ? rag_rows_per_tile<G>(n, a.tile_rows) : 1;
      const int nt = n <= a.tile_rows ? (n > 0 ? 1 : 0) : (n + per - 1) / per;
      const unsigned has = __ballot_sync(0xffffffffu, n > 0);
      int inc = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (n > 0) {
        const int s = nseg + __popc(has & ((1u << lane) - 1u));
        tile0[s] = tiles + inc - nt;
        row0[s] = mx;
        cnt[s] = n;
        exp[s] = e;
      }
      nseg += __popc(has);
      tiles += __shfl_sync(0xffffffffu, inc, 31);
      top = __shfl_sync(0xffffffffu, end, 31);
    }
    if (lane == 0) {
      tile0[nseg] = tiles;
      hdr[0] = nseg;
    }
    if (bad && blockIdx.x == 0) set_dev_error(a.err, kDevErrBadIndex);
  }
  fence_proxy_async_smem();   // scratch lies where TMA writes next
  __syncwarp();
  __syncthreads();
  RagSched s;
  s.tile0 = tile0;
  s.row0 = row0;
  s.cnt = cnt;
  s.exp = exp;
  s.nseg = hdr[0];
  return s;
}

// One tile of forward or dgrad: rows [row0, row0 + rows) of expert e, columns
// from 128 w_tile (256 w_tile on SM pairs).
struct RagTile {
  int e, row0, rows, w_tile;
  int tok;               // number of the token tile, counted over all segments
};

// Tile t: segment by segment; inside a segment groups of group_max token
// tiles, weight tile by weight tile, the group's token tiles inner, so that
// the CTAs running together share weight tiles and token rows in L2.
template <int G>
__device__ __forceinline__ RagTile rag_tile(const RagSched& s, const RagArgs& a, int t) {
  const int q = t / a.w_tiles;
  const int w_tiles = a.w_tiles.d;
  int lo = 0, hi = s.nseg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.tile0[mid] <= q) lo = mid; else hi = mid - 1;
  }
  const int nt = s.tile0[lo + 1] - s.tile0[lo];
  const int local = t - s.tile0[lo] * w_tiles;
  RagTile T;
  int tok;
  if (nt == 1) {               // no divisions for the short segments
    T.w_tile = local;
    tok = 0;
  } else {
    const int c = nt <= a.group_max ? 0 : local / (a.group_max * w_tiles);
    const int gm = min(a.group_max, nt - c * a.group_max);
    const int l2 = local - c * a.group_max * w_tiles;
    T.w_tile = l2 / gm;
    tok = c * a.group_max + (l2 - T.w_tile * gm);
  }
  const int per = rag_rows_per_tile<G>(s.cnt[lo], a.tile_rows);
  T.e = s.exp[lo];
  T.row0 = s.row0[lo] + tok * per;
  T.rows = min(per, s.cnt[lo] - tok * per);
  T.tok = s.tile0[lo] + tok;
  return T;
}

// Whether a double tile of 512 weights has a second half (SM pairs).
template <int MT>
__device__ __forceinline__ bool rag_second_tile(const RagArgs& a, int w_tile) {
  return MT == 2 && w_tile * 512 + 256 < a.W;
}

// One tile of wgrad: expert e, rows n_tile of N and columns k_tile of K, over
// the expert's cnt rows.  Groups of 2^kRagGroupShift n tiles, k tile by k tile, the
// group's n tiles inner.
constexpr int kRagGroupShift = 3;
struct RagWTile {
  int e, n_tile, k_tile;
};
__device__ __forceinline__ RagWTile rag_wtile(const RagArgs& a, int t) {
  RagWTile T;
  T.e = t / a.e_tiles;
  const int local = t - T.e * a.e_tiles.d;
  // groups of 8 n tiles x all k tiles
  const int g = (local >> kRagGroupShift) / a.k_tiles;
  const int n0 = g << kRagGroupShift;
  const int gm = min(1 << kRagGroupShift, a.w_tiles.d - n0);
  const int l2 = local - n0 * a.k_tiles.d;
  T.k_tile = gm == 1 << kRagGroupShift ? l2 >> kRagGroupShift : l2 / gm;
  T.n_tile = n0 + (l2 - T.k_tile * gm);
  return T;
}

// {first row, rows} of every expert, with and without rows, for wgrad, which
// visits them all.  Takes the table's memory (the schedule's arrays are gone
// afterwards); scratch: E int2 of shared memory free until this returns.  Every
// thread calls it.
__device__ __forceinline__ const int2* rag_rows_by_expert(const RagSched& s, int E, int* mem,
                                                          int2* scratch) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) scratch[e] = make_int2(0, 0);
  __syncthreads();
  for (int i = threadIdx.x; i < s.nseg; i += blockDim.x)
    scratch[s.exp[i]] = make_int2(s.row0[i], s.cnt[i]);
  __syncthreads();
  int2* out = reinterpret_cast<int2*>(mem + 4);
  for (int e = threadIdx.x; e < E; e += blockDim.x) out[e] = scratch[e];
  fence_proxy_async_smem();   // scratch lies where TMA writes next
  __syncthreads();
  return out;
}

// Zeros rows [from, to) of BOXES consecutive 64-row boxes (128 bytes a row;
// swizzling permutes within a row) at shared address base, by one warp, before
// the MMA that reads them.
template <int BOXES>
__device__ __forceinline__ void rag_zero_rows(uint32_t base, int from, int to, int lane) {
  if (from >= to) return;
  const int per = (to - from) * 8;       // 16-byte pieces of a box
  for (int b = 0; b < BOXES; ++b)
    for (int i = lane; i < per; i += 32)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + b * 8192 + from * 128 +
                                                                   i * 16),
                   "r"(0)
                   : "memory");
  fence_proxy_async_smem();
  __syncwarp();
}

// Descriptor of an MN-major tile written by TMA with 128-byte swizzling: 64
// values of M (or N) a row, one row for each step of the reduction, 64 rows a
// box; 8-row atoms of 1024 bytes follow one another along the reduction
// (stride byte offset), the box of the next 64 values of M lies 8192 bytes on
// (leading byte offset).  Sixteen steps of the reduction are 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(8192u >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;   // MN-major operands

// 3-D tiled load (the weights [E, N, K]) into this CTA's shared memory.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t cluster_bar, int32_t c0, int32_t c1,
                                                 int32_t c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(cluster_bar),
      "l"(policy)
      : "memory");
}
// 4-D tiled load: an MN-major operand with its 64-value chunks as a dimension
// (make_tmap_rag_wide), so that one copy brings several chunks.  A copy costs
// its issuing thread some 150 cycles, and a step has 512 cycles of MMA work.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar),
      "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t cluster_bar, int32_t c0, int32_t c1,
                                                 int32_t c2, int32_t c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(cluster_bar), "l"(policy)
      : "memory");
}

// 5-D tiled load: gate and up weights interleaved (make_tmap_rag_gated).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c3, int32_t c4,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(0), "r"(c3), "r"(c4), "r"(bar),
      "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t cluster_bar, int32_t c0, int32_t c3,
                                                 int32_t c4, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(0), "r"(c3), "r"(c4), "r"(cluster_bar),
      "l"(policy)
      : "memory");
}

// True in one lane of a warp whose lanes are all here.  The producers and the
// MMA issuers run their loops with the whole warp and issue from this lane: with
// the loop inside one lane's branch the compiler keeps descriptors and
// coordinates in per-thread registers and moves them to the uniform ones that
// the instructions take, ~600 cycles a step against 512 of MMA work (5% of a
// long forward).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b32 r;\n\t"
      "elect.sync r|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// fp32 <-> the operands' 16-bit types.
template <typename T>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
  static constexpr uint32_t kFmt = kFmtBF16;
  static __device__ __forceinline__ uint16_t bits(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float value(uint16_t b) {
    return __bfloat162float(__ushort_as_bfloat16(b));
  }
};
template <>
struct Half16<__half> {
  static constexpr uint32_t kFmt = 0;   // kind::f16 operand format code for fp16
  static __device__ __forceinline__ uint16_t bits(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float value(uint16_t b) {
    return __half2float(__ushort_as_half(b));
  }
};

// Forward / dgrad epilogue of 32 tokens: r[j] is this lane's column w of token
// row0 + j; the lanes of a warp hold 32 neighbouring columns.  Two neighbouring
// lanes swap halves so that each holds both columns of every other token, and
// a store instruction writes two tokens' 64 bytes (two full sectors each) in
// 4-byte pieces.  `live` tokens are stored, columns below W (W is even: a
// multiple of 8).  Packed conversion, one shuffle and one byte permute for two
// tokens: the warps are bound by instruction issue here, not by the stores.
template <bool ALL>
__device__ __forceinline__ void rag_store_pairs(const uint32_t* pk, uint16_t* p, long long ldo,
                                                int live, bool inside, int lane) {
  const uint32_t sel = (lane & 1) ? 0x3276u : 0x5410u;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, pk[j], 1);
    const uint32_t v = __byte_perm(pk[j], other, sel);
    if (ALL || (inside && 2 * j + (lane & 1) < live)) *reinterpret_cast<uint32_t*>(p) = v;
    p += 2 * ldo;
  }
}
// The 32 tokens as 16 packed pairs: pk[j] holds tokens 2j and 2j + 1 of this
// lane's column w, out points at (first token, w).
__device__ __forceinline__ void rag_store_packed32(const uint32_t* pk, uint16_t* out,
                                                   long long ldo, int live, int w, int W,
                                                   int lane) {
  // odd lanes: the next token, from the column before
  uint16_t* p = out + ((lane & 1) ? ldo - 1 : 0);
  const bool inside = w < W;
  if (live >= 32 && __all_sync(0xffffffffu, inside))
    rag_store_pairs<true>(pk, p, ldo, live, inside, lane);
  else
    rag_store_pairs<false>(pk, p, ldo, live, inside, lane);
}
template <typename T>
__device__ __forceinline__ void rag_store_tokens32(uint32_t (&r)[32], bool has_bias, float bias,
                                                   uint16_t* out, long long ldo, int live, int w,
                                                   int W, int lane) {
  if (has_bias) {
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + bias);
  }
  uint32_t pk[16];
#pragma unroll
  for (int j = 0; j < 16; ++j)
    pk[j] = Half16<T>::pack(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
  rag_store_packed32(pk, out, ldo, live, w, W, lane);
}

// A reduction that the CTAs of a cluster share (splits > 1; one tile for each
// cluster).  N tokens from token c of this CTA's sums of tile t: column col.
template <int N>
__device__ __forceinline__ void rag_store_part(const RagArgs& a, const uint32_t (&r)[N], int t,
                                               int rank, int c, int rows, int col) {
  float* p = a.part + (((size_t)t * a.splits + rank) * a.tile_rows + c) * 128 + col;
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (c + j < rows) p[128 * j] = __uint_as_float(r[j]);
}
// After the cluster barrier: this CTA's share of tile t's tokens, the slices
// added in order; a lane takes four columns of a token.
template <typename T, bool BIAS>
__device__ __forceinline__ void rag_join_tokens(const RagArgs& a, const RagTile& D, int t,
                                                int rank, int warp, int warps, int lane) {
  const int w = D.w_tile * 128 + 4 * lane;
  float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (BIAS && a.bias != nullptr && w < a.W) {
    const uint16_t* b = static_cast<const uint16_t*>(a.bias) + (size_t)D.e * a.W + w;
    bias = make_float4(Half16<T>::value(b[0]), Half16<T>::value(b[1]), Half16<T>::value(b[2]),
                       Half16<T>::value(b[3]));
  }
  const float* p = a.part + (size_t)t * a.splits * a.tile_rows * 128 + 4 * lane;
  for (int j = rank * warps + warp; j < D.rows; j += a.splits * warps) {
    float4 v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < a.splits)
        v[s] = *reinterpret_cast<const float4*>(p + ((size_t)s * a.tile_rows + j) * 128);
    float4 x = v[0];
#pragma unroll
    for (int s = 1; s < 8; ++s)
      if (s < a.splits)
        x = make_float4(x.x + v[s].x, x.y + v[s].y, x.z + v[s].z, x.w + v[s].w);
    if (w < a.W)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (D.row0 + j) * a.ldo + w) =
          make_uint2(Half16<T>::pack(x.x + bias.x, x.y + bias.y),
                     Half16<T>::pack(x.z + bias.z, x.w + bias.w));
  }
}
// CTAs that share one tile's reduction of `steps` steps: as many as have at
// least `least` steps each and as clusters run at the same time (of 2 CTAs 76,
// of 4 36, of 8 15 on a GB300's 152 SMs: a 16th tile of eight would wait).  The
// limits are that GPU's on purpose: sizes of workspaces follow from them, which
// are asked for without one too, and only speed would differ on another.
constexpr int kRagClusters[3] = {15, 36, 76};     // tiles that take 8, 4, 2 CTAs each
inline int rag_slices(long long tiles, int steps, int least) {
  for (int i = 0; i < 3; ++i)
    if (tiles <= kRagClusters[i] && steps >= (8 >> i) * least) return 8 >> i;
  return 1;
}
// Bytes for the sums of a sliced product of R rows, at least what any number of
// rows up to R takes, so that a workspace for the largest batch serves the
// smaller ones (fewer rows can mean more slices).  Even segments make
// tok <= limit / w_tiles token tiles, and any segments at most min(E, R) +
// R / tile_rows <= 2 tok; all terms grow with R, as tile_rows does.
inline size_t rag_part_bytes(int R, int E, int w_tiles, int steps, int least, int tile_rows) {
  size_t most = 0;
  for (int i = 0; i < 3; ++i) {
    if (steps < (8 >> i) * least) continue;
    const long long even = 2ll * (kRagClusters[i] / w_tiles) * tile_rows;
    const long long any = (long long)(E < R ? E : R) * tile_rows + R;
    const size_t b = (size_t)(8 >> i) * w_tiles * (size_t)(even < any ? even : any);
    if (b > most) most = b;
  }
  return most * 128 * sizeof(float);
}

// A 128-byte wide box of shared memory (128-byte swizzled) to a 3-D tensor,
// clipped at its ends; with `add`, added to it (fp32, one rounding).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t c0,
                                             int32_t c1, int32_t c2, bool add) {
  if (add)
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group "
        "[%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group "
        "[%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until at most N of this thread's stores still read shared memory / are not
// complete.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// dw of an expert without rows: part `part` of `parts` of its zeros, by the
// epilogue's threads, as one run of 16-byte pieces.  (As tiles, rows that do not
// start on a sector took partial writes: 1160 columns 488 us, 1152 276.)
__device__ __forceinline__ void rag_zero_expert(const RagArgs& a, int e, int part, int parts,
                                                int tid, int threads) {
  const long long pieces = (long long)a.N * a.K * (a.out_f32 ? 4 : 2) / 16;
  uint4* dw = static_cast<uint4*>(a.out) + e * pieces;
  const long long end = pieces * (part + 1) / parts;
  for (long long i = pieces * part / parts + tid; i < end; i += threads)
    dw[i] = make_uint4(0, 0, 0, 0);
}

// wgrad epilogue of one warp: its 32 accumulator rows (one a lane) x SPAN
// columns from taddr to rows n0 .. n0 + 31 and columns from k0 of dw[e].  Each
// lane packs 128 bytes of its row (64 16-bit or 32 fp32 values) into a swizzled
// box of shared memory, which goes out as one TMA store: whole 128-byte lines,
// clipped at N and K by the tensor map.  (Stores from the lanes, 32 bytes in each
// of 32 rows, kept the weight gradient of 256 experts at 4.3 TB/s.)  buf: BUFS
// boxes of 4 KB used in turn, `turn` counting them.  fp32 sums are added to dw
// by the store; 16-bit ones here, so that they are rounded once.
// release() is called by the whole warp when the accumulator has been read.
template <typename T, int BUFS, int SPAN, class Release>
__device__ __forceinline__ void rag_wgrad_epilogue(const RagArgs& a, const CUtensorMap* tmD,
                                                   uint32_t buf, int& turn, uint32_t taddr,
                                                   int e, int n0, int k0, int lane,
                                                   Release&& release) {
  const int cols = a.out_f32 ? 32 : 64;
  const int width = min(SPAN, a.K - k0);
  // Nothing of it inside dw.  A box that is not stored must not be filled either:
  // the wait below counts the warp's stores, one for each turn.
  if (width <= 0 || n0 >= a.N) {
    release();
    return;
  }
  const bool add16 = a.accumulate && !a.out_f32;
#pragma unroll 1
  for (int c = 0; c < width; c += cols) {
    const uint32_t box = buf + 4096u * (BUFS == 1 ? 0 : turn % BUFS);
    ++turn;
    uint32_t w[32];           // this lane's 128 bytes
    if (a.out_f32) {
      tmem_ld_32x32b_x32(taddr + c, w);
      tmem_ld_wait();
    } else {
      uint32_t r[32], s[32];
      tmem_ld_32x32b_x32(taddr + c, r);
      tmem_ld_32x32b_x32(taddr + c + 32, s);
      tmem_ld_wait();
      if (add16 && n0 + lane < a.N) {
        const uint16_t* old = static_cast<const uint16_t*>(a.out) +
                              ((size_t)e * a.N + n0 + lane) * a.K + k0 + c;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (c + 8 * q < width) {
            const uint4 o = *reinterpret_cast<const uint4*>(old + 8 * q);
            const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float lo = Half16<T>::value((uint16_t)(ow[i] & 0xFFFFu));
              const float hi = Half16<T>::value((uint16_t)(ow[i] >> 16));
              uint32_t& x = q < 4 ? r[8 * q + 2 * i] : s[8 * (q - 4) + 2 * i];
              uint32_t& y = q < 4 ? r[8 * q + 2 * i + 1] : s[8 * (q - 4) + 2 * i + 1];
              x = __float_as_uint(__uint_as_float(x) + lo);
              y = __float_as_uint(__uint_as_float(y) + hi);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = Half16<T>::pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        w[16 + i] = Half16<T>::pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
      }
    }
    if (c + cols >= width) release();
    if (lane == 0) tma_store_wait_read<BUFS - 1>();     // the box's last store has read it
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 128 +
                                                                   ((q ^ (lane & 7)) * 16)),
                   "r"(w[4 * q]), "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                   : "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0)
      tma_store_3d(tmD, box, k0 + c, n0, e, a.accumulate && a.out_f32);
  }
}

}  // namespace moe
