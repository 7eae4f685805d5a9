// Fused epilogues of the ragged products' kernels (ragged_one.cuh,
// ragged_pair.cuh), and the tiles of a batch of dense products.
//
// EPI_GATED, on the forward product with w13 [E, 2 I, K], gate rows first:
//   h = x W^T (+ bias),  z = g' s(alpha g') (u' + beta),   s(v) = 1 / (1 + e^-v),
//   g' = min(g, limit), u' = clamp(u, -limit, limit), g and u the halves of h.
// A tile's weights are gate and up rows in turn, eight of each
// (make_tmap_rag_gated), so that g and u of a column meet in lanes l and l ^ 8 of one
// warp and the tile, its accumulators and its slices stay those of the plain
// product.  The two lanes swap half of their tokens, and each computes z for half.
// (Gate and up rows in an accumulator each would need both until a tile ends.)
// z is computed from the fp32 sums, not from h's rounded values.
//
// EPI_GATED_GRAD, on the gradient product dz = dy W2 with w2 [E, K, I]:
//   dg = dz (u' + beta) s (1 + alpha g' (1 - s))  where g <= limit, else 0,
//   du = dz g' s                                  where |u| <= limit, else 0,
//   z as above, for the gradient of w2.
// dz itself is never rounded or stored.  Two neighbouring lanes swap tokens first,
// so that each reads and writes both columns of a token as 4-byte pieces, 64 bytes
// of a row a half-warp.
//
// EPI_DENSE: E products of matrices of m rows, in fp16 with hi and lo parts where
// that is asked for (mat_lo, out_lo): v = c_acc sum + c_mat mat + c_diag (row ==
// column), rounded to fp16 (lo = v - hi), or the last product in bf16.
#pragma once

#include "moe_internal.h"
#include "ragged.cuh"

namespace moe {

// ---------------------------------------------------------------- activation
// CLAMP: with a limit (the comparisons are a fifth of a gradient's instructions).
template <bool CLAMP>
__device__ __forceinline__ float gated_min(float v, float limit) {
  return CLAMP && v > limit ? limit : v;
}
template <bool CLAMP>
__device__ __forceinline__ float gated_clamp(float v, float limit) {
  return !CLAMP ? v : v > limit ? limit : v < -limit ? -limit : v;      // NaN stays
}
__device__ __forceinline__ float gated_sigmoid(float v) {
  return __fdividef(1.0f, 1.0f + __expf(-v));
}
template <bool CLAMP>
__device__ __forceinline__ float gated_value(const RagGated& a, float g, float u) {
  g = gated_min<CLAMP>(g, a.limit);
  return g * gated_sigmoid(a.alpha * g) * (gated_clamp<CLAMP>(u, a.limit) + a.beta);
}
struct GatedGrad {
  float dg, du, z;
};
template <bool CLAMP>
__device__ __forceinline__ GatedGrad gated_grad(const RagGated& a, float dz, float g, float u) {
  const float gc = gated_min<CLAMP>(g, a.limit), uc = gated_clamp<CLAMP>(u, a.limit) + a.beta;
  const float s = gated_sigmoid(a.alpha * gc), act = gc * s;
  GatedGrad r;
  // (act (1 - s) first: alpha act may be past fp32's range where 1 - s is 0)
  r.dg = CLAMP && g > a.limit ? 0.0f : dz * uc * (s + a.alpha * (act * (1.0f - s)));
  r.du = CLAMP && fabsf(u) > a.limit ? 0.0f : dz * act;
  r.z = act * uc;
  return r;
}
template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  return make_float2(Half16<T>::value((uint16_t)(w & 0xFFFFu)), Half16<T>::value((uint16_t)(w >> 16)));
}

inline void gated_args(const GatedProblem& g, RagGated& a) {
  a.h = g.h;
  a.h_out = g.h_out;
  a.z = g.z;
  a.ldh = g.ldh;
  a.ldh_out = g.ldh_out;
  a.ldz = g.ldz;
  a.inter = g.inter;
  a.alpha = g.alpha;
  a.beta = g.beta;
  a.limit = g.limit > 0.0f ? g.limit : __builtin_huge_valf();
}

// Interleaved row w of the gate and up weights: column w of the tile is column
// gated_col(w) of the gate (up = 0) or up half.
__device__ __forceinline__ int gated_col(int w) { return ((w >> 4) << 3) + (w & 7); }

// All fused epilogues take sixteen tokens at a time: with 32, twice the unrolled code and
// registers, the gated product and its gradient took 1 to 8% longer (512 rows, 16
// experts, 776 -> 520: 9.5 us instead of 8.7), the steps of the update's short products a
// sixth (16 x 517 x 1031: 58 us instead of 50).
//
// 16 tokens from row row0 of this lane's interleaved column w.
template <typename T, bool CLAMP>
__device__ __forceinline__ void rag_gated_tokens16(const RagArgs& a, uint32_t (&r)[16], float bias,
                                                   long long row0, int live, int w, int lane) {
  const RagGated& q = a.gated;
  const int up = (w >> 3) & 1, col = gated_col(w), odd = lane & 1;
  const bool inside = w < a.W;
  const uint32_t sel = odd ? 0x3276u : 0x5410u;
#pragma unroll
  for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + bias);
  if (q.h_out != nullptr) {      // neighbouring columns swap: 4-byte pieces of two tokens
    uint16_t* p = static_cast<uint16_t*>(q.h_out) + (row0 + odd) * q.ldh_out + up * q.inter + col - odd;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t pk = Half16<T>::pack(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
      const uint32_t v = __byte_perm(pk, __shfl_xor_sync(0xffffffffu, pk, 1), sel);
      if (inside && 2 * j + odd < live) *reinterpret_cast<uint32_t*>(p) = v;
      p += 2 * q.ldh_out;
    }
  }
  // the gate's lane takes the even tokens, the up half's the odd ones; then of
  // neighbouring columns an even lane both columns of the first token
  const int tok0 = up + 2 * odd;
  uint16_t* p = static_cast<uint16_t*>(q.z) + (row0 + tok0) * q.ldz + (col - odd);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float z[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = 2 * i + k;
      const uint32_t other = __shfl_xor_sync(0xffffffffu, up ? r[2 * j] : r[2 * j + 1], 8);
      z[k] = gated_value<CLAMP>(q, __uint_as_float(up ? other : r[2 * j]),
                                __uint_as_float(up ? r[2 * j + 1] : other));
    }
    const uint32_t pk = Half16<T>::pack(z[0], z[1]);     // tokens 4 i + up and 4 i + up + 2
    const uint32_t v = __byte_perm(pk, __shfl_xor_sync(0xffffffffu, pk, 1), sel);
    if (inside && tok0 + 4 * i < live) *reinterpret_cast<uint32_t*>(p) = v;
    p += 4 * q.ldz;
  }
}

// Two words at a lane's two columns of every other of 16 tokens, read a chunk ahead (the
// first before the sums are complete): read where they are used, they kept the gradient
// of 8 x (2048, 1024), 256 rows each, at 28 us instead of 20.
struct Words16 {
  uint32_t a[8], b[8];
};
// h for the gradient.  c: tokens of the tile before the 16.
__device__ __forceinline__ void rag_gated_load(const RagArgs& a, const RagTile& D, Words16& x, int c,
                                               int w, int lane) {
  const RagGated& q = a.gated;
  const int odd = lane & 1, live = D.rows - c;
  const bool inside = w < a.W;
  const uint16_t* h = static_cast<const uint16_t*>(q.h) + (long long)(D.row0 + c + odd) * q.ldh +
                      (w - odd);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = inside && 2 * j + odd < live;
    x.a[j] = in ? *reinterpret_cast<const uint32_t*>(h) : 0u;
    x.b[j] = in ? *reinterpret_cast<const uint32_t*>(h + q.inter) : 0u;
    h += 2 * q.ldh;
  }
}

// 16 tokens from row row0 of this lane's column w of dz.
template <typename T, bool CLAMP>
__device__ __forceinline__ void rag_gated_grad_tokens16(const RagArgs& a, const uint32_t (&r)[16],
                                                        const Words16& h, long long row0, int live,
                                                        int w, int lane) {
  const RagGated& q = a.gated;
  const int odd = lane & 1, c0 = w - odd;
  const bool inside = w < a.W;
  uint16_t* dh = static_cast<uint16_t*>(q.h_out) + (row0 + odd) * q.ldh_out + c0;
  uint16_t* z = static_cast<uint16_t*>(q.z) + (row0 + odd) * q.ldz + c0;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? r[2 * t] : r[2 * t + 1], 1);
    const float dz0 = __uint_as_float(odd ? other : r[2 * t]);
    const float dz1 = __uint_as_float(odd ? r[2 * t + 1] : other);
    const float2 g = unpack16<T>(h.a[t]), u = unpack16<T>(h.b[t]);
    const GatedGrad x = gated_grad<CLAMP>(q, dz0, g.x, u.x), y = gated_grad<CLAMP>(q, dz1, g.y, u.y);
    if (inside && 2 * t + odd < live) {
      *reinterpret_cast<uint32_t*>(dh) = Half16<T>::pack(x.dg, y.dg);
      *reinterpret_cast<uint32_t*>(dh + q.inter) = Half16<T>::pack(x.du, y.du);
      if (q.z != nullptr) *reinterpret_cast<uint32_t*>(z) = Half16<T>::pack(x.z, y.z);
    }
    dh += 2 * q.ldh_out;
    z += 2 * q.ldz;
  }
}

// --------------------------------------------------------------- dense products
// Tile t of the batch.  rows: of a symmetric product those of its padded output,
// which has zeros there.  tri: the tiles (w_tile, tok) with tok <= w_tile; else
// groups of 8 token tiles, as rag_tile.
__device__ __forceinline__ void rag_triangle(int l, RagTile& T) {
  // l = i (i + 1) / 2 + tok: i from the square root, which is off by one at most
  int i = (int)((sqrtf(8.0f * (float)l + 1.0f) - 1.0f) * 0.5f);
  if (i * (i + 1) / 2 > l) --i;
  if ((i + 1) * (i + 2) / 2 <= l) ++i;
  T.w_tile = i;
  T.tok = l - i * (i + 1) / 2;
}
__device__ __forceinline__ RagTile rag_dense_tile(const RagArgs& a, int t) {
  const RagDense& q = a.dense;
  RagTile T;
  T.e = t / q.e_tiles;
  const int l = t - T.e * q.e_tiles.d;
  if (q.tri) {
    rag_triangle(l, T);
    T.rows = min(q.per, q.mp - T.tok * q.per);
  } else {
    const int w_tiles = a.w_tiles.d;
    const int c = q.tok_tiles <= 8 ? 0 : l / (8 * w_tiles);
    const int gm = min(8, q.tok_tiles - 8 * c);
    const int l2 = l - 8 * c * w_tiles;
    T.w_tile = l2 / gm;
    T.tok = 8 * c + (l2 - T.w_tile * gm);
    T.rows = min(q.per, (q.sym ? q.mp : q.m) - T.tok * q.per);
  }
  T.row0 = T.e * q.m + T.tok * q.per;
  return T;
}

__device__ __forceinline__ uint32_t half_hi2(float& x, float& y) {
  const uint32_t p = Half16<__half>::pack(x, y);
  const float2 v = unpack16<__half>(p);
  x -= v.x;
  y -= v.y;
  return p;
}

// mat and its lo part at two columns of 16 tokens.
template <bool FULL, bool LO>
__device__ __forceinline__ void rag_load_mat(Words16& x, const uint16_t* mat, long long lo,
                                             long long ld, int live, int odd) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = FULL || 2 * j + odd < live;
    x.a[j] = in ? __ldcg(reinterpret_cast<const uint32_t*>(mat)) : 0u;
    x.b[j] = LO && in ? __ldcg(reinterpret_cast<const uint32_t*>(mat + lo)) : 0u;
    mat += 2 * ld;
  }
}
__device__ __forceinline__ void rag_dense_load(const RagArgs& a, const RagTile& D, Words16& x, int c,
                                               int w, int lane) {
  const RagDense& q = a.dense;
  const int odd = lane & 1, live = min(D.rows - c, q.m - (D.row0 - D.e * q.m) - c);
  const bool inside = w < a.W, full = w - lane + 32 <= a.W && live >= 16;
  const uint16_t* mat = reinterpret_cast<const uint16_t*>(q.mat) +
                        (long long)(D.row0 + c + odd) * a.ldo + (w - odd);
  if (q.mat_lo == 0) {
    if (full)
      rag_load_mat<true, false>(x, mat, 0, a.ldo, 16, odd);
    else
      rag_load_mat<false, false>(x, mat, 0, a.ldo, inside ? live : 0, odd);
  } else {
    if (full)
      rag_load_mat<true, true>(x, mat, q.mat_lo, a.ldo, 16, odd);
    else
      rag_load_mat<false, true>(x, mat, q.mat_lo, a.ldo, inside ? live : 0, odd);
  }
}

// The last product: 16 tokens from row tok (of the matrix) of this lane's column w,
// `live` of them to be stored.
__device__ __forceinline__ void rag_dense_final16(const RagArgs& a, const RagTile& D,
                                                  const uint32_t (&r)[16], int tok, int live, int w,
                                                  int lane) {
  const RagDense& q = a.dense;
  uint32_t pk[8];              // tokens 2 j and 2 j + 1
#pragma unroll
  for (int j = 0; j < 8; ++j)
    pk[j] = Half16<__nv_bfloat16>::pack(q.c_acc * __uint_as_float(r[2 * j]),
                                        q.c_acc * __uint_as_float(r[2 * j + 1]));
  uint16_t* out = reinterpret_cast<uint16_t*>(q.final_out);
  if (!q.transposed) {
    out += ((long long)D.e * q.m + tok) * a.W + w;
    if (a.W % 2 == 0) {        // neighbouring columns swap: 4-byte pieces of two tokens
      const int odd = lane & 1;
      out += odd ? a.W - 1 : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t v = __byte_perm(pk[j], __shfl_xor_sync(0xffffffffu, pk[j], 1),
                                       odd ? 0x3276u : 0x5410u);
        if (w < a.W && 2 * j + odd < live) *reinterpret_cast<uint32_t*>(out) = v;
        out += 2 * a.W;
      }
    } else if (w < a.W) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < live) out[(long long)j * a.W] = (uint16_t)(pk[j >> 1] >> (16 * (j & 1)));
    }
    return;
  }
  // a lane's tokens lie side by side
  if (q.m % 8 == 0 && live >= 16) {
    uint4* to = reinterpret_cast<uint4*>(out + ((long long)D.e * a.W + w) * q.m + tok);
    if (w < a.W) {
      to[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      to[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
    }
    return;
  }
  // Rows that start anywhere, or end here: the warp's 32 x 16 values are turned, so that a
  // store writes two rows' 16 tokens.  (From each lane's own row they went out as 32
  // sectors for 64 bytes: 16 matrices of 1031 x 517 took 90 us here instead of 22.)
#pragma unroll
  for (int o = 8; o >= 2; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j & (o >> 1)) continue;
      const int k = j | (o >> 1);
      const uint32_t x = __shfl_xor_sync(0xffffffffu, up ? pk[j] : pk[k], o);
      if (up) pk[j] = x; else pk[k] = x;
    }
  }
  // now pk[j]: a pair of tokens of row 2 j + (lane & 17); the low half after the swap
  // this lane's token of row 2 j + (lane & 16), the high half that of the next row
  const int row0 = w - lane + (lane & 16), t = lane & 15;
  uint16_t* to = out + ((long long)D.e * a.W + row0) * q.m + tok + t;
  const uint32_t sel = (lane & 1) ? 0x3276u : 0x5410u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t x = __byte_perm(pk[j], __shfl_xor_sync(0xffffffffu, pk[j], 1), sel);
    if (t < live && row0 + 2 * j < a.W) to[(long long)2 * j * q.m] = (uint16_t)(x & 0xFFFFu);
    if (t < live && row0 + 2 * j + 1 < a.W) to[(long long)(2 * j + 1) * q.m] = (uint16_t)(x >> 16);
  }
}

// The others: two neighbouring lanes swap tokens first.  A lo part of mat may be the
// output's own: each word is read and written by one lane.  Of a symmetric product's
// tiles beside the diagonal (tri) the values are stored once more as rows from the
// columns: lanes swap back, and two of them put 32 bytes of a row together.
template <bool SYM, bool LO, bool FULL>
__device__ __forceinline__ void rag_dense_pairs16(const RagArgs& a, const RagTile& D,
                                                  const uint32_t (&r)[16], const Words16& h,
                                                  bool loads, int tok, int live, int w, int lane) {
  const RagDense& q = a.dense;
  const int odd = lane & 1;
  const long long base = (long long)D.e * q.m;
  uint16_t* out = static_cast<uint16_t*>(a.out) + (base + tok + odd) * a.ldo + w - odd;
  uint32_t pk[8], lo[8];
  const int diagonal = SYM ? w - tok : -1;       // this lane's token in its column
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? r[2 * t] : r[2 * t + 1], 1);
    float x = q.c_acc * __uint_as_float(odd ? other : r[2 * t]);
    float y = q.c_acc * __uint_as_float(odd ? r[2 * t + 1] : other);
    if (loads) {
      const float2 mh = unpack16<__half>(h.a[t]), ml = unpack16<__half>(h.b[t]);
      x += q.c_mat * (LO || !SYM ? mh.x + ml.x : mh.x);
      y += q.c_mat * (LO || !SYM ? mh.y + ml.y : mh.y);
    }
    if (SYM && diagonal == 2 * t + odd) {
      if (odd) y += q.c_diag; else x += q.c_diag;
    }
    const bool in = FULL || 2 * t + odd < live;
    if (SYM && !FULL) {       // rows behind the matrix (the next one's) are zero columns
      x = in ? x : 0.0f;
      y = in ? y : 0.0f;
    }
    pk[t] = half_hi2(x, y);
    if (in && (FULL || w < a.W)) *reinterpret_cast<uint32_t*>(out) = pk[t];
    if (LO) {
      lo[t] = Half16<__half>::pack(x, y);
      if (in && (FULL || w < a.W)) *reinterpret_cast<uint32_t*>(out + q.out_lo) = lo[t];
    }
    out += 2 * a.ldo;
  }
  if (!SYM || !q.tri || D.tok == D.w_tile) return;
#pragma unroll
  for (int part = 0; part < (LO ? 2 : 1); ++part) {
    // tokens 2 t and 2 t + 1 of this lane's column w
    uint32_t p[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t v = part == 0 ? pk[t] : lo[t];
      p[t] = __byte_perm(v, __shfl_xor_sync(0xffffffffu, v, 1), odd ? 0x3276u : 0x5410u);
    }
    // the two 16-byte pieces of two lanes' rows: one piece of both rows each
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __shfl_xor_sync(0xffffffffu, odd ? p[i] : p[4 + i], 1);
    const int w0 = w - odd;
    uint16_t* to = static_cast<uint16_t*>(a.out) + (base + w0) * a.ldo + tok + 8 * odd +
                   (part == 0 ? 0 : q.out_lo);
    if (w0 < q.m)
      *reinterpret_cast<uint4*>(to) = odd ? make_uint4(u[0], u[1], u[2], u[3])
                                          : make_uint4(p[0], p[1], p[2], p[3]);
    if (w0 + 1 < q.m)
      *reinterpret_cast<uint4*>(to + a.ldo) = odd ? make_uint4(p[4], p[5], p[6], p[7])
                                                  : make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// 16 tokens from row tok (of the matrix) of this lane's column w; left: the tile's
// (the next tile's may be among the 16).
template <bool SYM>
__device__ __forceinline__ void rag_dense_store16(const RagArgs& a, const RagTile& D,
                                                  const uint32_t (&r)[16], const Words16& h,
                                                  bool loads, int tok, int left, int w, int lane) {
  const int live = min(a.dense.m - tok, left);
  const bool full = live >= 16 && w - lane + 32 <= a.W;
  if (!SYM && a.dense.final_out != nullptr)
    rag_dense_final16(a, D, r, tok, live, w, lane);
  else if (full && a.dense.out_lo == 0)
    rag_dense_pairs16<SYM, false, true>(a, D, r, h, loads, tok, 16, w, lane);
  else if (full)
    rag_dense_pairs16<SYM, true, true>(a, D, r, h, loads, tok, 16, w, lane);
  else if (a.dense.out_lo == 0)
    rag_dense_pairs16<SYM, false, false>(a, D, r, h, loads, tok, live, w, lane);
  else
    rag_dense_pairs16<SYM, true, false>(a, D, r, h, loads, tok, live, w, lane);
}

// ------------------------------------------------------------- joining slices
// As rag_join_tokens, with the fused epilogues: a lane has the sums of the four
// columns from w of row D.row0 + j.  Loads of what other CTAs of the cluster wrote
// in this launch bypass L1 (__ldcg).
template <int EPI, typename T>
__device__ __forceinline__ void rag_join_store(const RagArgs& a, const RagTile& D, int j, int w,
                                               float4 x) {
  const long long row = D.row0 + j;
  if (EPI == EPI_GATED) {
    const RagGated& q = a.gated;
    const int up = (w >> 3) & 1, col = gated_col(w);
    if (a.bias != nullptr && w < a.W) {
      const uint16_t* b =
          static_cast<const uint16_t*>(a.bias) + (long long)D.e * a.W + up * q.inter + col;
      x = make_float4(x.x + Half16<T>::value(b[0]), x.y + Half16<T>::value(b[1]),
                      x.z + Half16<T>::value(b[2]), x.w + Half16<T>::value(b[3]));
    }
    // the same columns of the other half are two lanes on
    const float4 o = make_float4(__shfl_xor_sync(0xffffffffu, x.x, 2),
                                 __shfl_xor_sync(0xffffffffu, x.y, 2),
                                 __shfl_xor_sync(0xffffffffu, x.z, 2),
                                 __shfl_xor_sync(0xffffffffu, x.w, 2));
    if (w >= a.W) return;
    if (q.h_out != nullptr)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(q.h_out) + row * q.ldh_out + up * q.inter +
                                col) =
          make_uint2(Half16<T>::pack(x.x, x.y), Half16<T>::pack(x.z, x.w));
    if (!up)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(q.z) + row * q.ldz + col) =
          make_uint2(Half16<T>::pack(gated_value<true>(q, x.x, o.x), gated_value<true>(q, x.y, o.y)),
                     Half16<T>::pack(gated_value<true>(q, x.z, o.z), gated_value<true>(q, x.w, o.w)));
  } else if (EPI == EPI_GATED_GRAD) {
    const RagGated& q = a.gated;
    if (w >= a.W) return;
    const uint16_t* h = static_cast<const uint16_t*>(q.h) + row * q.ldh + w;
    const uint2 hg = *reinterpret_cast<const uint2*>(h);
    const uint2 hu = *reinterpret_cast<const uint2*>(h + q.inter);
    const float2 g0 = unpack16<T>(hg.x), g1 = unpack16<T>(hg.y);
    const float2 u0 = unpack16<T>(hu.x), u1 = unpack16<T>(hu.y);
    const GatedGrad r0 = gated_grad<true>(q, x.x, g0.x, u0.x), r1 = gated_grad<true>(q, x.y, g0.y, u0.y);
    const GatedGrad r2 = gated_grad<true>(q, x.z, g1.x, u1.x), r3 = gated_grad<true>(q, x.w, g1.y, u1.y);
    uint16_t* dh = static_cast<uint16_t*>(q.h_out) + row * q.ldh_out + w;
    *reinterpret_cast<uint2*>(dh) =
        make_uint2(Half16<T>::pack(r0.dg, r1.dg), Half16<T>::pack(r2.dg, r3.dg));
    *reinterpret_cast<uint2*>(dh + q.inter) =
        make_uint2(Half16<T>::pack(r0.du, r1.du), Half16<T>::pack(r2.du, r3.du));
    if (q.z != nullptr)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(q.z) + row * q.ldz + w) =
          make_uint2(Half16<T>::pack(r0.z, r1.z), Half16<T>::pack(r2.z, r3.z));
  } else {
    const RagDense& q = a.dense;
    if (w >= a.W) return;
    float v[4] = {q.c_acc * x.x, q.c_acc * x.y, q.c_acc * x.z, q.c_acc * x.w};
    const int tok = (int)(row - (long long)D.e * q.m);
    if (tok >= q.m) return;                   // sym: rows of the padded output only
    if (q.final_out != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (w + i < a.W)
          q.final_out[q.transposed ? ((long long)D.e * a.W + w + i) * q.m + tok
                                   : row * a.W + w + i] = __float2bfloat16_rn(v[i]);
      return;
    }
    if (q.mat != nullptr) {
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (part == 0 || q.mat_lo != 0) {
          const uint2 m =
              __ldcg(reinterpret_cast<const uint2*>(q.mat + row * a.ldo + w + part * q.mat_lo));
          const float2 m0 = unpack16<__half>(m.x), m1 = unpack16<__half>(m.y);
          v[0] += q.c_mat * m0.x;
          v[1] += q.c_mat * m0.y;
          v[2] += q.c_mat * m1.x;
          v[3] += q.c_mat * m1.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (tok == w + i) v[i] += q.c_diag;
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.ldo + w;
    uint2 hi;
    hi.x = half_hi2(v[0], v[1]);
    hi.y = half_hi2(v[2], v[3]);
    *reinterpret_cast<uint2*>(out) = hi;
    if (q.out_lo != 0)
      *reinterpret_cast<uint2*>(out + q.out_lo) =
          make_uint2(Half16<__half>::pack(v[0], v[1]), Half16<__half>::pack(v[2], v[3]));
  }
}
template <int EPI, typename T>
__device__ __forceinline__ void rag_join_fused(const RagArgs& a, const RagTile& D, int t, int rank,
                                               int ctas, int warp, int warps, int lane) {
  const int w = D.w_tile * 128 + 4 * lane;
  const float* p = a.part + (size_t)t * a.splits * a.tile_rows * 128 + 4 * lane;
  for (int j = rank * warps + warp; j < D.rows; j += ctas * warps) {
    float4 x = __ldcg(reinterpret_cast<const float4*>(p + (size_t)j * 128));
    for (int s = 1; s < a.splits; ++s) {
      const float4 v =
          __ldcg(reinterpret_cast<const float4*>(p + ((size_t)s * a.tile_rows + j) * 128));
      x = make_float4(x.x + v.x, x.y + v.y, x.z + v.z, x.w + v.w);
    }
    rag_join_store<EPI, T>(a, D, j, w, x);
  }
}

// Tile t of a product, whatever its epilogue.
template <int EPI, int G>
__device__ __forceinline__ RagTile rag_any_tile(const RagSched& s, const RagArgs& a, int t) {
  if constexpr (EPI == EPI_DENSE) return rag_dense_tile(a, t);
  return rag_tile<G>(s, a, t);
}

}  // namespace moe
