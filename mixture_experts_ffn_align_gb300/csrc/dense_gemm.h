// Products of E matrices of one size in fp16, fp32 sums (dense_gemm.cu on one SM a
// tile, dense_gemm_2sm.cu on SM pairs):
//   nt:   out[e][r, c] = sum_k rows[e][r, k] w[e][c, k]
//   else  out[e][r, c] = sum_k rows[e][r, k] w[e][k, c]
// and v = c_acc out + c_mat mat + c_diag (r == c), stored in fp16 or, the last
// product, in bf16.  Matrices have m rows; widths of rows and w are multiples of 64
// with zeros behind the values.  segs 1: the operands have fp16's 11 bits; segs 3:
// every matrix is a hi and a lo part side by side, and hi hi + hi lo + lo hi is
// summed, about 22 bits of each operand.
#pragma once

#include "moe_internal.h"
#include "ragged.cuh"

namespace moe {

struct DenseProduct {
  bool nt;                   // rows == w: the output is symmetric
  int E, m;
  int width;                 // columns of the output
  const void* rows;
  int rows_ld, rows_lo;      // row stride, columns from the hi to the lo part
  const void* w;
  int w_ld, w_lo;
  int segs, seg_kb;          // 1 or 3; 64-deep steps of each
  float c_acc, c_mat, c_diag;
  const void* mat;           // as out, or null
  long long mat_lo;          // elements from mat to its lo part, 0: none
  void* out;
  int out_ld;
  long long out_lo;          // as mat_lo
  void* final_out;           // bf16 [E, m, width], transposed [E, width, m]; out unused
  bool transposed;
};

size_t dense_part_bytes(const DenseProduct& d);
// Modelled cycles of the product on its own, and whether SM pairs take fewer.
long long dense_cycles(const DenseProduct& d);
bool dense_on_pairs(const DenseProduct& d);
cudaError_t launch_dense(const DenseProduct& d, void* workspace, cudaStream_t stream);
cudaError_t launch_dense_2sm(const DenseProduct& d, cudaStream_t stream);

inline void dense_args(const DenseProduct& d, bool tri, int per, int tok_tiles, long long e_tiles,
                       RagArgs& a) {
  a.R = d.E * d.m;
  a.E = d.E;
  a.W = d.width;
  a.num_kb = d.segs * d.seg_kb;
  a.group_max = 8;
  a.wide_a = 1;
  a.out = d.out;
  a.ldo = d.out_ld;
  RagDense& q = a.dense;
  q.m = d.m;
  q.mp = d.width;
  q.sym = d.nt;
  q.tri = tri;
  q.per = per;
  q.tok_tiles = tok_tiles;
  q.e_tiles = fast_div((int)e_tiles);
  q.seg_kb = d.seg_kb;
  q.a_lo = d.w_lo;
  q.b_lo = d.rows_lo;
  q.c_acc = d.c_acc;
  q.c_mat = d.c_mat;
  q.c_diag = d.c_diag;
  q.mat = static_cast<const __half*>(d.mat);
  q.mat_lo = d.mat_lo;
  q.out_lo = d.out_lo;
  q.final_out = static_cast<__nv_bfloat16*>(d.final_out);
  q.transposed = d.transposed;
}

}  // namespace moe
