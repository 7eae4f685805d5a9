// One launch for all steps of the orthogonalised update (ortho_cluster.cu): clusters for
// small matrices, the whole grid for those between small and large.
#pragma once

#include "../../include/moe_ffn.h"
#include "moe_internal.h"

namespace moe {

// Tiles of a product of one matrix, and slices of their reduction.
struct OrthoTiles {
  int per, tok_tiles, w_tiles, splits;
  int tri, tiles;            // tri: on and below the diagonal
};
struct OrthoClusterPlan {
  int ctas;                  // of a cluster; 0: the whole grid
  int stages, stage_bytes;
  OrthoTiles t[3];           // A = X X^T, B, X = B X
  long long cycles;          // modelled
};
struct OrthoClusterProblem {
  OrthoClusterPlan plan;
  int E, m, M, mp, Mp, parts, steps;
  bool transposed;
  void *x[2], *lo, *a, *b, *out, *part;
  int kept;                  // steps that add a X from x and lo
  float c_gram, c_apply, c_last;
  const float* coef;         // of each step: a (kept) or c_diag, c_mat and c_acc of B
  uint32_t* done;            // [E], zeros: tiles finished (whole grid)
};
OrthoClusterPlan ortho_cluster_plan(int E, int m, int mp, int M, int Mp, int parts, int steps);
OrthoClusterPlan ortho_grid_plan(int E, int m, int mp, int M, int Mp, int parts, int steps);
size_t ortho_cluster_part_bytes(const OrthoClusterPlan& p, int E);
cudaError_t launch_ortho_cluster(const OrthoClusterProblem& d, cudaStream_t stream);

}  // namespace moe
