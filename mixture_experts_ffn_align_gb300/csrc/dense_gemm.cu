// Products of E matrices of one size in fp16, on one SM per tile: plan and launch
// (the kernel is in ragged_one.cuh, tiles and epilogue in ragged_epi.cuh).
#include "dense_gemm.h"
#include "ragged_one.cuh"

namespace moe {

namespace {

// Tiles, and CTAs that share the reduction of one.  Symmetric outputs are computed
// in square tiles on and below the diagonal, unless there are so few tiles that the
// reduction is sliced.
struct DensePlan {
  int tile_rows, per, tok_tiles, w_tiles, splits;
  bool tri;
  long long e_tiles;
};
DensePlan plan_of(const DenseProduct& d) {
  DensePlan r;
  r.tile_rows = d.m <= 32 ? 32 : d.m <= 64 ? 64 : d.m <= 128 ? 128 : 256;
  r.w_tiles = (d.width + 127) / 128;
  r.tok_tiles = (d.m + r.tile_rows - 1) / r.tile_rows;
  r.per = ((d.m + r.tok_tiles - 1) / r.tok_tiles + 15) / 16 * 16;
  r.e_tiles = (long long)r.w_tiles * r.tok_tiles;
  r.splits = rag_slices(r.e_tiles * d.E, d.segs * d.seg_kb, kLeastSteps);
  r.tri = d.symmetric && r.splits == 1;
  if (r.tri) {
    r.tile_rows = r.per = 128;
    r.tok_tiles = r.w_tiles;
    r.e_tiles = (long long)r.w_tiles * (r.w_tiles + 1) / 2;
  }
  return r;
}

}  // namespace

size_t dense_part_bytes(const DenseProduct& d) {
  const DensePlan r = plan_of(d);
  return r.splits > 1 ? (size_t)r.e_tiles * d.E * r.splits * r.tile_rows * 128 * sizeof(float) : 0;
}

bool dense_on_pairs(const DenseProduct& d) {
  if (ragged_form() != 0) return ragged_form() != 1;
  const DensePlan r = plan_of(d);
  const long long kb = (long long)d.segs * d.seg_kb;
  // Cycles as the ragged products' model has them: a step's operands at 50 bytes a
  // cycle from L2 or its MMAs, and a tile's fixed cost.
  const auto step = [](int a, int b, int n) { return std::max((a + b) / 50, 53 * n / 20); };
  const int n1 = r.tri ? 128 : r.per;
  const long long tiles1 = r.e_tiles * d.E;
  const long long one = r.splits > 1
                            ? kb / r.splits * step(16384, n1 * 128, n1) + 4000 + 50 * n1
                            : (tiles1 + 151) / 152 * (kb * step(16384, n1 * 128, n1) + 1200);
  const int w2 = (d.width + 255) / 256, t2 = (d.m + 255) / 256;
  const int n2 = d.symmetric ? 256 : ((d.m + t2 - 1) / t2 + 31) / 32 * 32;
  const long long tiles2 = (d.symmetric ? (long long)w2 * (w2 + 1) / 2 : (long long)w2 * t2) * d.E;
  const long long two = (tiles2 + 75) / 76 * (kb * step(16384, n2 * 64, n2) + 1400) + 3000;
  return two < one;
}

cudaError_t launch_dense(const DenseProduct& d, void* workspace, cudaStream_t stream) {
  CUtensorMap tmA, tmB;
  if (!(d.nt ? make_tmap_rag(&tmA, d.w, true, 3, d.w_ld, d.m, d.E, d.w_ld, 128)
             : make_tmap_rag_wide(&tmA, d.w, true, d.m, d.w_ld, d.E, d.w_ld, 2)) ||
      !make_tmap_rag(&tmB, d.rows, true, 2, d.rows_ld, (uint64_t)d.E * d.m, 0, d.rows_ld, 32))
    return cudaErrorInvalidValue;
  const DensePlan r = plan_of(d);
  RagArgs a{};
  dense_args(d, r.tri, r.per, r.tok_tiles, r.e_tiles, a);
  a.tile_rows = r.tile_rows;
  a.w_tiles = fast_div(r.w_tiles);
  a.splits = r.splits;
  a.part = static_cast<float*>(workspace);
  a.stages = std::min(MAX_STAGES, RING_BYTES / (A_BYTES + a.tile_rows * BK * 2));
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  const long long tiles = r.e_tiles * d.E;
  const int grid = a.splits > 1 ? (int)tiles * a.splits
                                : (int)std::min<long long>(num_sms(), tiles);
  return d.nt ? launch_one<RAG_FWD, __half, EPI_DENSE>(tmA, tmB, tmB, a, grid, stream)
              : launch_one<RAG_DGRAD, __half, EPI_DENSE>(tmA, tmB, tmB, a, grid, stream);
}

}  // namespace moe
