// Products of E matrices of one size in fp16, on one SM per tile: plan and launch
// (the kernel is in ragged_one.cuh, tiles and epilogue in ragged_epi.cuh).
#include "dense_gemm.h"
#include "ragged_one.cuh"

namespace moe {

namespace {

// Tiles, and CTAs that share the reduction of one, and the cycles that takes.
struct DensePlan {
  int tile_rows, per, tok_tiles, w_tiles, splits;
  bool tri;
  long long e_tiles, cycles;
};
// The plan of least modelled time.  A step takes its operands from L2 at some 55 bytes
// a cycle, or its MMAs; a tile's epilogue runs under the next tile's steps, the last
// one's and a kernel's start do not; a sliced reduction adds its sums' way through L2.
// Small products want narrow token tiles (more SMs, fewer bytes a step) and slices,
// long ones wide tiles; a symmetric output square ones on and below the diagonal.
// (8 matrices of 256 x 512, a step of 3 products: 38 us with 256 tokens a tile.)
DensePlan plan_of(const DenseProduct& d) {
  DensePlan best{};
  const long long kb = (long long)d.segs * d.seg_kb;
  for (int tile = 32; tile <= 256; tile *= 2) {
    if (tile > 32 && tile >= 2 * d.m) break;
    for (int mode = 0; mode < 5; ++mode) {            // slices, or the triangle
      DensePlan r;
      r.tri = mode == 4;
      r.splits = r.tri ? 1 : 1 << mode;
      if (r.tri && (!d.nt || tile != 128)) continue;
      r.tile_rows = tile;
      r.w_tiles = (d.width + 127) / 128;
      const int rows = d.nt ? d.width : d.m, unit = d.nt ? 32 : 16;
      r.tok_tiles = (rows + tile - 1) / tile;
      r.per = r.tri ? tile : ((rows + r.tok_tiles - 1) / r.tok_tiles + unit - 1) / unit * unit;
      r.e_tiles = r.tri ? (long long)r.w_tiles * (r.w_tiles + 1) / 2
                        : (long long)r.w_tiles * r.tok_tiles;
      const long long tiles = r.e_tiles * d.E;
      if (r.splits > 1 && (tiles > kRagClusters[3 - mode] || kb < 2 * r.splits)) continue;
      const long long steps = (kb + r.splits - 1) / r.splits;
      const long long step = std::max((16384 + (r.per + 31) / 32 * 4096) / 55, 53 * r.per / 20);
      const long long epilogue = (r.tri ? 1500 : 1000) * ((r.per + 63) / 64);
      r.cycles = r.splits > 1 ? 9500 + steps * step + 600 * ((r.per + 63) / 64)
                              : 5000 + (tiles + 151) / 152 * std::max(steps * step, epilogue) + epilogue;
      if (best.cycles == 0 || r.cycles < best.cycles) best = r;
    }
  }
  return best;
}

}  // namespace

size_t dense_part_bytes(const DenseProduct& d) {
  const DensePlan r = plan_of(d);
  return r.splits > 1 ? (size_t)r.e_tiles * d.E * r.splits * r.tile_rows * 128 * sizeof(float) : 0;
}

static long long pairs_cycles(const DenseProduct& d) {
  const long long kb = (long long)d.segs * d.seg_kb;
  const int w = (d.width + 255) / 256, t = (d.m + 255) / 256;
  const int n = d.nt ? 256 : ((d.m + t - 1) / t + 31) / 32 * 32;
  const long long tiles = (d.nt ? (long long)w * (w + 1) / 2 : (long long)w * t) * d.E;
  const long long step = std::max((16384 + n * 64) / 55, 53 * n / 20);
  const long long epilogue = (d.nt ? 1500 : 1000) * ((n + 63) / 64);
  return 8000 + (tiles + 75) / 76 * std::max(kb * step, epilogue) + epilogue;
}
long long dense_cycles(const DenseProduct& d) {
  return std::min(plan_of(d).cycles, pairs_cycles(d));
}
bool dense_on_pairs(const DenseProduct& d) {
  if (ragged_form() != 0) return ragged_form() != 1;
  return pairs_cycles(d) < plan_of(d).cycles;
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
