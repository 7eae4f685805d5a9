// Products of E matrices of one size in fp16, on SM pairs: launch (the kernel is in
// ragged_pair.cuh, tiles and epilogue in ragged_epi.cuh).
#include "dense_gemm.h"
#include "ragged_pair.cuh"

namespace moe {

cudaError_t launch_dense_2sm(const DenseProduct& d, cudaStream_t stream) {
  CUtensorMap tmA, tmB, tmC;
  const uint64_t rows = (uint64_t)d.E * d.m;
  if (!(d.nt ? make_tmap_rag(&tmA, d.w, true, 3, d.w_ld, d.m, d.E, d.w_ld, 128)
             : make_tmap_rag_wide(&tmA, d.w, true, d.m, d.w_ld, d.E, d.w_ld, 2)) ||
      !make_tmap_rag(&tmB, d.rows, true, 2, d.rows_ld, rows, 0, d.rows_ld, 128) ||
      !make_tmap_rag(&tmC, d.rows, true, 2, d.rows_ld, rows, 0, d.rows_ld, 32))
    return cudaErrorInvalidValue;
  RagArgs a{};
  const int w_tiles = (d.width + 255) / 256;
  int tok_tiles = (d.m + 255) / 256, per = ((d.m + tok_tiles - 1) / tok_tiles + 31) / 32 * 32;
  long long e_tiles = (long long)w_tiles * tok_tiles;
  if (d.nt) {
    per = 256;
    tok_tiles = w_tiles;
    e_tiles = (long long)w_tiles * (w_tiles + 1) / 2;
  }
  dense_args(d, d.nt, per, tok_tiles, e_tiles, a);
  a.tile_rows = 256;
  a.w_tiles = fast_div(w_tiles);
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  const long long tiles = e_tiles * d.E;
  return d.nt ? launch_pair<RAG_FWD, __half, 1, EPI_DENSE>(tmA, tmB, tmC, a, tiles, stream)
              : launch_pair<RAG_DGRAD, __half, 1, EPI_DENSE>(tmA, tmB, tmC, a, tiles, stream);
}

}  // namespace moe
