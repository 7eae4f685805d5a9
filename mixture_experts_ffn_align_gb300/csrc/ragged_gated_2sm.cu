// The gated forward product and its gradient on SM pairs: launches (the kernel is
// in ragged_pair.cuh, the epilogues in ragged_epi.cuh).
#include "ragged_pair.cuh"

namespace moe {

cudaError_t launch_ragged_gated_2sm(const RaggedProblem& p, const GatedProblem& g,
                                    const void* rows, const void* w, const void* bias,
                                    cudaStream_t stream) {
  const bool fwd = !g.grad;
  CUtensorMap tmA, tmB, tmC;
  const int red = fwd ? p.K : p.N;
  const long long ld = fwd ? p.ldx : p.ldy;
  const bool wide = !fwd && p.K % 64 == 0;
  if (!(fwd    ? make_tmap_rag_gated(&tmA, w, p.half, p.K, p.N / 2, p.E)
        : wide ? make_tmap_rag_wide(&tmA, w, p.half, p.N, p.K, p.E, p.K, 2)
               : make_tmap_rag(&tmA, w, p.half, 3, p.K, p.N, p.E, p.K, 64)) ||
      !make_tmap_rag(&tmB, rows, p.half, 2, red, p.R, 0, ld, 128) ||
      !make_tmap_rag(&tmC, rows, p.half, 2, red, p.R, 0, ld, 32))
    return cudaErrorInvalidValue;
  RagArgs a{};
  if (!pair_args(p, a)) return cudaErrorInvalidDevice;
  a.W = fwd ? p.N : p.K;
  a.num_kb = (red + BK - 1) / BK;
  a.w_tiles = fast_div((a.W + 255) / 256);
  a.wide_a = wide;
  a.bias = bias;
  gated_args(g, a.gated);
  const long long tiles = ((long long)std::min(p.E, p.R) + p.R / 256) * a.w_tiles.d;   // at most
  const auto launch = fwd ? (p.half ? launch_pair<RAG_FWD, __half, 1, EPI_GATED>
                                    : launch_pair<RAG_FWD, __nv_bfloat16, 1, EPI_GATED>)
                          : (p.half ? launch_pair<RAG_DGRAD, __half, 1, EPI_GATED_GRAD>
                                    : launch_pair<RAG_DGRAD, __nv_bfloat16, 1, EPI_GATED_GRAD>);
  return launch(tmA, tmB, tmC, a, tiles, stream);
}

}  // namespace moe
