// The gated forward product and its gradient on one SM per tile: launches (the
// kernel is in ragged_one.cuh, the epilogues in ragged_epi.cuh).
#include "ragged_one.cuh"

namespace moe {

cudaError_t launch_ragged_gated(const RaggedProblem& p, const GatedProblem& g, const void* rows,
                                const void* w, const void* bias, void* workspace,
                                cudaStream_t stream) {
  const bool fwd = !g.grad;
  CUtensorMap tmA, tmB;
  const int red = fwd ? p.K : p.N, width = fwd ? p.N : p.K;
  const bool wide = !fwd && p.K % 64 == 0;
  if (!(fwd    ? make_tmap_rag_gated(&tmA, w, p.half, p.K, p.N / 2, p.E)
        : wide ? make_tmap_rag_wide(&tmA, w, p.half, p.N, p.K, p.E, p.K, 2)
               : make_tmap_rag(&tmA, w, p.half, 3, p.K, p.N, p.E, p.K, 64)) ||
      !make_tmap_rag(&tmB, rows, p.half, 2, red, p.R, 0, fwd ? p.ldx : p.ldy, 32))
    return cudaErrorInvalidValue;
  RagArgs a{};
  const RowsPlan r = rows_plan(p.R, p.E, width, red);
  a.offsets = p.offsets;
  a.R = p.R;
  a.E = p.E;
  a.W = width;
  a.num_kb = (red + BK - 1) / BK;
  a.tile_rows = r.tile_rows;
  a.w_tiles = fast_div(r.w_tiles);
  a.splits = r.splits;
  a.part = static_cast<float*>(workspace);
  a.stages = std::min(MAX_STAGES, RING_BYTES / (A_BYTES + a.tile_rows * BK * 2));
  a.group_max = 8;
  a.wide_a = wide;
  a.bias = bias;
  gated_args(g, a.gated);
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  const int grid = a.splits > 1 ? (int)r.tiles * a.splits
                                : (int)std::min<long long>(num_sms(), r.tiles);
  const auto launch = fwd ? (p.half ? launch_one<RAG_FWD, __half, EPI_GATED>
                                    : launch_one<RAG_FWD, __nv_bfloat16, EPI_GATED>)
                          : (p.half ? launch_one<RAG_DGRAD, __half, EPI_GATED_GRAD>
                                    : launch_one<RAG_DGRAD, __nv_bfloat16, EPI_GATED_GRAD>);
  return launch(tmA, tmB, tmB, a, grid, stream);
}

}  // namespace moe
