// Ragged grouped products on SM pairs: launches (the kernel is in
// ragged_pair.cuh).
#include "ragged_pair.cuh"

namespace moe {

namespace {

template <int OP, int MT>
cudaError_t launch_op(bool half, const CUtensorMap& tmA, const CUtensorMap& tmB,
                      const CUtensorMap& tmC, const RagArgs& a,
                      long long tiles, cudaStream_t stream) {
  return half ? launch_pair<OP, __half, MT>(tmA, tmB, tmC, a, tiles, stream)
              : launch_pair<OP, __nv_bfloat16, MT>(tmA, tmB, tmC, a, tiles, stream);
}

}  // namespace

// double_tiles: a CTA then takes in 24 KB a tile and step instead of 32, which
// counts where the pairs run at the rate L2 feeds them (or at the power limit);
// but both accumulators are in use until a tile ends, so it costs the time to
// read them, 2500 to 8000 cycles.  Pairs / double tiles, 8 experts of 1030 rows:
// 4096 -> 28672 forward 1211 / 1185 us, of 128 rows: 6704 -> 2968 dgrad 77 / 62;
// 8192 rows, 4096 -> 14336 forward 518 / 559.
cudaError_t launch_ragged_rows_2sm(const RaggedProblem& p, int op, bool double_tiles,
                                   const void* rows, const void* w,
                                   const void* bias, void* out,
                                   cudaStream_t stream) {
  const bool fwd = op == RAG_FWD;
  CUtensorMap tmA, tmB, tmC;
  const int red = fwd ? p.K : p.N;
  const bool wide = !fwd && p.K % 64 == 0;
  if (!(wide ? make_tmap_rag_wide(&tmA, w, p.half, p.N, p.K, p.E, p.K, 2)
             : make_tmap_rag(&tmA, w, p.half, 3, p.K, p.N, p.E, p.K, fwd ? 128 : 64)) ||
      !make_tmap_rag(&tmB, rows, p.half, 2, red, p.R, 0, fwd ? p.ldx : p.ldy, 128) ||
      !make_tmap_rag(&tmC, rows, p.half, 2, red, p.R, 0, fwd ? p.ldx : p.ldy, 32))
    return cudaErrorInvalidValue;
  RagArgs a{};
  if (!pair_args(p, a)) return cudaErrorInvalidDevice;
  a.W = fwd ? p.N : p.K;
  a.num_kb = (red + BK - 1) / BK;
  const int mt = double_tiles ? 2 : 1;
  a.w_tiles = fast_div((a.W + 256 * mt - 1) / (256 * mt));
  a.wide_a = wide;
  a.out = out;
  a.ldo = fwd ? p.ldy : p.ldx;
  a.bias = bias;
  const long long tiles = ((long long)std::min(p.E, p.R) + p.R / 256) * a.w_tiles.d;   // at most
  const auto launch = fwd ? (mt == 2 ? launch_op<RAG_FWD, 2> : launch_op<RAG_FWD, 1>)
                          : (mt == 2 ? launch_op<RAG_DGRAD, 2> : launch_op<RAG_DGRAD, 1>);
  return launch(p.half, tmA, tmB, tmC, a, tiles, stream);
}

cudaError_t launch_ragged_wgrad_2sm(const RaggedProblem& p, const void* dy, const void* x,
                                    void* dw, bool out_f32, bool accumulate,
                                    cudaStream_t stream) {
  CUtensorMap tmA, tmB, tmC;
  const bool wide_a = p.N % 64 == 0, wide_b = p.K % 64 == 0;
  if (!(wide_a ? make_tmap_rag_wide(&tmA, dy, p.half, p.R, p.N, 1, p.ldy, 2)
               : make_tmap_rag(&tmA, dy, p.half, 2, p.N, p.R, 0, p.ldy, 64)) ||
      !(wide_b ? make_tmap_rag_wide(&tmB, x, p.half, p.R, p.K, 1, p.ldx, 2)
               : make_tmap_rag(&tmB, x, p.half, 2, p.K, p.R, 0, p.ldx, 64)) ||
      !make_tmap_rag_store(&tmC, dw, out_f32 ? 2 : p.half ? 1 : 0, p.K, p.N, p.E))
    return cudaErrorInvalidValue;
  RagArgs a{};
  if (!pair_args(p, a)) return cudaErrorInvalidDevice;
  a.N = p.N;
  a.K = p.K;
  a.w_tiles = fast_div((p.N + 255) / 256);
  a.k_tiles = fast_div((p.K + 255) / 256);
  a.e_tiles = fast_div(a.w_tiles.d * a.k_tiles.d);
  a.wide_a = wide_a;
  a.wide_b = wide_b;
  a.out = dw;
  a.out_f32 = out_f32;
  a.accumulate = accumulate;
  return launch_op<RAG_WGRAD, 1>(p.half, tmA, tmB, tmC, a, (long long)p.E * a.e_tiles.d, stream);
}

}  // namespace moe
