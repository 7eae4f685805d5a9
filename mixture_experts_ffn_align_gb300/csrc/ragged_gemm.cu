// Ragged grouped products on one SM per tile: launches (the kernel is in
// ragged_one.cuh).
#include "ragged_one.cuh"

namespace moe {

namespace {

template <int OP>
cudaError_t launch_op(bool half, const CUtensorMap& tmA, const CUtensorMap& tmB,
                      const CUtensorMap& tmD, const RagArgs& a,
                      int grid, cudaStream_t stream) {
  return half ? launch_one<OP, __half>(tmA, tmB, tmD, a, grid, stream)
              : launch_one<OP, __nv_bfloat16>(tmA, tmB, tmD, a, grid, stream);
}

}  // namespace

int ragged_wgrad_splits(int R, int N, int K, int E) {
  return rag_slices((long long)E * ((N + 127) / 128) * ((K + 255) / 256), R / E / BK, kLeastSteps);
}
size_t ragged_wgrad_bytes(int R, int N, int K, int E) {
  const int s = ragged_wgrad_splits(R, N, K, E);
  return s > 1 ? (size_t)E * ((N + 127) / 128) * ((K + 255) / 256) * s * 128 * 256 * sizeof(float)
               : 0;
}
int ragged_rows_splits(int R, int E, int width, int red) {
  return rows_plan(R, E, width, red).splits;
}
size_t ragged_split_bytes(int R, int E, int width, int red) {
  const RowsPlan r = rows_plan(R, E, width, red);
  return rag_part_bytes(R, E, r.w_tiles, (red + BK - 1) / BK, kLeastSteps, r.tile_rows);
}

cudaError_t launch_ragged_rows(const RaggedProblem& p, int op, const void* rows, const void* w,
                               const void* bias, void* out, void* workspace,
                               cudaStream_t stream) {
  const bool fwd = op == RAG_FWD;
  CUtensorMap tmA, tmB;
  const int red = fwd ? p.K : p.N;
  const bool wide = !fwd && p.K % 64 == 0;
  if (!(wide ? make_tmap_rag_wide(&tmA, w, p.half, p.N, p.K, p.E, p.K, 2)
             : make_tmap_rag(&tmA, w, p.half, 3, p.K, p.N, p.E, p.K, fwd ? 128 : 64)) ||
      !make_tmap_rag(&tmB, rows, p.half, 2, red, p.R, 0, fwd ? p.ldx : p.ldy, 32))
    return cudaErrorInvalidValue;
  RagArgs a{};
  a.offsets = p.offsets;
  a.R = p.R;
  a.E = p.E;
  a.W = fwd ? p.N : p.K;
  a.num_kb = (red + BK - 1) / BK;
  const RowsPlan r = rows_plan(p.R, p.E, a.W, red);
  a.tile_rows = r.tile_rows;
  a.w_tiles = fast_div(r.w_tiles);
  a.splits = r.splits;
  a.part = static_cast<float*>(workspace);
  a.stages = std::min(MAX_STAGES, RING_BYTES / (A_BYTES + a.tile_rows * BK * 2));
  a.group_max = 8;
  a.wide_a = wide;
  a.out = out;
  a.ldo = fwd ? p.ldy : p.ldx;
  a.bias = bias;
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  const int grid = a.splits > 1 ? (int)r.tiles * a.splits
                                : (int)std::min<long long>(num_sms(), r.tiles);
  return fwd ? launch_op<RAG_FWD>(p.half, tmA, tmB, tmB, a, grid, stream)
             : launch_op<RAG_DGRAD>(p.half, tmA, tmB, tmB, a, grid, stream);
}

cudaError_t launch_ragged_wgrad(const RaggedProblem& p, const void* dy, const void* x, void* dw,
                                bool out_f32, bool accumulate, void* workspace,
                                cudaStream_t stream) {
  CUtensorMap tmA, tmB, tmD;
  const bool wide_a = p.N % 64 == 0, wide_b = p.K % 64 == 0;
  if (!(wide_a ? make_tmap_rag_wide(&tmA, dy, p.half, p.R, p.N, 1, p.ldy, 2)
               : make_tmap_rag(&tmA, dy, p.half, 2, p.N, p.R, 0, p.ldy, 64)) ||
      !(wide_b ? make_tmap_rag_wide(&tmB, x, p.half, p.R, p.K, 1, p.ldx, 4)
               : make_tmap_rag(&tmB, x, p.half, 2, p.K, p.R, 0, p.ldx, 64)) ||
      !make_tmap_rag_store(&tmD, dw, out_f32 ? 2 : p.half ? 1 : 0, p.K, p.N, p.E))
    return cudaErrorInvalidValue;
  RagArgs a{};
  a.offsets = p.offsets;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.K = p.K;
  a.w_tiles = fast_div((p.N + 127) / 128);
  a.k_tiles = fast_div((p.K + 255) / 256);
  a.e_tiles = fast_div(a.w_tiles.d * a.k_tiles.d);
  a.tile_rows = 256;
  a.stages = W_STAGES;
  a.wide_a = wide_a;
  a.wide_b = wide_b;
  a.out = dw;
  a.out_f32 = out_f32;
  a.accumulate = accumulate;
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  a.splits = ragged_wgrad_splits(p.R, p.N, p.K, p.E);
  a.part = static_cast<float*>(workspace);
  const long long tiles = (long long)p.E * a.e_tiles.d;
  const int grid = a.splits > 1 ? (int)tiles * a.splits
                                : (int)std::min<long long>(num_sms(), tiles);
  return launch_op<RAG_WGRAD>(p.half, tmA, tmB, tmD, a, grid, stream);
}

}  // namespace moe
