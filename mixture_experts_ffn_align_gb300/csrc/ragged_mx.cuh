// Pieces shared by the 4-bit ragged products on one SM (ragged_mxfp4.cu) and on
// SM pairs (ragged_mxfp4_2sm.cu).
#pragma once

#include "ragged.cuh"

namespace moe {

// 128-row scale blocks of a token tile, and bytes of one tile's scales.
__host__ __device__ constexpr int tile_groups(int tile_rows) { return (tile_rows + 127) / 128; }
__host__ __device__ constexpr size_t tile_scale_bytes(int tile_rows, int K) {
  return (size_t)(K / 128) * tile_groups(tile_rows) * 512;
}

struct Mx44Args {
  RagArgs r;
  const uint8_t* x_scale;    // [R, K/32]
  const uint8_t* w_packed;   // [E][K/128][W/128][512]
  uint8_t* x_packed;         // [token tiles][K/128][tile_groups][512]
  int K;
};

// kind::mxf4: as make_idesc_block_scaled, E2M1 operands (format code 1), scale
// bytes sf and sf + 1 (0 or 2) of the words.
constexpr uint32_t kFmtMxf4 = 1;

// Brings the tokens' scales into operand blocks for tiles rounded up to G rows.
template <int G>
cudaError_t launch_pack_token_scales(const Mx44Args& a, long long most_tiles, cudaStream_t stream);

int ragged_mxfp4_tile_rows(int R, int E);

// Token tiles at most, whatever the segments.
inline long long most_token_tiles(int R, int E, int tile_rows) {
  return (long long)(E < R ? E : R) + R / tile_rows;
}

}  // namespace moe
