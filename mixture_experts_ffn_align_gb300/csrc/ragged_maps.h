// Tensor maps of the ragged products' operands (ragged_maps.cu).  Each returns
// false when the driver refuses the map.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace moe {

// A 16-bit matrix [d1, d0] (rank 2) or a stack of d2 of them (rank 3), rows ld
// elements apart: boxes of 64 x box1 (x 1) values.
bool make_tmap_rag(CUtensorMap* map, const void* base, bool half, int rank, uint64_t d0,
                   uint64_t d1, uint64_t d2, uint64_t ld, uint32_t box1);
// The same for an MN-major operand whose width is a multiple of 64: one copy
// brings `chunks` boxes of 64 x 64 values, side by side in the matrix.
bool make_tmap_rag_wide(CUtensorMap* map, const void* base, bool half, uint64_t rows,
                        uint64_t cols, uint64_t batch, uint64_t ld, uint32_t chunks);
// dw [E, N, K] for stores (elem 0 bf16, 1 fp16, 2 fp32; dense): boxes of 128
// bytes x 32 rows.
bool make_tmap_rag_store(CUtensorMap* map, const void* base, int elem, uint64_t K, uint64_t N,
                         uint64_t E);
// Packed 4-bit values ([d1, d0 / 2] bytes, or d2 of them): boxes of 128 bytes x
// box1 rows.
bool make_tmap_rag_fp4(CUtensorMap* map, const void* base, int rank, uint64_t d0, uint64_t d1,
                       uint64_t d2, uint32_t box1);
// 512-byte scale blocks ([d1] or [d2, d1] of them): boxes of box1 (x box2) blocks.
bool make_tmap_scale_blocks(CUtensorMap* map, const void* base, int rank, uint64_t d1, uint64_t d2,
                            uint32_t box1, uint32_t box2);

}  // namespace moe
