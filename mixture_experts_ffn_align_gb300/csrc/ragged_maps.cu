// Tensor maps of the ragged products (ragged_maps.h).  Operand tiles are 128
// bytes wide with 128-byte swizzle, as the MMA reads them; what lies outside a
// tensor reads as zero and is not written.  The same map serves K-major and
// MN-major operands: the MMA's descriptors tell them apart.
#include "ragged_maps.h"

#include <cuda_runtime.h>

#include <mutex>

namespace moe {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool encode(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
            const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box, bool swizzle,
            CUtensorMapL2promotion promotion) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, promotion,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

CUtensorMapDataType type16(bool half) {
  return half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

}  // namespace

bool make_tmap_rag(CUtensorMap* map, const void* base, bool half, int rank, uint64_t d0,
                   uint64_t d1, uint64_t d2, uint64_t ld, uint32_t box1) {
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {ld * 2, d1 * ld * 2};
  const cuuint32_t box[3] = {64, box1, 1};
  return encode(map, type16(half), rank, base, dims, strides, box, true,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// [batch, rows, cols] seen as [batch, cols / 64, rows, 64].
bool make_tmap_rag_wide(CUtensorMap* map, const void* base, bool half, uint64_t rows,
                        uint64_t cols, uint64_t batch, uint64_t ld, uint32_t chunks) {
  if (cols % 64 != 0) return false;
  const cuuint64_t dims[4] = {64, rows, cols / 64, batch};
  const cuuint64_t strides[3] = {ld * 2, 128, rows * ld * 2};
  const cuuint32_t box[4] = {64, 64, chunks, 1};
  return encode(map, type16(half), 4, base, dims, strides, box, true,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// [E, 2, inter, K] seen as [E, inter / 8, 2, 8, K]: boxes of eight 8-row groups of
// gate weights, each followed by the same rows of the up weights.
bool make_tmap_rag_gated(CUtensorMap* map, const void* base, bool half, uint64_t K,
                         uint64_t inter, uint64_t E) {
  if (inter % 8 != 0) return false;
  const cuuint64_t dims[5] = {K, 8, 2, inter / 8, E};
  const cuuint64_t strides[4] = {K * 2, inter * K * 2, 8 * K * 2, 2 * inter * K * 2};
  const cuuint32_t box[5] = {64, 8, 2, 8, 1};
  return encode(map, type16(half), 5, base, dims, strides, box, true,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

bool make_tmap_rag_store(CUtensorMap* map, const void* base, int elem, uint64_t K, uint64_t N,
                         uint64_t E) {
  const uint64_t size = elem == 2 ? 4 : 2;
  const cuuint64_t dims[3] = {K, N, E};
  const cuuint64_t strides[2] = {K * size, N * K * size};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), 32, 1};
  return encode(map, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type16(elem == 1), 3, base,
                dims, strides, box, true, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

bool make_tmap_rag_fp4(CUtensorMap* map, const void* base, int rank, uint64_t d0, uint64_t d1,
                       uint64_t d2, uint32_t box1) {
  const cuuint64_t dims[3] = {d0 / 2, d1, d2};
  const cuuint64_t strides[2] = {d0 / 2, d1 * (d0 / 2)};
  const cuuint32_t box[3] = {128, box1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, base, dims, strides, box, true,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Rows of 128 words.
bool make_tmap_scale_blocks(CUtensorMap* map, const void* base, int rank, uint64_t d1, uint64_t d2,
                            uint32_t box1, uint32_t box2) {
  const cuuint64_t dims[3] = {128, d1, d2};
  const cuuint64_t strides[2] = {512, d1 * 512};
  const cuuint32_t box[3] = {128, box1, box2};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, rank, base, dims, strides, box, false,
                CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

}  // namespace moe
