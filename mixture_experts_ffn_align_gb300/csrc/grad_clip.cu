// Global norm over many gradient tensors, and clipping:
//   norm = sqrt(sum_i sum_j g_i[j]^2),  c = min(1, max_norm / (norm + 1e-6)),
//   out_i = c * g_i   (bf16, fp16 or fp32 each; out_i may be g_i itself).
//
// Two launches.  k_clip_norm sums squares: a thread squares the values of one
// chunk in fp32 (at most 64 in 4 sums) and carries its total from chunk to
// chunk in fp64, the block's total goes to partial[block].  k_clip_scale adds
// the partials in every block again, in the same order (they are in L2 by
// then), so no third launch and no atomics are needed and the norm does not
// depend on the order in which blocks ran.  It walks the chunks in the other
// direction, so that what the first pass read last is still in L2, and in
// place with c == 1 it writes nothing.
//
// Bound by HBM: read once for the norm, read and written for the scaling.  1.2 GB
// of bf16: 173 us (7.0 TB/s) and 356 us (6.7 TB/s).
//
// The list of tensors travels in the kernel's parameters (up to kMaxList a
// launch), so a captured graph holds it and nothing is copied to the device.
#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "pdl.cuh"
#include "ragged.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kChunkBytes = 32768;
constexpr int kSmallList = 64, kMaxList = 1024;
constexpr int kMaxBlocks = 1024;      // partial sums of one launch
constexpr int kMaxLaunches = 64;      // lists of up to kMaxList each

struct Item {
  const void* in;
  void* out;
  int64_t n;
};
template <int CAP>
struct List {
  Item item[CAP];
  uint8_t type[CAP];
  int32_t chunk0[CAP + 1];   // first chunk of each tensor
  int n;
};

template <int CAP>
__device__ __forceinline__ int tensor_of(const List<CAP>& L, int chunk) {
  int lo = 0, hi = L.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.chunk0[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The two (16-bit) or one (fp32) values of a 32-bit word.
template <int TYPE>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if (TYPE == 0) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return make_float2(Half16<__half>::value((uint16_t)(w & 0xFFFFu)),
                     Half16<__half>::value((uint16_t)(w >> 16)));
}
template <int TYPE>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (TYPE == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return TYPE == 0 ? Half16<__nv_bfloat16>::value(b) : Half16<__half>::value(b);
}
template <int TYPE>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (TYPE == 2)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] =
        TYPE == 0 ? Half16<__nv_bfloat16>::bits(v) : Half16<__half>::bits(v);
}

constexpr int kVec = kChunkBytes / 16 / kThreads;   // 16-byte loads a thread and chunk

template <int TYPE>
__device__ __forceinline__ float chunk_squares(const Item& t, int64_t begin, int64_t end) {
  constexpr int per = TYPE == 2 ? 4 : 8;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if ((reinterpret_cast<uintptr_t>(t.in) & 15u) == 0) {
    const uint4* p = reinterpret_cast<const uint4*>(t.in) + begin / per;
    const int nv = (int)((end - begin) / per);
    uint4 v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = i * kThreads + threadIdx.x;
      v[i] = at < nv ? __ldg(p + at) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (TYPE == 2) {
          const float f = __uint_as_float(w[j]);
          s[j] += f * f;
        } else {
          const float2 f = unpack<TYPE>(w[j]);
          s[j] += f.x * f.x;
          s[j] += f.y * f.y;
        }
      }
    }
    begin += (int64_t)nv * per;
  }
  for (int64_t i = begin + threadIdx.x; i < end; i += kThreads) {
    const float f = load1<TYPE>(t.in, i);
    s[0] += f * f;
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <int TYPE>
__device__ __forceinline__ void chunk_scale(const Item& t, int64_t begin, int64_t end, float c) {
  constexpr int per = TYPE == 2 ? 4 : 8;
  if (((reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out)) & 15u) == 0) {
    const uint4* p = reinterpret_cast<const uint4*>(t.in) + begin / per;
    uint4* d = reinterpret_cast<uint4*>(t.out) + begin / per;
    const int nv = (int)((end - begin) / per);
    uint4 v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = i * kThreads + threadIdx.x;
      if (at < nv) v[i] = p[at];
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = i * kThreads + threadIdx.x;
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (TYPE == 2) {
          w[j] = __float_as_uint(__uint_as_float(w[j]) * c);
        } else {
          using T = typename std::conditional<TYPE == 1, __half, __nv_bfloat16>::type;
          const float2 f = unpack<TYPE>(w[j]);
          w[j] = Half16<T>::pack(f.x * c, f.y * c);
        }
      }
      if (at < nv) d[at] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    begin += (int64_t)nv * per;
  }
  for (int64_t i = begin + threadIdx.x; i < end; i += kThreads)
    store1<TYPE>(t.out, i, load1<TYPE>(t.in, i) * c);
}

// Sum of v over the block, in every thread; the same order every time.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  double r = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) r += s[i];
  return r;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    k_clip_norm(const __grid_constant__ List<CAP> L, double* partial) {
  griddep_launch();
  griddep_wait();
  double sum = 0.0;
  const int chunks = L.chunk0[L.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(L, c);
    const Item t = L.item[i];
    const int type = L.type[i];
    const int64_t per = kChunkBytes / (type == 2 ? 4 : 2);
    const int64_t begin = (c - L.chunk0[i]) * per, end = min(t.n, begin + per);
    sum += type == 0 ? chunk_squares<0>(t, begin, end)
                     : type == 1 ? chunk_squares<1>(t, begin, end) : chunk_squares<2>(t, begin, end);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    k_clip_scale(const __grid_constant__ List<CAP> L, const double* partial, int partials,
                 float max_norm, float* norm_out, int in_place) {
  griddep_launch();
  griddep_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) sum += partial[i];
  const float norm = (float)sqrt(block_sum(sum));
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float q = max_norm / (norm + 1e-6f);
  const float c = q < 1.0f || q != q ? q : 1.0f;     // a NaN norm stays visible
  if (in_place && c == 1.0f) return;
  const int chunks = L.chunk0[L.n];
  for (int k = blockIdx.x; k < chunks; k += gridDim.x) {
    const int chunk = chunks - 1 - k;
    const int i = tensor_of(L, chunk);
    const Item t = L.item[i];
    const int type = L.type[i];
    const int64_t per = kChunkBytes / (type == 2 ? 4 : 2);
    const int64_t begin = (chunk - L.chunk0[i]) * per, end = min(t.n, begin + per);
    if (type == 0) chunk_scale<0>(t, begin, end, c);
    else if (type == 1) chunk_scale<1>(t, begin, end, c);
    else chunk_scale<2>(t, begin, end, c);
  }
}

// Fills L with tensors [at, at + count) and returns their chunks.
template <int CAP>
int fill(List<CAP>& L, int at, int count, const void* const* grads, void* const* outs,
         const int64_t* numel, const int32_t* types) {
  int chunks = 0;
  L.n = count;
  for (int i = 0; i < count; ++i) {
    const int64_t per = kChunkBytes / (types[at + i] == 2 ? 4 : 2);
    L.item[i] = Item{grads[at + i], outs[at + i], numel[at + i]};
    L.type[i] = (uint8_t)types[at + i];
    L.chunk0[i] = chunks;
    chunks += (int)((numel[at + i] + per - 1) / per);
  }
  L.chunk0[count] = chunks;
  return chunks;
}

template <int CAP>
cudaError_t clip_lists(int n, const void* const* grads, void* const* outs, const int64_t* numel,
                       const int32_t* types, float max_norm, float* norm, double* partial,
                       cudaStream_t stream) {
  const int most = std::min(kMaxBlocks, num_sms() * 4);
  int partials = 0, in_place = 1;
  for (int i = 0; i < n; ++i)
    if (grads[i] != outs[i]) in_place = 0;
  List<CAP> L;
  const int lists = std::max(1, (n + CAP - 1) / CAP);   // no tensors: the norm is 0
  for (int l = 0; l < lists; ++l) {
    const int at = l * CAP;
    const int chunks = fill(L, at, std::min(CAP, n - at), grads, outs, numel, types);
    const int grid = std::max(1, std::min(chunks, most));
    const cudaError_t e =
        launch_dependent(k_clip_norm<CAP>, grid, kThreads, 0, stream, 1, L, partial + partials);
    if (e != cudaSuccess) return e;
    partials += grid;
  }
  for (int l = lists - 1; l >= 0; --l) {      // last read first: still in L2
    const int at = l * CAP;
    const int chunks = fill(L, at, std::min(CAP, n - at), grads, outs, numel, types);
    const int grid = std::max(1, std::min(chunks, most));
    const cudaError_t e =
        launch_dependent(k_clip_scale<CAP>, grid, kThreads, 0, stream, 1, L, partial, partials,
                         max_norm, l == 0 ? norm : nullptr, in_place);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t clip_workspace_bytes() { return sizeof(double) * kMaxBlocks * kMaxLaunches; }

cudaError_t launch_clip_grad_norm(int n, const void* const* grads, void* const* outs,
                                  const int64_t* numel, const int32_t* types, float max_norm,
                                  float* norm, void* workspace, cudaStream_t stream) {
  double* partial = static_cast<double*>(workspace);
  // the short list's parameters are 2 KB, the long one's 30 KB, which every
  // launch carries to the device
  return n <= kSmallList
             ? clip_lists<kSmallList>(n, grads, outs, numel, types, max_norm, norm, partial, stream)
             : clip_lists<kMaxList>(n, grads, outs, numel, types, max_norm, norm, partial, stream);
}

}  // namespace moe
