// MXFP4: E2M1 codes, two a byte (even k in the low nibble), with one E8M0
// scale per 32 values along K -- the weight format of MOE_Q_MXFP4_W4A8.
//
// Quantise, for each group of 32 values with a = max |v| = 1.m * 2^x:
//   scale 2^s with s = x - 2 (floor form: 2 is the exponent of 6 = 1.5 * 2^2, the
//   largest E2M1 value; values between 6 and 8 of the scaled group saturate),
//   or the smallest s with a <= 6 * 2^s (ceil form: s = x - 2, or x - 1 when
//   1.m > 1.5; nothing saturates); s >= -127.
//   code = E2M1 nearest to v / 2^s, ties to even, saturating at +-6.  The
//   quotient is an exact fp32 product unless it underflows, far below the
//   smallest tie at 0.25.
// A group holding an infinity or NaN gets scale 255 (E8M0's NaN) and codes 0:
// E2M1 has neither, and every product with the group is then NaN.
//
// Bound by HBM: 2 (4) bytes read and 0.53 written a value.  Each thread takes
// 8 values (one 16-byte load of 16-bit input), four threads share a group, and
// kUnroll such loads are in flight a thread.  bf16, 65536 x 4096: quantise 106 us,
// dequantise 98 us, 6.3 TB/s both.
#include <cuda_fp16.h>

#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "pdl.cuh"
#include "ragged.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

// 8 values as fp32.
template <int TYPE>
struct Load8 {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* x, size_t at) {
    if constexpr (TYPE == 2) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(x) + at);
      a = __ldg(p);
      b = __ldg(p + 1);
    } else {
      a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    if constexpr (TYPE == 2) {
      const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(w[i]);
        v[4 + i] = __uint_as_float(u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == 0) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
          v[2 * i] = Half16<__half>::value((uint16_t)(w[i] & 0xFFFFu));
          v[2 * i + 1] = Half16<__half>::value((uint16_t)(w[i] >> 16));
        }
      }
    }
  }
};

// Eight fp32 values -> eight E2M1 codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// E8M0 code of a group from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t group_scale(uint32_t amax_bits, bool ceil_scale) {
  const int x = (int)(amax_bits >> 23);
  if (x == 255) return 255;
  const int up = ceil_scale && (amax_bits & 0x7FFFFFu) > 0x400000u ? 1 : 0;
  return (uint32_t)max(x - 2 + up, 0);
}

template <int TYPE, bool DENSE>
__global__ void __launch_bounds__(kThreads)
    k_mxfp4_quantize(const void* __restrict__ x, size_t units, int units_per_row, long long ldx,
                     int ceil_scale, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_launch();
  griddep_wait();
  constexpr int step = kThreads;      // a block's units are consecutive
  // every lane of a group of four has a unit or none has: units % 4 == 0
  for (size_t u0 = (size_t)blockIdx.x * kThreads * kUnroll + threadIdx.x; u0 < units;
       u0 += (size_t)gridDim.x * kThreads * kUnroll) {
    Load8<TYPE> in[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const size_t u = u0 + i * step;
      if (u < units) {
        size_t at = u * 8;
        if (!DENSE) {
          const size_t row = u / (unsigned)units_per_row;
          at = row * ldx + (u - row * units_per_row) * 8;
        }
        in[i].load(x, at);
      } else {
        in[i].a = in[i].b = make_uint4(0, 0, 0, 0);
      }
    }
    const unsigned act = 0xFu << (threadIdx.x & 28);   // the group's four lanes
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const size_t u = u0 + i * step;
      float v[8];
      in[i].get(v);
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      m = max(m, __shfl_xor_sync(act, m, 1));
      m = max(m, __shfl_xor_sync(act, m, 2));
      const uint32_t s = group_scale(m, ceil_scale);
      const float inv = __uint_as_float((254u - min(s, 253u)) << 23);   // 2^(127 - s)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= inv;
      if (u < units) {
        codes[u] = s == 255u ? 0u : e2m1x8(v);
        if ((threadIdx.x & 3) == 0) scales[u >> 2] = (uint8_t)s;
      }
    }
  }
}

// Eight codes a thread: E2M1 -> fp16 pairs (exact) -> fp32 times the scale.
template <int TYPE, bool DENSE>
__global__ void __launch_bounds__(kThreads)
    k_mxfp4_dequantize(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                       size_t units, int units_per_row, long long ldo, void* __restrict__ out) {
  griddep_launch();
  griddep_wait();
  constexpr int step = kThreads;
  for (size_t u0 = (size_t)blockIdx.x * kThreads * kUnroll + threadIdx.x; u0 < units;
       u0 += (size_t)gridDim.x * kThreads * kUnroll) {
    uint32_t c[kUnroll], s[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const size_t u = u0 + i * step;
      c[i] = u < units ? __ldg(codes + u) : 0u;
      s[i] = u < units ? __ldg(scales + (u >> 2)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const size_t u = u0 + i * step;
      if (u >= units) break;
      // E8M0 0 is 2^-127, a subnormal fp32; 255 is NaN
      const float scale =
          __uint_as_float(s[i] == 0u ? 0x400000u : s[i] == 255u ? 0x7FC00000u : s[i] << 23);
      float v[8];
      uint32_t h[4];
      asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
          "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
          "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
          "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
          : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
          : "r"(c[i]));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = Half16<__half>::value((uint16_t)(h[j] & 0xFFFFu)) * scale;
        v[2 * j + 1] = Half16<__half>::value((uint16_t)(h[j] >> 16)) * scale;
      }
      size_t at = u * 8;
      if (!DENSE) {
        const size_t row = u / (unsigned)units_per_row;
        at = row * ldo + (u - row * units_per_row) * 8;
      }
      if constexpr (TYPE == 2) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        using T = typename std::conditional<TYPE == 1, __half, __nv_bfloat16>::type;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = Half16<T>::pack(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// A block for every kThreads * kUnroll units.  (A grid of a few blocks an SM
// striding over the tensor ran 451 us for 229376 x 4096 bf16 against 360: its
// loads lie 20 MB apart, and eight blocks an SM are one and a third waves.)
int codec_grid(size_t units) {
  const size_t want = (units + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  return (int)std::min<size_t>(want, 1u << 30);
}

template <int TYPE>
cudaError_t quantize_of(const void* x, size_t units, int upr, long long ldx, int K,
                        bool ceil_scale, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  return launch_dependent(ldx == K ? k_mxfp4_quantize<TYPE, true> : k_mxfp4_quantize<TYPE, false>,
                          codec_grid(units), kThreads, 0, st, 1, x, units, upr, ldx,
                          ceil_scale ? 1 : 0, reinterpret_cast<uint32_t*>(codes), scales);
}
template <int TYPE>
cudaError_t dequantize_of(const uint8_t* codes, const uint8_t* scales, size_t units, int upr,
                          long long ldo, int K, void* out, cudaStream_t st) {
  return launch_dependent(
      ldo == K ? k_mxfp4_dequantize<TYPE, true> : k_mxfp4_dequantize<TYPE, false>,
      codec_grid(units), kThreads, 0, st, 1, reinterpret_cast<const uint32_t*>(codes), scales,
      units, upr, ldo, out);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int type, long long rows, int K, long long ldx,
                                  bool ceil_scale, uint8_t* codes, uint8_t* scales,
                                  cudaStream_t stream) {
  const size_t units = (size_t)rows * (K / 8);
  return (type == 0 ? quantize_of<0> : type == 1 ? quantize_of<1> : quantize_of<2>)(
      x, units, K / 8, ldx, K, ceil_scale, codes, scales, stream);
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, long long rows,
                                    int K, void* out, int type, long long ldo,
                                    cudaStream_t stream) {
  const size_t units = (size_t)rows * (K / 8);
  return (type == 0 ? dequantize_of<0> : type == 1 ? dequantize_of<1> : dequantize_of<2>)(
      codes, scales, units, K / 8, ldo, K, out, stream);
}

}  // namespace moe
