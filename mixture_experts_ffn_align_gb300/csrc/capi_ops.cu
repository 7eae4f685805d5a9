// C ABI (include/moe_ffn.h) of the training and 4-bit operators: ragged
// grouped products, the MXFP4 codec and product, gradient norm and clip.
// Argument validation and launch order; the kernels are in ragged_gemm.cu,
// ragged_mxfp4.cu, mxfp4_codec.cu and grad_clip.cu.
#include <algorithm>

#include "../../include/moe_ffn.h"
#include "moe_internal.h"

using namespace moe;

namespace {

moe_status done(cudaError_t e) { return static_cast<moe_status>(record_cuda_status(e)); }
bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
size_t pad256(size_t v) { return (v + 255) / 256 * 256; }

constexpr int64_t kMaxDim = 1 << 20;

bool valid_ragged(const moe_ragged* p) {
  if (p == nullptr) return false;
  if (p->R < 0 || p->R > MOE_MAX_RAGGED_ROWS || p->E < 1 || p->E > MOE_MAX_EXPERTS) return false;
  if (p->N < 8 || p->N % 8 || p->N > kMaxDim || p->K < 8 || p->K % 8 || p->K > kMaxDim) return false;
  // tiles and weights within the kernels' 32-bit tile numbers
  if ((int64_t)p->E * ((p->N + 127) / 128) * ((p->K + 127) / 128) > (1ll << 30)) return false;
  if (((int64_t)p->R / 128 + p->E) * ((std::max(p->N, p->K) + 127) / 128) > (1ll << 30)) return false;
  if (p->dtype != MOE_T_BF16 && p->dtype != MOE_T_FP16) return false;
  if (p->ldx != 0 && (p->ldx < p->K || p->ldx % 8 || p->ldx > (1ll << 32))) return false;
  if (p->ldy != 0 && (p->ldy < p->N || p->ldy % 8 || p->ldy > (1ll << 32))) return false;
  return true;
}

RaggedProblem ragged_problem(const moe_ragged* p, const int32_t* offsets) {
  RaggedProblem q;
  q.half = p->dtype == MOE_T_FP16;
  q.R = p->R;
  q.N = p->N;
  q.K = p->K;
  q.E = p->E;
  q.ldx = p->ldx != 0 ? p->ldx : p->K;
  q.ldy = p->ldy != 0 ? p->ldy : p->N;
  q.offsets = offsets;
  return q;
}

bool mxfp4_shape(const moe_ragged* p) { return p->N % 128 == 0 && p->K % 128 == 0; }

size_t ragged_bytes(const moe_ragged* p) {
  size_t b = std::max({(size_t)1, ragged_split_bytes(p->R, p->E, p->N, p->K),
                       ragged_split_bytes(p->R, p->E, p->K, p->N),
                       ragged_wgrad_bytes(p->R, p->N, p->K, p->E)});
  if (mxfp4_shape(p)) b = std::max(b, ragged_mxfp4_scale_bytes(p->R, p->K, p->E));
  return pad256(b);
}

// SM pairs (256-wide tiles) unless that leaves fewer tiles than two for each
// pair: then the one-SM form's 128-wide tiles spread over twice as many CTAs.
bool use_pairs(const moe_ragged* p, int width) {
  const int form = ragged_form();
  const int64_t tiles = ((int64_t)std::min(p->E, p->R) + p->R / 256) * ((width + 255) / 256);
  return form >= 2 || (form == 0 && tiles >= num_sms());
}

// wgrad on SM pairs from segments of about 192 rows up: 16 experts, 4096 x 4096,
// one SM / pairs: 130 rows each 119 / 125 us, 257 rows 192 / 158 us.
bool wgrad_pairs(const moe_ragged* p) {
  const int form = ragged_form();
  const int64_t tiles = (int64_t)p->E * ((p->N + 255) / 256) * ((p->K + 255) / 256);
  return form >= 2 || (form == 0 && p->R >= 192ll * p->E && 2 * tiles >= num_sms());
}

cudaError_t ragged_rows(const moe_ragged* p, int op, const void* rows, const void* w,
                        const void* bias, const int32_t* offsets, void* out, void* workspace,
                        void* stream) {
  const RaggedProblem q = ragged_problem(p, offsets);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return use_pairs(p, op == 0 ? p->N : p->K)
             ? launch_ragged_rows_2sm(q, op, rows, w, bias, out, st)
             : launch_ragged_rows(q, op, rows, w, bias, out, workspace, st);
}

// Checks shared by the products; MOE_OK to go on.
moe_status ragged_args(const moe_ragged* p, const void* a, const void* b, const int32_t* offsets,
                       const void* out, const void* workspace, size_t workspace_bytes) {
  if (!valid_ragged(p)) return MOE_ERR_INVALID_ARG;
  if (p->R == 0) return MOE_OK;
  if (!a || !b || !offsets || !out || !workspace) return MOE_ERR_INVALID_ARG;
  if (misaligned(a, 16) || misaligned(b, 16) || misaligned(out, 16) || misaligned(offsets, 4) ||
      misaligned(workspace, 128))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < ragged_bytes(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return MOE_OK;
}

bool valid_dtype(int t) { return t >= MOE_T_BF16 && t <= MOE_T_FP32; }

}  // namespace

extern "C" {

size_t moe_ragged_workspace_bytes(const moe_ragged* p) {
  return valid_ragged(p) ? ragged_bytes(p) : 0;
}

moe_status ragged_gemm(const moe_ragged* p, const void* x, const void* w, const void* bias,
                       const int32_t* expert_offsets, void* y, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const moe_status s = ragged_args(p, x, w, expert_offsets, y, workspace, workspace_bytes);
  if (s != MOE_OK || p->R == 0) return s;
  if (misaligned(bias, 2)) return MOE_ERR_INVALID_ARG;
  return done(ragged_rows(p, 0, x, w, bias, expert_offsets, y, workspace, stream));
}

moe_status ragged_gemm_dgrad(const moe_ragged* p, const void* dy, const void* w,
                             const int32_t* expert_offsets, void* dx, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const moe_status s = ragged_args(p, dy, w, expert_offsets, dx, workspace, workspace_bytes);
  if (s != MOE_OK || p->R == 0) return s;
  return done(ragged_rows(p, 1, dy, w, nullptr, expert_offsets, dx, workspace, stream));
}

moe_status ragged_gemm_wgrad(const moe_ragged* p, const void* dy, const void* x,
                             const int32_t* expert_offsets, void* dw, int dw_dtype,
                             int accumulate, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const moe_status s = ragged_args(p, dy, x, expert_offsets, dw, workspace, workspace_bytes);
  if (s != MOE_OK) return s;
  if (dw_dtype != p->dtype && dw_dtype != MOE_T_FP32) return MOE_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p->R == 0) {             // no rows: the gradient is zero
    if (accumulate) return MOE_OK;
    if (!dw) return MOE_ERR_INVALID_ARG;
    const size_t bytes = (size_t)p->E * p->N * p->K * (dw_dtype == MOE_T_FP32 ? 4 : 2);
    return done(cudaMemsetAsync(dw, 0, bytes, st));
  }
  const RaggedProblem q = ragged_problem(p, expert_offsets);
  const bool f32 = dw_dtype == MOE_T_FP32;
  return done(wgrad_pairs(p) ? launch_ragged_wgrad_2sm(q, dy, x, dw, f32, accumulate != 0, st)
                             : launch_ragged_wgrad(q, dy, x, dw, f32, accumulate != 0, workspace, st));
}

moe_status ragged_gemm_mxfp4(const moe_ragged* p, const void* x_codes, const void* x_scales,
                             const void* w_codes, const void* w_scales_packed,
                             const int32_t* expert_offsets, void* y, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const moe_status s = ragged_args(p, x_codes, w_codes, expert_offsets, y, workspace, workspace_bytes);
  if (s != MOE_OK) return s;
  if (!mxfp4_shape(p)) return MOE_ERR_UNSUPPORTED;
  if (p->ldx != 0 && p->ldx != p->K) return MOE_ERR_INVALID_ARG;   // codes are dense
  if (p->R == 0) return MOE_OK;
  if (!x_scales || !w_scales_packed || misaligned(x_scales, 4) || misaligned(w_scales_packed, 16))
    return MOE_ERR_INVALID_ARG;
  const auto launch = use_pairs(p, p->N) ? launch_ragged_mxfp4_2sm : launch_ragged_mxfp4;
  return done(launch(ragged_problem(p, expert_offsets), x_codes,
                     static_cast<const uint8_t*>(x_scales), w_codes, w_scales_packed, y,
                     workspace, static_cast<cudaStream_t>(stream)));
}

moe_status moe_mxfp4_quantize(const void* x, int x_dtype, int64_t rows, int K, int64_t ldx,
                              int scale_mode, void* codes, void* scales, void* stream) {
  if (!valid_dtype(x_dtype) || rows < 0 || K < 32 || K % 32 ||
      (scale_mode != MOE_MXFP4_FLOOR && scale_mode != MOE_MXFP4_CEIL))
    return MOE_ERR_INVALID_ARG;
  if (ldx == 0) ldx = K;
  if (ldx < K || ldx % 8) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || misaligned(x, 16) || misaligned(codes, 16))
    return MOE_ERR_INVALID_ARG;
  return done(launch_mxfp4_quantize(x, x_dtype, rows, K, ldx, scale_mode == MOE_MXFP4_CEIL,
                                    static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                                    static_cast<cudaStream_t>(stream)));
}

moe_status moe_mxfp4_dequantize(const void* codes, const void* scales, int64_t rows, int K,
                                void* out, int out_dtype, int64_t ldo, void* stream) {
  if (!valid_dtype(out_dtype) || rows < 0 || K < 32 || K % 32) return MOE_ERR_INVALID_ARG;
  if (ldo == 0) ldo = K;
  if (ldo < K || ldo % 8) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!out || !codes || !scales || misaligned(out, 16) || misaligned(codes, 16))
    return MOE_ERR_INVALID_ARG;
  return done(launch_mxfp4_dequantize(static_cast<const uint8_t*>(codes),
                                      static_cast<const uint8_t*>(scales), rows, K, out,
                                      out_dtype, ldo, static_cast<cudaStream_t>(stream)));
}

moe_status moe_mxfp4_pack_scales(const void* scales, int E, int N, int K, void* packed,
                                 void* stream) {
  if (E < 1 || E > MOE_MAX_EXPERTS || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (N % 128 || K % 128) return MOE_ERR_UNSUPPORTED;
  if (!scales || !packed || misaligned(scales, 4) || misaligned(packed, 16))
    return MOE_ERR_INVALID_ARG;
  return done(launch_prepack_mx_scales(static_cast<const uint8_t*>(scales), E, N, K, packed,
                                       static_cast<cudaStream_t>(stream)));
}

size_t moe_clip_workspace_bytes(void) { return clip_workspace_bytes(); }

moe_status moe_clip_grad_norm(int n, const void* const* grads, void* const* outs,
                              const int64_t* numel, const int32_t* dtypes, float max_norm,
                              float* norm, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (n < 0 || n > MOE_MAX_CLIP_TENSORS || !(max_norm >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (n > 0 && (!grads || !outs || !numel || !dtypes)) return MOE_ERR_INVALID_ARG;
  if (!norm || !workspace || misaligned(norm, 4) || misaligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] > (1ll << 40) || !valid_dtype(dtypes[i])) return MOE_ERR_INVALID_ARG;
    const uintptr_t size = dtypes[i] == MOE_T_FP32 ? 4 : 2;
    if (numel[i] > 0 &&
        (!grads[i] || !outs[i] || misaligned(grads[i], size) || misaligned(outs[i], size)))
      return MOE_ERR_INVALID_ARG;
  }
  if (workspace_bytes < clip_workspace_bytes()) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return done(launch_clip_grad_norm(n, grads, outs, numel, dtypes, max_norm, norm, workspace,
                                    static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
