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
  if (mxfp4_shape(p)) b = std::max(b, ragged_mxfp4_bytes(p->R, p->N, p->K, p->E));
  return pad256(b);
}

// Choice of the kernels' form.  A form's time is modelled in rounds of its CTAs
// (or pairs) on segments of the average length.  A round takes a tile's cycles,
// which are the slower of what its operands take at the ~50 bytes a cycle that an
// SM gets from L2 and of its MMAs, and a fixed cost; or, if that is longer, what
// HBM takes for the round's share of the bytes that are read and written once.
// The constants are fitted to the three forms' times at 184 products each of
// forward and dgrad (1 to 128 experts of 1 to 2048 rows).  The form taken is slower
// than the best by 0.8% on average for forward and wgrad (single products up to
// 13%), 0.5% for dgrad (8%) and 0.4% for 4-bit operands (14%).  In us, one SM /
// pairs / double tiles:
//   forward, 8 x (28672, 4096): 32 rows each 275 / 287 / 282, 256 351 / 313 / 326;
//   forward, 8 x (6704, 2968): 128 rows each 79 / 63 / 66, 400 185 / 148 / 124;
//   dgrad, 8 x (28672, 4096): 32 rows each 269 / 281 / 256, 400 785 / 568 / 569;
//   dgrad, 8 x (6704, 2968): 32 rows each 66 / 70 / 57, 256 102 / 82 / 72;
//   forward, 1 x (4096, 4096), one SM in slices: 128 rows 14 / 20 / 26, 400 24 /
//   21 / 38.
// wgrad of 16 experts, 4096 x 4096: one SM / pairs 140 / 145 at 130 rows each,
// 192 / 158 at 257.
enum Form { ONE_SM = 1, PAIRS = 2, DOUBLE = 3 };
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// A GB300's, which the model is fitted to (and the host may have no GPU).
constexpr int kSms = 152, kBytesPerCycle = 50;

// Cycles of `tiles` tiles on `units` CTAs or pairs: a tile's own, or those of its
// bytes at HBM's bytes a cycle.
int64_t tiles_cycles(int64_t tiles, int64_t units, int64_t tile, int64_t bytes, int64_t hbm) {
  const int64_t full = tiles / units, rest = tiles % units;
  return full * std::max(tile, bytes * units / tiles / hbm) +
         (rest ? std::max(tile, bytes * rest / tiles / hbm) : 0);
}
// Bytes as L2 serves them: rows that do not start on a 32-byte sector cost 1.4
// times theirs (11592 against 11584 columns: 619 / 417 us).
int64_t l2_bytes(int64_t bytes, int64_t pitch_bytes) {
  return pitch_bytes % 32 ? bytes * 7 / 5 : bytes;
}

// Forward (w_cols: columns of the output, red: of the reduction) or dgrad.
// step_deep: 64, or 256 4-bit values, whose 16 KB operand tiles are alike;
// extra: bytes of scales a step.  hbm, hbm_double: bytes a cycle (hbm_double unused
// for 4-bit operands); dgrad's boxes of the weights are 256 bytes to 1 KB wide in
// memory against forward's 128 bytes.
Form rows_form(const moe_ragged* p, int w_cols, int red, int64_t w_pitch, int64_t x_pitch,
               int step_deep, int extra, int hbm, int hbm_double) {
  const int form = ragged_form();
  const bool fp4 = step_deep != 64;
  if (form == DOUBLE) return fp4 ? PAIRS : DOUBLE;
  if (form != 0) return static_cast<Form>(form);
  const int64_t segs = std::min(p->E, p->R), rows = ceil_div(p->R, segs);
  const int64_t per_seg = ceil_div(rows, 256), tok = segs * per_seg;
  const int64_t n = ceil_div(ceil_div(rows, per_seg), 32) * 32;    // tokens of a tile
  const int64_t steps = ceil_div(red, step_deep);
  const int64_t a = l2_bytes(16384, w_pitch);
  const int64_t half = n / 2 <= 64 ? ceil_div(n / 2, 32) * 4096 : 16384;
  const int64_t b1 = l2_bytes(n / 32 * 4096, x_pitch) + extra, b2 = l2_bytes(half, x_pitch) + extra;
  const int64_t w1 = ceil_div(w_cols, 128), w2 = ceil_div(w_cols, 256), w4 = ceil_div(w_cols, 512);
  // 2 n at the tensor cores' full rate, and a third more for the clock under power
  const int64_t mma = 53 * n / 20;
  const auto step = [&](int64_t bytes, int64_t cycles) {
    return std::max(bytes / kBytesPerCycle, cycles);
  };
  const int64_t values = segs * w_cols * red, io = static_cast<int64_t>(p->R) * (w_cols + red);
  const int64_t bytes = fp4 ? values * 17 / 32 + io / 2 : 2 * values + io;
  // 4-bit tiles of more than 128 tokens leave room for one accumulator only
  const bool one_acc = fp4 && p->R > 64ll * p->E && p->R > 128;
  const int splits = fp4 ? ragged_mxfp4_splits(p->R, w_cols, red, p->E)
                         : ragged_rows_splits(p->R, p->E, w_cols, red);
  // What they were fitted on started while the kernel before ended; kernels of
  // clusters no longer do (515 rows, 16 experts, 1032 -> 776: one SM 9.6, pairs
  // 12.4).  Few rows stream from HBM a little faster on one SM, more rows on pairs.
  const int64_t launch = fp4 ? 0 : 3000;
  const int64_t hbm_one = fp4 || n <= 64 ? hbm : hbm * 23 / 25;
  const int64_t hbm_two = fp4 || n > 64 ? hbm : hbm * 97 / 100;
  int64_t one;
  if (splits > 1)
    one = ceil_div(tok * w1 * splits, kSms) *
              (ceil_div(steps, splits) * step(a + b1, mma) + 4000 + 50 * n) + launch;
  else
    one = tiles_cycles(tok * w1, kSms, steps * step(a + b1, mma) + (one_acc ? 4000 : 1200), bytes,
                       hbm_one) * (fp4 ? 21 : 20) / 20;
  const int64_t two =
      tiles_cycles(tok * w2, kSms / 2,
                   steps * step(a + b2, mma) + (one_acc ? 2000 : fp4 ? 1900 : 1400), bytes,
                   hbm_two) + launch;
  if (!fp4 && steps >= 16) {   // no double tiles of 4-bit operands, and no rate for them
    // both accumulators are drained before the next tile's MMAs
    const int64_t dbl =
        tiles_cycles(tok * w4, kSms / 2, steps * step(2 * a + b2, 2 * mma) + 2500 + 24 * n, bytes,
                     hbm_double) + launch;
    if (dbl < std::min(one, two)) return DOUBLE;
  }
  return two <= one && w_cols > 128 ? PAIRS : ONE_SM;
}

Form wgrad_form(const moe_ragged* p) {
  const int form = ragged_form();
  if (form != 0) return form == ONE_SM ? ONE_SM : PAIRS;
  const int64_t segs = std::min(p->E, p->R), steps = ceil_div(ceil_div(p->R, segs), 64);
  const int64_t k = ceil_div(p->K, 256);
  const int splits = ragged_wgrad_splits(p->R, p->N, p->K, p->E);
  const int64_t t1 = p->E * ceil_div(p->N, 128) * k, t2 = p->E * ceil_div(p->N, 256) * k;
  // a tile's output: 64 KB a CTA at an SM's share of the HBM rate
  const int64_t out = 2800;
  const int64_t load1 = 49152 / kBytesPerCycle, load2 = 32768 / kBytesPerCycle;
  const int64_t one = splits > 1 ? ceil_div(steps, splits) * load1 + 8000
                                 : ceil_div(t1, kSms) * std::max(steps * load1, out);
  const int64_t two = ceil_div(t2, kSms / 2) * std::max(steps * load2, out * 21 / 20);
  return two < one ? PAIRS : ONE_SM;
}

cudaError_t ragged_rows(const moe_ragged* p, int op, const void* rows, const void* w,
                        const void* bias, const int32_t* offsets, void* out, void* workspace,
                        void* stream) {
  const RaggedProblem q = ragged_problem(p, offsets);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool fwd = op == 0;
  const Form f = rows_form(p, fwd ? p->N : p->K, fwd ? p->K : p->N, 2ll * p->K,
                           2 * (fwd ? q.ldx : q.ldy), 64, 0, fwd ? 3400 : 3600, fwd ? 3400 : 3650);
  return f == ONE_SM ? launch_ragged_rows(q, op, rows, w, bias, out, workspace, st)
                     : launch_ragged_rows_2sm(q, op, f == DOUBLE, rows, w, bias, out, st);
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
  return done(wgrad_form(p) == PAIRS ? launch_ragged_wgrad_2sm(q, dy, x, dw, f32, accumulate != 0, st)
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
  const Form f = rows_form(p, p->N, p->K, p->K / 2, p->K / 2, 256, 3072, 3400, 0);
  const auto launch = f == PAIRS ? launch_ragged_mxfp4_2sm : launch_ragged_mxfp4;
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
