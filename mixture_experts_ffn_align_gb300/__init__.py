"""Python binding of the GB300 fused MoE expert forward (libmoe_ffn.so).

Argument marshalling only: every function here has the name of a C entry
point in ``include/moe_ffn.h``, takes torch tensors (device memory) or None,
passes their data pointers and the current CUDA stream to the library, and
raises ``MoEError`` on a non-OK status.  All computation happens in the CUDA
kernels of the library; there is no fallback.  The library must have been
built (``__graft_entry__.build()`` or ``python -m
mixture_experts_ffn_align_gb300._build``); importing a function that needs it
raises if it is missing.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from dataclasses import dataclass
from functools import cache, cached_property, lru_cache
from types import SimpleNamespace

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_ffn.so")

QUANT = {"bf16": 0, "fp8": 1, "mxfp4": 2, "mxfp8": 3}
SCALE_FMT = {"fp32": 0, "ue8m0": 1}

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_CUDA",
          4: "MOE_ERR_DEVICE_TIMEOUT", 5: "MOE_ERR_WORKSPACE_TOO_SMALL",
          6: "MOE_ERR_DEVICE_BAD_INDEX"}

EXPORTS = ["moe_m_sum_bound", "moe_align_workspace_bytes", "moe_align_permute_launches",
           "moe_workspace_bytes",
           "moe_host_workspace_bytes", "moe_align_permute", "grouped_gemm_w13", "act_mul_quant",
           "grouped_gemm_w2", "unpermute_reduce", "fused_experts", "fused_experts_from_host",
           "moe_sync_status", "moe_status_string", "moe_debug_set_watchdog",
           "moe_debug_set_bf16_gemm_form", "moe_debug_set_grid_ctas",
           "moe_align_permute_noalloc", "moe_last_error_string", "moe_topk_router",
           "moe_batched_workspace_bytes", "fused_experts_batched", "grouped_gemm_w13_ex",
           "grouped_gemm_w2_ex", "fused_experts_ex", "moe_gemm2_splits",
           "moe_gemm2_partial_bytes", "grouped_gemm_w2_split", "unpermute_reduce_split",
           "moe_prepacked_scale_bytes", "moe_prepack_weights",
           "moe_ragged_workspace_bytes", "ragged_gemm", "ragged_gemm_dgrad", "ragged_gemm_wgrad",
           "moe_mxfp4_quantize", "moe_mxfp4_dequantize", "moe_mxfp4_pack_scales",
           "ragged_gemm_mxfp4", "moe_clip_workspace_bytes", "moe_clip_grad_norm",
           "ragged_gated", "ragged_gated_dgrad", "moe_orthogonalize_workspace_bytes",
           "moe_orthogonalize"]

NOALLOC_SCRATCH_BYTES = 1 << 20   # MOE_NOALLOC_SCRATCH_BYTES in include/moe_ffn.h


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}" + (f" ({detail})" if detail else ""))


class CProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("M", "H", "I", "E", "topk", "block_size", "quant", "act_scale_fmt",
                 "apply_router_weight_on_input", "router_weight_in_gemm2", "act_recipe")] + \
               [(n, ctypes.c_float) for n in ("gemm1_alpha", "gemm1_beta", "gemm1_clamp_limit")] + \
               [("weight_scales_prepacked", ctypes.c_int32)]


@dataclass(frozen=True)
class Problem:
    """Mirror of ``moe_problem``."""
    M: int
    H: int
    I: int
    E: int
    topk: int
    block_size: int = 128
    quant: str = "bf16"
    act_scale_fmt: str = "fp32"
    apply_router_weight_on_input: bool = False
    router_weight_in_gemm2: bool = False
    # None: SiLU(gate) * up; else (alpha, beta, clamp_limit) of the gemm1 recipe
    act_recipe: tuple | None = None
    # MXFP4 / MXFP8: the weight scales passed are moe_prepack_weights' output
    weight_scales_prepacked: bool = False

    def c(self) -> CProblem:
        a, b, lim = self.act_recipe if self.act_recipe is not None else (0.0, 0.0, 0.0)
        return CProblem(self.M, self.H, self.I, self.E, self.topk, self.block_size,
                        QUANT[self.quant], SCALE_FMT[self.act_scale_fmt],
                        int(self.apply_router_weight_on_input),
                        int(self.router_weight_in_gemm2), int(self.act_recipe is not None),
                        float(a), float(b), float(lim), int(self.weight_scales_prepacked))

    @classmethod
    def from_config(cls, cfg, **kw):
        d = dict(M=cfg.M, H=cfg.H, I=cfg.I, E=cfg.E, topk=cfg.topk, block_size=cfg.block_size,
                 quant=cfg.quant, act_scale_fmt=cfg.act_scale_fmt,
                 apply_router_weight_on_input=cfg.apply_router_weight_on_input)
        d.update(kw)
        return cls(**d)


DTYPE = {"bfloat16": 0, "float16": 1, "float32": 2}
MXFP4_SCALE = {"floor": 0, "ceil": 1}


class CRagged(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "N", "K", "E", "dtype")] + \
               [(n, ctypes.c_int64) for n in ("ldx", "ldy")]


@dataclass(frozen=True)
class Ragged:
    """Mirror of ``moe_ragged``: R rows grouped by expert, weights [E, N, K]."""
    R: int
    N: int
    K: int
    E: int
    dtype: str = "bfloat16"     # of x, w, y and the 16-bit gradients
    ldx: int = 0                # row strides in elements, 0: dense
    ldy: int = 0

    @cached_property
    def _v(self):
        """Shapes, strides and types that the binding checks."""
        import torch
        R, N, K, E = self.R, self.N, self.K, self.E
        return SimpleNamespace(
            x=(R, K), y=(R, N), w=(E, N, K), bias=(E, N), offsets=(E + 1,),
            half_n=(R, N // 2), twice_k=(R, 2 * K),
            x_codes=(R, K // 2), x_scales=(R, K // 32), w_codes=(E, N, K // 2),
            packed=E * N * (K // 32), ldx=self.ldx or K, ldy=self.ldy or N,
            dtype=getattr(torch, self.dtype), int32=torch.int32, uint8=torch.uint8,
            float32=torch.float32)

    @cached_property
    def _ref(self):
        return ctypes.byref(CRagged(self.R, self.N, self.K, self.E, DTYPE[self.dtype], self.ldx,
                                    self.ldy))


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe_ffn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(CProblem)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        for n in ("moe_m_sum_bound", "moe_align_workspace_bytes", "moe_workspace_bytes",
                  "moe_host_workspace_bytes"):
            getattr(L, n).argtypes, getattr(L, n).restype = [P], sz
        L.moe_align_permute.argtypes = [P] + [vp] * 10 + [vp, sz, vp]
        L.moe_align_permute_noalloc.argtypes = [P] + [vp] * 10 + [vp]
        L.moe_align_permute_noalloc.restype = i32
        L.grouped_gemm_w13.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp]
        L.act_mul_quant.argtypes = [P, vp, vp, vp, vp, vp]
        L.grouped_gemm_w2.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
        L.unpermute_reduce.argtypes = [P, vp, vp, vp, vp, vp]
        L.fused_experts.argtypes = [P] + [vp] * 9 + [sz, vp]
        L.fused_experts_from_host.argtypes = [P] + [vp] * 9 + [sz, vp]
        L.moe_sync_status.argtypes = [vp]
        L.moe_prepacked_scale_bytes.argtypes = [P, i32]
        L.moe_prepacked_scale_bytes.restype = sz
        L.moe_prepack_weights.argtypes = [P, vp, vp, vp, vp, vp]
        L.moe_topk_router.argtypes = [i32, i32, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp]
        L.moe_batched_workspace_bytes.argtypes = [P, i32]
        L.moe_batched_workspace_bytes.restype = sz
        L.fused_experts_batched.argtypes = [P, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.grouped_gemm_w13_ex.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp]
        L.grouped_gemm_w2_ex.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.fused_experts_ex.argtypes = [P] + [vp] * 11 + [sz, vp]
        L.moe_gemm2_splits.argtypes, L.moe_gemm2_splits.restype = [P], i32
        L.moe_align_permute_launches.argtypes = [P]
        L.moe_align_permute_launches.restype = i32
        L.moe_gemm2_partial_bytes.argtypes, L.moe_gemm2_partial_bytes.restype = [P, i32], sz
        L.grouped_gemm_w2_split.argtypes = [P, vp, vp, vp, vp, vp, i32, vp, vp]
        L.unpermute_reduce_split.argtypes = [P, vp, i32, vp, vp, vp, vp]
        L.moe_status_string.argtypes, L.moe_status_string.restype = [i32], ctypes.c_char_p
        L.moe_last_error_string.argtypes, L.moe_last_error_string.restype = [], ctypes.c_char_p
        L.moe_debug_set_watchdog.argtypes, L.moe_debug_set_watchdog.restype = \
            [ctypes.c_int64, i32], None
        L.moe_debug_set_bf16_gemm_form.argtypes, L.moe_debug_set_bf16_gemm_form.restype = \
            [i32], None
        L.moe_debug_set_grid_ctas.argtypes, L.moe_debug_set_grid_ctas.restype = [i32], None
        G, i64, f32 = ctypes.POINTER(CRagged), ctypes.c_int64, ctypes.c_float
        L.moe_ragged_workspace_bytes.argtypes, L.moe_ragged_workspace_bytes.restype = [G], sz
        L.ragged_gemm.argtypes = [G] + [vp] * 6 + [sz, vp]
        L.ragged_gemm_dgrad.argtypes = [G] + [vp] * 5 + [sz, vp]
        L.ragged_gemm_wgrad.argtypes = [G] + [vp] * 4 + [i32, i32, vp, sz, vp]
        L.ragged_gemm_mxfp4.argtypes = [G] + [vp] * 7 + [sz, vp]
        L.moe_mxfp4_quantize.argtypes = [vp, i32, i64, i32, i64, i32, vp, vp, vp]
        L.moe_mxfp4_dequantize.argtypes = [vp, vp, i64, i32, vp, i32, i64, vp]
        L.moe_mxfp4_pack_scales.argtypes = [vp, i32, i32, i32, vp, vp]
        L.moe_clip_workspace_bytes.argtypes, L.moe_clip_workspace_bytes.restype = [], sz
        L.moe_clip_grad_norm.argtypes = [i32] + [vp] * 4 + [f32, vp, vp, sz, vp]
        L.ragged_gated.argtypes = [G] + [vp] * 4 + [f32] * 3 + [vp, i64, vp, vp, sz, vp]
        L.ragged_gated_dgrad.argtypes = \
            [G, vp, vp, vp, i64, vp] + [f32] * 3 + [vp, i64, vp, vp, sz, vp]
        L.moe_orthogonalize_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_orthogonalize_workspace_bytes.restype = sz
        L.moe_orthogonalize.argtypes = [i32, i32, i32, vp, i32, vp, i32, vp, f32, f32, vp, sz, vp]
        for n in ("ragged_gemm", "ragged_gemm_dgrad", "ragged_gemm_wgrad", "ragged_gemm_mxfp4",
                  "moe_mxfp4_quantize", "moe_mxfp4_dequantize", "moe_mxfp4_pack_scales",
                  "moe_clip_grad_norm", "ragged_gated", "ragged_gated_dgrad",
                  "moe_orthogonalize"):
            getattr(L, n).restype = i32
        for n in ("moe_align_permute", "grouped_gemm_w13", "act_mul_quant", "grouped_gemm_w2",
                  "unpermute_reduce", "fused_experts", "fused_experts_from_host",
                  "moe_sync_status", "moe_topk_router", "fused_experts_batched",
                  "grouped_gemm_w13_ex", "grouped_gemm_w2_ex", "fused_experts_ex",
                  "grouped_gemm_w2_split", "unpermute_reduce_split", "moe_prepack_weights"):
            getattr(L, n).restype = i32
        _lib = L
    return _lib


def _p(t):
    """Data pointer of a tensor (or None -> NULL)."""
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        detail = moe_last_error_string() if status == 3 else ""
        raise MoEError(status, where, detail)


def _cp(p: Problem):
    return ctypes.byref(p.c())


# ------------------------------------------------------------------ sizes
def moe_m_sum_bound(p: Problem) -> int:
    return int(lib().moe_m_sum_bound(_cp(p)))


def moe_align_workspace_bytes(p: Problem) -> int:
    return int(lib().moe_align_workspace_bytes(_cp(p)))


def moe_align_permute_launches(p: Problem) -> int:
    """Kernels moe_align_permute launches for p (routing + permute)."""
    return int(lib().moe_align_permute_launches(_cp(p)))


def moe_workspace_bytes(p: Problem) -> int:
    return int(lib().moe_workspace_bytes(_cp(p)))


def moe_host_workspace_bytes(p: Problem) -> int:
    return int(lib().moe_host_workspace_bytes(_cp(p)))


def moe_prepacked_scale_bytes(p: Problem, which: int) -> int:
    """Bytes of the prepacked w13 (which=0) or w2 (which=1) weight scales."""
    return int(lib().moe_prepacked_scale_bytes(_cp(p), int(which)))


def moe_prepack_weights(p: Problem, w13_scale, w2_scale, w13_scale_packed, w2_scale_packed,
                        stream=None):
    _check(lib().moe_prepack_weights(_cp(p), _p(w13_scale), _p(w2_scale), _p(w13_scale_packed),
                                     _p(w2_scale_packed), _stream(stream)),
           "moe_prepack_weights")


# ------------------------------------------------------------------ stages
def moe_align_permute(p: Problem, x, topk_ids, topk_weights, sorted_ids, block_expert_ids,
                      expert_offsets, num_post_padded, inv_perm, x_perm, x_perm_scale,
                      workspace, stream=None):
    _check(lib().moe_align_permute(
        _cp(p), _p(x), _p(topk_ids), _p(topk_weights), _p(sorted_ids), _p(block_expert_ids),
        _p(expert_offsets), _p(num_post_padded), _p(inv_perm), _p(x_perm), _p(x_perm_scale),
        _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
        "moe_align_permute")


def moe_align_permute_noalloc(p: Problem, x, topk_ids, topk_weights, sorted_ids,
                              block_expert_ids, expert_offsets, num_post_padded, inv_perm,
                              x_perm, x_perm_scale, stream=None):
    """moe_align_permute without a workspace, for callers that may not
    allocate device memory at call time (for instance an engine that owns the
    whole device through its own memory pool).  Its scratch is a fixed
    MOE_NOALLOC_SCRATCH_BYTES array inside the library, shared by every call on
    a device; larger problems raise MoEError(MOE_ERR_WORKSPACE_TOO_SMALL).
    Make the first call on a device before any stream capture, and keep calls
    ordered on one stream (overlapping calls race on the shared array)."""
    _check(lib().moe_align_permute_noalloc(
        _cp(p), _p(x), _p(topk_ids), _p(topk_weights), _p(sorted_ids), _p(block_expert_ids),
        _p(expert_offsets), _p(num_post_padded), _p(inv_perm), _p(x_perm), _p(x_perm_scale),
        _stream(stream)), "moe_align_permute_noalloc")


def grouped_gemm_w13(p: Problem, x_perm, x_scale, w13, w13_scale, block_expert_ids,
                     num_post_padded, out, out_scale=None, fuse_act=False, stream=None):
    _check(lib().grouped_gemm_w13(
        _cp(p), _p(x_perm), _p(x_scale), _p(w13), _p(w13_scale), _p(block_expert_ids),
        _p(num_post_padded), _p(out), _p(out_scale), int(bool(fuse_act)), _stream(stream)),
        "grouped_gemm_w13")


def act_mul_quant(p: Problem, h1, num_post_padded, z, z_scale=None, stream=None):
    _check(lib().act_mul_quant(_cp(p), _p(h1), _p(num_post_padded), _p(z), _p(z_scale),
                               _stream(stream)), "act_mul_quant")


def grouped_gemm_w2(p: Problem, z, z_scale, w2, w2_scale, block_expert_ids, num_post_padded,
                    y2, stream=None):
    _check(lib().grouped_gemm_w2(_cp(p), _p(z), _p(z_scale), _p(w2), _p(w2_scale),
                                 _p(block_expert_ids), _p(num_post_padded), _p(y2),
                                 _stream(stream)), "grouped_gemm_w2")


def unpermute_reduce(p: Problem, y2, inv_perm, topk_weights, y, stream=None):
    _check(lib().unpermute_reduce(_cp(p), _p(y2), _p(inv_perm), _p(topk_weights), _p(y),
                                  _stream(stream)), "unpermute_reduce")


def grouped_gemm_w13_ex(p: Problem, x_perm, x_scale, w13, w13_scale, w13_bias, block_expert_ids,
                        num_post_padded, out, out_scale=None, fuse_act=False, stream=None):
    _check(lib().grouped_gemm_w13_ex(
        _cp(p), _p(x_perm), _p(x_scale), _p(w13), _p(w13_scale), _p(w13_bias),
        _p(block_expert_ids), _p(num_post_padded), _p(out), _p(out_scale), int(bool(fuse_act)),
        _stream(stream)), "grouped_gemm_w13_ex")


def grouped_gemm_w2_ex(p: Problem, z, z_scale, w2, w2_scale, w2_bias, block_expert_ids,
                       num_post_padded, sorted_ids, topk_weights, y2, stream=None):
    _check(lib().grouped_gemm_w2_ex(
        _cp(p), _p(z), _p(z_scale), _p(w2), _p(w2_scale), _p(w2_bias), _p(block_expert_ids),
        _p(num_post_padded), _p(sorted_ids), _p(topk_weights), _p(y2), _stream(stream)),
        "grouped_gemm_w2_ex")


def fused_experts_ex(p: Problem, x, w13, w13_scale, w13_bias, w2, w2_scale, w2_bias,
                     topk_weights, topk_ids, y, workspace, stream=None):
    _check(lib().fused_experts_ex(
        _cp(p), _p(x), _p(w13), _p(w13_scale), _p(w13_bias), _p(w2), _p(w2_scale), _p(w2_bias),
        _p(topk_weights), _p(topk_ids), _p(y), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)), "fused_experts_ex")


def moe_batched_workspace_bytes(p: Problem, max_tokens: int) -> int:
    return int(lib().moe_batched_workspace_bytes(_cp(p), int(max_tokens)))


def fused_experts_batched(p: Problem, x, expert_num_tokens, w13, w13_scale, w2, w2_scale, y,
                          workspace, expected_m=0, stream=None):
    """Expert MLPs on the batched layout x [E, max_tokens, H] (bf16) with
    per-expert counts (int32 [E]) into y of the same shape."""
    E, T, _ = x.shape
    _check(lib().fused_experts_batched(
        _cp(p), _p(x), _p(expert_num_tokens), int(T), int(expected_m), _p(w13), _p(w13_scale),
        _p(w2), _p(w2_scale), _p(y), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "fused_experts_batched")


SCORING = {"softmax": 0, "sigmoid": 1}


def moe_topk_router(logits, topk, topk_weights, topk_ids, token_expert_indices=None,
                    scoring="softmax", renormalize=True, expert_map=None, stream=None):
    """Router (softmax or sigmoid scores, top-k, optional renormalisation and
    expert map) into caller-allocated [M, topk] float32 / int32 tensors;
    logits [M, E] float32 or bfloat16, all on the device."""
    import torch
    M, E = logits.shape
    bf16 = logits.dtype == torch.bfloat16
    if not bf16 and logits.dtype != torch.float32:
        raise TypeError("logits must be float32 or bfloat16")
    _check(lib().moe_topk_router(int(M), int(E), int(topk), _p(logits), int(bf16),
                                 SCORING[scoring], int(bool(renormalize)), _p(expert_map),
                                 _p(topk_weights), _p(topk_ids), _p(token_expert_indices),
                                 _stream(stream)), "moe_topk_router")


def fused_experts(p: Problem, x, w13, w13_scale, w2, w2_scale, topk_weights, topk_ids, y,
                  workspace, stream=None):
    _check(lib().fused_experts(
        _cp(p), _p(x), _p(w13), _p(w13_scale), _p(w2), _p(w2_scale), _p(topk_weights),
        _p(topk_ids), _p(y), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "fused_experts")


def fused_experts_from_host(p: Problem, host_x, host_topk_ids, host_topk_weights, host_y,
                            w13, w13_scale, w2, w2_scale, workspace, stream=None):
    _check(lib().fused_experts_from_host(
        _cp(p), _p(host_x), _p(host_topk_ids), _p(host_topk_weights), _p(host_y), _p(w13),
        _p(w13_scale), _p(w2), _p(w2_scale), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "fused_experts_from_host")


# --------------------------------------- ragged products, 4-bit operands, clip
# The checks below run on every call of kernels that take a few microseconds:
# each tests everything in one expression and looks for the reason only when
# it fails.
def _fail(name: str, t, shape, dtype, stride, dev):
    """Raises for a tensor argument that is not as the call needs it."""
    if t.get_device() < 0 or dev < 0:
        raise ValueError(f"{name if dev >= 0 else 'every tensor'} must be on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, not cuda:{t.get_device()}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if stride is not None:
        raise ValueError(f"{name} must have strides ({stride}, 1), not {t.stride()}")
    raise ValueError(f"{name} must be dense")


def _dense(name: str, t, shape, dtype, dev) -> int:
    """Data pointer of a dense tensor of this shape and type on GPU dev."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _fail(name, t, shape, dtype, None, dev)


def _rows(name: str, t, shape, dtype, ld, dev) -> int:
    """Data pointer of a matrix on GPU dev whose rows lie ld elements apart."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and (
            t.stride() == (ld, 1) or shape[0] <= 1 and t.stride(1) == 1):
        return t.data_ptr()
    _fail(name, t, shape, dtype, ld, dev)


def _overlap(name: str, ld, cols):
    """Raises for rows that lie closer than they are long.  (An expanded row's
    stride is 0, which the C entry points take for "dense".)"""
    raise ValueError(f"rows of {name} must not overlap (stride {ld} for {cols} columns)")


def _bytes(name: str, t, dev):
    """Data pointer and size of a dense buffer of any type on GPU dev."""
    if t.get_device() == dev and t.is_contiguous():
        return t.data_ptr(), t.nbytes
    _fail(name, t, None, None, None, dev)


def _raw_stream(stream, dev) -> int:
    """The stream given, or PyTorch's current one on GPU dev, the call's leading
    tensor's (-1: not on a GPU).  The library launches on the current GPU."""
    t = _t()
    if dev < 0:
        raise ValueError("every tensor must be on the GPU")
    if dev != t.device():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{t.device()}")
    if stream is None:
        return t.raw_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def moe_ragged_workspace_bytes(p: Ragged) -> int:
    return int(lib().moe_ragged_workspace_bytes(p._ref))


def ragged_gemm(p: Ragged, x, w, expert_offsets, y, workspace, bias=None, stream=None):
    """y[r] = W_e x[r] (+ bias_e) for the rows r of each expert e; x [R, K],
    w [E, N, K], y [R, N], bias [E, N], expert_offsets int32 [E + 1]."""
    v = p._v
    dev = x.get_device()
    ws, n = _bytes("workspace", workspace, dev)
    _check(lib().ragged_gemm(
        p._ref, _rows("x", x, v.x, v.dtype, v.ldx, dev), _dense("w", w, v.w, v.dtype, dev),
        None if bias is None else _dense("bias", bias, v.bias, v.dtype, dev),
        _dense("expert_offsets", expert_offsets, v.offsets, v.int32, dev),
        _rows("y", y, v.y, v.dtype, v.ldy, dev), ws, n, _raw_stream(stream, dev)), "ragged_gemm")


def ragged_gemm_dgrad(p: Ragged, dy, w, expert_offsets, dx, workspace, stream=None):
    """dx[r] = W_e^T dy[r]: the gradient of ragged_gemm's x."""
    v = p._v
    dev = dy.get_device()
    ws, n = _bytes("workspace", workspace, dev)
    _check(lib().ragged_gemm_dgrad(
        p._ref, _rows("dy", dy, v.y, v.dtype, v.ldy, dev), _dense("w", w, v.w, v.dtype, dev),
        _dense("expert_offsets", expert_offsets, v.offsets, v.int32, dev),
        _rows("dx", dx, v.x, v.dtype, v.ldx, dev), ws, n, _raw_stream(stream, dev)),
        "ragged_gemm_dgrad")


def ragged_gemm_wgrad(p: Ragged, dy, x, expert_offsets, dw, workspace, accumulate=False,
                      stream=None):
    """dw[e] (+)= sum over e's rows of dy[r] x[r]^T: the gradient of
    ragged_gemm's w, in the operands' type or float32 (dw's)."""
    v = p._v
    f32 = dw.dtype is v.float32
    dev = dy.get_device()
    ws, n = _bytes("workspace", workspace, dev)
    _check(lib().ragged_gemm_wgrad(
        p._ref, _rows("dy", dy, v.y, v.dtype, v.ldy, dev), _rows("x", x, v.x, v.dtype, v.ldx, dev),
        _dense("expert_offsets", expert_offsets, v.offsets, v.int32, dev),
        _dense("dw", dw, v.w, v.float32 if f32 else v.dtype, dev),
        DTYPE["float32"] if f32 else DTYPE[p.dtype], 1 if accumulate else 0, ws, n,
        _raw_stream(stream, dev)), "ragged_gemm_wgrad")


def _matrix(name: str, t, shape, dtype, dev):
    """Data pointer and row stride (in elements, any that holds a row) of a matrix on GPU
    dev."""
    rows, cols = shape
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        ld, one = t.stride()
        if one == 1 and ld >= cols:
            return t.data_ptr(), ld
        if rows <= 1 and (one == 1 or cols == 1):      # PyTorch leaves it open
            return t.data_ptr(), cols
        if one == 1:
            _overlap(name, ld, cols)
    _fail(name, t, shape, dtype, "any", dev)


def ragged_gated(p: Ragged, x, w13, expert_offsets, z, workspace, h=None, bias=None, alpha=1.0,
                 beta=0.0, limit=0.0, stream=None):
    """z = g' sigmoid(alpha g') (u' + beta) of h = W13_e x (+ bias_e) for the rows of
    each expert e: g' = min(g, limit), u' = clamp(u, -limit, limit), limit <= 0: as they
    are; the default is SiLU(g) u.  p: the gate/up product, N = 2 I; x [R, K], w13
    [E, 2 I, K] (gate rows first), bias [E, 2 I], z [R, I]; h [R, 2 I] is written if
    given, for ragged_gated_dgrad."""
    v = p._v
    dev = x.get_device()
    ws, n = _bytes("workspace", workspace, dev)
    zp, ldz = _matrix("z", z, v.half_n, v.dtype, dev)
    _check(lib().ragged_gated(
        p._ref, _rows("x", x, v.x, v.dtype, v.ldx, dev), _dense("w13", w13, v.w, v.dtype, dev),
        None if bias is None else _dense("bias", bias, v.bias, v.dtype, dev),
        _dense("expert_offsets", expert_offsets, v.offsets, v.int32, dev), alpha, beta, limit,
        zp, ldz,
        None if h is None else _rows("h", h, v.y, v.dtype, v.ldy, dev), ws, n,
        _raw_stream(stream, dev)), "ragged_gated")


def ragged_gated_dgrad(p: Ragged, dy, w2, h, expert_offsets, dh, workspace, z=None, alpha=1.0,
                       beta=0.0, limit=0.0, stream=None):
    """Gradient of the gated block from dy, that of its output W2_e z: dh, that of
    ragged_gated's h, and, if given, z once more.  p: the down projection, K = I;
    dy [R, N], w2 [E, N, I], h and dh [R, 2 I] (may be one), z [R, I]; alpha, beta and
    limit as in ragged_gated."""
    v = p._v
    dev = dy.get_device()
    ws, n = _bytes("workspace", workspace, dev)
    hp, ldh = _matrix("h", h, v.twice_k, v.dtype, dev)
    dhp, lddh = _matrix("dh", dh, v.twice_k, v.dtype, dev)
    _check(lib().ragged_gated_dgrad(
        p._ref, _rows("dy", dy, v.y, v.dtype, v.ldy, dev), _dense("w2", w2, v.w, v.dtype, dev),
        hp, ldh, _dense("expert_offsets", expert_offsets, v.offsets, v.int32, dev), alpha, beta, limit,
        dhp, lddh,
        None if z is None else _rows("z", z, v.x, v.dtype, v.ldx, dev), ws, n,
        _raw_stream(stream, dev)), "ragged_gated_dgrad")


@cache
def _t():
    """torch, and the library's codes of its floating types."""
    import torch
    return SimpleNamespace(
        uint8=torch.uint8, float32=torch.float32, bfloat16=torch.bfloat16, Tensor=torch.Tensor,
        raw_stream=torch._C._cuda_getCurrentRawStream, device=torch._C._cuda_getDevice,
        code={getattr(torch, k): v for k, v in DTYPE.items()})


def _float_code(name: str, t) -> int:
    """moe_dtype of a bfloat16, float16 or float32 tensor."""
    code = _t().code.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, not {t.dtype}")
    return code


def moe_mxfp4_quantize(x, codes, scales, scale_mode="floor", stream=None):
    """E2M1 codes (uint8 [rows, K/2]) and E8M0 scales (uint8 [rows, K/32]) of
    x [rows, K] (bfloat16, float16 or float32; rows may lie apart)."""
    rows, K = x.shape
    ld = x.stride(0) if rows > 1 else K
    if ld < K:
        _overlap("x", ld, K)
    dev, u8 = x.get_device(), _t().uint8
    _check(lib().moe_mxfp4_quantize(
        _rows("x", x, (rows, K), x.dtype, ld, dev), _float_code("x", x), rows, K, ld,
        MXFP4_SCALE[scale_mode], _dense("codes", codes, (rows, K // 2), u8, dev),
        _dense("scales", scales, (rows, K // 32), u8, dev), _raw_stream(stream, dev)),
        "moe_mxfp4_quantize")


def moe_mxfp4_dequantize(codes, scales, out, stream=None):
    """out [rows, K] (bfloat16, float16 or float32) = value * 2^(scale - 127)."""
    rows, K = out.shape
    ld = out.stride(0) if rows > 1 else K
    if ld < K:
        _overlap("out", ld, K)
    dev, u8 = out.get_device(), _t().uint8
    _check(lib().moe_mxfp4_dequantize(
        _dense("codes", codes, (rows, K // 2), u8, dev),
        _dense("scales", scales, (rows, K // 32), u8, dev), rows, K,
        _rows("out", out, (rows, K), out.dtype, ld, dev), _float_code("out", out), ld,
        _raw_stream(stream, dev)), "moe_mxfp4_dequantize")


def moe_mxfp4_pack_scales(scales, packed, stream=None):
    """Weight scales (uint8 [E, N, K/32]) in the block form that
    ragged_gemm_mxfp4 reads; packed has as many bytes."""
    E, N, G = scales.shape
    dev = scales.get_device()
    src = _dense("scales", scales, (E, N, G), _t().uint8, dev)
    dst = _dense("packed", packed, packed.shape, _t().uint8, dev)
    if packed.numel() != scales.numel():
        raise ValueError("packed must have as many bytes as scales")
    _check(lib().moe_mxfp4_pack_scales(src, E, N, 32 * G, dst, _raw_stream(stream, dev)),
           "moe_mxfp4_pack_scales")


def ragged_gemm_mxfp4(p: Ragged, x_codes, x_scales, w_codes, w_scales_packed, expert_offsets, y,
                      workspace, stream=None):
    """y[r] = W_e x[r] with both operands in MXFP4; p.dtype is y's."""
    v = p._v
    dev = x_codes.get_device()
    packed, have = _bytes("w_scales_packed", w_scales_packed, dev)
    if have != v.packed:
        raise ValueError("w_scales_packed must have E * N * K / 32 bytes")
    ws, n = _bytes("workspace", workspace, dev)
    _check(lib().ragged_gemm_mxfp4(
        p._ref, _dense("x_codes", x_codes, v.x_codes, v.uint8, dev),
        _dense("x_scales", x_scales, v.x_scales, v.uint8, dev),
        _dense("w_codes", w_codes, v.w_codes, v.uint8, dev), packed,
        _dense("expert_offsets", expert_offsets, v.offsets, v.int32, dev),
        _rows("y", y, v.y, v.dtype, v.ldy, dev), ws, n, _raw_stream(stream, dev)),
        "ragged_gemm_mxfp4")


def moe_clip_workspace_bytes() -> int:
    return int(lib().moe_clip_workspace_bytes())


def _tensor_arrays(name: str, tensors, norm):
    """Pointers, lengths and types of a list of dense tensors on norm's GPU.  (map over
    the descriptors: lists have dozens of tensors, and this is most of the
    call's time.)"""
    T = _t().Tensor
    types = [*map(_t().code.get, map(T.dtype.__get__, tensors))]
    if None in types:
        raise TypeError(f"{name} must be bfloat16, float16 or float32")
    dev = norm.get_device()
    if not ({*map(T.get_device, tensors)} <= {dev} and all(map(T.is_contiguous, tensors))):
        for t in tensors:
            if not (t.get_device() == dev and t.is_contiguous()):
                _fail(name, t, None, None, None, dev)
    return [*map(T.data_ptr, tensors)], [*map(T.numel, tensors)], types


def moe_clip_grad_norm(grads, max_norm, norm, workspace, out=None, stream=None):
    """Global L2 norm of the gradients (into the float32 scalar tensor norm)
    and clipping to max_norm, in place or into the tensors of ``out``."""
    n = len(grads)
    src, numel, types = _tensor_arrays("grads", grads, norm)
    src = array("Q", src)
    dst = src
    if out is not None:
        dst, n2, t2 = _tensor_arrays("out", out, norm)
        if n2 != numel or t2 != types:
            raise ValueError("out must match grads in number, lengths and types")
        dst = array("Q", dst)
    numel, types = array("q", numel), array("i", types)
    dev = norm.get_device()
    ws, size = _bytes("workspace", workspace, dev)
    _check(lib().moe_clip_grad_norm(
        n, src.buffer_info()[0], dst.buffer_info()[0], numel.buffer_info()[0],
        types.buffer_info()[0], max_norm,
        _dense("norm", norm, norm.shape, _t().float32, dev), ws, size, _raw_stream(stream, dev)),
        "moe_clip_grad_norm")


def moe_orthogonalize_workspace_bytes(E: int, N: int, K: int) -> int:
    return int(lib().moe_orthogonalize_workspace_bytes(int(E), int(N), int(K)))


MAX_ORTHOGONALIZE_STEPS = 64      # MOE_MAX_ORTHOGONALIZE_STEPS in include/moe_ffn.h


@lru_cache(64)
def _coefficients(steps, coefficients):
    """The steps' coefficients as an array: three numbers for all, or three a step."""
    flat = array("f")
    if not coefficients:
        raise ValueError("coefficients must not be empty")
    for c in coefficients if isinstance(coefficients[0], tuple) else (coefficients,) * steps:
        flat.extend(c)
    if len(flat) != 3 * steps:
        raise ValueError(f"coefficients must be three numbers, or three for each of {steps} steps")
    return flat


def _numbers(c):
    """The sequence c, or a sequence of such, with floats in place of what it holds:
    tensors and arrays of one number hash by identity, and may change between calls."""
    c = tuple(c)
    try:
        return tuple(map(float, c))
    except (TypeError, ValueError, RuntimeError):       # not numbers: a triple a step
        return tuple(tuple(map(float, row)) for row in c)


def moe_orthogonalize(g, out, workspace, steps=5, coefficients=(3.4445, -4.7750, 2.0315),
                      eps=1e-7, scale=1.0, stream=None):
    """out = scale X of every matrix of g [E, N, K] (or [N, K]; bfloat16, float16 or
    float32): X = g / (|g|_F + eps), then in each step X = (a I + b A + c A^2) X with
    A = X X^T.  coefficients: (a, b, c), or a sequence of such triples, one a step; steps:
    1 to 64.  out: bfloat16, of g's shape.  Products take operands of 22 bits where the
    steps or short sides need them, else of 11 (include/moe_ffn.h has the errors)."""
    shape = g.shape
    if not 2 <= len(shape) <= 3:
        raise ValueError(f"g must be [E, N, K] or [N, K], not {tuple(shape)}")
    E, N, K = shape if len(shape) == 3 else (1, *shape)
    dev = g.get_device()
    ws, n = _bytes("workspace", workspace, dev)
    if not 1 <= steps <= MAX_ORTHOGONALIZE_STEPS:
        raise ValueError(f"steps must be 1 to {MAX_ORTHOGONALIZE_STEPS}, not {steps}")
    if type(coefficients) is not tuple or set(map(type, coefficients)) != {float}:
        coefficients = _numbers(coefficients)
    c = _coefficients(steps, coefficients)
    _check(lib().moe_orthogonalize(
        E, N, K, _dense("g", g, shape, g.dtype, dev), _float_code("g", g),
        _dense("out", out, shape, _t().bfloat16, dev), steps, c.buffer_info()[0], eps, scale, ws,
        n, _raw_stream(stream, dev)), "moe_orthogonalize")


def moe_gemm2_splits(p: Problem) -> int:
    return int(lib().moe_gemm2_splits(_cp(p)))


def moe_gemm2_partial_bytes(p: Problem, splits: int) -> int:
    return int(lib().moe_gemm2_partial_bytes(_cp(p), int(splits)))


def grouped_gemm_w2_split(p: Problem, z, w2, block_expert_ids, num_post_padded, sorted_ids,
                          splits, partial, stream=None):
    _check(lib().grouped_gemm_w2_split(
        _cp(p), _p(z), _p(w2), _p(block_expert_ids), _p(num_post_padded), _p(sorted_ids),
        int(splits), _p(partial), _stream(stream)), "grouped_gemm_w2_split")


def unpermute_reduce_split(p: Problem, partial, splits, inv_perm, topk_weights, y, stream=None):
    _check(lib().unpermute_reduce_split(
        _cp(p), _p(partial), int(splits), _p(inv_perm), _p(topk_weights), _p(y),
        _stream(stream)), "unpermute_reduce_split")


def moe_sync_status(stream=None) -> int:
    return int(lib().moe_sync_status(_stream(stream)))


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def moe_last_error_string() -> str:
    return lib().moe_last_error_string().decode()


def moe_debug_set_watchdog(limit_ns: int, never_arrive: bool = False):
    lib().moe_debug_set_watchdog(int(limit_ns), int(bool(never_arrive)))


# "clusters" is "pairs_double", under what it is for the orthogonalised update
BF16_GEMM_FORMS = {"auto": 0, "single": 1, "pairs": 2, "pairs_double": 3, "clusters": 3,
                   "whole_grid": 4}


def moe_debug_set_bf16_gemm_form(form: str = "auto"):
    """Force the single-SM or the SM-pair GEMMs (tests), or restore the
    size-based choice; "pairs_double" or "clusters": ragged forward and dgrad on double
    tiles, the orthogonalised update in one launch of clusters; "whole_grid": that update
    in one launch over the whole grid, all else by size."""
    lib().moe_debug_set_bf16_gemm_form(BF16_GEMM_FORMS[form])


def moe_debug_set_grid_ctas(ctas: int = 0):
    """CTAs of the orthogonalised update's launch over the whole grid (tests; 0: one an
    SM).  More than the GPU runs at once are refused as where a context has few SMs."""
    lib().moe_debug_set_grid_ctas(int(ctas))


# ------------------------------------------------- buffer allocation helper
def stage_buffers(p: Problem, device="cuda"):
    """Allocates (torch.empty) the outputs of the staged entry points for
    problem ``p``, sized by the library's own bound; returns a dict."""
    import torch
    cap = moe_m_sum_bound(p)
    q = p.quant != "bf16"
    g = 32 if p.quant == "mxfp8" else 128      # activation quantisation group
    xb = torch.uint8 if q else torch.bfloat16
    i32 = dict(dtype=torch.int32, device=device)
    return {
        "sorted_ids": torch.empty(cap, **i32),
        "block_expert_ids": torch.empty(cap // p.block_size, **i32),
        "expert_offsets": torch.empty(p.E + 1, **i32),
        "num_post_padded": torch.empty(1, **i32),
        "inv_perm": torch.empty(p.M, p.topk, **i32),
        "x_perm": torch.empty(cap, p.H, dtype=xb, device=device),
        "x_perm_scale": torch.empty(cap, p.H // g, dtype=torch.float32, device=device)
        if q else None,
        "h1": torch.empty(cap, 2 * p.I, dtype=torch.bfloat16, device=device),
        "z": torch.empty(cap, p.I, dtype=xb, device=device),
        "z_scale": torch.empty(cap, p.I // g, dtype=torch.float32, device=device)
        if q else None,
        "y2": torch.empty(cap, p.H, dtype=torch.bfloat16, device=device),
        "y": torch.empty(p.M, p.H, dtype=torch.bfloat16, device=device),
        "align_ws": torch.empty(max(moe_align_workspace_bytes(p), 1), dtype=torch.uint8,
                                device=device),
    }
