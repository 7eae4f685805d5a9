"""Ragged grouped products, the MXFP4 codec and gradient clipping -- fp64
oracle (test infrastructure only), from the formulas:

* forward  y[r] = W_e x[r] + b_e, dgrad dx[r] = W_e^T dy[r],
  wgrad dW_e = sum_r dy[r] x[r]^T over the rows offsets[e] .. offsets[e+1]-1;
* MXFP4: per 32 values a power-of-two scale and E2M1 codes (OCP Microscaling
  Formats specification v1.0, section 6.3, for the floor form);
* clip: c = min(1, max_norm / (norm + 1e-6)) over all tensors' L2 norm.
"""
from __future__ import annotations

import numpy as np

from . import codecs


def _segments(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def forward(x, w, offsets, bias=None):
    y = np.zeros((x.shape[0], w.shape[1]))
    for e, a, b in _segments(offsets):
        y[a:b] = x[a:b] @ w[e].T + (0.0 if bias is None else bias[e])
    return y


def dgrad(dy, w, offsets):
    dx = np.zeros((dy.shape[0], w.shape[2]))
    for e, a, b in _segments(offsets):
        dx[a:b] = dy[a:b] @ w[e]
    return dx


def wgrad(dy, x, offsets):
    return np.stack([dy[a:b].T @ x[a:b] for _, a, b in _segments(offsets)])


def mxfp4_quantize(x, scale_mode="floor"):
    """x [R, K] finite or not -> (codes [R, K] E2M1 nibbles, scales [R, K/32])."""
    v = np.asarray(x, dtype=np.float64)
    R, K = v.shape
    g = v.reshape(R, K // 32, 32)
    amax = np.abs(g).max(-1)
    bad = ~np.isfinite(amax)
    a = np.where(bad | (amax == 0), 1.0, amax)
    m, e = np.frexp(a)                          # a = m 2^e, 0.5 <= m < 1
    s = e - 1 - 2
    if scale_mode == "ceil":
        s = np.where(2 * m > 1.5, s + 1, s)
    s = np.where(amax == 0, -127, np.maximum(s, -127))
    with np.errstate(invalid="ignore"):
        q = np.ldexp(np.abs(g), -s[..., None])
    grid = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    q = np.where(bad[..., None], 0.0, q)
    d = np.abs(q[..., None] - grid)
    best = d.min(-1, keepdims=True)
    # of two equally near values the one with the even code
    near = d == best
    code = np.where(near[..., ::2].any(-1), 2 * near[..., ::2].argmax(-1), near.argmax(-1))
    code = np.where(q >= 6.0, 7, code)
    sign = np.where(np.signbit(g) & ~bad[..., None], 8, 0)
    return ((code | sign).reshape(R, K).astype(np.uint8),
            np.where(bad, 255, s + 127).astype(np.uint8))


def pack_fp4(codes):
    c = np.asarray(codes, dtype=np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def mxfp4_dequantize(packed, scales):
    k = packed.shape[-1] * 2
    v = codecs.e2m1_decode(codecs.unpack_fp4(packed, k))
    s = np.asarray(scales)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return v * np.repeat(f, 32, axis=-1)


def pack_scales(scales):
    """[E, N, K/32] -> [E, K/128, N/128, 512]: byte 16 l + 4 c + j of a block is
    the scale of row 32 c + l, chunk j."""
    E, N, G = scales.shape
    v = scales.reshape(E, N // 128, 4, 32, G // 4, 4)
    return np.ascontiguousarray(v.transpose(0, 4, 1, 3, 2, 5)).reshape(E, G // 4, N // 128, 512)


def clip(grads, max_norm):
    norm = float(np.sqrt(sum(np.sum(np.square(g)) for g in grads)))
    c = min(1.0, max_norm / (norm + 1e-6))
    return norm, [g * c for g in grads]
