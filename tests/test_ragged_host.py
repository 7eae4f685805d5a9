"""Training and 4-bit operators without a GPU: refusals of the C ABI (nothing
is launched), and the oracle against differences and hand-worked values."""
import ctypes
import os

import numpy as np
import pytest

import mixture_experts_ffn_align_gb300 as moe
from oracle import codecs, ragged

OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 5
PTR = ctypes.c_void_p(4096)      # aligned, never dereferenced: validation fails first
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(moe.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()


def problem(**kw):
    d = dict(R=16, N=128, K=128, E=4)
    d.update(kw)
    return moe.Ragged(**d)


def calls(p, ptr=PTR, ws=PTR, ws_bytes=BIG, offsets=PTR):
    """Status of every ragged entry point for the same arguments."""
    L = moe.lib()
    return {
        "fwd": L.ragged_gemm(p._ref, ptr, PTR, None, offsets, PTR, ws, ws_bytes, None),
        "dgrad": L.ragged_gemm_dgrad(p._ref, ptr, PTR, offsets, PTR, ws, ws_bytes, None),
        "wgrad": L.ragged_gemm_wgrad(p._ref, ptr, PTR, offsets, PTR, 0, 0, ws, ws_bytes, None),
        "mxfp4": L.ragged_gemm_mxfp4(p._ref, ptr, PTR, PTR, PTR, offsets, PTR, ws, ws_bytes, None),
    }


@pytest.mark.parametrize("bad", [dict(R=-1), dict(R=(1 << 22) + 1), dict(N=0), dict(N=12),
                                 dict(K=4), dict(K=(1 << 20) + 8), dict(E=0), dict(E=1025),
                                 dict(ldx=120), dict(ldx=132), dict(ldy=64), dict(ldy=-8),
                                 dict(dtype="float32"),
                                 dict(N=1 << 20, K=1 << 20, E=1024)])
def test_invalid_ragged_problems_rejected(bad):
    p = problem(**bad)
    assert moe.moe_ragged_workspace_bytes(p) == 0
    assert set(calls(p).values()) == {INVALID}


def test_null_and_misaligned_pointers_rejected():
    p = problem()
    odd = ctypes.c_void_p(4096 + 8)
    assert set(calls(p, ptr=None).values()) == {INVALID}
    assert set(calls(p, ptr=odd).values()) == {INVALID}
    assert set(calls(p, offsets=None).values()) == {INVALID}
    assert set(calls(p, offsets=ctypes.c_void_p(4098)).values()) == {INVALID}
    assert set(calls(p, ws=None).values()) == {INVALID}
    assert set(calls(p, ws=ctypes.c_void_p(4096 + 64)).values()) == {INVALID}
    assert set(calls(p, ws_bytes=moe.moe_ragged_workspace_bytes(p) - 1).values()) == {SMALL}


def test_empty_problem_is_a_noop():
    L, p = moe.lib(), problem(R=0)
    assert L.ragged_gemm(p._ref, None, None, None, None, None, None, 0, None) == OK
    assert L.ragged_gemm_dgrad(p._ref, None, None, None, None, None, 0, None) == OK
    assert L.ragged_gemm_mxfp4(p._ref, None, None, None, None, None, None, None, 0, None) == OK
    assert L.ragged_gemm_wgrad(p._ref, None, None, None, None, 0, 1, None, 0, None) == OK
    # without accumulation the gradient would have to be zeroed
    assert L.ragged_gemm_wgrad(p._ref, None, None, None, None, 0, 0, None, 0, None) == INVALID


def test_wgrad_output_types():
    L, p = moe.lib(), problem(dtype="float16")
    for dt, acc in ((0, 0), (3, 0), (2, 2), (1, -1)):
        assert L.ragged_gemm_wgrad(p._ref, PTR, PTR, PTR, PTR, dt, acc, PTR, BIG, None) == INVALID


@pytest.mark.parametrize("kw, status", [(dict(N=136), UNSUPPORTED), (dict(K=192), UNSUPPORTED),
                                        (dict(ldx=256), INVALID)])
def test_mxfp4_product_shapes(kw, status):
    assert calls(problem(**kw))["mxfp4"] == status


def test_mxfp4_codec_refusals():
    L = moe.lib()
    odd = ctypes.c_void_p(4096 + 8)

    def q(x=PTR, dt=0, rows=4, K=64, ld=0, mode=0, codes=PTR, scales=PTR):
        return L.moe_mxfp4_quantize(x, dt, rows, K, ld, mode, codes, scales, None)

    def d(codes=PTR, scales=PTR, rows=4, K=64, out=PTR, dt=0, ld=0):
        return L.moe_mxfp4_dequantize(codes, scales, rows, K, out, dt, ld, None)

    for bad in (dict(dt=3), dict(rows=-1), dict(K=48), dict(K=0), dict(ld=56), dict(ld=68),
                dict(x=None), dict(x=odd), dict(codes=odd), dict(scales=None)):
        assert q(**bad) == INVALID, bad
    assert q(mode=2) == INVALID
    for bad in (dict(dt=-1), dict(rows=-1), dict(K=33), dict(ld=60), dict(ld=66), dict(out=None),
                dict(out=odd), dict(codes=odd), dict(scales=None)):
        assert d(**bad) == INVALID, bad
    assert q(rows=0, x=None, codes=None, scales=None) == OK
    assert d(rows=0, out=None, codes=None, scales=None) == OK
    assert L.moe_mxfp4_pack_scales(PTR, 0, 128, 128, PTR, None) == INVALID
    assert L.moe_mxfp4_pack_scales(PTR, 1, 136, 128, PTR, None) == UNSUPPORTED
    assert L.moe_mxfp4_pack_scales(PTR, 1, 128, 64, PTR, None) == UNSUPPORTED
    assert L.moe_mxfp4_pack_scales(None, 1, 128, 128, PTR, None) == INVALID


def test_clip_refusals():
    L = moe.lib()

    def c(n=1, ptr=4096, out=4096, numel=8, dt=0, max_norm=1.0, norm=PTR, ws=PTR, nbytes=BIG):
        one = max(n, 1) if n < 100 else 1
        g, o = (ctypes.c_void_p * one)(*[ptr] * one), (ctypes.c_void_p * one)(*[out] * one)
        m, t = (ctypes.c_int64 * one)(*[numel] * one), (ctypes.c_int32 * one)(*[dt] * one)
        return L.moe_clip_grad_norm(n, g, o, m, t, max_norm, norm, ws, nbytes, None)

    for bad in (dict(n=-1), dict(n=65537), dict(ptr=None), dict(out=None), dict(ptr=4097),
                dict(dt=2, ptr=4098), dict(dt=2, out=4098), dict(numel=-1), dict(dt=3),
                dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None), dict(ws=None),
                dict(ws=ctypes.c_void_p(4104))):
        assert c(**bad) == INVALID, bad
    assert c(nbytes=moe.moe_clip_workspace_bytes() - 1) == SMALL
    assert L.moe_clip_grad_norm(1, None, None, None, None, 1.0, PTR, PTR, BIG, None) == INVALID


def test_binding_refuses_wrong_tensors():
    import torch
    p = problem()
    x = torch.zeros(16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        moe.ragged_gemm(p, x, x, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_mxfp4_quantize(x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_clip_grad_norm([x], 1.0, x, x)
    with pytest.raises(TypeError):
        moe.moe_clip_grad_norm([x.int()], 1.0, x, x)


# ------------------------------------------------------------------- oracle
def test_oracle_gradients_match_differences():
    rng = np.random.default_rng(0)
    off = [0, 3, 3, 8]
    x, w, g = rng.normal(size=(8, 5)), rng.normal(size=(3, 4, 5)), rng.normal(size=(8, 4))

    def loss(x, w):
        return float(np.sum(np.tanh(ragged.forward(x, w, off)) * g))

    dy = g * (1 - np.tanh(ragged.forward(x, w, off)) ** 2)
    dx, dw = ragged.dgrad(dy, w, off), ragged.wgrad(dy, x, off)
    h = 1e-6
    for grad, t, f in ((dx, x, lambda t: loss(t, w)), (dw, w, lambda t: loss(x, t))):
        for i in np.ndindex(t.shape):
            up, dn = t.copy(), t.copy()
            up[i] += h
            dn[i] -= h
            # central difference: error h^2 / 6 |f'''| + 2 eps |f| / h < 1e-8 here
            assert abs((f(up) - f(dn)) / (2 * h) - grad[i]) < 1e-7
    assert not dw[1].any()


def test_oracle_mxfp4_hand_worked():
    x = np.zeros((1, 64))
    # floor: a = 6.5 -> scale 1; ties 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2,
    # 3.5 -> 4, 5 -> 4; 6.5 saturates at 6
    vals = [6.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.3, 0.1]
    x[0, :len(vals)] = vals
    c, s = ragged.mxfp4_quantize(x)
    assert list(codecs.e2m1_decode(c[0, :len(vals)])) == [6, 0, 1, 1, 2, 2, 4, 4, 0, -0.5, 0]
    assert list(s[0]) == [127, 0]
    # ceil: 6.5 > 6 -> scale 2
    c, s = ragged.mxfp4_quantize(x, "ceil")
    assert s[0, 0] == 128 and codecs.e2m1_decode(c[0, :1])[0] == 3     # 3.25 -> 3
    x[0, 3] = np.inf
    c, s = ragged.mxfp4_quantize(x)
    assert s[0, 0] == 255 and not c[0, :32].any()
    assert np.isnan(ragged.mxfp4_dequantize(ragged.pack_fp4(c), s)[0, :32]).all()


def test_oracle_pack_scales_positions():
    E, N, K = 2, 256, 256
    s = np.random.default_rng(1).integers(0, 255, (E, N, K // 32), dtype=np.uint8)
    p = ragged.pack_scales(s)
    for e, kb, g, l, c, j in ((0, 0, 0, 0, 0, 0), (1, 1, 1, 31, 3, 3), (1, 0, 1, 7, 2, 1)):
        assert p[e, kb, g, 16 * l + 4 * c + j] == s[e, 128 * g + 32 * c + l, 4 * kb + j]


def test_oracle_clip():
    norm, out = ragged.clip([np.array([3.0]), np.array([4.0])], 1.0)
    assert norm == 5.0 and abs(out[0][0] - 0.6) < 1e-6
    assert ragged.clip([np.array([3.0])], 10.0)[1][0][0] == 3.0
