"""The gated block and the orthogonalised update without a GPU: refusals of the C ABI
(nothing is launched), workspaces, and the oracle against differences and known cases."""
import ctypes
import os

import numpy as np
import pytest

import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

OK, INVALID, SMALL = 0, 1, 5
PTR = ctypes.c_void_p(4096)      # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(4096 + 8)
BIG = 1 << 50
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(moe.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()


def gated(x=PTR, w=PTR, bias=None, offsets=PTR, alpha=1.0, beta=0.0, limit=0.0, z=PTR, ldz=0, h=PTR,
          ws=PTR, size=BIG, **kw):
    p = moe.Ragged(**{**dict(R=16, N=128, K=128, E=4), **kw})
    return moe.lib().ragged_gated(p._ref, x, w, bias, offsets, alpha, beta, limit, z, ldz, h, ws,
                                  size, None)


def grad(dy=PTR, w=PTR, h=PTR, ldh=0, offsets=PTR, alpha=1.0, beta=0.0, limit=0.0,
         dh=ctypes.c_void_p(8192), lddh=0,
         z=PTR, ws=PTR, size=BIG, **kw):
    p = moe.Ragged(**{**dict(R=16, N=128, K=128, E=4), **kw})
    return moe.lib().ragged_gated_dgrad(p._ref, dy, w, h, ldh, offsets, alpha, beta, limit, dh, lddh,
                                        z, ws, size, None)


def ortho(E=2, N=64, K=96, g=PTR, dtype=2, out=PTR, steps=5, c=(3.0, -3.0, 1.0), eps=1e-7, scale=1.0,
          ws=PTR, size=BIG):
    flat = None if c is None else (ctypes.c_float * max(1, 3 * steps))(*(list(c) * max(steps, 0)))
    return moe.lib().moe_orthogonalize(E, N, K, g, dtype, out, steps, flat, eps, scale, ws, size,
                                       None)


@pytest.mark.parametrize("bad", [dict(N=136), dict(N=8), dict(R=-1), dict(K=12), dict(E=0),
                                 dict(dtype="float32"), dict(ldx=120), dict(ldy=120),
                                 dict(alpha=NAN), dict(alpha=INF), dict(beta=NAN), dict(limit=NAN),
                                 dict(ldz=56), dict(ldz=68), dict(ldz=-64), dict(x=None), dict(w=None),
                                 dict(z=None), dict(offsets=None), dict(ws=None), dict(x=ODD),
                                 dict(w=ODD), dict(z=ODD), dict(h=ODD),
                                 dict(bias=ctypes.c_void_p(4097))], ids=str)
def test_gated_refusals(bad):
    assert gated(**bad) == INVALID


@pytest.mark.parametrize("bad", [dict(N=12), dict(K=12), dict(R=(1 << 22) + 1), dict(alpha=NAN),
                                 dict(beta=INF), dict(limit=NAN), dict(ldh=248), dict(ldh=260),
                                 dict(lddh=128), dict(lddh=-256), dict(dy=None), dict(w=None),
                                 dict(h=None), dict(dh=None), dict(ws=None), dict(offsets=None),
                                 dict(dy=ODD), dict(h=ODD), dict(dh=ODD), dict(z=ODD),
                                 dict(dh=PTR, lddh=264)], ids=str)
def test_gated_grad_refusals(bad):
    assert grad(**bad) == INVALID


def test_workspaces_and_empty_problems():
    need = moe.moe_ragged_workspace_bytes(moe.Ragged(R=16, N=128, K=128, E=4))
    assert gated(size=need - 1) == SMALL and grad(size=need - 1) == SMALL
    none = dict(R=0, ws=None, size=0)
    assert gated(x=None, w=None, z=None, h=None, **none) == OK
    assert grad(dy=None, w=None, h=None, dh=None, z=None, **none) == OK


@pytest.mark.parametrize("bad", [dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(K=(1 << 18) + 1), dict(N=(1 << 18) + 1),
                                 dict(E=1024, N=1 << 18, K=1 << 18), dict(dtype=3), dict(dtype=-1),
                                 dict(steps=0), dict(steps=65), dict(c=None), dict(c=(1.0, NAN, 0.0)),
                                 dict(c=(INF, 0.0, 0.0)), dict(eps=0.0), dict(eps=-1.0),
                                 dict(eps=NAN), dict(eps=INF), dict(scale=NAN), dict(scale=INF),
                                 dict(g=None), dict(out=None), dict(ws=None), dict(out=ODD),
                                 dict(g=ctypes.c_void_p(4098)), dict(ws=ctypes.c_void_p(4096 + 128))],
                         ids=str)
def test_orthogonalize_refusals(bad):
    assert ortho(**bad) == INVALID


def test_orthogonalize_workspace():
    need = moe.moe_orthogonalize_workspace_bytes(2, 64, 96)
    assert need > 0 and ortho(size=need - 1) == SMALL
    for bad in ((0, 64, 96), (2, 0, 96), (2, 64, 0), (1025, 8, 8), (1, 1 << 21, 1)):
        assert moe.moe_orthogonalize_workspace_bytes(*bad) == 0
    # two copies of X, its lower bits and two squares, in fp16, and little beside
    E, N, K = 8, 4096, 14336
    need = moe.moe_orthogonalize_workspace_bytes(E, N, K)
    assert need == moe.moe_orthogonalize_workspace_bytes(E, K, N)
    assert 0 <= need - E * (6 * N * K + 4 * N * N) < 1 << 20


def test_coefficient_forms():
    one = moe._coefficients(2, (1.0, 2.0, 3.0))
    assert list(one) == [1.0, 2.0, 3.0] * 2
    assert list(moe._coefficients(2, ((1.0, 2.0, 3.0), (4.0, 5.0, 6.0)))) == [1, 2, 3, 4, 5, 6]
    for bad in (((1.0, 2.0, 3.0),) * 3, (1.0, 2.0), ((1.0, 2.0),) * 2, ()):
        with pytest.raises(ValueError):
            moe._coefficients(2, bad)


@pytest.mark.parametrize("recipe", [(1.0, 0.0, 0.0), (1.702, 1.0, 1.2), (0.5, -0.3, 0.0)])
def test_oracle_gradient_against_differences(recipe):
    rng = np.random.default_rng(0)
    h, dz = rng.standard_normal((4, 12)), rng.standard_normal((4, 6))
    got, step = ragged.gated_grad(dz, h, *recipe), 1e-6
    for i in range(4):
        for j in range(12):
            e = np.zeros_like(h)
            e[i, j] = step
            want = (dz * (ragged.gated(h + e, *recipe) - ragged.gated(h - e, *recipe))).sum() / (2 * step)
            assert abs(got[i, j] - want) < 1e-8


def test_oracle_orthogonalize_known_cases():
    # a scalar goes through the polynomial
    x = 1.0
    for _ in range(5):
        x = 3.4445 * x - 4.7750 * x ** 3 + 2.0315 * x ** 5
    assert abs(ragged.orthogonalize(np.array([[5.0]]), eps=0.0)[0, 0] - x) < 1e-12
    # orthogonal rows stay so, and the cubic form converges to the polar factor
    rng = np.random.default_rng(1)
    g = rng.standard_normal((6, 9))
    u, _, v = np.linalg.svd(g, full_matrices=False)
    got = ragged.orthogonalize(g, steps=30, coefficients=(1.5, -0.5, 0.0))
    assert np.abs(got - u @ v).max() < 1e-9
    assert np.allclose(ragged.orthogonalize(g.T), ragged.orthogonalize(g).T)
