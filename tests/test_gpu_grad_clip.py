"""Global gradient norm and clipping against fp64.

Norm: squares in fp32 (2^-24 each), at most 64 added in fp32 (64 * 2^-24 of the
sum), fp64 beyond, one rounding to fp32: relative error of the square sum below
66 * 2^-24, so of the norm below 34 * 2^-24.  Outputs: the coefficient's error
(the norm's and three fp32 roundings) and half a step of the type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
NORM_TOL = 34 * 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def workspace():
    return torch.empty(moe.moe_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")


def check(grads, max_norm, in_place=False):
    before = [f64(g) for g in grads]
    out = None if in_place else [torch.full_like(g, 7.0) for g in grads]
    norm = torch.full((), -1.0, device="cuda")
    moe.moe_clip_grad_norm(grads, max_norm, norm, workspace(), out=out)
    ref, clipped = ragged.clip(before, max_norm)
    assert abs(float(norm) - ref) <= NORM_TOL * ref
    for g, o, r, b in zip(grads, grads if in_place else out, clipped, before):
        fi = torch.finfo(g.dtype)
        tol = (fi.eps / 2 + NORM_TOL + 3 * 2.0 ** -24) * np.abs(r) + fi.tiny * fi.eps
        assert (np.abs(f64(o) - r) <= tol).all()
        if not in_place:
            assert np.array_equal(f64(g), b)
    return float(norm)


def rand(n, dtype, seed, scale=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6])
def test_mixed_list(max_norm, in_place):
    sizes = [1, 7, 8, 9, 1023, 16384, 16385, 70001, 3, 8192, 300000, 2, 5]
    check([rand(n, TYPES[i % 3], i) for i, n in enumerate(sizes)], max_norm, in_place)


@pytest.mark.parametrize("dtype", TYPES)
def test_alignment_and_empty_tensors(dtype):
    base = rand(40000, dtype, 1)
    grads = [base[1:20000], base[20003:20003], base[20004:39999], rand(0, dtype, 2)]
    check(grads, 1.0)
    check([g.clone() for g in grads], 1.0, in_place=True)
    check([base[1:20000], base[20001:]], 1.0, in_place=True)


@pytest.mark.parametrize("n", [64, 65, 1024, 1025, 2500])
def test_long_lists(n):
    check([rand(1 + 37 * (i % 50), TYPES[i % 3], i) for i in range(n)], 1.0, in_place=True)


def test_no_tensors_and_zero_gradients():
    norm = torch.full((), -1.0, device="cuda")
    moe.moe_clip_grad_norm([], 1.0, norm, workspace())
    assert float(norm) == 0
    z = torch.zeros(1000, device="cuda")
    moe.moe_clip_grad_norm([z], 1.0, norm, workspace())
    assert float(norm) == 0 and not z.any()


def test_below_the_limit_is_untouched():
    g = [rand(100000, t, 5) for t in TYPES]
    before = [t.clone() for t in g]
    norm = torch.empty((), device="cuda")
    moe.moe_clip_grad_norm(g, 1e9, norm, workspace())
    assert all(bool((a == b).all()) for a, b in zip(g, before))


def test_large_and_non_finite_values():
    # bf16 values whose squares pass fp16's range but not fp32's
    check([rand(5000, torch.bfloat16, 1, 1e15)], 1.0)
    norm = torch.empty((), device="cuda")
    for bad in (float("inf"), float("nan")):
        g = rand(5000, torch.float32, 2)
        g[77] = bad
        moe.moe_clip_grad_norm([g], 1.0, norm, workspace())
        if bad != bad:
            assert norm.isnan() and bool(g.isnan().all())
        else:
            assert norm.isinf() and g[77].isnan() and float(g[0]) == 0.0


def test_same_result_every_time_and_in_a_graph():
    g = [rand(1000003, TYPES[i], i) for i in range(3)]
    out = [torch.empty_like(t) for t in g]
    norm, ws = torch.empty((), device="cuda"), workspace()
    moe.moe_clip_grad_norm(g, 1.0, norm, ws, out=out)
    first = [norm.clone()] + [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_clip_grad_norm(g, 1.0, norm, ws, out=out)
    for _ in range(5):
        norm.zero_()
        graph.replay()
        assert all(bool((a == b).all()) for a, b in zip(first, [norm] + out))
    for t in g:
        t.mul_(2)
    graph.replay()
    assert abs(float(norm) - 2 * float(first[0])) <= 1e-6 * float(norm)
