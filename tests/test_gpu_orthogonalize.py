"""The orthogonalised update against the fp64 oracle.

Tolerances.  The kernels round X, A and B to fp16's 11 bits where the shorter side is
longer than 128 (and add a X with 22 bits, in all steps but the last).  The oracle
with the same rounding points (of scaled values, powers of two as the kernels take)
shows what these cost on the same inputs; another order of the
sums turns single roundings over, but not their number or size, so the kernels' rms
error is held to 1.3 times the rounded oracle's (with the result's rounding to bf16 in
both).  A value out of place would be off by its own size: single errors are held to
25 times the rms of the errors (5 deviations of the largest, which are up to 4 to 5 times
the typical value).
Up to 128 the operands have 22 bits, errors of 2^-23 relative to sums of magnitudes, and
accumulation truncates once per 16 products: (L / 16 + 20) 2^-23 of a sum over L.  In a
step |a| + |b| + |c| = 10.3 (for singular values of 1) enters a value of 0.7: a gain
of 15; three products in each of five steps: at most 225 (L / 16 + 20) 2^-23 relative to
the singular values' scale, L three times the longer side.  Beyond half a step of bf16,
errors are held to that times the largest value.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

pytestmark = pytest.mark.gpu
DT = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


@pytest.fixture(params=["auto", "single", "pairs", "pairs_double", "whole_grid"])
def form(request):
    """By size; products one launch each, on one SM or SM pairs; all steps in one launch,
    in clusters or over the whole grid."""
    moe.moe_debug_set_bf16_gemm_form(request.param)
    yield request.param
    moe.moe_debug_set_bf16_gemm_form("auto")


def f64(t):
    return t.double().cpu().numpy()


def gradient(shape, dtype, seed, strong=0.02):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, n, k = shape
    v = 0.01 * torch.randn(shape, generator=g, device="cuda")
    v += strong * torch.randn(E, n, 1, generator=g, device="cuda") * \
        torch.randn(E, 1, k, generator=g, device="cuda")
    return v.to(DT[dtype])


def call(g, out=None, **kw):
    shape = g.shape if g.dim() == 3 else (1, *g.shape)
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(*shape), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)                       # NaN patterns: nothing of it may be read before it is written
    if out is None:
        out = torch.full(g.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_orthogonalize(g, out, ws, **kw)
    assert moe.moe_sync_status() == 0
    return out


def fp16(v):
    """Rounded to 11 bits as at a scale well inside fp16's range."""
    m, e = np.frexp(v)
    return np.ldexp(np.round(m * 2.0 ** 11), e - 11)


def bf16(v):
    return f64(torch.tensor(v).to(torch.bfloat16))


def check(got, g, scale=1.0, **kw):
    for i in range(g.shape[0]):
        G, y = f64(g[i]), f64(got[i])
        ref = scale * ragged.orthogonalize(G, **kw)
        assert np.isfinite(y).all()
        err = np.abs(y - ref)
        if min(G.shape) <= 128:
            tol = 225 * (3 * max(G.shape) / 16 + 20) * 2.0 ** -23 * np.abs(ref).max()
            # half a step of bf16: 8 bits, so 2^-8 of a value just above a power of two
            half = torch.finfo(torch.bfloat16).eps / 2
            assert (err <= half * np.abs(ref) + tol).all(), (i, err.max(), tol)
            continue
        kept = kw.get("steps", 5) - 1
        rounded = scale * ragged.orthogonalize(G, rounded=fp16, kept=kept, **kw)
        cost = np.sqrt(np.mean((bf16(rounded) - ref) ** 2))
        rms = np.sqrt(np.mean(err ** 2))
        assert rms <= 1.3 * cost, (i, rms / cost)
        assert err.max() <= 25 * cost, (i, err.max() / cost)


SMALL = [(1, 1, 1), (2, 1, 77), (2, 77, 1), (3, 2, 50), (2, 8, 264), (2, 33, 31), (3, 64, 64),
         (2, 65, 129), (2, 200, 96), (1, 256, 512), (2, 255, 257), (1, 500, 130), (1, 16, 3000)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SMALL, ids=str)
def test_short_sides(shape, dtype, form):
    g = gradient(shape, dtype, sum(shape))
    check(call(g), g)


LARGE = [(1, 257, 257), (2, 264, 600), (2, 600, 264), (1, 512, 1031), (1, 777, 513), (1, 1024, 640)]


@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_long_sides(shape, form):
    for dtype, strong in (("bfloat16", 0.02), ("float32", 0.0)):
        g = gradient(shape, dtype, sum(shape), strong)
        check(call(g), g)


@pytest.mark.parametrize("strong", [0.1, 0.5, 2.0])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_one_strong_direction(strong, dtype, form):
    """A direction 10 to 200 times as strong as the rest: the rest grows most, and what
    is lost beside the strong one with it."""
    for shape in ((1, 200, 400), (1, 520, 300)):
        g = gradient(shape, dtype, 21, strong)
        check(call(g), g)


@pytest.mark.parametrize("rank", [1, 3, 40])
def test_few_rows_gradients(rank, form):
    """Of low rank, as an expert's gradient of few rows: what the products lose in the null
    space grows in every step."""
    for shape in ((150, 300), (400, 260)):
        g = torch.randn(shape[0], rank, generator=torch.Generator("cuda").manual_seed(rank),
                        device="cuda") @ torch.randn(
            rank, shape[1], generator=torch.Generator("cuda").manual_seed(9), device="cuda")
        g = g[None].contiguous()
        got = call(g)
        check(got, g)
        ref = ragged.orthogonalize(f64(g[0]))
        err = np.sqrt(np.mean((f64(got[0]) - ref) ** 2) / np.mean(ref ** 2))
        assert err <= 0.0025                   # what the library states


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 8])
def test_steps_with_long_sides(steps, form):
    g = gradient((2, 300, 200), "float32", 4, 0.1)
    check(call(g, steps=steps), g, steps=steps)


@pytest.mark.parametrize("shape", [(12, 300, 130), (40, 70, 40), (5, 300, 520)], ids=str)
def test_many_matrices(shape, form):
    g = gradient(shape, "bfloat16", 5)
    check(call(g), g)


@pytest.mark.parametrize("size", [(270, 300), (20, 90), (90, 20), (3, 7), (1, 5)])
def test_each_matrix_by_itself(size, form):
    """A matrix of another scale, a zero one and one of NaN beside the others."""
    g = gradient((5, *size), "float32", 8)
    alone = [call(g[i:i + 1].contiguous())[0] for i in range(5)]
    g2 = g.clone()
    g2[1] *= 1e6
    g2[2] = 0
    g2[3, size[0] // 2, size[1] // 2] = float("nan")
    out = call(g2)
    assert torch.equal(out[0], call(g)[0]) and torch.equal(out[4], call(g)[4])
    check(out[:2], g2[:2])
    assert bool((out[2] == 0).all()) and bool(out[3].isnan().all())
    for i in (0, 4):
        check(alone[i][None], g[i:i + 1])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("size", [(300, 140), (12, 40)])
def test_infinities_stay_in_their_matrix(size, bad):
    g = gradient((3, *size), "bfloat16", 5)
    want = call(g)
    g[1, -1, 0] = bad
    out = call(g)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    assert bool(out[1].isnan().all())


@pytest.mark.parametrize("shape", [(1024, 1, 1), (1024, 9, 5), (300, 40, 24), (1, 1, 1 << 18),
                                   (1, 1 << 18, 1), (2, 3, 100003), (1, 60001, 70), (1, 130, 30011)],
                         ids=str)
def test_extreme_shapes(shape):
    g = gradient(shape, "bfloat16", 13)
    out = call(g)
    some = sorted({0, shape[0] // 2, shape[0] - 1})
    for e in some:
        G, y = f64(g[e]), f64(out[e])
        ref = ragged.orthogonalize(G)
        err = np.sqrt(np.mean((y - ref) ** 2) / np.mean(ref ** 2))
        assert err <= 0.0025, (e, err)             # what the library states
    assert bool(out.isfinite().all())


def test_options():
    g = gradient((2, 40, 90), "float32", 3)
    check(call(g, steps=1), g, steps=1)
    check(call(g, scale=0.2), g, scale=0.2)
    check(call(g, eps=1.0), g, eps=1.0)
    cubic = (1.5, -0.5, 0.0)
    check(call(g, steps=12, coefficients=cubic), g, steps=12, coefficients=cubic)
    each = ((4.0, -6.0, 3.0), (3.0, -3.5, 1.4), (2.0, -1.5, 0.5))
    check(call(g, steps=3, coefficients=each), g, steps=3, coefficients=each)
    check(call(g, steps=3, coefficients=[list(c) for c in each]), g, steps=3, coefficients=each)


def test_plain_matrix_and_in_place():
    g = gradient((1, 96, 300), "bfloat16", 4)
    want = call(g)
    assert torch.equal(call(g[0].contiguous()), want[0])
    h = g.clone()
    assert torch.equal(call(h, out=h), want)


def test_unaligned_input():
    base = gradient((1, 1, 2 * 70 * 130 + 3), "bfloat16", 6).flatten()
    for at in (1, 2, 3):
        g = base[at:at + 2 * 70 * 130].view(2, 70, 130)
        assert torch.equal(call(g), call(g.clone()))


def test_small_and_large_values():
    g = gradient((1, 48, 64), "float32", 7)
    want = call(g)
    for s in (2.0 ** 40, 2.0 ** -10):
        a = f64(call(g * s, eps=1e-12))
        # scaled by a power of two: the same, but for eps and one rounding of 1 / norm
        assert np.abs(a - f64(want)).max() <= 2.0 ** -8 * np.abs(f64(want)).max()
    huge = torch.full((1, 48, 64), 1e30, device="cuda")
    assert bool((call(huge) == 0).all())             # the norm's square is past fp32


def test_repeats_and_graphs(form):
    g = gradient((2, 300, 400), "bfloat16", 9)
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(2, 300, 400), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty_like(g)
    moe.moe_orthogonalize(g, out, ws)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out, ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    g.mul_(-1)
    graph.replay()
    assert torch.equal(out, -first)
    assert moe.moe_sync_status() == 0


def test_singular_values_near_one():
    g = gradient((1, 300, 700), "float32", 11)
    s = np.linalg.svd(f64(call(g)[0]), compute_uv=False)
    assert s.min() > 0.3 and s.max() < 1.3
