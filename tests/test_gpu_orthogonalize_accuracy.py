"""The orthogonalised update's error over the schedules, sizes and values that the library
takes, against the fp64 oracle.

Tolerances are what the library states.  22-bit operands (shorter sides up to 128, or steps
that enlarge roundings more than five of the default triple do): 0.25% of the result's rms,
of which its rounding to bf16 is 2^-8 / sqrt(12) .. 2^-8 / sqrt(3) of a value, 0.17% on
average.  The rest is sqrt(0.25^2 - 0.17^2) = 0.18%; sums of L products are truncated by
(L / 16 + 17) 2^-24, 4e-6 for 3 x 300, which the schedules below enlarge up to 100-fold
where all singular values are equal (2.5% from the roundings of 11-bit operands alone,
2^-12 each, restated in fp64).  Single values: half a step of bf16 and five deviations of the rest, 1% of the
rms.
11-bit operands: 1.3 times the error of the oracle with the same rounding points, as in
test_gpu_orthogonalize.py, and 0.35%, between what the library states for broad spectra and
for equal singular values.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

from .test_gpu_orthogonalize import DT, call, check, f64, form, gradient  # noqa: F401

pytestmark = pytest.mark.gpu

DEFAULT = (3.4445, -4.7750, 2.0315)
# singular values below 3, the polynomials below 8.3, all within the stated range
STEEP = ((8.287, -23.596, 17.300), (4.107, -2.948, 0.545), (3.949, -2.909, 0.552),
         (3.318, -2.488, 0.510), (2.301, -1.669, 0.419))
FINE = {"steep": STEEP, "default_6": (DEFAULT,) * 6, "default_8": (DEFAULT,) * 8,
        "default_20": (DEFAULT,) * 20, "settled": (DEFAULT,) * 5 + ((2.0, -1.5, 0.5), (1.5, -0.5, 0.0))}
# 11 bits: unlike triples in every step
COARSE = {"settling": (DEFAULT, (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)),
          "falling": (DEFAULT, DEFAULT, (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)),
          "cubic_12": ((1.5, -0.5, 0.0),) * 12}


def equal(shape, seed):
    """Matrices whose singular values are all the same."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, n, k = shape
    q = [torch.linalg.qr(torch.randn(max(n, k), min(n, k), generator=g, device="cuda",
                                     dtype=torch.float64))[0] for _ in range(E)]
    return torch.stack([v if n >= k else v.T for v in q]).float().contiguous()


SPECTRA = {"broad": lambda s, seed: gradient(s, "float32", seed, 0.0), "equal": equal,
           "strong": lambda s, seed: gradient(s, "float32", seed, 0.1)}


def stated(got, g, limit=0.0025, **kw):
    for i in range(g.shape[0]):
        y, ref = f64(got[i]), ragged.orthogonalize(f64(g[i]), **kw)
        rms, err = np.sqrt(np.mean(ref ** 2)), np.abs(y - ref)
        assert np.sqrt(np.mean(err ** 2)) <= limit * rms, (i, np.sqrt(np.mean(err ** 2)) / rms)
        if limit == 0.0025:
            assert (err <= 2.0 ** -8 * np.abs(ref) + 0.01 * rms).all(), (i, err.max() / rms)


def schedule(c):
    return dict(steps=len(c), coefficients=c)


@pytest.mark.parametrize("spectrum", list(SPECTRA))
@pytest.mark.parametrize("name", list(FINE))
def test_steep_and_long_schedules(name, spectrum, form):
    for shape in ((1, 129, 300), (2, 400, 200), (1, 300, 500)):
        g = SPECTRA[spectrum](shape, sum(shape))
        stated(call(g, **schedule(FINE[name])), g, **schedule(FINE[name]))


@pytest.mark.parametrize("name", list(COARSE))
def test_unlike_triples_of_11_bits(name, form):
    for shape in ((1, 129, 300), (2, 400, 200), (1, 300, 520)):
        for spectrum in SPECTRA:
            g = SPECTRA[spectrum](shape, sum(shape))
            got = call(g, **schedule(COARSE[name]))
            check(got, g, **schedule(COARSE[name]))
            stated(got, g, 0.0035, **schedule(COARSE[name]))


@pytest.mark.parametrize("spectrum", list(SPECTRA))
def test_short_sides_at_any_number_of_steps(spectrum, form):
    for shape in ((2, 100, 260), (1, 128, 128)):
        g = SPECTRA[spectrum](shape, sum(shape))
        for name in ("steep", "default_20"):
            stated(call(g, **schedule(FINE[name])), g, **schedule(FINE[name]))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(2, 300, 200), (3, 136, 264), (7, 150, 333), (16, 333, 150)],
                         ids=str)
def test_stacks_of_22_bits(shape, dtype, form):
    """Of every type, wider and taller, in place too."""
    g = gradient(shape, dtype, 3, 0.05)
    got = call(g, **schedule(STEEP))
    stated(got, g, **schedule(STEEP))
    if dtype == "bfloat16":
        h = g.clone()
        assert torch.equal(call(h, out=h, **schedule(STEEP)), got)


@pytest.mark.parametrize("dtype", list(DT))
def test_groups_of_22_bits(dtype, form):
    """Seven matrices of 1056 x 1000: more than the workspace holds at a time with both
    parts, so four and three go through the steps together.  Nothing behind it is written."""
    g = gradient((7, 1056, 1000), dtype, 3, 0.05)
    n = moe.moe_orthogonalize_workspace_bytes(*g.shape)
    space = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    got = torch.empty_like(g, dtype=torch.bfloat16)
    moe.moe_orthogonalize(g, got, space[:n], coefficients=STEEP)
    assert moe.moe_sync_status() == 0
    assert bool((space[n:] == 0xAB).all())
    some = [0, 3, 4, 6]
    stated(got[some], g[some], **schedule(STEEP))
    if dtype == "bfloat16":
        moe.moe_orthogonalize(g, g, space[:n], coefficients=STEEP)
        assert torch.equal(g, got)


def test_stacks_of_22_bits_keep_to_themselves(form):
    """A zero matrix, one of another scale and one of NaN beside the others."""
    g = gradient((6, 150, 220), "float32", 8)
    want = call(g, **schedule(STEEP))
    h = g.clone()
    h[1] = 0
    h[2] *= 2.0 ** 20
    h[4, 17, 3] = float("nan")
    out = call(h, **schedule(STEEP))
    for i in (0, 3, 5):
        assert torch.equal(out[i], want[i])
    stated(out[2:3], h[2:3], **schedule(STEEP))
    assert bool((out[1] == 0).all()) and bool(out[4].isnan().all())


def test_graph_of_22_bits():
    g = gradient((5, 200, 300), "bfloat16", 9)
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(*g.shape), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(g)
    moe.moe_orthogonalize(g, out, ws, coefficients=STEEP)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out, ws, coefficients=STEEP)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    assert moe.moe_sync_status() == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape", [(1, 48, 64), (2, 140, 300), (1, 3, 7), (1, 60, 33)], ids=str)
def test_sums_of_squares_past_fp32(shape, dtype):
    """Each square is below fp32's largest value, a sum of 32 of them is not."""
    u = torch.rand(shape, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    g = ((2 * u - 1) * 1.8e19).to(DT[dtype])
    check(call(g), g)


@pytest.mark.parametrize("shape", [(1, 48, 64), (1, 200, 300)], ids=str)
@pytest.mark.parametrize("below", [1e-2, 1e-4])
def test_norms_below_eps(below, shape):
    """X is g / eps, and its smallest steps (2^-24 / 4096 a value, in fp16's subnormals) are
    2^-36: within the stated error while its values are well above that."""
    g = gradient(shape, "float32", 6, 0.0)
    g *= below / g.norm()
    stated(call(g, eps=1.0), g, eps=1.0)
