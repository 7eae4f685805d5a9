"""Ragged products with several tiles for each CTA or SM pair in turn, and the
default choice of form.

Accumulators, rings and scale slots pass from tile to tile here: a GB300 holds
152 CTAs or 76 pairs, and each product below has several hundred tiles in every
form.  References are in fp64 on the GPU; the tolerances are those that
test_gpu_ragged.py and test_gpu_mxfp4_ops.py derive (half a step of the output's
type; one fp32 step of the magnitudes' sum for each instruction's addition and
for each product aligned in one)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe

from .test_gpu_mxfp4_ops import product
from .test_gpu_ragged import SEGMENTS, run_all

pytestmark = pytest.mark.gpu
FORMS = ["auto", "single", "pairs", "pairs_double"]


@pytest.fixture
def form(request):
    moe.moe_debug_set_bf16_gemm_form(request.param)
    yield request.param
    moe.moe_debug_set_bf16_gemm_form("auto")


def every_form(f):
    return pytest.mark.parametrize("form", FORMS, indirect=True)(f)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets(counts):
    o = np.concatenate([[0], np.cumsum(counts)])
    return o, torch.tensor(o, dtype=torch.int32, device="cuda")


def workspace(p):
    """Filled with NaN: no call may rely on what it finds there."""
    return torch.full((moe.moe_ragged_workspace_bytes(p),), 255, dtype=torch.uint8, device="cuda")


def check(got, ref, mag, terms, what):
    """terms: additions of the magnitudes' sum mag, in fp32 steps."""
    fi = torch.finfo(got.dtype)
    tol = fi.eps / 2 * ref.abs() + fi.tiny * fi.eps + terms * 2.0 ** -23 * mag
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                                 f"{bad.nonzero()[0].tolist()}, worst {float((err / tol).max()):.2f}")


# ------------------------------------------------------------ 16-bit operands
@every_form
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forward_and_dgrad_of_many_tiles(form, dtype):
    """110 experts: 440 double tiles forward (the last of a row without its
    second half) and 330 dgrad (the last second half 8 columns wide)."""
    n, k = 1544, 1288
    counts = [(37 * e) % 90 + 1 if e % 9 else 300 for e in range(110)]
    o, od = offsets(counts)
    rows = int(o[-1])
    p = moe.Ragged(R=rows, N=n, K=k, E=len(counts), dtype=str(dtype)[6:])
    g = generator(1)
    x, dy = (torch.randn(rows, c, generator=g, device="cuda").to(dtype) for c in (k, n))
    w = torch.randn(len(counts), n, k, generator=g, device="cuda").mul_(0.1).to(dtype)
    b = torch.randn(len(counts), n, generator=g, device="cuda").to(dtype)
    y, dx, ws = torch.empty_like(dy), torch.empty_like(x), workspace(p)
    moe.ragged_gemm(p, x, w, od, y, ws, bias=b)
    moe.ragged_gemm_dgrad(p, dy, w, od, dx, ws)
    assert moe.moe_sync_status() == 0
    for e in range(len(counts)):
        at = slice(int(o[e]), int(o[e + 1]))
        X, D, W, B = x[at].double(), dy[at].double(), w[e].double(), b[e].double()
        check(y[at], X @ W.T + B, X.abs() @ W.abs().T + B.abs(), (k + 16) / 16 + 17, f"y of {e}")
        check(dx[at], D @ W, D.abs() @ W.abs(), n / 16 + 17, f"dx of {e}")


@every_form
def test_same_result_every_time(form):
    """Sums are joined in a fixed order: outputs repeat bit for bit, beside other
    work on the GPU, whatever the workspace held."""
    n, k = 1032, 2056
    counts = [700, 5, 0, 256, 33, 129]
    o, od = offsets(counts)
    rows = int(o[-1])
    p = moe.Ragged(R=rows, N=n, K=k, E=len(counts))
    g = generator(2)
    x, dy = (torch.randn(rows, c, generator=g, device="cuda").bfloat16() for c in (k, n))
    w = torch.randn(len(counts), n, k, generator=g, device="cuda").bfloat16()
    first = None
    noise = torch.randn(2048, 2048, device="cuda")
    for i in range(6):
        y, dx = torch.empty_like(dy), torch.empty_like(x)
        dw, ws = torch.empty_like(w), workspace(p)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        if i % 2:
            with torch.cuda.stream(side):
                noise @ noise
        moe.ragged_gemm(p, x, w, od, y, ws)
        moe.ragged_gemm_dgrad(p, dy, w, od, dx, ws)
        moe.ragged_gemm_wgrad(p, dy, x, od, dw, ws)
        torch.cuda.synchronize()
        first = first or [y, dx, dw]
        assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw)))
    assert moe.moe_sync_status() == 0


def test_one_workspace_for_all_batches():
    """A workspace for the largest batch serves the smaller ones, which take more
    slices and more of it."""
    n = k = 1032
    g = generator(3)
    w = torch.randint(-2, 3, (1, n, k), generator=g, device="cuda").bfloat16()
    ws = workspace(moe.Ragged(R=2000, N=n, K=k, E=1))
    for rows in (2000, 1000, 256, 100, 1):
        p = moe.Ragged(R=rows, N=n, K=k, E=1)
        x, dy = (torch.randint(-2, 3, (rows, c), generator=g, device="cuda").bfloat16()
                 for c in (k, n))
        o = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        y, dx = torch.empty_like(dy), torch.empty_like(x)
        dw = torch.empty(1, n, k, device="cuda")
        moe.ragged_gemm(p, x, w, o, y, ws)
        moe.ragged_gemm_dgrad(p, dy, w, o, dx, ws)
        moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws)
        assert moe.moe_sync_status() == 0
        # small integers: every partial sum is exact in fp32
        X, D, W = x.double(), dy.double(), w[0].double()
        assert torch.equal(y, (X @ W.T).bfloat16())
        assert torch.equal(dx, (D @ W).bfloat16())
        assert torch.equal(dw[0], (D.T @ X).float())


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("name", list(SEGMENTS))
def test_segments_in_the_default_form(name, dtype):
    run_all(SEGMENTS[name], 264, 200, dtype)


@pytest.mark.parametrize("counts, n, k", [([5, 0, 200, 33], 8, 1032), ([1], 2056, 4104),
                                          ([300, 0, 7], 2056, 4104), ([2500, 5], 136, 264),
                                          ([130] * 40, 520, 264), ([600] * 8, 1032, 520),
                                          ([700, 1, 900], 2056, 1032)])
def test_sizes_in_the_default_form(counts, n, k):
    run_all(counts, n, k, "bfloat16", lead=1, tail=2, bias=True, dw_type=torch.float32)


# ------------------------------------------------------------- 4-bit operands
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def values(codes, scales):
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device="cuda")
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scales.double() - 127)[..., None]).flatten(-2)


@pytest.mark.parametrize("form", FORMS[:3], indirect=True)
@pytest.mark.parametrize("counts", [[1 + 7 * e % 39 for e in range(64)],
                                    [300 - 11 * e for e in range(12)] + [0, 513]])
def test_product_of_many_tiles(form, counts):
    """Tiles of up to 128 tokens in two accumulators in turn (64 experts: 2048 tiles
    on one SM, 1024 on pairs) and of up to 256 in the one (12 experts), over a
    reduction of four and a half steps."""
    n, k = 4096, 1152
    o, od = offsets(counts)
    rows, E = int(o[-1]), len(counts)
    g = generator(4)

    def u8(shape, a, b):
        return torch.randint(a, b, shape, dtype=torch.uint8, generator=g, device="cuda")

    xc, xs = u8((rows, k // 2), 0, 256), u8((rows, k // 32), 118, 130)
    wc, wsc = u8((E, n, k // 2), 0, 256), u8((E, n, k // 32), 112, 124)
    packed = torch.empty_like(wsc)
    moe.moe_mxfp4_pack_scales(wsc, packed)
    p = moe.Ragged(R=rows, N=n, K=k, E=E)
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    ws = workspace(p)
    for _ in range(2):
        y.fill_(7.0)
        moe.ragged_gemm_mxfp4(p, xc, xs, wc, packed, od, y, ws)
        assert moe.moe_sync_status() == 0
        for e in range(E):
            at = slice(int(o[e]), int(o[e + 1]))
            X, W = values(xc[at], xs[at]), values(wc[e], wsc[e])
            check(y[at], X @ W.T, X.abs() @ W.abs().T, k / 64 + 65, f"y of {e}")


@pytest.mark.parametrize("counts, n, k", [([1], 128, 128), ([0, 3, 0, 1, 130, 0], 256, 384),
                                          ([16, 32, 64, 127, 128, 129], 384, 640),
                                          ([700, 5, 256], 1152, 1152), ([200], 256, 8576),
                                          ([300] * 9, 512, 2048), ([20] * 60, 256, 512)])
def test_product_in_the_default_form(counts, n, k):
    product(counts, n, k, lead=1, tail=2, lo=122, hi=126)
