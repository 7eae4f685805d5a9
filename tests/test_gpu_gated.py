"""The gated expert block and its gradient against the fp64 oracle.

Tolerances, derived from the arithmetic.  A sum of n products of magnitudes' sum m is
off by at most d = (n / 16 + 17) 2^-23 m (the tensor core adds 16 products at a time and
may truncate), and a stored value by half a step of its type besides.
* Activation in fp32: __expf(v) is within 2 + 1.2 |v| steps, the division within 2,
  and four products of half a step each: relative to s = sigmoid(alpha g) and so to z at
  most r = (10 + 1.2 |alpha g|) 2^-23; below e^-87 s is 0, off by less than 2^-118.
* z = act(g) (u + beta): |act'| <= 1.1, so sums off by dg and du move it by at most
  1.1 dg |u' + beta| + |act| du + 1.1 dg du.
* dh from exact h: dz's d times the derivative, and the derivative's own error.  That by g
  is s + (alpha g s)(1 - s), whose terms cancel and whose 1 - s is off by 2^-22 s:
  at most (s + |alpha g| s)(12 + 1.2 |alpha g|) 2^-23.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

pytestmark = pytest.mark.gpu
DT = {"bfloat16": torch.bfloat16, "float16": torch.float16}
CANARY = 7.0
RECIPES = {"silu": (1.0, 0.0, 0.0), "clamped": (1.702, 1.0, 2.0), "shifted": (0.5, -0.25, -1.0)}


@pytest.fixture(params=["auto", "single", "pairs"])
def form(request):
    moe.moe_debug_set_bf16_gemm_form(request.param)
    yield request.param
    moe.moe_debug_set_bf16_gemm_form("auto")


SEGMENTS = {
    "one_row": [1],
    "empties": [0, 3, 0, 0, 1, 130, 0],
    "tile_ends": [16, 32, 64, 127, 128, 129],
    "long": [700, 5, 256],
    "none": [0, 0, 0],
}


def f64(t):
    return t.double().cpu().numpy()


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


def check(got, ref, extra, dtype, what):
    fi = torch.finfo(dtype)
    got = f64(got)
    tol = fi.eps / 2 * 1.001 * np.abs(ref) + fi.tiny * fi.eps + extra
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at "
                           f"{np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(got - ref) / tol):.2f}")


def sum_error(n, mag):
    return (n / 16 + 17) * 2.0 ** -23 * mag


def clamped(h, limit):
    g, u = np.split(h, 2, axis=1)
    return (np.minimum(g, limit), np.clip(u, -limit, limit)) if limit > 0 else (g, u)


def parts(h, recipe):
    """act, sigmoid, clamped g and u + beta, and alpha |g|."""
    alpha, beta, limit = recipe
    g, u = clamped(h, limit)
    s = 1 / (1 + np.exp(-alpha * g))
    return g * s, s, g, u + beta, alpha * np.abs(g)


def z_error(h, recipe, dh):
    act, _, g, ub, ag = parts(h, recipe)
    dg, du = np.split(dh, 2, axis=1)
    return ((10 + 1.2 * ag) * 2.0 ** -23 * np.abs(act * ub) + 2.0 ** -118 * np.abs(g * ub)
            + 1.1 * dg * np.abs(ub) + np.abs(act) * du + 1.1 * dg * du)


def offsets_of(counts, lead=0):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64) + lead


def buffer(rows, ld, dtype):
    return torch.full((rows, ld), CANARY, dtype=DT[dtype], device="cuda")


def workspace(p):
    return torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")


def run_forward(counts, inter, hidden, dtype, recipe="silu", lead=0, tail=0, ldx=0, ldh=0, ldz=0,
                bias=False, keep=True, seed=0):
    off = offsets_of(counts, lead)
    rows, E, n = int(off[-1]) + tail, len(counts), 2 * inter
    p = moe.Ragged(R=rows, N=n, K=hidden, E=E, dtype=dtype, ldx=ldx, ldy=ldh)
    x = randn((rows, ldx or hidden), dtype, seed)[:, :hidden]
    w = randn((E, n, hidden), dtype, seed + 1, 1.5 / hidden ** 0.5)
    b = randn((E, n), dtype, seed + 2) if bias else None
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    z, h = buffer(rows, ldz or inter, dtype), buffer(rows, ldh or n, dtype)
    alpha, beta, limit = RECIPES[recipe]
    moe.ragged_gated(p, x, w, o, z[:, :inter], workspace(p), h=h[:, :n] if keep else None, bias=b,
                     alpha=alpha, beta=beta, limit=limit)
    assert moe.moe_sync_status() == 0
    live = np.zeros(rows, bool)
    live[off[0]:off[-1]] = True
    X, W = f64(x), f64(w)
    B = None if b is None else f64(b)
    ref = ragged.forward(X, W, off, B)
    d = sum_error(hidden + 16, ragged.forward(abs(X), abs(W), off, None if B is None else abs(B)))
    r = RECIPES[recipe]
    check(z[live][:, :inter], ragged.gated(ref, *r)[live], z_error(ref, r, d)[live], DT[dtype], "z")
    if keep:
        check(h[live][:, :n], ref[live], d[live], DT[dtype], "h")
    else:
        assert bool((h == CANARY).all())
    assert bool((z[~live] == CANARY).all()) and bool((h[~live] == CANARY).all())
    assert bool((z[:, inter:] == CANARY).all()) and bool((h[:, n:] == CANARY).all())


def run_grad(counts, inter, hidden, dtype, recipe="silu", lead=0, tail=0, ldy=0, ldh=0, lddh=0,
             ldz=0, again=True, in_place=False, seed=0, h=None):
    off = offsets_of(counts, lead)
    rows, E, n = int(off[-1]) + tail, len(counts), 2 * inter
    p = moe.Ragged(R=rows, N=hidden, K=inter, E=E, dtype=dtype, ldx=ldz, ldy=ldy)
    dy = randn((rows, ldy or hidden), dtype, seed)[:, :hidden]
    w = randn((E, hidden, inter), dtype, seed + 1, 1 / hidden ** 0.5)
    if h is None:
        h = randn((rows, ldh or n), dtype, seed + 2, 2.0)
    H = f64(h[:, :n])
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    dh = h if in_place else buffer(rows, lddh or n, dtype)
    before = dh.clone()
    z = buffer(rows, ldz or inter, dtype)
    alpha, beta, limit = RECIPES[recipe]
    moe.ragged_gated_dgrad(p, dy, w, h[:, :n], o, dh[:, :n], workspace(p),
                           z=z[:, :inter] if again else None, alpha=alpha, beta=beta, limit=limit)
    assert moe.moe_sync_status() == 0
    live = np.zeros(rows, bool)
    live[off[0]:off[-1]] = True
    D, W = f64(dy), f64(w)
    dz = ragged.dgrad(D, W, off)
    d = sum_error(hidden, ragged.dgrad(abs(D), abs(W), off))
    r = RECIPES[recipe]
    act, s, g, ub, ag = parts(H, r)
    slope = s * (1 + alpha * g * (1 - s))
    off_slope = (s + ag * s) * (12 + 1.2 * ag) * 2.0 ** -23
    tol_g = np.abs(ub * slope) * d + np.abs(dz * ub) * off_slope + 2.0 ** -118 * np.abs(dz * ub * g)
    tol_u = (np.abs(act) * d + (10 + 1.2 * ag) * 2.0 ** -23 * np.abs(dz * act)
             + 2.0 ** -118 * np.abs(dz * g))
    ref = ragged.gated_grad(dz, H, *r)
    check(dh[live][:, :n], ref[live], np.concatenate([tol_g, tol_u], 1)[live] * 1.001, DT[dtype],
          "dh")
    if again:
        zero = np.zeros_like(H)
        check(z[live][:, :inter], ragged.gated(H, *r)[live], z_error(H, r, zero)[live], DT[dtype],
              "z")
    else:
        assert bool((z == CANARY).all())
    keep = torch.tensor(~live, device="cuda")
    assert torch.equal(dh[keep], before[keep]) and torch.equal(dh[:, n:], before[:, n:])
    assert bool((z[keep] == CANARY).all()) and bool((z[:, inter:] == CANARY).all())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("name", list(SEGMENTS))
def test_segments(name, dtype, form):
    run_forward(SEGMENTS[name], 136, 200, dtype)
    run_grad(SEGMENTS[name], 136, 200, dtype)


@pytest.mark.parametrize("inter, hidden", [(8, 8), (8, 1032), (1032, 8), (64, 64), (72, 136),
                                           (264, 520), (128, 4104), (1032, 128)])
def test_odd_sizes(inter, hidden, form):
    run_forward([5, 0, 200, 33], inter, hidden, "bfloat16", seed=5)
    run_grad([5, 0, 200, 33], inter, hidden, "bfloat16", seed=5)


@pytest.mark.parametrize("recipe", list(RECIPES))
@pytest.mark.parametrize("dtype", list(DT))
def test_activations(recipe, dtype, form):
    run_forward([40, 300], 72, 136, dtype, recipe=recipe, bias=True)
    run_grad([40, 300], 72, 136, dtype, recipe=recipe)


@pytest.mark.parametrize("bias", [False, True])
def test_strides_lead_and_tail_rows(bias, form):
    run_forward([50, 0, 281], 72, 136, "float16", "clamped", lead=3, tail=70, ldx=144, ldh=160,
                ldz=88, bias=bias)
    run_grad([50, 0, 281], 72, 136, "float16", "clamped", lead=3, tail=70, ldy=144, ldh=160,
             lddh=152, ldz=88)


def test_without_h_and_without_z(form):
    run_forward([50, 0, 281], 72, 136, "bfloat16", keep=False)
    run_grad([50, 0, 281], 72, 136, "bfloat16", again=False)


def test_gradient_in_place(form):
    run_grad([50, 0, 281], 136, 264, "bfloat16", tail=5, ldh=280, in_place=True)


@pytest.mark.parametrize("rows", [1, 2, 3, 17, 33, 100])
def test_sliced_reductions(rows):
    """One expert, few rows, a long reduction: the clusters' form."""
    run_forward([rows], 264, 4104, "bfloat16", "clamped", bias=True, seed=rows)
    run_grad([rows], 264, 4104, "bfloat16", "clamped", seed=rows)


def test_many_experts():
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 7, 300).tolist()
    run_forward(counts, 40, 72, "bfloat16")
    run_grad(counts, 40, 72, "bfloat16")


@pytest.mark.parametrize("counts, inter, hidden", [
    ([0] * 1000 + [1] + [0] * 23, 8, 8), ([1] * 1024, 16, 24), ([3000, 0, 2000], 8, 24),
    ([5], 2056, 8), ([2], 8, 8200)])
def test_extreme_shapes(counts, inter, hidden, form):
    run_forward(counts, inter, hidden, "bfloat16", "clamped", bias=True)
    run_grad(counts, inter, hidden, "bfloat16", "clamped")


def test_the_limit_itself_passes_gradients(form):
    """h of exactly the limit, just beyond it, and of large values of both signs."""
    v = torch.tensor([2.0, -2.0, 2.015625, -2.015625, 0.0, 100.0, -100.0, 1.0], device="cuda")
    h = torch.cat([v.repeat(48, 9), v.flip(0).repeat(48, 9)], 1).to(torch.bfloat16).contiguous()
    run_grad([48], 72, 136, "bfloat16", "clamped", h=h)


def test_gradient_against_differences():
    """Loss sum(dy * W2 z(h)): central differences of the kernel's own forward chain,
    in directions of one element of h each."""
    rows, inter, hidden = 3, 8, 16
    p = moe.Ragged(R=rows, N=hidden, K=inter, E=1, dtype="float16")
    dy, w = randn((rows, hidden), "float16", 1), randn((1, hidden, inter), "float16", 2)
    h = randn((rows, 2 * inter), "float16", 3)
    o = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    dh = torch.empty_like(h)
    moe.ragged_gated_dgrad(p, dy, w, h, o, dh, workspace(p), alpha=1.3, beta=0.5, limit=3.0)
    H, D, W = f64(h), f64(dy), f64(w)

    def loss(hh):
        return (D * (ragged.gated(hh, 1.3, 0.5, 3.0) @ W[0].T)).sum()

    step = 1e-5
    for i in range(rows):
        for j in range(2 * inter):
            e = np.zeros_like(H)
            e[i, j] = step
            want = (loss(H + e) - loss(H - e)) / (2 * step)
            # differences: third derivatives times step^2, and 1e-16 |loss| / step
            assert abs(f64(dh)[i, j] - want) <= 2.0 ** -11 * abs(want) + 1e-5


def test_nan_and_inf_stay_in_their_rows(form):
    """Rows of NaN and infinities beside a segment and of another expert change nothing
    of the others'."""
    counts, inter, hidden = [40, 90], 72, 136
    off = torch.tensor([2, 42, 132], dtype=torch.int32, device="cuda")
    p = moe.Ragged(R=140, N=2 * inter, K=hidden, E=2)
    q = moe.Ragged(R=140, N=hidden, K=inter, E=2)
    x, dy = randn((140, hidden), "bfloat16", 1), randn((140, hidden), "bfloat16", 2)
    w13, w2 = randn((2, 2 * inter, hidden), "bfloat16", 3, 0.1), randn((2, hidden, inter), "bfloat16", 4)

    def run(x, dy):
        z, h = buffer(140, inter, "bfloat16"), buffer(140, 2 * inter, "bfloat16")
        dh = torch.zeros_like(h)
        moe.ragged_gated(p, x, w13, off, z, workspace(p), h=h, limit=7.0)
        moe.ragged_gated_dgrad(q, dy, w2, h, off, dh, workspace(q), limit=7.0)
        return z, h, dh

    clean = run(x, dy)
    x2, dy2 = x.clone(), dy.clone()
    for t in (x2, dy2):
        t[:2], t[41], t[132:] = float("nan"), float("nan"), float("inf")
    dirty = run(x2, dy2)
    assert moe.moe_sync_status() == 0
    keep = torch.ones(140, dtype=torch.bool, device="cuda")
    keep[41] = False
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])
    for t in dirty:
        assert bool(t[41].isnan().all())


def test_bad_offsets_are_reported():
    p = moe.Ragged(R=64, N=144, K=136, E=2)
    q = moe.Ragged(R=64, N=136, K=72, E=2)
    x, w13, w2 = (randn(s, "bfloat16", 1) for s in ((64, 136), (2, 144, 136), (2, 136, 72)))
    h = randn((64, 144), "bfloat16", 2)
    z, dh = buffer(64, 72, "bfloat16"), buffer(64, 144, "bfloat16")
    for bad in ([0, 40, 30], [0, 40, 65], [-1, 3, 64]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        moe.ragged_gated(p, x, w13, off, z, workspace(p))
        assert moe.moe_sync_status() == 6
        moe.ragged_gated_dgrad(q, x, w2, h, off, dh, workspace(q))
        assert moe.moe_sync_status() == 6


@pytest.mark.parametrize("rows", [2, 700])
def test_forms_and_repeats_agree(rows):
    """Twice the same call gives the same bits; the forms differ by their sums' order at
    most (checked against the oracle above)."""
    inter, hidden = 264, 1032
    p = moe.Ragged(R=rows, N=2 * inter, K=hidden, E=1)
    x, w = randn((rows, hidden), "bfloat16", 1), randn((1, 2 * inter, hidden), "bfloat16", 2, 0.05)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out = []
    for _ in range(3):
        z, h = buffer(rows, inter, "bfloat16"), buffer(rows, 2 * inter, "bfloat16")
        moe.ragged_gated(p, x, w, off, z, workspace(p), h=h)
        out.append((z, h))
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(out[0], o))


def test_graph_replay_reads_the_offsets_of_the_moment():
    inter, hidden, rows = 72, 136, 96
    p = moe.Ragged(R=rows, N=2 * inter, K=hidden, E=2)
    q = moe.Ragged(R=rows, N=hidden, K=inter, E=2)
    x, dy = randn((rows, hidden), "bfloat16", 1), randn((rows, hidden), "bfloat16", 2)
    w13, w2 = randn((2, 2 * inter, hidden), "bfloat16", 3, 0.1), randn((2, hidden, inter), "bfloat16", 4)
    off = torch.tensor([0, 96, 96], dtype=torch.int32, device="cuda")
    wp, wq = workspace(p), workspace(q)

    def both(z, h, dh):
        moe.ragged_gated(p, x, w13, off, z, wp, h=h)
        moe.ragged_gated_dgrad(q, dy, w2, h, off, dh, wq)

    def buffers():
        return (torch.zeros(rows, inter, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(rows, 2 * inter, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(rows, 2 * inter, dtype=torch.bfloat16, device="cuda"))

    kept = buffers()
    both(*kept)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(*kept)
    for o in ([0, 30, 96], [5, 5, 40], [0, 0, 0]):
        off.copy_(torch.tensor(o, dtype=torch.int32))
        for t in kept:
            t.zero_()
        graph.replay()
        want = buffers()
        both(*want)
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
    assert moe.moe_sync_status() == 0
