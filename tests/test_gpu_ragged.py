"""Ragged grouped products (forward, dgrad, wgrad) against the fp64 oracle.

Tolerance of one output value v = sum of n products p_i (|p| their magnitudes'
sum), derived from the arithmetic:
* rounding to the output's type: half a step, eps / 2 * |v| (plus the type's
  smallest step, for values below its normal range);
* accumulation: the tensor core adds 16 products at a time to an fp32
  accumulator and may truncate: at most one fp32 step (2^-23) of the partial
  sum each time, and one for each product aligned to the largest in a step; all
  partial sums are at most |p|: (n / 16 + 17) 2^-23 |p|.
Integer inputs small enough for every partial sum to be exact have to match
exactly.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

pytestmark = pytest.mark.gpu
DT = {"bfloat16": torch.bfloat16, "float16": torch.float16}


@pytest.fixture(autouse=True, params=["single", "pairs", "pairs_double"])
def form(request):
    """Every test in every form of the kernels."""
    moe.moe_debug_set_bf16_gemm_form(request.param)
    yield
    moe.moe_debug_set_bf16_gemm_form("auto")


# rows of each expert; offsets may leave rows in front (lead) and behind (tail)
SEGMENTS = {
    "one_row": [1],
    "empties": [0, 3, 0, 0, 1, 130, 0],
    "tile_ends": [16, 32, 64, 127, 128, 129],
    "long": [700, 5, 256],
    "even": [257, 513],
    "none": [0, 0, 0],
}


def offsets_of(counts, lead=0):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64) + lead


def f64(t):
    return t.double().cpu().numpy()


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


def check(got, ref, mag, n_terms, dtype, what):
    fi = torch.finfo(dtype)
    got = f64(got)
    tol = (fi.eps / 2 * np.abs(ref) + fi.tiny * fi.eps
           + (np.asarray(n_terms) / 16 + 17) * 2.0 ** -23 * mag)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at "
                           f"{np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(got - ref) / tol):.2f}")


def run_all(counts, n, k, dtype, lead=0, tail=0, ldx=0, ldy=0, bias=False, dw_type=None, seed=0):
    off = offsets_of(counts, lead)
    rows, E = int(off[-1]) + tail, len(counts)
    p = moe.Ragged(R=rows, N=n, K=k, E=E, dtype=dtype, ldx=ldx, ldy=ldy)
    x = randn((rows, ldx or k), dtype, seed)[:, :k]
    dy = randn((rows, ldy or n), dtype, seed + 1)[:, :n]
    w = randn((E, n, k), dtype, seed + 2, 0.1)
    b = randn((E, n), dtype, seed + 3) if bias else None
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    canary = 7.0
    y = torch.full((rows, ldy or n), canary, dtype=DT[dtype], device="cuda")
    dx = torch.full((rows, ldx or k), canary, dtype=DT[dtype], device="cuda")
    dw = torch.full((E, n, k), canary, dtype=dw_type or DT[dtype], device="cuda")
    moe.ragged_gemm(p, x, w, o, y[:, :n], ws, bias=b)
    moe.ragged_gemm_dgrad(p, dy, w, o, dx[:, :k], ws)
    moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws)
    assert moe.moe_sync_status() == 0
    live = np.zeros(rows, bool)
    live[off[0]:off[-1]] = True
    X, D, W = f64(x), f64(dy), f64(w)
    B = None if b is None else f64(b)
    ref = ragged.forward(X, W, off, B)
    mag = ragged.forward(abs(X), abs(W), off, None if B is None else abs(B))
    check(y[live][:, :n], ref[live], mag[live], k + 16, DT[dtype], "y")
    check(dx[live][:, :k], ragged.dgrad(D, W, off)[live], ragged.dgrad(abs(D), abs(W), off)[live],
          n, DT[dtype], "dx")
    check(dw, ragged.wgrad(D, X, off), ragged.wgrad(abs(D), abs(X), off),
          np.asarray(counts)[:, None, None], dw.dtype, "dw")
    # rows of no expert and the columns behind a strided row keep what they held
    assert bool((y[~live] == canary).all()) and bool((dx[~live] == canary).all())
    assert bool((y[:, n:] == canary).all()) and bool((dx[:, k:] == canary).all())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("name", list(SEGMENTS))
def test_segments(name, dtype):
    run_all(SEGMENTS[name], 264, 200, dtype)


@pytest.mark.parametrize("n, k", [(192, 320), (320, 192), (8, 8), (8, 1032), (1032, 8), (128, 64), (136, 72), (520, 264),
                                  (256, 4104), (2056, 128)])
def test_odd_sizes(n, k):
    run_all([5, 0, 200, 33], n, k, "bfloat16", seed=5)


@pytest.mark.parametrize("rows", [1, 17, 31, 33, 64, 65, 128, 129, 255, 256, 257, 1000])
def test_one_expert(rows):
    run_all([rows], 136, 136, "float16", seed=rows)


def test_rows_of_no_expert_and_strides():
    run_all([40, 0, 90], 136, 72, "bfloat16", lead=3, tail=9, ldx=80, ldy=152)


def test_bias():
    run_all([40, 0, 290], 264, 72, "float16", bias=True)


@pytest.mark.parametrize("rows", [1, 31, 300])
def test_long_reduction_of_few_tiles(rows):
    """Few tiles, long reductions in both directions: slices that are joined."""
    run_all([rows, 0, 7], 2056, 4104, "bfloat16", bias=True, ldx=4112, ldy=2064, lead=1, tail=2)
    run_all([rows], 1032, 72, "float16", bias=True)


@pytest.mark.parametrize("counts", [[2100], [5, 0, 2500], [4096, 1, 64, 1500]])
@pytest.mark.parametrize("dw_type", [None, torch.float32])
def test_long_segments_of_few_weights(counts, dw_type):
    """wgrad of few tiles: a long segment's rows in slices that are joined."""
    run_all(counts, 136, 264, "bfloat16", lead=1, dw_type=dw_type)


def test_many_experts():
    rng = np.random.default_rng(3)
    run_all(list(rng.integers(0, 6, 1024)), 72, 40, "bfloat16")


@pytest.mark.parametrize("dtype", list(DT))
def test_wgrad_fp32_output(dtype):
    run_all([5, 0, 200, 700], 136, 264, dtype, dw_type=torch.float32)


@pytest.mark.parametrize("counts", [[20, 0, 300], [2100, 0, 1500]])
@pytest.mark.parametrize("dw_type", [None, torch.float32])
def test_wgrad_accumulates(dw_type, counts):
    n, k, rows = 136, 72, sum(counts)
    off = offsets_of(counts)
    p = moe.Ragged(R=rows, N=n, K=k, E=3)
    x, dy = randn((rows, k), "bfloat16", 1), randn((rows, n), "bfloat16", 2)
    start = randn((3, n, k), "bfloat16", 3, 4.0).to(dw_type or torch.bfloat16)
    dw = start.clone()
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws, accumulate=True)
    assert moe.moe_sync_status() == 0
    ref = f64(start) + ragged.wgrad(f64(dy), f64(x), off)
    mag = abs(f64(start)) + ragged.wgrad(abs(f64(dy)), abs(f64(x)), off)
    check(dw, ref, mag, max(counts) + 16, dw.dtype, "dw")
    assert bool((dw[1] == start[1]).all())


@pytest.mark.parametrize("n, k, experts", [(296, 12536, 29), (1984, 14104, 4), (1040, 5840, 60)])
@pytest.mark.parametrize("dw_type", [None, torch.float32])
def test_wgrad_tiles_past_the_last_row(n, k, experts, dw_type):
    """Many short tiles a CTA in turn, some with rows past N, at HBM's pace: what
    is not stored of one must not touch the stores of the one before that are still
    on their way.  Small integers: every value is exact."""
    counts = [(5 * e + 1) % 31 for e in range(experts)]
    off = offsets_of(counts)
    rows = int(off[-1])
    g = torch.Generator(device="cuda").manual_seed(n)
    x, dy = (torch.randint(-4, 5, (rows, c), generator=g, device="cuda").bfloat16() for c in (k, n))
    p = moe.Ragged(R=rows, N=n, K=k, E=experts)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    dw = torch.empty((experts, n, k), dtype=dw_type or torch.bfloat16, device="cuda")
    for _ in range(3):
        dw.fill_(7.0)
        moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws)
        assert moe.moe_sync_status() == 0
        for e in range(experts):
            ref = dy[off[e]:off[e + 1]].double().T @ x[off[e]:off[e + 1]].double()
            assert bool((dw[e] == ref.to(dw.dtype)).all()), f"expert {e}"


def test_many_lone_calls_end():
    """Calls that find the GPU idle, one after another: none may wait for a signal
    that was lost at the end of the one before."""
    p = moe.Ragged(R=24, N=1080, K=456, E=40)
    off = [min(24, e) for e in range(41)]
    x, dy, w = (torch.ones(s, dtype=torch.bfloat16, device="cuda")
                for s in ((24, 456), (24, 1080), (40, 1080, 456)))
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)
    for _ in range(300):
        y.fill_(0.0)
        moe.ragged_gemm(p, x, w, o, y, ws)
        torch.cuda.synchronize()
        moe.ragged_gemm_dgrad(p, dy, w, o, dx, ws)
        moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws)
        torch.cuda.synchronize()
    assert moe.moe_sync_status() == 0
    assert bool((y == 456).all()) and bool((dx == 1080).all()) and bool((dw[:24] == 1).all())


def test_other_rows_cannot_leak():
    """Infinities and NaN in another expert's rows, in rows of no expert and in
    the columns behind a strided row stay there."""
    counts, n, k = [33, 70, 1], 136, 72
    off = offsets_of(counts, 2)
    rows = int(off[-1]) + 5
    p = moe.Ragged(R=rows, N=n, K=k, E=3, ldx=80, ldy=144)
    x, dy = randn((rows, 80), "bfloat16", 1), randn((rows, 144), "bfloat16", 2)
    w = randn((3, n, k), "bfloat16", 3)
    for t, c in ((x, k), (dy, n)):
        t[:2], t[-5:], t[:, c:] = float("nan"), float("inf"), float("nan")
        t[off[1]:off[2]] = float("nan")
    w[1] = float("inf")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y, dx = torch.zeros_like(dy), torch.zeros_like(x)
    dw = torch.zeros(3, n, k, dtype=torch.bfloat16, device="cuda")
    moe.ragged_gemm(p, x[:, :k], w, o, y[:, :n], ws)
    moe.ragged_gemm_dgrad(p, dy[:, :n], w, o, dx[:, :k], ws)
    moe.ragged_gemm_wgrad(p, dy[:, :n], x[:, :k], o, dw, ws)
    assert moe.moe_sync_status() == 0
    for e in (0, 2):
        at = slice(off[e], off[e + 1])
        X, D, W = f64(x[at, :k]), f64(dy[at, :n]), f64(w[e:e + 1])
        one = [0, counts[e]]
        check(y[at, :n], ragged.forward(X, W, one), ragged.forward(abs(X), abs(W), one), k,
              torch.bfloat16, "y")
        check(dx[at, :k], ragged.dgrad(D, W, one), ragged.dgrad(abs(D), abs(W), one), n,
              torch.bfloat16, "dx")
        check(dw[e], ragged.wgrad(D, X, one)[0], ragged.wgrad(abs(D), abs(X), one)[0], counts[e],
              torch.bfloat16, "dw")
    assert bool(dw[1].isnan().all()) and bool(y[off[1]:off[2], :n].isnan().all())


def test_gradients_match_differences():
    """Integer inputs: every sum is exact, so the difference of the forward
    outputs along a direction equals the gradient's product with it."""
    counts, n, k = [3, 0, 17, 40], 72, 136
    off = offsets_of(counts)
    rows = 60
    p = moe.Ragged(R=rows, N=n, K=k, E=4, dtype="float16")
    g = torch.Generator(device="cuda").manual_seed(11)

    def ints(shape, top):
        return torch.randint(-top, top + 1, shape, generator=g, device="cuda").half()

    x, w, dy = ints((rows, k), 1), ints((4, n, k), 1), ints((rows, n), 1)
    u, v = ints((rows, k), 1), ints((4, n, k), 1)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")

    def loss(x, w):
        y = torch.empty(rows, n, dtype=torch.float16, device="cuda")
        moe.ragged_gemm(p, x, w, o, y, ws)
        return float((y.double() * dy.double()).sum())

    dx, dw = torch.empty_like(x), torch.empty_like(w)
    moe.ragged_gemm_dgrad(p, dy, w, o, dx, ws)
    moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws)
    assert loss(x + u, w) - loss(x, w) == float((dx.double() * u.double()).sum())
    assert loss(x, w + v) - loss(x, w) == float((dw.double() * v.double()).sum())
    assert moe.moe_sync_status() == 0


def test_bad_offsets_are_reported_and_stay_inside():
    n, k, rows = 136, 72, 64
    p = moe.Ragged(R=rows, N=n, K=k, E=3)
    x, dy, w = (randn((rows, k), "bfloat16", 1), randn((rows, n), "bfloat16", 2),
                randn((3, n, k), "bfloat16", 3))
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)
    for off in ([0, 10, 5, 64], [-3, 10, 20, 64], [0, 10, 20, 65], [0, 1 << 30, -(1 << 30), 64]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        for call in (lambda: moe.ragged_gemm(p, x, w, o, y, ws),
                     lambda: moe.ragged_gemm_dgrad(p, dy, w, o, dx, ws),
                     lambda: moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws)):
            call()
            assert moe.moe_status_string(moe.moe_sync_status()) == "MOE_ERR_DEVICE_BAD_INDEX"
    assert moe.moe_sync_status() == 0


def test_empty_input_zeroes_dw():
    p = moe.Ragged(R=0, N=16, K=8, E=2)
    t = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, moe.moe_ragged_workspace_bytes(p)), dtype=torch.uint8, device="cuda")
    dw = torch.ones(2, 16, 8, device="cuda")
    moe.ragged_gemm_wgrad(p, t, x, o, dw, ws, accumulate=True)
    assert bool((dw == 1).all())
    moe.ragged_gemm_wgrad(p, t, x, o, dw, ws)
    assert bool((dw == 0).all())


def test_graph_replay_and_side_stream():
    """Captured once, replayed with other offsets and inputs in place."""
    n, k, rows = 136, 72, 200
    p = moe.Ragged(R=rows, N=n, K=k, E=3)
    x, dy, w = (randn((rows, k), "bfloat16", 1), randn((rows, n), "bfloat16", 2),
                randn((3, n, k), "bfloat16", 3))
    o = torch.tensor([0, 50, 50, 200], dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)

    def step():
        moe.ragged_gemm(p, x, w, o, y, ws)
        moe.ragged_gemm_dgrad(p, dy, w, o, dx, ws)
        moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    off = [0, 20, 130, 200]
    o.copy_(torch.tensor(off))
    x.copy_(randn((rows, k), "bfloat16", 9))
    graph.replay()
    assert moe.moe_sync_status() == 0
    got = [t.clone() for t in (y, dx, dw)]
    step()
    assert all(bool((a == b).all()) for a, b in zip(got, (y, dx, dw)))
    X, W = f64(x), f64(w)
    check(y, ragged.forward(X, W, off), ragged.forward(abs(X), abs(W), off), k, torch.bfloat16, "y")
    D = f64(dy)
    check(dx, ragged.dgrad(D, W, off), ragged.dgrad(abs(D), abs(W), off), n, torch.bfloat16, "dx")
    check(dw, ragged.wgrad(D, X, off), ragged.wgrad(abs(D), abs(X), off), 110, torch.bfloat16, "dw")


def test_watchdog_reports_and_recovers():
    p = moe.Ragged(R=64, N=128, K=128, E=2)
    x, w = randn((64, 128), "bfloat16", 1), randn((2, 128, 128), "bfloat16", 2)
    o = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y = torch.empty(64, 128, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty_like(w)
    for call in (lambda: moe.ragged_gemm(p, x, w, o, y, ws),
                 lambda: moe.ragged_gemm_dgrad(p, x, w, o, y, ws),
                 lambda: moe.ragged_gemm_wgrad(p, x, x, o, dw, ws)):
        try:
            moe.moe_debug_set_watchdog(50_000_000, True)
            call()
            assert moe.moe_status_string(moe.moe_sync_status()) == "MOE_ERR_DEVICE_TIMEOUT"
        finally:
            moe.moe_debug_set_watchdog(0, False)
        call()
        assert moe.moe_sync_status() == 0


def test_binding_refuses_wrong_tensors():
    p = moe.Ragged(R=8, N=16, K=8, E=2, ldx=16)
    x = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")[:, :8]
    w, y = torch.zeros(2, 16, 8, device="cuda").bfloat16(), torch.zeros(8, 16, device="cuda").bfloat16()
    o = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    moe.ragged_gemm(p, x, w, o, y, ws)
    for kind, bad in ((TypeError, (x.half(), w, o, y)), (ValueError, (x.contiguous(), w, o, y)),
                      (ValueError, (x, w[:1], o, y)), (TypeError, (x, w, o.long(), y)),
                      (ValueError, (x, w, o[:2], y)), (ValueError, (x, w, o, y.T.contiguous().T)),
                      (ValueError, (x, w, o, y.cpu())), (ValueError, (x, w.transpose(1, 2), o, y))):
        with pytest.raises(kind):
            moe.ragged_gemm(p, *bad, ws)
    with pytest.raises(TypeError):
        moe.ragged_gemm_wgrad(p, y, x, o, w.half(), ws)
    with pytest.raises(moe.MoEError, match="WORKSPACE"):
        moe.ragged_gemm(p, x, w, o, y, ws[:128])
    assert moe.moe_sync_status() == 0
