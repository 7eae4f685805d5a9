"""The gated block, its gradient and the orthogonalised update as a program uses them:
a training step of a routed layer against fp64 and against differences, on several
streams and in graphs, with a wait that runs out, past 2^32 elements, and as a process's
first call inside a capture."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def f64(t):
    return t.double().cpu().numpy()


def randn(shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def space(n):
    return torch.empty(int(n), dtype=torch.uint8, device="cuda")


class Block:
    """One expert layer on rows grouped by expert: forward, backward and update."""

    def __init__(self, counts, inter, hidden, dtype="bfloat16", seed=0):
        dt = getattr(torch, dtype)
        self.off = np.concatenate([[0], np.cumsum(counts)])
        rows, E = int(self.off[-1]), len(counts)
        self.o = torch.tensor(self.off, dtype=torch.int32, device="cuda")
        self.up = moe.Ragged(R=rows, N=2 * inter, K=hidden, E=E, dtype=dtype)
        self.down = moe.Ragged(R=rows, N=hidden, K=inter, E=E, dtype=dtype)
        self.ws = space(max(moe.moe_ragged_workspace_bytes(p) for p in (self.up, self.down)))
        self.x = randn((rows, hidden), dt, seed)
        self.dy = randn((rows, hidden), dt, seed + 1)
        self.w13 = randn((E, 2 * inter, hidden), dt, seed + 2, hidden ** -0.5)
        self.w2 = randn((E, hidden, inter), dt, seed + 3, inter ** -0.5)
        self.h, self.dh = (torch.empty(rows, 2 * inter, dtype=dt, device="cuda") for _ in range(2))
        self.z = torch.empty(rows, inter, dtype=dt, device="cuda")
        self.y, self.dx = torch.empty_like(self.x), torch.empty_like(self.x)
        self.dw13, self.dw2 = (torch.empty(w.shape, device="cuda") for w in (self.w13, self.w2))
        self.u13, self.u2 = (torch.empty(w.shape, dtype=torch.bfloat16, device="cuda")
                             for w in (self.w13, self.w2))
        self.wo = [space(moe.moe_orthogonalize_workspace_bytes(*w.shape)) for w in (self.w13, self.w2)]

    def outputs(self):
        return [self.y, self.h, self.z, self.dh, self.dx, self.dw13, self.dw2, self.u13, self.u2]

    def clear(self):
        for t in self.outputs():
            t.fill_(float("nan"))

    def forward(self):
        moe.ragged_gated(self.up, self.x, self.w13, self.o, self.z, self.ws, h=self.h)
        moe.ragged_gemm(self.down, self.z, self.w2, self.o, self.y, self.ws)

    def backward(self):
        moe.ragged_gated_dgrad(self.down, self.dy, self.w2, self.h, self.o, self.dh, self.ws, z=self.z)
        moe.ragged_gemm_wgrad(self.down, self.dy, self.z, self.o, self.dw2, self.ws)
        moe.ragged_gemm_dgrad(self.up, self.dh, self.w13, self.o, self.dx, self.ws)
        moe.ragged_gemm_wgrad(self.up, self.dh, self.x, self.o, self.dw13, self.ws)

    def update(self):
        moe.moe_orthogonalize(self.dw13, self.u13, self.wo[0])
        moe.moe_orthogonalize(self.dw2, self.u2, self.wo[1])

    def step(self):
        self.forward()
        self.backward()
        self.update()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_training_step_against_fp64(dtype):
    """Each stage from the stage before as the library rounded it, so that one rounding of
    the output (half a step) and the sums' error remain: (n / 16 + 17) steps of 2^-23 of
    the magnitudes, for at most 300 terms 2^-17.8 of some 14 times the values' scale,
    which 2^-12 of that scale covers.  (The gradient writes z from h's rounded values, so
    y is held against the z it was made of.)"""
    b = Block([70, 0, 300, 1, 129], 136, 264, dtype)
    b.clear()
    b.forward()
    forward_z = f64(b.z)
    b.backward()
    b.update()
    assert moe.moe_sync_status() == 0
    x, dy, w13, w2, h, z, dh = map(f64, (b.x, b.dy, b.w13, b.w2, b.h, b.z, b.dh))
    half = torch.finfo(getattr(torch, dtype)).eps / 2

    def close(got, ref, step=half):
        scale = np.sqrt(np.mean(ref ** 2))
        assert (np.abs(f64(got) - ref) <= step * np.abs(ref) + 2.0 ** -12 * scale).all()

    close(b.h, ragged.forward(x, w13, b.off))
    close(b.z, ragged.gated(h))
    close(b.y, ragged.forward(forward_z, w2, b.off))
    close(b.dh, ragged.gated_grad(ragged.dgrad(dy, w2, b.off), h))
    close(b.dx, ragged.dgrad(dh, w13, b.off))
    close(b.dw2, ragged.wgrad(dy, z, b.off), 0.0)
    close(b.dw13, ragged.wgrad(dh, x, b.off), 0.0)
    for u, d in ((b.u13, b.dw13), (b.u2, b.dw2)):
        for e in range(5):
            ref = ragged.orthogonalize(f64(d[e]))
            err = np.sqrt(np.mean((f64(u[e]) - ref) ** 2))
            assert err <= 0.0035 * np.sqrt(np.mean(ref ** 2)) + 1e-12     # twice bf16's own 0.0017


def test_gradients_against_differences():
    """Directional derivatives of sum(dy * y) by x, w13 and w2, in fp64, against the
    kernels' gradients in bf16: relative to the gradients' norms times the direction's
    (a random direction of n values meets errors of 2^-8 each as their rms / sqrt n)."""
    b = Block([33, 0, 95], 40, 72, seed=9)
    b.step()
    assert moe.moe_sync_status() == 0
    base = dict(x=f64(b.x), w13=f64(b.w13), w2=f64(b.w2))
    dy = f64(b.dy)

    def loss(x, w13, w2):
        return (dy * ragged.forward(ragged.gated(ragged.forward(x, w13, b.off)), w2, b.off)).sum()

    rng = np.random.default_rng(0)
    for name, grad in (("x", b.dx), ("w13", b.dw13), ("w2", b.dw2)):
        g = f64(grad)
        for _ in range(4):
            d = rng.standard_normal(g.shape)
            e = 1e-6
            up, down = ({**base, name: base[name] + s * e * d} for s in (1, -1))
            want = (loss(**up) - loss(**down)) / (2 * e)
            # three roundings (h, z or dh, and dx) of 2^-9 rms each, 4 deviations
            assert abs((g * d).sum() - want) <= 4 * 3 * 2.0 ** -9 * np.sqrt((g ** 2).sum())


@pytest.mark.parametrize("form", ["auto", "single", "pairs", "pairs_double", "whole_grid"])
def test_streams_and_graphs_give_the_same_bits(form):
    """Two layers on two streams at once, eager and captured into one graph together,
    against each by itself."""
    moe.moe_debug_set_bf16_gemm_form(form)
    try:
        blocks = [Block([70, 0, 300, 1, 129], 136, 264, seed=1), Block([400, 37], 72, 520, seed=2)]
        want = []
        for b in blocks:
            b.clear()
            b.step()
            want.append([t.clone() for t in b.outputs()])
        torch.cuda.synchronize()
        sides = [torch.cuda.Stream() for _ in blocks]

        def both():
            main = torch.cuda.current_stream()
            for s, b in zip(sides, blocks):
                s.wait_stream(main)
                with torch.cuda.stream(s):
                    b.clear()
                    b.step()
            for s in sides:
                main.wait_stream(s)

        def check():
            torch.cuda.synchronize()
            assert moe.moe_sync_status() == 0
            for b, w in zip(blocks, want):
                assert all(torch.equal(t, v) for t, v in zip(b.outputs(), w))

        for _ in range(10):
            both()
        check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
        for b in blocks:
            b.clear()
        for _ in range(10):
            graph.replay()
        check()
    finally:
        moe.moe_debug_set_bf16_gemm_form("auto")


def test_two_graphs_share_a_workspace_in_turn():
    """Captured calls that never overlap may use one workspace: nothing is kept in it."""
    a, b = Block([90, 11], 72, 136, seed=3), Block([90, 11], 72, 136, seed=4)
    b.ws, b.wo = a.ws, a.wo
    graphs, want = [], []
    for block in (a, b):
        block.clear()
        block.step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in block.outputs()])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            block.step()
        graphs.append(g)
    for _ in range(3):
        for g, block, w in zip(graphs, (a, b), want):
            block.clear()
            a.ws.fill_(0xFF)
            for s in a.wo:
                s.fill_(0xFF)
            g.replay()
            assert all(torch.equal(t, v) for t, v in zip(block.outputs(), w))


@pytest.mark.parametrize("form", ["single", "pairs", "pairs_double", "whole_grid"])
def test_wait_that_runs_out_is_reported(form):
    """The producer leaves its first copy out, the waits run out and are reported, and the
    next calls give the same bits as before."""
    b = Block([200, 40], 136, 264)
    calls = [lambda: moe.ragged_gated(b.up, b.x, b.w13, b.o, b.z, b.ws, h=b.h),
             lambda: moe.ragged_gated_dgrad(b.down, b.dy, b.w2, b.h, b.o, b.dh, b.ws),
             lambda: moe.moe_orthogonalize(b.w2, b.u2, b.wo[1], steps=1)]
    outs = [b.z, b.dh, b.u2]
    moe.moe_debug_set_bf16_gemm_form(form)
    try:
        want = []
        for call, out in zip(calls, outs):
            call()
            want.append(out.clone())
        assert moe.moe_sync_status() == 0
        for call, out, w in zip(calls, outs, want):
            moe.moe_debug_set_watchdog(20_000_000, never_arrive=True)       # 20 ms
            call()
            assert moe.moe_sync_status() == 4          # MOE_ERR_DEVICE_TIMEOUT
            moe.moe_debug_set_watchdog(0)
            assert moe.moe_sync_status() == 0
            b.ws.fill_(0xFF)
            b.wo[1].fill_(0xFF)
            out.fill_(float("nan"))
            call()
            assert moe.moe_sync_status() == 0 and torch.equal(out, w)
    finally:
        moe.moe_debug_set_watchdog(0)
        moe.moe_debug_set_bf16_gemm_form("auto")


ROWS, INTER, HIDDEN = 300007, 8192, 72           # h: 4.9e9 elements


@pytest.mark.parametrize("form", ["single", "pairs"])
def test_gated_past_32_bits(form):
    """Rows on both sides of 2^31 and 2^32 elements of h, dh and z; those of no expert
    stay as they were."""
    torch.cuda.empty_cache()
    off = [3, 7, 131000, 131100, 262200, 300000]
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, w13 = randn((ROWS, HIDDEN), seed=1), randn((5, 2 * INTER, HIDDEN), seed=2, scale=0.2)
    up = moe.Ragged(R=ROWS, N=2 * INTER, K=HIDDEN, E=5)
    down = moe.Ragged(R=ROWS, N=HIDDEN, K=INTER, E=5)
    h = torch.full((ROWS, 2 * INTER), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((ROWS, INTER), 7.0, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 2, 3, ROWS - 1, ROWS - 7, ROWS - 8]
    for width in (INTER, 2 * INTER):
        for p in (1 << 31, 1 << 32):
            at += [min(p // width + d, ROWS - 1) for d in range(-2, 3)]
    at = torch.tensor(sorted(set(at + list(range(777, ROWS, 30011)))), device="cuda")
    e = torch.bucketize(at, o[1:].long(), right=True).clamp(max=4)
    live = (at >= 3) & (at < 300000)
    moe.moe_debug_set_bf16_gemm_form(form)
    try:
        moe.ragged_gated(up, x, w13, o, z, space(moe.moe_ragged_workspace_bytes(up)), h=h)
        assert moe.moe_sync_status() == 0
        ref = torch.einsum("rk,rnk->rn", x[at].double(), w13[e].double())
        g, u = ref.split(INTER, 1)
        want = g * torch.sigmoid(g) * u

        def close(got, ref):
            # half a step, and 2^-14 of the scale for 22 steps of 2^-23 of magnitudes
            tol = 2.0 ** -8 * ref.abs() + 2.0 ** -14 * ref.square().mean().sqrt()
            assert bool(((got.double() - ref).abs() <= tol)[live].all())
            assert bool((got[~live] == 7.0).all())

        close(h[at], ref)
        close(z[at], want)
        dy, w2 = randn((ROWS, HIDDEN), seed=3), randn((5, HIDDEN, INTER), seed=4, scale=0.2)
        H = h[at].double()
        moe.ragged_gated_dgrad(down, dy, w2, h, o, h, space(moe.moe_ragged_workspace_bytes(down)),
                               z=z.fill_(7.0))
        assert moe.moe_sync_status() == 0
        dz = torch.einsum("rn,rnk->rk", dy[at].double(), w2[e].double())
        g, u = H.split(INTER, 1)
        s = torch.sigmoid(g)
        close(h[at], torch.cat([dz * u * s * (1 + g * (1 - s)), dz * g * s], 1))
        close(z[at], g * s * u)
    finally:
        moe.moe_debug_set_bf16_gemm_form("auto")


@pytest.mark.parametrize("shape", [(80, 256, 1 << 18), (80, 1 << 18, 224)], ids=str)
def test_orthogonalize_past_32_bits(shape):
    """Matrices before, across and past 2^32 elements against fp64 on the GPU."""
    torch.cuda.empty_cache()
    E, N, K = shape
    g = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    g.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    out = torch.empty_like(g)
    ws = space(moe.moe_orthogonalize_workspace_bytes(*shape))
    moe.moe_orthogonalize(g, out, ws)
    assert moe.moe_sync_status() == 0
    del ws
    for e in (0, (1 << 31) // (N * K), (1 << 32) // (N * K), E - 1):
        x = g[e].double() if N <= K else g[e].double().T
        x = x / (x.square().sum().sqrt() + 1e-7)
        for _ in range(5):
            a = x @ x.T
            p = -4.7750 * a + 2.0315 * a @ a
            p.diagonal().add_(3.4445)
            x = p @ x
        ref = x if N <= K else x.T
        err = (out[e].double() - ref).square().mean().sqrt() / ref.square().mean().sqrt()
        assert float(err) <= 0.0025          # 0.0017 of bf16's rounding, at most as much again
        del x, ref


FIRST = """
import torch, mixture_experts_ffn_align_gb300 as moe
g = torch.Generator(device="cuda").manual_seed(0)
x, w, w2 = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((300, 256), (3, 512, 256), (3, 256, 256)))
o = torch.tensor([0, 100, 130, 300], dtype=torch.int32, device="cuda")
p, q = moe.Ragged(R=300, N=512, K=256, E=3), moe.Ragged(R=300, N=256, K=256, E=3)
ws = torch.empty(moe.moe_ragged_workspace_bytes(p) + moe.moe_ragged_workspace_bytes(q), dtype=torch.uint8, device="cuda")
z, h, dh = (torch.empty(300, n, dtype=torch.bfloat16, device="cuda") for n in (256, 512, 512))
u, wo = torch.empty_like(w), torch.empty(moe.moe_orthogonalize_workspace_bytes(3, 512, 256), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
moe.moe_debug_set_bf16_gemm_form({form!r})

def run():
    moe.ragged_gated(p, x, w, o, z, ws, h=h)
    moe.ragged_gated_dgrad(q, x, w2, h, o, dh, ws)
    moe.moe_orthogonalize(w, u, wo)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
assert moe.moe_sync_status() == 0
got = [t.clone() for t in (z, h, dh, u)]
run()
assert moe.moe_sync_status() == 0
assert all(torch.equal(a, b) and bool(b.isfinite().all()) for a, b in zip(got, (z, h, dh, u)))
print("done")
"""


@pytest.mark.parametrize("form", ["auto", "single", "pairs", "pairs_double", "whole_grid"])
def test_first_call_of_a_process_in_a_capture(form):
    r = subprocess.run([sys.executable, "-c", FIRST.replace("{form!r}", repr(form))], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-2000:]


def test_example_with_orthogonalised_updates():
    """It runs, its gradients are those of its layer (by differences of the layer's own
    loss in fp64), and its update is the oracle's."""
    path = os.path.join(ROOT, "examples", "finetune_experts.py")
    spec = importlib.util.spec_from_file_location("finetune_experts_orthogonal", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(steps=3, update="orthogonal", verbose=False)
    assert len(r["losses"]) == 3 and all(np.isfinite(r["losses"] + r["norms"]))
    layer = m.ExpertLayer()
    x, logits = randn((m.M, m.H), seed=1), randn((m.M, m.E), torch.float32, seed=2)
    layer.route(x, logits)
    w13, w2 = randn((m.E, 2 * m.I, m.H), seed=3, scale=0.06), randn((m.E, m.H, m.I), seed=4, scale=0.06)
    layer.forward(w13, w2)
    dy = randn((m.M, m.H), torch.float32, seed=5)
    dw13, dw2 = torch.empty(w13.shape, device="cuda"), torch.empty(w2.shape, device="cuda")
    layer.backward(dy, w13, w2, dw13, dw2)
    assert moe.moe_sync_status() == 0
    X, D, ids, pw = x.double(), dy.double(), layer.ids.long(), layer.weights.double()

    def loss(a13, a2):
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for e in range(m.E):
            t, k = (ids == e).nonzero(as_tuple=True)
            g, u = (X[t] @ a13[e].T).split(m.I, 1)
            y = (g * torch.sigmoid(g) * u) @ a2[e].T
            total += (pw[t, k, None] * y * D[t]).sum()
        return float(total)

    gen = torch.Generator(device="cuda").manual_seed(6)
    W13, W2 = w13.double(), w2.double()
    for which, grad in ((0, dw13), (1, dw2)):
        d = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
        e = 1e-5
        args = [(W13 + s * e * d, W2) if which == 0 else (W13, W2 + s * e * d) for s in (1, -1)]
        want = (loss(*args[0]) - loss(*args[1])) / (2 * e)
        norm = float(grad.double().square().sum().sqrt())
        # roundings of h, z or dh and dy of 2^-9 rms each, met by a random direction
        assert abs(float((grad.double() * d).sum()) - want) <= 4 * 3 * 2.0 ** -9 * norm
    opt = m.Orthogonal(dw13)
    opt.step(W13.float(), dw13, 0.1)
    ref = opt.scale * ragged.orthogonalize(f64(dw13[0]))
    assert np.sqrt(np.mean((f64(opt.out[0]) - ref) ** 2) / np.mean(ref ** 2)) <= 0.0025
