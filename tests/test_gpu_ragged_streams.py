"""The training and 4-bit operators on several streams, eager and in one graph.

Their kernels may start while the one before on the stream ends (programmatic
launches); what a stream waits for by an event has to be complete all the same.
Small integers throughout: every value is exact."""
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe

pytestmark = pytest.mark.gpu
R, N, K, E = 700, 520, 264, 6


class Step:
    """Forward on this stream, the weight gradient and its clipping on another,
    the input gradient on a third; each stream reads what another wrote."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(0)

        def ints(*shape):
            return torch.randint(-2, 3, shape, generator=g, device="cuda").bfloat16()

        self.x, self.dy, self.w = ints(R, K), ints(R, N), ints(E, N, K)
        self.o = torch.tensor([0, 90, 90, 300, 333, 690, 700], dtype=torch.int32, device="cuda")
        self.p = moe.Ragged(R=R, N=N, K=K, E=E)
        n = moe.moe_ragged_workspace_bytes(self.p)
        self.ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(3)]
        self.cw = torch.empty(moe.moe_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
        self.y, self.dx = torch.empty_like(self.dy), torch.empty_like(self.x)
        self.dw, self.norm = torch.empty(E, N, K, device="cuda"), torch.empty((), device="cuda")
        self.y2, self.src = torch.empty_like(self.y), torch.empty_like(self.x)
        self.sides = [torch.cuda.Stream() for _ in range(2)]

    def clear(self):
        for t in (self.y, self.dx, self.dw, self.norm, self.y2, self.src):
            t.fill_(float("nan"))

    def __call__(self):
        main, (a, b) = torch.cuda.current_stream(), self.sides
        self.src.copy_(self.x)
        a.wait_stream(main)
        b.wait_stream(main)
        with torch.cuda.stream(a):
            moe.ragged_gemm_wgrad(self.p, self.dy, self.src, self.o, self.dw, self.ws[0])
            moe.moe_clip_grad_norm([self.dw], 1e30, self.norm, self.cw)
        with torch.cuda.stream(b):
            moe.ragged_gemm_dgrad(self.p, self.dy, self.w, self.o, self.dx, self.ws[1])
        moe.ragged_gemm(self.p, self.src, self.w, self.o, self.y, self.ws[2])
        main.wait_stream(a)
        main.wait_stream(b)
        # reads what all three wrote, and frees src for the next step
        moe.ragged_gemm(self.p, self.dx, self.w, self.o, self.y2, self.ws[2])
        self.src.fill_(float("nan"))

    def check(self):
        assert moe.moe_sync_status() == 0
        o = self.o.tolist()
        squares = 0.0
        for e in range(E):
            at = slice(o[e], o[e + 1])
            X, D, W = self.x[at].double(), self.dy[at].double(), self.w[e].double()
            assert torch.equal(self.y[at], (X @ W.T).bfloat16())
            assert torch.equal(self.dx[at], (D @ W).bfloat16())
            assert torch.equal(self.dw[e].double(), D.T @ X)
            assert torch.equal(self.y2[at], (self.dx[at].double() @ W.T).bfloat16())
            squares += float((D.T @ X).square().sum())
        assert abs(float(self.norm) - squares ** 0.5) <= 34 * 2.0 ** -24 * squares ** 0.5


@pytest.mark.parametrize("form", ["auto", "single", "pairs", "pairs_double"])
def test_streams_that_wait_for_each_other(form):
    moe.moe_debug_set_bf16_gemm_form(form)
    try:
        step = Step()
        for _ in range(20):
            step.clear()
            step()
        torch.cuda.synchronize()
        step.check()
        step.clear()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        step.clear()
        for _ in range(20):
            graph.replay()
        torch.cuda.synchronize()
        step.check()
    finally:
        moe.moe_debug_set_bf16_gemm_form("auto")


def test_codec_and_product_on_two_streams_in_a_graph():
    """Two quantisations on two streams, joined by a product of both."""
    n = k = 256
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-1, 2, (300, k), generator=g, device="cuda").bfloat16()
    w = torch.randint(-1, 2, (2, n, k), generator=g, device="cuda").bfloat16()
    x[:, ::32] = w[:, :, ::32] = 4        # every group's scale is 2^0: the values are exact
    o = torch.tensor([0, 130, 300], dtype=torch.int32, device="cuda")
    p = moe.Ragged(R=300, N=n, K=k, E=2)
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")

    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device="cuda")

    xc, xs, wc, wsc, packed = u8(300, k // 2), u8(300, k // 32), u8(2 * n, k // 2), \
        u8(2 * n, k // 32), u8(2, n, k // 32)
    y = torch.empty(300, n, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            moe.moe_mxfp4_quantize(w.view(2 * n, k), wc, wsc)
            moe.moe_mxfp4_pack_scales(wsc.view(2, n, k // 32), packed)
        moe.moe_mxfp4_quantize(x, xc, xs)
        main.wait_stream(side)
        moe.ragged_gemm_mxfp4(p, xc, xs, wc.view(2, n, k // 2), packed, o, y, ws)

    ref = torch.cat([x[:130].double() @ w[0].double().T, x[130:].double() @ w[1].double().T])
    step()
    assert moe.moe_sync_status() == 0 and torch.equal(y, ref.bfloat16())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (xc, xs, wc, wsc, packed):
        t.zero_()
    for _ in range(10):
        y.fill_(float("nan"))
        graph.replay()
    assert moe.moe_sync_status() == 0 and torch.equal(y, ref.bfloat16())
