"""Training and 4-bit operators on tensors of more than 2^32 elements, and as a
process's very first call inside a graph capture.

Offsets into inputs and outputs pass 32 bits; rows on both sides of 2^31 and 2^32
elements are compared.  Small integers: every value is exact."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROWS, WIDE, NARROW = 300007, 16384, 72         # ROWS * WIDE = 4.9e9


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def ints(*shape, seed=0, top=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda", dtype=torch.int8).bfloat16()


def u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def sample(width):
    """Rows at both ends, around 2^31 and 2^32 elements, and a few between."""
    at = [0, 1, ROWS - 1, ROWS - 2]
    for p in (1 << 31, 1 << 32):
        at += [p // width + d for d in range(-2, 3)]
    return torch.tensor(at + list(range(777, ROWS, 30011)), device="cuda").clamp(max=ROWS - 1)


def of_rows(t, at):
    return t[at].double()


@pytest.mark.parametrize("form", ["single", "pairs", "pairs_double"])
def test_products_past_32_bits(form):
    off = [0, 7, 131000, 131100, 262200, 300000]           # a few rows of no expert behind
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, w = ints(ROWS, NARROW), ints(5, WIDE, NARROW, seed=1)
    p = moe.Ragged(R=ROWS, N=WIDE, K=NARROW, E=5)
    ws = u8(moe.moe_ragged_workspace_bytes(p))
    y = torch.full((ROWS, WIDE), 7.0, dtype=torch.bfloat16, device="cuda")
    at = sample(WIDE)
    e = torch.bucketize(at, o[1:].long(), right=True)
    live = e < 5
    moe.moe_debug_set_bf16_gemm_form(form)
    try:
        moe.ragged_gemm(p, x, w, o, y, ws)
        assert moe.moe_sync_status() == 0
        ref = torch.einsum("rk,rnk->rn", of_rows(x, at), w[e.clamp(max=4)].double())
        ref[~live] = 7.0
        assert torch.equal(y[at], ref.bfloat16())
        # y as dy: the input gradient reads past 32 bits
        dx = torch.full((ROWS, NARROW), 7.0, dtype=torch.bfloat16, device="cuda")
        dy = y.clamp_(-1, 1)
        moe.ragged_gemm_dgrad(p, dy, w, o, dx, ws)
        assert moe.moe_sync_status() == 0
        ref = torch.einsum("rn,rnk->rk", of_rows(dy, at), w[e.clamp(max=4)].double())
        ref[~live] = 7.0
        assert torch.equal(dx[at], ref.bfloat16())
        # and the weight gradient: each expert's sum over all its rows
        dw = torch.empty(5, WIDE, NARROW, device="cuda")
        moe.ragged_gemm_wgrad(p, dy, x, o, dw, ws)
        assert moe.moe_sync_status() == 0
        for i in range(5):
            ref = torch.zeros(64, NARROW, dtype=torch.float64, device="cuda")
            for a in range(off[i], off[i + 1], 65536):
                b = min(a + 65536, off[i + 1])
                ref += dy[a:b, -64:].double().T @ x[a:b].double()
            assert torch.equal(dw[i, -64:].double(), ref)
        # the wide side as the reduction's rows: dx past 32 bits
        q = moe.Ragged(R=ROWS, N=NARROW, K=WIDE, E=5)
        ws = u8(moe.moe_ragged_workspace_bytes(q))
        w2 = w.view(5, NARROW, WIDE)
        moe.ragged_gemm_dgrad(q, x, w2, o, y.fill_(7.0), ws)
        assert moe.moe_sync_status() == 0
        ref = torch.einsum("rn,rnk->rk", of_rows(x, at), w2[e.clamp(max=4)].double())
        ref[~live] = 7.0
        assert torch.equal(y[at], ref.bfloat16())
    finally:
        moe.moe_debug_set_bf16_gemm_form("auto")


def test_codec_product_and_clip_past_32_bits():
    k = WIDE
    x = torch.empty(ROWS, k, dtype=torch.bfloat16, device="cuda")
    for a in range(0, ROWS, 50000):
        x[a:a + 50000] = ints(min(50000, ROWS - a), k, seed=a)
    x[:, ::32] = 4                        # every group's scale is 2^0: the values are exact
    codes, scales = u8(ROWS, k // 2), u8(ROWS, k // 32)
    moe.moe_mxfp4_quantize(x, codes, scales)
    assert bool((scales == 127).all())
    back = torch.empty_like(x)
    moe.moe_mxfp4_dequantize(codes, scales, back)
    assert moe.moe_sync_status() == 0 and torch.equal(back, x)
    # clip: one tensor of 4.9e9 values, c = 1 / 2 exactly (up to the norm's 1e-6)
    norm = torch.empty((), device="cuda")
    cw = u8(moe.moe_clip_workspace_bytes())
    moe.moe_clip_grad_norm([x], 1e30, norm, cw, out=[back])
    assert torch.equal(back, x)
    ref = sum(float(x[a:a + 20000].float().square().sum(dtype=torch.float64))
              for a in range(0, ROWS, 20000)) ** 0.5
    assert abs(float(norm) - ref) <= 34 * 2.0 ** -24 * ref
    moe.moe_clip_grad_norm([x], ref / 2, norm, cw, out=[back])
    at = sample(k)
    # half the value, its error that of the norm and of bf16's half step
    want, got = x[at].double() / 2, back[at].double()
    assert bool(((got - want).abs() <= (2.0 ** -8 + 40 * 2.0 ** -24) * want.abs()).all())
    assert bool(((back == 0) == (x == 0)).all())
    # the 4-bit product reads the codes past 2^31 bytes, and writes past 2^32 values
    del back
    n = 256
    wc, wsc = u8(3, n, k // 2), torch.full((3, n, k // 32), 127, dtype=torch.uint8, device="cuda")
    w = ints(3, n, k, seed=5)
    w[:, :, ::32] = 4
    moe.moe_mxfp4_quantize(w.view(3 * n, k), wc.view(3 * n, -1), wsc.view(3 * n, -1))
    packed = torch.empty_like(wsc)
    moe.moe_mxfp4_pack_scales(wsc, packed)
    o = torch.tensor([0, 100, 150000, ROWS], dtype=torch.int32, device="cuda")
    e = torch.bucketize(at, o[1:].long(), right=True)
    for form in ("single", "pairs"):
        # rows of y lie far apart: the last ones are past 2^32 values
        y = torch.empty(ROWS, WIDE, dtype=torch.bfloat16, device="cuda")[:, :n]
        p = moe.Ragged(R=ROWS, N=n, K=k, E=3, ldy=WIDE)
        ws = u8(moe.moe_ragged_workspace_bytes(p))
        moe.moe_debug_set_bf16_gemm_form(form)
        try:
            moe.ragged_gemm_mxfp4(p, codes, scales, wc, packed, o, y, ws)
            assert moe.moe_sync_status() == 0
        finally:
            moe.moe_debug_set_bf16_gemm_form("auto")
        ref = torch.einsum("rk,rnk->rn", x[at].double(), w[e].double())
        assert torch.equal(y[at], ref.bfloat16())
        del y


FIRST = """
import torch, mixture_experts_ffn_align_gb300 as moe
g = torch.Generator(device="cuda").manual_seed(0)
x, w = (torch.randint(-1, 2, s, generator=g, device="cuda").bfloat16() for s in ((300, 256), (3, 1024, 256)))
o = torch.tensor([0, 100, 130, 300], dtype=torch.int32, device="cuda")
p = moe.Ragged(R=300, N=1024, K=256, E=3)
ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
y, dw = torch.empty(300, 1024, dtype=torch.bfloat16, device="cuda"), torch.empty_like(w)
c, s = (torch.empty(300, n, dtype=torch.uint8, device="cuda") for n in (128, 8))
norm, cw = torch.empty((), device="cuda"), torch.empty(moe.moe_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
moe.moe_debug_set_bf16_gemm_form({form!r})
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.ragged_gemm(p, x, w, o, y, ws)
    moe.ragged_gemm_wgrad(p, y, x, o, dw, ws)
    moe.moe_mxfp4_quantize(x, c, s)
    moe.moe_clip_grad_norm([dw], 1.0, norm, cw)
graph.replay()
assert moe.moe_sync_status() == 0
for e, (a, b) in enumerate(((0, 100), (100, 130), (130, 300))):
    assert torch.equal(y[a:b], (x[a:b].double() @ w[e].double().T).bfloat16())
print("done")
"""


@pytest.mark.parametrize("form", ["auto", "single", "pairs", "pairs_double"])
def test_first_call_of_a_process_in_a_capture(form):
    r = subprocess.run([sys.executable, "-c", FIRST.replace("{form!r}", repr(form))], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-2000:]
