"""MXFP4 codec (bit for bit against the fp64 oracle) and the 4-bit product.

Tolerance of the product: operands are what the codes stand for, so only the
accumulation and the output's rounding differ from fp64: eps / 2 * |v| for the
output and, as the block-scaled MMA adds 64 scaled products at a time to an
fp32 accumulator, (K / 64 + 65) 2^-23 of the magnitudes' sum.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

pytestmark = pytest.mark.gpu
DT = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


@pytest.fixture(params=["single", "pairs"])
def form(request):
    """The products in both forms of the kernel."""
    moe.moe_debug_set_bf16_gemm_form(request.param)
    yield
    moe.moe_debug_set_bf16_gemm_form("auto")


def f64(t):
    return t.double().cpu().numpy()


def quantize(x, mode="floor"):
    rows, k = x.shape
    codes = torch.full((rows, k // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, k // 32), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_mxfp4_quantize(x, codes, scales, scale_mode=mode)
    return codes, scales


@pytest.mark.parametrize("mode", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows, k", [(1, 32), (3, 96), (17, 2880), (257, 7168), (1000, 64)])
def test_quantize_bits(rows, k, dtype, mode):
    g = torch.Generator(device="cuda").manual_seed(rows * 31 + k)
    x = torch.randn(rows, k, generator=g, device="cuda")
    x = (x * torch.exp2(torch.randint(-12, 12, (rows, k // 32), generator=g, device="cuda")
                        .float()).repeat_interleave(32, 1)).to(DT[dtype])
    codes, scales = quantize(x, mode)
    c, s = ragged.mxfp4_quantize(f64(x), mode)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), ragged.pack_fp4(c))


@pytest.mark.parametrize("mode", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_edges(dtype, mode):
    """Ties, zeros of both signs, the type's extremes and subnormals, infinity
    and NaN; every value with each of several largest magnitudes."""
    fi = torch.finfo(DT[dtype])
    specials = [0.0, -0.0, fi.tiny, fi.tiny * fi.eps, -fi.tiny * fi.eps, fi.max, -fi.max, 1.0]
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375, -0.25, -5.0]
    groups = []
    for top in (6.0, 4.0, 7.5, 7.9375, fi.max, fi.tiny, fi.tiny * fi.eps, 0.0):
        groups.append((ties + specials)[:20] + [0.0] * 11 + [top])
        groups.append([t * top / 8 for t in ties] + [0.0] * 19 + [top])
        groups.append([fi.tiny * fi.eps * i for i in range(31)] + [min(top, fi.tiny * 4)])
    for bad in (float("inf"), -float("inf"), float("nan")):
        groups.append([1.0] * 31 + [bad])
        groups.append([bad] + [0.0] * 31)
    x = torch.tensor(groups, dtype=torch.float64).to(DT[dtype]).cuda()
    codes, scales = quantize(x, mode)
    c, s = ragged.mxfp4_quantize(f64(x), mode)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), ragged.pack_fp4(c))


def test_quantize_strided_rows():
    x = torch.randn(37, 200, device="cuda").to(torch.bfloat16)
    a = quantize(x[:, 8:168])
    b = quantize(x[:, 8:168].contiguous())
    assert all(bool((i == j).all()) for i, j in zip(a, b))


@pytest.mark.parametrize("dtype", list(DT))
def test_dequantize_every_code_and_scale(dtype):
    """All 16 codes under all 256 scales; the type's own rounding beyond its
    range, NaN under scale 255."""
    codes = (torch.arange(256, device="cuda")[:, None] * 0
             + torch.tensor([0x10 * (2 * i + 1) + 2 * i for i in range(8)] * 2, device="cuda"))
    codes = codes.to(torch.uint8).contiguous()
    scales = torch.arange(256, device="cuda").to(torch.uint8)[:, None].contiguous()
    out = torch.empty(256, 40, dtype=DT[dtype], device="cuda")
    moe.moe_mxfp4_dequantize(codes, scales, out[:, :32])
    ref = ragged.mxfp4_dequantize(codes.cpu().numpy(), scales.cpu().numpy())
    # exact in fp32 (its subnormals reach 2^-149), then the type's cast
    want = torch.from_numpy(ref).float().to(DT[dtype]).float().numpy()
    got = out[:, :32].float().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_pack_scales():
    s = torch.randint(0, 256, (3, 256, 12), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(s)
    moe.moe_mxfp4_pack_scales(s, out)
    assert np.array_equal(out.cpu().numpy().ravel(), ragged.pack_scales(s.cpu().numpy()).ravel())


def product(counts, n, k, dtype="bfloat16", lead=0, tail=0, ldy=0, seed=0, lo=118, hi=130):
    off = np.concatenate([[0], np.cumsum(counts)]) + lead
    rows, E = int(off[-1]) + tail, len(counts)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def u8(shape, a, b):
        return torch.randint(a, b, shape, dtype=torch.uint8, generator=g, device="cuda")

    xc, xs = u8((rows, k // 2), 0, 256), u8((rows, k // 32), lo, hi)
    wc, wsc = u8((E, n, k // 2), 0, 256), u8((E, n, k // 32), lo - 6, hi - 6)
    packed = torch.empty_like(wsc)
    moe.moe_mxfp4_pack_scales(wsc, packed)
    p = moe.Ragged(R=rows, N=n, K=k, E=E, dtype=dtype, ldy=ldy)
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y = torch.full((rows, ldy or n), 7.0, dtype=DT[dtype], device="cuda")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    moe.ragged_gemm_mxfp4(p, xc, xs, wc, packed, o, y[:, :n], ws)
    assert moe.moe_sync_status() == 0
    X = ragged.mxfp4_dequantize(xc.cpu().numpy(), xs.cpu().numpy())
    W = ragged.mxfp4_dequantize(wc.cpu().numpy(), wsc.cpu().numpy())
    ref, mag = ragged.forward(X, W, off), ragged.forward(abs(X), abs(W), off)
    fi = torch.finfo(DT[dtype])
    live = slice(int(off[0]), int(off[-1]))
    tol = (fi.eps / 2 * np.abs(ref) + fi.tiny * fi.eps + (k / 64 + 65) * 2.0 ** -23 * mag)[live]
    err = np.abs(f64(y[:, :n])[live] - ref[live])
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size}, worst {(err / tol).max():.2f}"
    keep = torch.ones(rows, dtype=torch.bool)
    keep[live] = False
    assert bool((y[keep.cuda()] == 7.0).all()) and bool((y[:, n:] == 7.0).all())


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1, 130, 0], [16, 32, 64, 127, 128, 129],
                                    [700, 5, 256], [0, 0], [300] * 9])
def test_product_segments(counts, form):
    product(counts, 256, 384)


@pytest.mark.parametrize("n, k", [(128, 128), (128, 256), (384, 640), (256, 2048), (1152, 1152)])
def test_product_sizes(n, k, form):
    product([5, 0, 40, 260], n, k, dtype="float16", seed=n, lo=122, hi=126)


@pytest.mark.parametrize("rows", [1, 31, 33, 127, 128, 129, 256, 257, 900])
def test_product_one_expert(rows, form):
    product([rows], 256, 512, seed=rows)


@pytest.mark.parametrize("counts", [[1], [200], [3, 0, 60]])
def test_product_long_reduction_of_few_tiles(counts, form):
    """Few tiles, a long reduction: slices that are joined."""
    product(counts, 256, 8576, lo=122, hi=126)


def test_product_rows_of_no_expert_and_stride(form):
    product([40, 0, 90], 128, 384, lead=3, tail=9, ldy=136)


def test_product_scales_of_their_rows_only(form):
    """A NaN scale poisons its own row (token) or column (weight) only."""
    n, k = 256, 256
    off = [0, 50, 200]
    p = moe.Ragged(R=200, N=n, K=k, E=2)
    xc = torch.full((200, k // 2), 0x22, dtype=torch.uint8, device="cuda")     # all ones
    wc = torch.full((2, n, k // 2), 0x22, dtype=torch.uint8, device="cuda")
    xs = torch.full((200, k // 32), 127, dtype=torch.uint8, device="cuda")
    wsc = torch.full((2, n, k // 32), 127, dtype=torch.uint8, device="cuda")
    xs[60, 3] = 255
    wsc[0, 17, 7] = 255
    packed = torch.empty_like(wsc)
    moe.moe_mxfp4_pack_scales(wsc, packed)
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y = torch.empty(200, n, dtype=torch.bfloat16, device="cuda")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    moe.ragged_gemm_mxfp4(p, xc, xs, wc, packed, o, y, ws)
    bad = torch.zeros(200, n, dtype=torch.bool, device="cuda")
    bad[60] = True
    bad[:50, 17] = True
    assert bool((y.isnan() == bad).all()) and bool((y[~bad] == 256).all())


def test_product_each_scale_lands_on_its_group(form):
    """One nonzero weight group at a time: y counts 32 scaled ones."""
    n, k = 128, 512
    p = moe.Ragged(R=130, N=n, K=k, E=1)
    g = torch.Generator(device="cuda").manual_seed(0)
    xs = torch.randint(120, 134, (130, k // 32), dtype=torch.uint8, generator=g, device="cuda")
    wsc = torch.randint(120, 134, (1, n, k // 32), dtype=torch.uint8, generator=g, device="cuda")
    packed = torch.empty_like(wsc)
    moe.moe_mxfp4_pack_scales(wsc, packed)
    xc = torch.full((130, k // 2), 0x22, dtype=torch.uint8, device="cuda")
    o = torch.tensor([0, 130], dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y = torch.empty(130, n, dtype=torch.bfloat16, device="cuda")
    for grp in range(k // 32):
        wc = torch.zeros(1, n, k // 2, dtype=torch.uint8, device="cuda")
        wc[:, :, 16 * grp:16 * grp + 16] = 0x22
        moe.ragged_gemm_mxfp4(p, xc, xs, wc, packed, o, y, ws)
        want = 32 * torch.exp2(xs[:, grp].float() - 127)[:, None] * torch.exp2(
            wsc[0, :, grp].float() - 127)[None]
        assert bool((y.float() == want).all()), grp


def test_product_watchdog_and_bad_offsets(form):
    p = moe.Ragged(R=64, N=128, K=256, E=2)
    xc = torch.zeros(64, 128, dtype=torch.uint8, device="cuda")
    xs = torch.full((64, 8), 127, dtype=torch.uint8, device="cuda")
    wc = torch.zeros(2, 128, 128, dtype=torch.uint8, device="cuda")
    packed = torch.full((2, 128, 8), 127, dtype=torch.uint8, device="cuda")
    ws = torch.empty(moe.moe_ragged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y = torch.ones(64, 128, dtype=torch.bfloat16, device="cuda")
    o = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    bad = torch.tensor([0, 70, 20], dtype=torch.int32, device="cuda")

    def call(off):
        moe.ragged_gemm_mxfp4(p, xc, xs, wc, packed, off, y, ws)
        return moe.moe_status_string(moe.moe_sync_status())

    assert call(bad) == "MOE_ERR_DEVICE_BAD_INDEX"
    try:
        moe.moe_debug_set_watchdog(50_000_000, True)
        assert call(o) == "MOE_ERR_DEVICE_TIMEOUT"
    finally:
        moe.moe_debug_set_watchdog(0, False)
    assert call(o) == "MOE_OK" and bool((y == 0).all())
