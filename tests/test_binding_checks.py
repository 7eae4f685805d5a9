"""What the Python binding of the training and 4-bit operators refuses before
anything is launched: no GPU is needed."""
import pytest

import mixture_experts_ffn_align_gb300 as moe

torch = pytest.importorskip("torch")


def codec_tensors(rows, k):
    return (torch.zeros(rows, k // 2, dtype=torch.uint8),
            torch.zeros(rows, k // 32, dtype=torch.uint8))


def overlapping(rows, k, stride):
    """[rows, k] whose rows lie `stride` < k elements apart."""
    base = torch.zeros(rows * max(stride, 1) + k, dtype=torch.bfloat16)
    return base.as_strided((rows, k), (stride, 1))


@pytest.mark.parametrize("stride", [0, 8, 56])
def test_codec_refuses_rows_that_overlap(stride):
    """An expanded row has stride 0, which the C entry points read as 'dense':
    they would go past the one row that exists."""
    codes, scales = codec_tensors(5, 64)
    with pytest.raises(ValueError, match="overlap"):
        moe.moe_mxfp4_quantize(overlapping(5, 64, stride), codes, scales)
    with pytest.raises(ValueError, match="overlap"):
        moe.moe_mxfp4_dequantize(codes, scales, overlapping(5, 64, stride))


def test_codec_takes_any_stride_of_a_single_row():
    """One row (or none) has no next row to overlap: only the device is wrong."""
    for rows in (0, 1):
        codes, scales = codec_tensors(rows, 64)
        with pytest.raises(ValueError, match="GPU"):
            moe.moe_mxfp4_quantize(overlapping(rows, 64, 0), codes, scales)
        with pytest.raises(ValueError, match="GPU"):
            moe.moe_mxfp4_dequantize(codes, scales, overlapping(rows, 64, 0))


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on cuda:<dev>; its pointer is never used."""

    @staticmethod
    def of(t, dev):
        t = t.as_subclass(OnDevice)
        t.dev = dev
        return t

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func is torch.Tensor.get_device:
            return args[0].dev
        if func == torch.Tensor.is_cuda.__get__:
            return True
        if func is torch.Tensor.data_ptr:
            return 4096
        with torch._C.DisableTorchFunctionSubclass():
            return func(*args, **(kwargs or {}))


def other_device_calls():
    """Every call of the binding, as (name, tensors -> call, tensors)."""
    bf, u8 = torch.bfloat16, torch.uint8
    p = moe.Ragged(R=16, N=128, K=128, E=2)
    n = moe.moe_ragged_workspace_bytes(p)
    x, y, w = torch.zeros(16, 128, dtype=bf), torch.zeros(16, 128, dtype=bf), torch.zeros(2, 128, 128, dtype=bf)
    b, o, ws = torch.zeros(2, 128, dtype=bf), torch.zeros(3, dtype=torch.int32), torch.zeros(n, dtype=u8)
    c, s = torch.zeros(16, 64, dtype=u8), torch.zeros(16, 4, dtype=u8)
    wc, wp = torch.zeros(2, 128, 64, dtype=u8), torch.zeros(2, 128, 4, dtype=u8)
    g, f = torch.zeros(10), torch.zeros(())
    cw = torch.zeros(moe.moe_clip_workspace_bytes(), dtype=u8)
    return [
        ("ragged_gemm", lambda x, w, o, y, ws, b: moe.ragged_gemm(p, x, w, o, y, ws, bias=b),
         (x, w, o, y, ws, b)),
        ("ragged_gemm_dgrad", lambda *t: moe.ragged_gemm_dgrad(p, *t), (y, w, o, x, ws)),
        ("ragged_gemm_wgrad", lambda *t: moe.ragged_gemm_wgrad(p, *t), (y, x, o, w, ws)),
        ("moe_mxfp4_quantize", moe.moe_mxfp4_quantize, (x, c, s)),
        ("moe_mxfp4_dequantize", moe.moe_mxfp4_dequantize, (c, s, x)),
        ("moe_mxfp4_pack_scales", moe.moe_mxfp4_pack_scales, (wp, wp.clone())),
        ("ragged_gemm_mxfp4", lambda *t: moe.ragged_gemm_mxfp4(p, *t), (c, s, wc, wp, o, y, ws)),
        ("moe_clip_grad_norm",
         lambda g, h, norm, ws, u, v: moe.moe_clip_grad_norm([g, h], 1.0, norm, ws, out=[u, v]),
         (g, g.clone(), f, cw, g.clone(), g.clone())),
    ]


@pytest.mark.skipif(torch.cuda.is_available(), reason="stand-ins for tensors of other devices")
@pytest.mark.parametrize("call", range(8))
def test_tensors_of_another_device_are_refused(call, monkeypatch):
    """Each tensor alone on cuda:1, then all of them, while cuda:0 is current."""
    monkeypatch.setattr(moe._t(), "raw_stream", lambda dev: 0)
    monkeypatch.setattr(moe._t(), "device", lambda: 0, raising=False)
    name, f, tensors = other_device_calls()[call]
    for i in range(len(tensors)):
        with pytest.raises(ValueError, match="cuda:1"):
            f(*(OnDevice.of(t.clone(), int(j == i)) for j, t in enumerate(tensors)))
    with pytest.raises(ValueError, match="current device"):
        f(*(OnDevice.of(t.clone(), 1) for t in tensors))
    with pytest.raises(moe.MoEError, match="MOE_ERR_CUDA"):      # no GPU here
        f(*(OnDevice.of(t.clone(), 0) for t in tensors))
