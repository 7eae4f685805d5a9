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
