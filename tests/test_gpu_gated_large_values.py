"""The gated block's gradient where h is near the largest values of its type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe
from oracle import ragged

from .test_gpu_gated import f64, form, randn, sum_error, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("alpha", [1.0, 1.702, 1e30])
def test_gradient_where_alpha_g_overflows(alpha, form):
    """g near bf16's largest value: s is 1 there and the derivative by g is u + beta, though
    alpha g is past fp32's range."""
    v = torch.tensor([3e38, -3e38, 1e30, -1e30, 1.0, -1.0, 0.0, 40.0], device="cuda")
    h = torch.cat([v.repeat(40, 9), randn((40, 72), "float16", 4).float()], 1)
    h = h.to(torch.bfloat16).contiguous()
    p = moe.Ragged(R=40, N=136, K=72, E=1)
    dy, w = randn((40, 136), "bfloat16", 1), randn((1, 136, 72), "bfloat16", 2, 0.1)
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    dh = torch.empty_like(h)
    moe.ragged_gated_dgrad(p, dy, w, h, off, dh, workspace(p), alpha=alpha)
    assert moe.moe_sync_status() == 0
    dz = ragged.dgrad(f64(dy), f64(w), np.array([0, 40]))
    want = dz * f64(h)[:, 72:]
    got = f64(dh)[:, :72]
    assert np.isfinite(got).all()
    large = np.tile(np.array([1, 0, 1, 0, 0, 0, 0, 1], bool), (40, 9))
    off_dz = sum_error(136, ragged.dgrad(abs(f64(dy)), abs(f64(w)), np.array([0, 40])))
    tol = 2.0 ** -8 * np.abs(want) * 1.001 + off_dz * np.abs(f64(h)[:, 72:]) * 1.001 \
        + 14 * 2.0 ** -23 * np.abs(want)
    assert (np.abs(got - want) <= tol)[large].all()
    low = np.tile(np.array([0, 1, 0, 1, 0, 0, 0, 0], bool), (40, 9))
    assert (got[low] == 0).all()
