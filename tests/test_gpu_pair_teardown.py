"""Launches on SM pairs end, however they follow one another.

A CTA of a pair may not end before the other's last signals to its barriers
have landed (commits that arrive in both CTAs, remote arrivals), so each waits
for them.  The calls here are short ones, in which a kernel's end is most of
its time: alone on an idle GPU, and many in a row on two streams."""
import pytest
import torch

import mixture_experts_ffn_align_gb300 as moe
from moe_synth import make_inputs

from .gpu_util import bf16_gemm_form
from .test_gpu_watchdog import CASES

pytestmark = pytest.mark.gpu


def _call(cfg, d):
    """The fused forward into the returned tensor, without allocations."""
    mx = cfg.quant in ("mxfp4", "mxfp8")
    p = moe.Problem.from_config(cfg, weight_scales_prepacked=True) if mx else \
        moe.Problem.from_config(cfg)
    s13, s2 = d["w13_scale"], d["w2_scale"]
    if mx:
        q = moe.Problem.from_config(cfg)
        s13, s2 = (torch.empty(moe.moe_prepacked_scale_bytes(q, i), dtype=torch.uint8,
                               device="cuda") for i in (0, 1))
        moe.moe_prepack_weights(q, d["w13_scale"], d["w2_scale"], s13, s2)
    ws = torch.empty(moe.moe_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(d["x"])

    def call():
        moe.fused_experts(p, d["x"], d["w13"], s13, d["w2"], s2, d["topk_weights"],
                          d["topk_ids"], y, ws)
    return call, y


@pytest.mark.parametrize("name", list(CASES))
def test_lone_calls_end(name):
    cfg = CASES[name]
    with bf16_gemm_form("pairs"):
        call, y = _call(cfg, make_inputs(cfg, "cuda"))
        call()
        assert moe.moe_sync_status() == 0
        first = y.clone()
        for _ in range(300):
            y.zero_()
            torch.cuda.synchronize()
            call()
            torch.cuda.synchronize()
            assert torch.equal(y, first)
        assert moe.moe_sync_status() == 0


@pytest.mark.parametrize("name", list(CASES))
def test_calls_in_a_row_end(name):
    cfg = CASES[name]
    d = make_inputs(cfg, "cuda")
    with bf16_gemm_form("pairs"):
        calls = [_call(cfg, d) for _ in range(2)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in calls]
        for _ in range(200):
            for (call, _), stream in zip(calls, streams):
                with torch.cuda.stream(stream):
                    call()
        torch.cuda.synchronize()
        assert moe.moe_sync_status() == 0
        assert torch.equal(calls[0][1], calls[1][1])
