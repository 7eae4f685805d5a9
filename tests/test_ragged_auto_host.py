"""The ragged products' default choice of form, without a GPU: past the checks
of arguments a call has to come back with a CUDA error, whatever the sizes."""
import os
import subprocess
import sys

import pytest

import mixture_experts_ffn_align_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A process of its own that sees no device: an arithmetic trap on the host ends
# it and not this one, and nothing can be launched.
CALLS = """
import ctypes, sys
import mixture_experts_ffn_align_gb300 as moe
L, P = moe.lib(), ctypes.c_void_p(4096)
for R in (1, 16, 130, 700, 8192, 1 << 22):
    for N in (128, 1024, 28672):
        for K in (128, 384, 7168):
            for E in (1, 4, 256, 1024):
                r = moe.Ragged(R=R, N=N, K=K, E=E)._ref
                for s in (L.ragged_gemm(r, P, P, None, P, P, P, 1 << 50, None),
                          L.ragged_gemm_dgrad(r, P, P, P, P, P, 1 << 50, None),
                          L.ragged_gemm_wgrad(r, P, P, P, P, 0, 0, P, 1 << 50, None),
                          L.ragged_gemm_mxfp4(r, P, P, P, P, P, P, P, 1 << 50, None)):
                    assert s == 3, (R, N, K, E, s)
print("done")
"""


@pytest.mark.parametrize("form", ["auto", "single", "pairs", "pairs_double"])
def test_every_size_reaches_the_launch(form):
    if not os.path.exists(moe.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    r = subprocess.run(
        [sys.executable, "-c",
         f"import mixture_experts_ffn_align_gb300 as m; m.moe_debug_set_bf16_gemm_form({form!r})\n"
         + CALLS],
        cwd=ROOT, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "done", (r.returncode, r.stderr[-500:])


def test_a_larger_batch_never_needs_less_workspace():
    """A workspace for the largest R serves every smaller one: the bytes do not
    fall as R grows, for bf16 and 4-bit shapes, few and many experts."""
    rows = sorted({*range(1, 1100), *range(1100, 9000, 37), *(1 << i for i in range(23)),
                   *((1 << i) + 1 for i in range(22))})
    for n, k in ((4096, 4096), (8, 4104), (264, 1032), (128, 8192), (1920, 7168), (28672, 4096),
                 (2048, 1024), (72, 72), (640, 16384), (16384, 128)):
        for e in (1, 2, 3, 8, 15, 60, 256, 1024):
            last = 0
            for r in rows:
                need = moe.moe_ragged_workspace_bytes(moe.Ragged(R=r, N=n, K=k, E=e))
                assert need >= last, (n, k, e, r, need, last)
                last = need
