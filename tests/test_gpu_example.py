"""The fine-tuning example: its loss falls, and the 4-bit layer is the bf16 one
up to the quantisation's error.

E2M1 rounds a value by at most half a step, 1/8 to 1/4 of its binade's start; on
the scaled values of a group that is about 0.1 rms, independent from value to
value, so each quantised operand adds some 0.1 of a product's rms.  Two products
with two (W4A4) or one (W4A8) operand in four bits: 0.2 and 0.15, the activation
between them amplifying by less than two."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_finetune_experts():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "finetune_experts.py")
    spec = importlib.util.spec_from_file_location("finetune_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(steps=60, verbose=False)
    assert all(n == n and n > 0 for n in r["norms"])
    assert r["losses"][-1] < 0.7 * r["losses"][0]
    assert r["w4a4"] < 0.4 and r["w4a8"] < 0.3
