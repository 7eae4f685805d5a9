"""Coefficients and steps of the orthogonalised update as the binding passes them on, with
a stand-in for the library: no GPU is needed."""
import ctypes

import numpy as np
import pytest

import mixture_experts_ffn_align_gb300 as moe

from .test_binding_checks import OnDevice

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="stand-ins for tensors on a GPU")


@pytest.fixture
def passed(monkeypatch):
    """Calls moe_orthogonalize on stand-ins of cuda:0 and gives the coefficients that
    reach the library."""
    seen = []

    class Library:
        @staticmethod
        def moe_orthogonalize(E, N, K, g, dtype, out, steps, coefficients, *rest):
            seen.append(list((ctypes.c_float * (3 * steps)).from_address(coefficients)))
            return 0

    monkeypatch.setattr(moe._t(), "raw_stream", lambda dev: 0)
    monkeypatch.setattr(moe._t(), "device", lambda: 0, raising=False)
    monkeypatch.setattr(moe, "lib", lambda: Library)
    g, out, ws = torch.zeros(2, 8, 24), torch.zeros(2, 8, 24, dtype=torch.bfloat16), \
        torch.zeros(64, dtype=torch.uint8)

    def call(**kw):
        moe.moe_orthogonalize(*(OnDevice.of(t, 0) for t in (g, out, ws)), **kw)
        return seen.pop()

    return call


@pytest.mark.parametrize("number", [torch.tensor, np.array, np.float32, float, int])
def test_coefficients_of_one_number_each_are_read_at_every_call(passed, number):
    """Tensors and arrays without dimensions hash by identity: the values of the moment
    count, not those of an earlier call with the same objects."""
    a, b, c = (number(v) for v in (3.0, -4.0, 2.0))
    assert passed(steps=2, coefficients=(a, b, c)) == [3, -4, 2] * 2
    assert passed(steps=2, coefficients=((a, b, c), (c, b, a))) == [3, -4, 2, 2, -4, 3]
    if hasattr(a, "fill_") or isinstance(a, np.ndarray):
        a[...] = 1.5
        assert passed(steps=2, coefficients=(a, b, c)) == [1.5, -4, 2] * 2
        assert passed(steps=2, coefficients=((a, b, c), (c, b, a))) == [1.5, -4, 2, 2, -4, 1.5]


@pytest.mark.parametrize("sequence", [list, tuple, torch.tensor, np.array])
def test_sequences_of_any_kind(passed, sequence):
    three, steps = [1.0, 2.0, 3.0], [[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]]
    assert passed(steps=2, coefficients=sequence(three)) == three * 2
    assert passed(steps=2, coefficients=sequence(steps)) == [1, 2, 3, 4, 5, 6]
    assert passed(steps=2, coefficients=[sequence(s) for s in steps]) == [1, 2, 3, 4, 5, 6]
    assert passed(steps=2, coefficients=tuple(sequence(s) for s in steps)) == [1, 2, 3, 4, 5, 6]


def test_sequences_that_are_read_once(passed):
    steps = ((1.0, 2.0, 3.0), (4.0, 5.0, 6.0))
    assert passed(steps=2, coefficients=iter(steps)) == [1, 2, 3, 4, 5, 6]
    assert passed(steps=2, coefficients=(iter(s) for s in steps)) == [1, 2, 3, 4, 5, 6]
    assert passed(steps=2, coefficients=iter(steps[0])) == [1, 2, 3] * 2
    with pytest.raises(ValueError, match="coefficients"):
        passed(steps=1, coefficients=iter(steps))


def test_default_and_longest(passed):
    f = np.float32([3.4445, -4.7750, 2.0315]).tolist()
    assert passed() == f * 5
    assert passed(steps=64) == f * 64


@pytest.mark.parametrize("steps", [-1, 0, 65, 1 << 32, (1 << 32) + 5, 1 << 60])
def test_step_counts_are_refused_before_anything_is_laid_out(passed, steps):
    """A count past 32 bits would wrap to another one, a huge one fill the memory."""
    with pytest.raises(ValueError, match="steps"):
        passed(steps=steps)


@pytest.mark.parametrize("bad", [(1.0, 2.0), (), ((1.0, 2.0),) * 5, ((1.0, 2.0, 3.0),) * 4])
def test_wrong_numbers_of_coefficients(passed, bad):
    with pytest.raises(ValueError, match="coefficients"):
        passed(coefficients=bad)
