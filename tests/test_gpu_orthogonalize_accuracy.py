"""The orthogonalised update's error over the values that the library takes, against the
fp64 oracle, with the tolerances of test_gpu_orthogonalize.py."""
import pytest

torch = pytest.importorskip("torch")

from .test_gpu_orthogonalize import DT, call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape", [(1, 48, 64), (2, 140, 300), (1, 3, 7), (1, 60, 33)], ids=str)
def test_sums_of_squares_past_fp32(shape, dtype):
    """Each square is below fp32's largest value, a sum of 32 of them is not."""
    u = torch.rand(shape, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    g = ((2 * u - 1) * 1.8e19).to(DT[dtype])
    check(call(g), g)
