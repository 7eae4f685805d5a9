"""The orthogonalised update's launch over the whole grid where the GPU has fewer SMs for it
than the device: smaller grids, and one that CUDA refuses."""
import pytest

torch = pytest.importorskip("torch")
import mixture_experts_ffn_align_gb300 as moe

from .test_gpu_orthogonalize import call, check, gradient

pytestmark = pytest.mark.gpu
MANY = 1 << 20            # CTAs: more than any GPU runs at once


@pytest.fixture
def grid():
    """Sets the form and the CTAs of the whole grid's launch."""
    def use(form, ctas):
        moe.moe_debug_set_bf16_gemm_form(form)
        moe.moe_debug_set_grid_ctas(ctas)
    yield use
    use("auto", 0)


@pytest.mark.parametrize("ctas", [1, 2, 7, 64])
@pytest.mark.parametrize("shape", [(3, 300, 200), (12, 140, 270)], ids=str)
def test_smaller_grids_give_the_same(ctas, shape, grid):
    g = gradient(shape, "bfloat16", 5)
    grid("whole_grid", 0)
    want = call(g)
    grid("whole_grid", ctas)
    got = call(g)
    assert torch.equal(got, want)
    check(got, g)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_a_refused_grid_runs_as_products(dtype, grid):
    """64 matrices of 300 x 520 are more tiles a product than a GPU has SMs."""
    g = gradient((64, 300, 520), dtype, 5)
    grid("whole_grid", MANY)
    got = call(g)
    check(got[:2], g[:2])
    grid("auto", MANY)            # a size that takes the whole grid by itself
    other = call(g)
    check(other[:2], g[:2])
    grid("auto", 0)
    after = call(g)
    check(after[:2], g[:2])
    assert moe.moe_sync_status() == 0


def test_a_refused_grid_in_a_graph(grid):
    g = gradient((64, 300, 520), "bfloat16", 6)
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(*g.shape), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(g)
    grid("whole_grid", MANY)
    moe.moe_orthogonalize(g, out, ws)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out, ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    assert moe.moe_sync_status() == 0
