"""The orthogonalised update's workspace against what the header states, on the CPU."""
import os

import pytest

import mixture_experts_ffn_align_gb300 as moe


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(moe.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()


def up(v):
    return (v + 63) // 64 * 64


@pytest.mark.parametrize("shape", [(64, 128, 4096), (8, 64, 64), (1024, 9, 5), (1, 1, 1), (256, 16, 2048),
                                   (1, 128, 1 << 18), (3, 77, 128), (2, 130, 2000), (1, 512, 256),
                                   (1, 4096, 14336), (8, 512, 256), (7, 1056, 1000), (2, 2048, 2048),
                                   (1024, 130, 130), (16, 7168, 2048), (300, 200, 4000),
                                   (610, 80, 13623), (321, 10503, 246)], ids=str)
def test_bytes_are_those_stated(shape):
    E, N, K = shape
    m, M = sorted((N, K))
    need = moe.moe_orthogonalize_workspace_bytes(E, N, K)
    assert need == moe.moe_orthogonalize_workspace_bytes(E, K, N)
    x, a = E * m * up(M), E * m * up(m)
    more = max(20 << 20, E << 19) + (1 << 20)   # sums of slices; of squares, counters, alignment
    if m <= 128 or E == 1:
        assert 8 * (x + a) <= need <= 8 * (x + a) + more
    else:
        assert 6 * x + 4 * a <= need <= 6 * x + 4 * a + (32 << 20) + more
        # one matrix at least with both parts
        assert need >= 8 * (x + a) // E
