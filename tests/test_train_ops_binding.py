"""What the binding of the gated block and the orthogonalised update refuses before
anything is launched: no GPU is needed."""
import pytest

import mixture_experts_ffn_align_gb300 as moe

from .test_binding_checks import OnDevice, overlapping

torch = pytest.importorskip("torch")
BF, U8 = torch.bfloat16, torch.uint8
P = dict(R=16, N=128, K=64, E=2)


def gated_tensors():
    p = moe.Ragged(**P)
    ws = torch.zeros(moe.moe_ragged_workspace_bytes(p), dtype=U8)
    return p, dict(x=torch.zeros(16, 64, dtype=BF), w13=torch.zeros(2, 128, 64, dtype=BF),
                   expert_offsets=torch.zeros(3, dtype=torch.int32), z=torch.zeros(16, 64, dtype=BF),
                   workspace=ws, h=torch.zeros(16, 128, dtype=BF), bias=torch.zeros(2, 128, dtype=BF))


def grad_tensors():
    p = moe.Ragged(**P)
    ws = torch.zeros(moe.moe_ragged_workspace_bytes(p), dtype=U8)
    return p, dict(dy=torch.zeros(16, 128, dtype=BF), w2=torch.zeros(2, 128, 64, dtype=BF),
                   h=torch.zeros(16, 128, dtype=BF), expert_offsets=torch.zeros(3, dtype=torch.int32),
                   dh=torch.zeros(16, 128, dtype=BF), workspace=ws, z=torch.zeros(16, 64, dtype=BF))


def ortho_tensors():
    return None, dict(g=torch.zeros(2, 8, 24), out=torch.zeros(2, 8, 24, dtype=BF),
                      workspace=torch.zeros(moe.moe_orthogonalize_workspace_bytes(2, 8, 24), dtype=U8))


CALLS = {"gated": (gated_tensors, lambda p, **t: moe.ragged_gated(p, **t)),
         "grad": (grad_tensors, lambda p, **t: moe.ragged_gated_dgrad(p, **t)),
         "ortho": (ortho_tensors, lambda p, **t: moe.moe_orthogonalize(**t))}


@pytest.fixture
def device_zero(monkeypatch):
    """Stand-ins for tensors of cuda:0, which is current."""
    monkeypatch.setattr(moe._t(), "raw_stream", lambda dev: 0)
    monkeypatch.setattr(moe._t(), "device", lambda: 0, raising=False)


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="stand-ins for tensors on a GPU")


@no_gpu
@pytest.mark.parametrize("name", list(CALLS))
def test_shapes_types_and_strides_are_checked(name, device_zero):
    make, call = CALLS[name]
    p, t = make()

    def refused(error, key, v):
        with pytest.raises(error, match=key):
            call(p, **{k: OnDevice.of(v if k == key else x, 0) for k, x in t.items()})

    for key, v in t.items():
        if key == "workspace":
            continue
        if key != "g":                       # out follows g's shape, g any
            refused(ValueError, key, v[:-1].clone())
        refused(TypeError, key, v.to(torch.float64 if v.dtype != torch.int32 else torch.int64))
        if v.dim() > 1:                      # last dimension not contiguous
            refused(ValueError, key, v.repeat_interleave(2, -1)[..., ::2])


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_on_the_host_are_refused(name):
    make, call = CALLS[name]
    p, t = make()
    with pytest.raises(ValueError, match="GPU"):
        call(p, **t)


@pytest.mark.parametrize("name, key, cols", [("gated", "z", 64), ("grad", "h", 128),
                                             ("grad", "dh", 128)])
@pytest.mark.parametrize("stride", [0, 8])
def test_rows_that_overlap_are_refused(name, key, cols, stride):
    make, call = CALLS[name]
    p, t = make()
    with pytest.raises(ValueError, match="overlap"):
        call(p, **{**t, key: overlapping(16, cols, stride)})


def test_orthogonalize_takes_matrices_and_stacks_of_them():
    for shape in ((5,), (1, 2, 3, 4)):
        with pytest.raises(ValueError, match=r"\[E, N, K\]"):
            moe.moe_orthogonalize(torch.zeros(shape), torch.zeros(shape, dtype=BF), torch.zeros(1))


@no_gpu
@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_another_device_are_refused(name, device_zero):
    """Each tensor alone on cuda:1, then all of them, while cuda:0 is current."""
    make, call = CALLS[name]
    p, t = make()
    for i in range(len(t)):
        with pytest.raises(ValueError, match="cuda:1"):
            call(p, **{k: OnDevice.of(v.clone(), int(j == i)) for j, (k, v) in enumerate(t.items())})
    with pytest.raises(ValueError, match="current device"):
        call(p, **{k: OnDevice.of(v.clone(), 1) for k, v in t.items()})
    with pytest.raises(moe.MoEError, match="MOE_ERR_CUDA"):      # no GPU here
        call(p, **{k: OnDevice.of(v.clone(), 0) for k, v in t.items()})
