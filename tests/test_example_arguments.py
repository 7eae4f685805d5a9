"""The fine-tuning example's arguments, refused before anything runs on a GPU."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")


def test_an_unknown_update_is_refused():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "finetune_experts.py")
    spec = importlib.util.spec_from_file_location("finetune_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for bad in ("orthogonalise", "Plain", ""):
        with pytest.raises(ValueError, match="update"):
            m.main(steps=1, update=bad)
