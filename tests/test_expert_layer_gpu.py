"""The expert-layer example: grouped, adapter and gradient calls together.

Each stage rounds its bf16 operands and results at 2^-9 of their size and the
stages' errors add at most linearly (four of them in the longest chain, with
random signs): 1.2e-2 bounds their relative 2-norm.
"""
import importlib.util
import os

import pytest

from tests._gpu import torch_cuda

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "expert_layer.py")


@pytest.mark.parametrize("kw", [dict(), dict(tokens=3, experts=16, k=4),
                                dict(tokens=1500, model=200, hidden=264, experts=5, rank=8)])
def test_example_matches_plain_torch(kw):
    torch_cuda()
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    off = layer.main(**kw)
    assert max(off) <= 1.2e-2, off
