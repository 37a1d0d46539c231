"""The training step of the expert-layer example: token rows, router balance, experts
and the vocabulary loss together, with the gradients of all weights (the table's from
both of its uses), against autograd in 64 bits.

Widths whose square root is a power of two make the token rows exact.  From them the
longest chain rounds six operands to bf16, at 2^-9 of their size in the mean, and each
enters its product beside exact weights: 6 2^-9 = 1.2e-2 of the 2-norm.  The router's
gradient is a difference of two such sums of similar size: twice that.
"""
import importlib.util
import os

import pytest

from tests._gpu import torch_cuda

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "expert_layer.py")


@pytest.fixture(scope="module")
def layer():
    torch_cuda()
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kw", [
    dict(), dict(tokens=5, model=64, hidden=40, experts=4, k=4, vocabulary=33),
    dict(tokens=2000, model=256, hidden=264, experts=16, k=3, vocabulary=12345),
    dict(tokens=700, model=1024, hidden=200, experts=5, k=1, vocabulary=30000, balance=1.0)])
def test_step_matches_autograd(layer, kw):
    off = layer.main_step(**kw)
    assert off[0] <= 4e-3, off          # the loss: a mean of logits of that error
    assert off[1] <= 1.2e-2 and off[2] <= 2.4e-2 and max(off[3:]) <= 1.2e-2, off


def test_step_in_a_graph(layer):
    """Captured on a reserved stream and replayed on other tokens, it gives what the
    eager step gives for those, bit for bit."""
    import torch
    tg = layer.tg
    gen = torch.Generator(device="cuda").manual_seed(3)
    tokens, model, hidden, experts, k, vocabulary = 500, 256, 136, 6, 2, 3000
    weight = lambda *s: (torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
                         * s[-1] ** -0.5).to(torch.bfloat16)
    w = (weight(vocabulary, model), weight(experts, model), weight(experts, hidden, model),
         weight(experts, model, hidden))
    ids, targets = (torch.randint(-1, vocabulary, (2, tokens), generator=gen, device="cuda",
                                  dtype=torch.int32) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tg.reserve_workspace(64 << 20, stream=s)
    with torch.cuda.stream(s):
        want = [layer.step(ids[i], targets[i], *w, k) for i in range(2)]
    s.synchronize()
    count = tg.workspace_alloc_count()
    now, aim = ids[0].clone(), targets[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = layer.step(now, aim, *w, k)
    for i in (0, 1, 0):
        now.copy_(ids[i])
        aim.copy_(targets[i])
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])
        assert all(torch.equal(a, b) for a, b in zip(got[3], want[i][3]))
    assert tg.workspace_alloc_count() == count
