"""The same grouped or adapter call returns the same bits, in a captured graph as
outside, once the stream has the tail scratch; and results that the calls
allocate have rows on 16-byte boundaries.

Sizes whose contractions are split between units, so that the order of the sums
depends on the scratch.
"""
import numpy as np
import pytest

from tests._gpu import torch_cuda
from tests.test_grouped_gpu import forward64, normal, offsets_of, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def calls(tg, torch, out):
    """Forward (few rows, pairs), both gradients, adapters for few rows and many."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    few, few_off = offsets_of([3, 1, 2])
    many, off = offsets_of([500, 900])
    x, X, G = normal(gen, 6, 4096), normal(gen, 1400, 6200), normal(gen, 1400, 264)
    w, W = normal(gen, 3, 128, 4096), normal(gen, 2, 264, 6200)
    long, long_off = offsets_of([7000])
    gl, xl = normal(gen, 7000, 300), normal(gen, 7000, 264)
    ids = torch.from_numpy(np.repeat(np.arange(5), 280).astype(np.int32)).cuda()
    down, up = normal(gen, 5, 24, 6200), normal(gen, 5, 264, 24)
    kw = dict(out_dtype=out)
    return few, (x, w), lambda: [
        tg.gemm_bf16_grouped(x, w, few_off, **kw), tg.gemm_bf16_grouped(X, W, off, **kw),
        tg.gemm_bf16_grouped_dgrad(G, W, off, **kw),
        tg.gemm_bf16_grouped_wgrad(gl, xl, long_off, **kw),
        tg.gemm_bf16_lora(X[:40], W[0], ids[:40], down, up, **kw),
        tg.gemm_bf16_lora(X, W[0], ids, down, up, **kw)]


@pytest.mark.parametrize("reserve", [False, True])
def test_a_graph_returns_the_bits_of_the_call(tg, reserve):
    torch = torch_cuda()
    for out in (torch.float32, torch.bfloat16):
        _, _, run = calls(tg, torch, out)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            if reserve:
                tg.reserve_workspace(tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_LORA, 1400, 24, 1))
            else:
                first = run()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got = run()
            g.replay()
            if reserve:
                first = run()
            s.synchronize()
        for a, b in zip(first, got):
            assert torch.equal(a, b)


def test_captured_without_scratch_the_result_is_as_good(tg):
    torch = torch_cuda()
    cut, (x, w), _ = calls(tg, torch, torch.float32)
    _, off = offsets_of([3, 1, 2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):           # on a stream of its own
        got = tg.gemm_bf16_grouped(x, w, off)
    g.replay()
    torch.cuda.synchronize()
    ref, mag = forward64(torch, x, w, cut)
    assert within(torch, got, ref, mag)


@pytest.mark.parametrize("width", [8, 12, 13, 100])
def test_allocated_results_start_rows_on_16_bytes(tg, width):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(1)
    A, B = normal(gen, 5, 16), normal(gen, 2, width, 16)
    _, off = offsets_of([2, 3])
    for dt, size in ((torch.float32, 4), (torch.bfloat16, 2)):
        D = tg.gemm_bf16_grouped(A, B, off, out_dtype=dt)
        assert D.shape == (5, width) and D.stride(1) == 1
        assert D.stride(0) * size % 16 == 0 and D.stride(0) - width < 16 // size
        assert torch.equal(D.reshape(-1), D.contiguous().view(-1))
