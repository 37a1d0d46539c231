"""tg_group_rows against numpy's stable sort: whole numbers, compared exactly."""
import numpy as np
import pytest

from tests._gpu import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def check(tg, ids, groups):
    torch = torch_cuda()
    offsets, order, slot = (t.cpu().numpy() for t in
                            tg.group_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), groups))
    key = np.where((ids >= 0) & (ids < groups), ids, groups)
    want = np.argsort(key, kind="stable")
    assert np.array_equal(order, want)
    assert np.array_equal(offsets, np.searchsorted(key[want], np.arange(groups + 1)))
    assert np.array_equal(slot[order], np.arange(len(ids)))


# Around a warp's step, the single-CTA limit and the chunk sizes; one group,
# groups around the widths of a warp and a block, and the most there are.
@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 257, 4096, 4097, 8193, 70001])
@pytest.mark.parametrize("groups", [1, 31, 32, 64, 1024, 1500, 4096])
def test_random_ids(tg, n, groups):
    rng = np.random.default_rng(n + groups)
    ids = rng.integers(-2, groups + 3, n)
    check(tg, ids, groups)


@pytest.mark.parametrize("n", [5000, 300000])
def test_skewed_sorted_and_extreme_ids(tg, n):
    rng = np.random.default_rng(n)
    check(tg, np.zeros(n, np.int64), 8)                        # one group takes all
    check(tg, np.full(n, -1), 8)                               # no row in any group
    check(tg, np.sort(rng.integers(0, 256, n)), 256)
    check(tg, np.sort(rng.integers(0, 256, n))[::-1].copy(), 256)
    ids = rng.integers(0, 16, n)
    ids[::7] = 2 ** 31 - 1
    ids[::11] = -2 ** 31
    check(tg, ids, 16)


def test_capture_and_streams(tg):
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    ids = torch.from_numpy(rng.integers(0, 64, 20000).astype(np.int32)).cuda()
    tg.group_rows(ids, 64)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        tg.reserve_workspace(tg.workspace_bytes(tg.TG_CALL_GROUP_ROWS, 20000, 64, 1))
        with torch.cuda.graph(g, stream=s):
            out = tg.group_rows(ids, 64)
    ids.copy_(torch.from_numpy(rng.integers(0, 64, 20000).astype(np.int32)).cuda())
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want = tg.group_rows(ids, 64)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
