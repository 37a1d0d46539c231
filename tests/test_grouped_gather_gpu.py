"""gemm_bf16_grouped with row_idx, on both sides of the rule that decides
whether the product's own loads gather the rows (M <= 16 * groups) or a copy
does.  Quarter-integer inputs: bit for bit.  Rows of the operand that no index
names hold NaN, and so does the operand's row padding.
"""
import numpy as np
import pytest

from tests._gpu import torch_cuda
from tests.test_grouped_gpu import forward64, offsets_of, quarters

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def sizes_of(kind, M, groups, rng):
    if kind == "one":                  # all rows in one group (tiles of 64 rows)
        sizes = np.zeros(groups, int)
        sizes[groups // 2] = M
        return sizes
    return np.bincount(rng.integers(0, groups, M), minlength=groups)


@pytest.mark.parametrize("M,groups", [(1, 1), (3, 64), (16, 1), (17, 1), (100, 7), (112, 7), (113, 7),
                                      (900, 64), (40, 4096)])
@pytest.mark.parametrize("kind", ["any", "one"])
@pytest.mark.parametrize("N,K", [(128, 64), (200, 1001), (520, 72)])
def test_rows_by_index(tg, M, groups, kind, N, K):
    torch = torch_cuda()
    if groups == 4096 and N * K > 20000:
        pytest.skip("weights of 4096 groups")
    gen = torch.Generator(device="cuda").manual_seed(M + groups + K)
    rng = np.random.default_rng(M + groups)
    rows = max(2, M // 3)
    A, B = quarters(gen, rows, K), quarters(gen, groups, N, K)
    idx = torch.from_numpy(rng.integers(0, max(1, rows - 1), M).astype(np.int32)).cuda()
    A[rows - 1] = float("nan")
    sizes = sizes_of(kind, M, groups, rng)
    cut, off = offsets_of(sizes)
    want, _ = forward64(torch, A, B, cut, idx)
    got = tg.gemm_bf16_grouped(A, B, off, row_idx=idx)
    assert torch.equal(got.double(), want)
    assert torch.equal(tg.gemm_bf16_grouped(A, B, off, row_idx=idx, out_dtype=torch.bfloat16),
                       got.to(torch.bfloat16))
    # Outside the operand on either side: a zero row, whatever the operand holds.
    far = idx.clone()
    out = torch.from_numpy(rng.random(M) < 0.4).cuda()
    out[0] = True
    far[out] = torch.from_numpy(rng.choice([-1, -2 ** 31, rows, rows + 5, 2 ** 31 - 1],
                                           int(out.sum())).astype(np.int32)).cuda()
    zero = tg.gemm_bf16_grouped(A, B, off, row_idx=far, epilogue_add=1.0)
    assert torch.equal(zero[~out].double(), want[~out] + 1.0)
    assert (zero[out] == 1.0).all()
    assert tg.tg_device_status()[0] == tg.TG_OK


def test_gathered_in_place_allocates_nothing(tg):
    """Once a stream has the tail scratch, few gathered rows need no more."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(1)
    A, B = quarters(gen, 50, 64), quarters(gen, 2, 64, 64)
    idx = torch.arange(32, device="cuda", dtype=torch.int32)
    cut, off = offsets_of([15, 17])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        tg.gemm_bf16_grouped(A[:32], B, off)
        before = tg.workspace_alloc_count()
        got = tg.gemm_bf16_grouped(A, B, off, row_idx=idx)
        assert tg.workspace_alloc_count() == before
    s.synchronize()
    assert torch.equal(got.double(), forward64(torch, A, B, cut, idx)[0])
