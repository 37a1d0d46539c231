"""Lengths of zero at widths that take the kernels' wide loads (two 64-element
chunks a box), and row plans far above one chunk per SM."""
import numpy as np
import pytest

from tests._gpu import torch_cuda
from tests.test_group_rows_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("N,K", [(128, 256), (300, 520), (1000, 130)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_nothing_to_contract(tg, N, K, out):
    torch = torch_cuda()
    bf = torch.bfloat16
    dt = torch.float32 if out == "f32" else bf
    empty = lambda *shape: torch.empty(*shape, dtype=bf, device="cuda")  # noqa: E731
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    off = torch.tensor([5, 5, 300, 640], dtype=torch.int32, device="cuda")
    # No rows: every group's gradient is zero.
    dW = torch.full((3, N, -(-K // 8) * 8), float("nan"), device="cuda", dtype=dt)[..., :K]
    tg.gemm_bf16_grouped_wgrad(empty(0, N), empty(0, K), zero, dW)
    assert (dW == 0).all()
    # Rows, none of them in a group, and a width of zero to sum over.
    G = torch.randn(700, -(-N // 8) * 8, device="cuda").to(bf)[:, :N]
    assert (tg.gemm_bf16_grouped_wgrad(G, empty(700, -(-K // 8) * 8).zero_()[:, :K], zero + 9,
                                       out_dtype=dt) == 0).all()
    assert (tg.gemm_bf16_grouped_dgrad(empty(700, 0), empty(3, 0, K), off, out_dtype=dt) == 0).all()
    got = tg.gemm_bf16_grouped(empty(700, 0), empty(3, N, 0), off, epilogue_add=2.0, out_dtype=dt)
    assert (got[5:640] == 2).all() and (got[:5] == 0).all() and (got[640:] == 0).all()
    few = torch.tensor([0, 1, 1, 3], dtype=torch.int32, device="cuda")
    idx = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = tg.gemm_bf16_grouped(empty(4, 0), empty(3, N, 0), few, row_idx=idx, epilogue_add=2.0,
                               out_dtype=dt)
    assert (got[:3] == 2).all() and (got[3:] == 0).all()
    assert tg.tg_device_status()[0] == tg.TG_OK


# 152 SMs x 2048 rows are 311296: above that the chunk of a warp grows.
@pytest.mark.parametrize("n", [311296, 311297, 1000003, 4200000])
@pytest.mark.parametrize("groups", [1, 64, 256, 4096])
def test_long_row_plans(tg, n, groups):
    rng = np.random.default_rng(n + groups)
    check(tg, rng.integers(-2, groups + 3, n), groups)
