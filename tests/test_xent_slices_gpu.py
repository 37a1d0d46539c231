"""The vocabulary loss's gradients where their contractions are cut into slices: few
columns of the operands, few rows, or both; the tolerances of tests/test_xent_gpu.py."""
import pytest

from tests._gpu import torch_cuda
from tests.test_xent_gpu import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("M,N,K", [
    (1, 69040, 149), (10, 55616, 320), (202, 60448, 384), (2259, 1281, 392), (640, 9912, 1546),
    (300, 33333, 7), (257, 1029, 256),        # the vocabulary
    (9001, 300, 72), (20000, 130, 257), (5181, 23, 179),    # the rows
    (7000, 3001, 33)])                                       # both
def test_sliced_contractions(tg, M, N, K):
    check(tg, *inputs(M + N + K, M, N, K))


@pytest.mark.parametrize("M,N,K", [(5181, 23373, 179), (17000, 16640, 40), (30000, 9001, 129)])
def test_slices_of_pieces(tg, M, N, K):
    """Several pieces of the vocabulary, the sums of each added to the slices'."""
    check(tg, *inputs(M, M, N, K, ignored=0.5))


def test_nan_rows_stay_in_their_row(tg):
    """With slices a row's NaN reaches its own gradient and the table's, no other row."""
    import torch
    A, B, t, grad = inputs(3, 140, 30011, 72, ignored=0.0)
    A[17] = float("nan")
    _, lse = tg.gemm_bf16_xent(A, B, t)
    for dtype in (torch.bfloat16, torch.float32):
        dA, dB = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, out_dtype=dtype)
        assert torch.isnan(dA[17]).all() and torch.isnan(dB).all()
        rest = torch.cat((dA[:17], dA[18:]))
        assert torch.isfinite(rest).all()
