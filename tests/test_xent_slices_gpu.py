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


@pytest.mark.parametrize("M,N,K", [(150, 20011, 300), (9001, 300, 72), (7000, 3001, 33)])
@pytest.mark.parametrize("f32", [False, True])
def test_captured_into_given_rows_with_what_it_asks_for(tg, M, N, K, f32):
    """On a stream that has the bytes the call asks for and no more, into results whose
    rows lie apart, replayed while another stream makes the same call: the eager bits, and
    what lies between the rows stays."""
    import torch
    A, B, t, grad = inputs(M + K, M, N, K)
    _, lse = tg.gemm_bf16_xent(A, B, t)
    dtype = torch.float32 if f32 else torch.bfloat16
    want = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, out_dtype=dtype)
    ld = -(-K // 8) * 8 + 8
    dA, dB = (torch.full((n, ld), 7.0, device="cuda", dtype=dtype) for n in (M, N))
    s = torch.cuda.Stream()
    need = tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_XENT_GRAD, M, N, K,
                              d_dtype=tg.TG_D_F32 if f32 else tg.TG_D_BF16)
    tg.reserve_workspace(need, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tg.gemm_bf16_xent_grad(A, B, t, lse, grad, dA[:, :K], dB[:, :K])
    for _ in range(3):
        with torch.cuda.stream(s):
            graph.replay()
        other = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, out_dtype=dtype)
    torch.cuda.synchronize()
    for got, tall, ref in zip(other, (dA, dB), want):
        assert torch.equal(got, ref) and torch.equal(tall[:, :K], ref)
        assert (tall[:, K:] == 7).all()
