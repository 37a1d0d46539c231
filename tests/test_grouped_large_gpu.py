"""Grouped and adapter calls on arrays of more than 2^31 elements: weights, rows,
results and adapters.  What is far from the start is compared bit for bit
(quarter integers); the rest of a large operand is zero.
"""
import pytest

from tests._gpu import torch_cuda
from tests.test_grouped_gpu import quarters

pytestmark = pytest.mark.gpu

BIG = 2 ** 31


@pytest.fixture(scope="module")
def tg():
    torch = torch_cuda()
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    yield m
    torch.cuda.empty_cache()


def gen_of(seed):
    return torch_cuda().Generator(device="cuda").manual_seed(seed)


def offsets(*cut):
    torch = torch_cuda()
    return torch.tensor(cut, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("M", [9, 2000])
def test_weights_past_32_bits(tg, M):
    """The first and the last of 36 experts of 8192 x 8192; few rows and many."""
    torch = torch_cuda()
    gen, groups, N, K = gen_of(M), 36, 8192, 8192
    B = torch.zeros(groups, N, K, device="cuda", dtype=torch.bfloat16)
    assert B.numel() > BIG
    B[0], B[-1] = quarters(gen, N, K), quarters(gen, N, K)
    A, G = quarters(gen, M, K), quarters(gen, M, N)
    a = M // 3
    off = offsets(*([0] + [a] * (groups - 1) + [M]))
    want = torch.cat([A[:a].double() @ B[0].double().T, A[a:].double() @ B[-1].double().T])
    assert torch.equal(tg.gemm_bf16_grouped(A, B, off).double(), want)
    idx = torch.arange(M, device="cuda", dtype=torch.int32)
    assert torch.equal(tg.gemm_bf16_grouped(A, B, off, row_idx=idx).double(), want)
    want = torch.cat([G[:a].double() @ B[0].double(), G[a:].double() @ B[-1].double()])
    assert torch.equal(tg.gemm_bf16_grouped_dgrad(G, B, off).double(), want)
    for dt in (torch.float32, torch.bfloat16):
        B = None
        dB = tg.gemm_bf16_grouped_wgrad(G, A, off, out_dtype=dt)
        assert torch.equal(dB[0].double(), (G[:a].double().T @ A[:a].double()).to(dt).double())
        assert torch.equal(dB[-1].double(), (G[a:].double().T @ A[a:].double()).to(dt).double())
        assert not dB[1:-1].any()
        dB = None
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_rows_past_32_bits(tg, out):
    """270000 rows of 8192 results, and of 8192 operand values."""
    torch = torch_cuda()
    dt = torch.float32 if out == "f32" else torch.bfloat16
    gen, M, W, S = gen_of(1), 270000, 8192, 72
    assert M * W > BIG
    off = offsets(0, 100000, 100000, M - 5)
    A, B = quarters(gen, M, S), quarters(gen, 3, W, S)
    pick = torch.cat([torch.arange(0, M, 9973, device="cuda"), torch.arange(M - 300, M, device="cuda")])
    group = (pick >= 100000).long() * 2

    def check(D, rows, weights):
        want = torch.einsum("ik,ink->in", rows[pick].double(), weights[group].double())
        want[pick >= M - 5] = 0
        assert torch.equal(D[pick].double(), want.to(dt).double())

    check(tg.gemm_bf16_grouped(A, B, off, out_dtype=dt), A, B)
    Bt = quarters(gen, 3, S, W)
    check(tg.gemm_bf16_grouped_dgrad(A, Bt, off, out_dtype=dt), A, Bt.transpose(1, 2))
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    ids[100000:], ids[M - 5:] = 1, -1
    down, up = quarters(gen, 2, 16, S), quarters(gen, 2, W, 16)
    D = tg.gemm_bf16_lora(A, B[0], ids, down, up, out_dtype=dt)
    own = ids[pick].clamp(0).long()
    h = torch.einsum("ik,irk->ir", A[pick].double(), down[own].double())
    h[pick >= M - 5] = 0
    want = A[pick].double() @ B[0].double().T + torch.einsum("ir,inr->in", h, up[own].double())
    assert torch.equal(D[pick].double(), want.to(dt).double())
    # Wide operands: rows of 8192 to contract.
    D = None
    X = torch.zeros(M, W, device="cuda", dtype=torch.bfloat16)
    X[pick] = quarters(gen, len(pick), W)
    V = quarters(gen, 3, S, W)
    check(tg.gemm_bf16_grouped(X, V, off, out_dtype=dt), X, V)
    order = torch.arange(M - 1, -1, -1, device="cuda", dtype=torch.int32)
    D = tg.gemm_bf16_grouped(X, V, off, row_idx=order, out_dtype=dt)
    check(D, X.flip(0), V)
    D = tg.gemm_bf16_grouped_wgrad(A, X, off, out_dtype=dt)
    for g, (lo, hi) in enumerate([(0, 100000), (100000, 100000), (100000, M - 5)]):
        inside = pick[(pick >= lo) & (pick < hi)].unique()
        want = A[inside].double().T @ X[inside].double()
        assert torch.equal(D[g].double(), want.to(dt).double())
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("M", [8, 100, 600, 3000])
def test_adapters_past_32_bits(tg, M):
    torch = torch_cuda()
    gen, N, K, rank, adapters = gen_of(2), 8192, 8192, 128, 2100
    down = torch.zeros(adapters, rank, K, device="cuda", dtype=torch.bfloat16)
    up = torch.zeros(adapters, N, rank, device="cuda", dtype=torch.bfloat16)
    assert down.numel() > BIG and up.numel() > BIG
    for t in (0, adapters - 1):
        # Few terms: the rank values fit two bf16 terms.
        down[t, :, 5000:5064], up[t] = quarters(gen, rank, 64), quarters(gen, N, rank)
    A, B = quarters(gen, M, K), quarters(gen, N, K)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    ids[M // 3:], ids[-1] = adapters - 1, adapters
    want = A.double() @ B.double().T
    for t in (0, adapters - 1):
        at = torch.nonzero(ids == t).flatten()
        want[at] += (A[at].double() @ down[t].double().T) @ up[t].double().T
    for dt in (torch.float32, torch.bfloat16):
        got = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt)
        assert torch.equal(got.double(), want.to(dt).double())
    assert tg.tg_device_status()[0] == tg.TG_OK
