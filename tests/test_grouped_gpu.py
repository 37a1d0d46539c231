"""GPU parity of the grouped products (gemm_bf16_grouped, _dgrad, _wgrad) with
their definitions in float64.

Quarter-integer inputs make every partial sum exact in f32, so f32 results
must equal the definition bit for bit whatever the order of the sums; that
covers layouts, ragged edges and masks.  Normal inputs are held to the
product's bound, rtol * sum |a b| + atol (tests/_gpu.py).  Rows that no
result may depend on (other groups, padding, rows in no group) hold NaN.
"""
import numpy as np
import pytest

from tests._gpu import (BF16_ATOL, BF16_RTOL, F32_ATOL, F32_RTOL, torch_cuda)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def quarters(gen, *shape):
    """bf16 quarter integers in [-1, 1] on rows of a 16-byte stride; the
    padding holds NaN."""
    torch = torch_cuda()
    width = -(-shape[-1] // 8) * 8
    t = torch.full((*shape[:-1], width), float("nan"), device="cuda", dtype=torch.bfloat16)
    t[..., :shape[-1]] = torch.randint(-4, 5, shape, generator=gen, device="cuda").float() / 4
    return t[..., :shape[-1]]


def normal(gen, *shape):
    torch = torch_cuda()
    width = -(-shape[-1] // 8) * 8
    t = torch.randn(*shape[:-1], width, generator=gen, device="cuda").to(torch.bfloat16)
    return t[..., :shape[-1]]


def offsets_of(sizes, first=0):
    torch = torch_cuda()
    cut = np.concatenate([[0], np.cumsum(sizes)]) + first
    return cut, torch.from_numpy(cut.astype(np.int32)).cuda()


def nan_rows(torch, t, lo, hi):
    t[:lo] = float("nan")
    t[hi:] = float("nan")


def forward64(torch, A, B, cut, rows=None):
    """The product, and sum |a b|, in float64; rows in no group zero."""
    if rows is not None:
        A = A[rows.long()]
    D = torch.zeros(A.shape[0], B.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(D)
    for g in range(len(cut) - 1):
        s = slice(int(cut[g]), int(cut[g + 1]))
        D[s] = A[s].double() @ B[g].double().T
        mag[s] = A[s].double().abs() @ B[g].double().abs().T
    return D, mag


def same(torch, got, want):
    return torch.equal(got.double(), want)


def within(torch, got, ref, mag):
    bf16 = got.dtype == torch.bfloat16
    tol = (BF16_RTOL if bf16 else F32_RTOL) * mag + (BF16_ATOL if bf16 else F32_ATOL)
    assert torch.isfinite(got).all()
    return float(((got.double() - ref).abs() / tol).max()) <= 1.0


# Sizes of the groups: empty ones first, last and between; one row; the tile
# sizes and one beyond; more groups than one warp holds.
SIZES = [
    [5],
    [0, 1, 0],
    [256, 0, 257, 31, 32, 33],
    [300, 700, 513],
    [1] * 40 + [0] * 3 + [2, 130],
    [3, 0] * 50 + [600],
]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}groups{sum(s)}rows")
@pytest.mark.parametrize("nk", [(8, 8), (130, 72), (257, 130), (999, 321)])
@pytest.mark.parametrize("first,after", [(0, 0), (3, 5)])
def test_all_three_exact(tg, sizes, nk, first, after):
    torch = torch_cuda()
    N, K = nk
    gen = torch.Generator(device="cuda").manual_seed(N + len(sizes))
    cut, off = offsets_of(sizes, first)
    M, groups = int(cut[-1]) + after, len(sizes)
    A, G = quarters(gen, M, K), quarters(gen, M, N)
    B = quarters(gen, groups, N, K)
    nan_rows(torch, A, first, int(cut[-1]))
    nan_rows(torch, G, first, int(cut[-1]))
    D = tg.gemm_bf16_grouped(A, B, off)
    want, _ = forward64(torch, A, B, cut)
    assert same(torch, D, want)
    dA = tg.gemm_bf16_grouped_dgrad(G, B, off)
    assert same(torch, dA, forward64(torch, G, B.transpose(1, 2), cut)[0])
    dB = tg.gemm_bf16_grouped_wgrad(G, A, off)
    for g in range(groups):
        s = slice(int(cut[g]), int(cut[g + 1]))
        assert same(torch, dB[g], G[s].double().T @ A[s].double()), g
    # bf16 results are the f32 ones, rounded once.
    bf = torch.bfloat16
    assert torch.equal(tg.gemm_bf16_grouped(A, B, off, out_dtype=bf), D.to(bf))
    assert torch.equal(tg.gemm_bf16_grouped_dgrad(G, B, off, out_dtype=bf), dA.to(bf))
    assert torch.equal(tg.gemm_bf16_grouped_wgrad(G, A, off, out_dtype=bf), dB.to(bf))
    assert tg.tg_device_status()[0] == tg.TG_OK
