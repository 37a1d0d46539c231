"""Infinite and NaN weights of `up` in gemm_bf16_lora: rows of their adapter get
what the definition gives (an infinity of the rank value's sign, NaN where the
rank value is zero), in every form of the call and whatever rows share a tile.

Quarter-integer inputs with few terms: the rank values are exact in two bf16
terms, and everything finite is compared bit for bit.
"""
import pytest

from tests._gpu import torch_cuda
from tests.test_grouped_gpu import quarters
from tests.test_lora_forms_gpu import WIDE, plan
from tests.test_lora_gpu import case, definition

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def same(torch, got, want):
    return bool(((got == want) | (torch.isnan(got) & torch.isnan(want))).all())


# Tiles of 64 and 128 columns, single CTAs over many rows, CTA pairs.
@pytest.mark.parametrize("M,N", [(5, 264), (40, 264), (100, 264), (300, 264), (300, WIDE[300]),
                                 (700, WIDE[700]), (2300, WIDE[2300])])
@pytest.mark.parametrize("kind", ["one", "requests", "any", "runs"])
@pytest.mark.parametrize("rank", [8, 24, 64, 136])
def test_infinite_weights_give_what_the_definition_gives(tg, M, N, kind, rank):
    torch = torch_cuda()
    K, adapters = 136, 4
    inf, nan = float("inf"), float("nan")
    gen = torch.Generator(device="cuda").manual_seed(M + rank)
    A, B, down, up = case(gen, quarters, M, N, K, adapters, rank)
    down[..., 64:] = 0
    ids = plan(kind, M, adapters, M)
    # One, two of one sign, two of different signs, next to a NaN; in every 128
    # columns, at both ends of the rank.
    for n in list(range(3, N, 128)) + [N - 1]:
        up[:, n, 0] = inf
        up[:, n - 1, rank - 1] = -inf
        up[1, n - 2, [1, rank - 2]] = inf
        up[2, n - 2, 1], up[2, n - 2, 2] = inf, -inf
        up[3, n - 2, 3] = nan
    want, _, _ = definition(torch, A, B, ids, down, up, None)
    if kind != "any" or M > 40:
        assert torch.isinf(want).any()
    got = tg.gemm_bf16_lora(A, B, ids, down, up)
    assert same(torch, got.double(), want)
    bf = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=torch.bfloat16)
    assert same(torch, bf, got.to(torch.bfloat16))
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("M,N,K", [(5, 264, 2048), (40, 136, 4096), (100, 264, 2048),
                                   (700, WIDE[700], 6208)])
@pytest.mark.parametrize("kind", ["one", "requests", "any"])
@pytest.mark.parametrize("rank", [16, 72])
def test_infinite_weights_in_split_tiles(tg, M, N, K, kind, rank):
    """Tiles whose contraction, and for few rows whose adapter steps, are shared
    out over several units: an infinity in one part, finite sums in the others."""
    torch = torch_cuda()
    adapters = 4
    inf = float("inf")
    gen = torch.Generator(device="cuda").manual_seed(M + rank)
    A, B, down, up = case(gen, quarters, M, N, K, adapters, rank)
    down[..., 64:] = 0
    ids = plan(kind, M, adapters, M)
    for n in list(range(3, N, 128)) + [N - 1]:
        up[:, n, 0] = inf
        up[:, n - 1, rank - 1] = -inf
        up[1, n - 2, [1, rank - 2]] = inf
        up[2, n - 2, 1], up[2, n - 2, rank - 1] = inf, -inf
    want, _, _ = definition(torch, A, B, ids, down, up, None)
    got = tg.gemm_bf16_lora(A, B, ids, down, up)
    assert same(torch, got.double(), want)
    bf = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=torch.bfloat16)
    assert same(torch, bf, got.to(torch.bfloat16))
    assert tg.tg_device_status()[0] == tg.TG_OK
