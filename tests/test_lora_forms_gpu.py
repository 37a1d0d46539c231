"""gemm_bf16_lora on the sizes that choose its forms: CTA pairs (more 128 x 128
tiles than SMs), single CTAs with many rows and few columns, the rank values of
both kernels, and the precision they are kept in.

Quarter-integer inputs as in test_lora_gpu: bit for bit.  f32 D keeps the rank
values in three bf16 terms (2^-26 of them, below f32's own rounding), so a
normal case's error is that of its two products:
|D - ref| <= rtol * (sum |a b| + 2 sum |h up|) + atol.
"""
import numpy as np
import pytest

from tests._gpu import BF16_ATOL, BF16_RTOL, F32_ATOL, F32_RTOL, torch_cuda
from tests.test_grouped_gpu import normal, quarters
from tests.test_lora_gpu import case, definition, ids_of

pytestmark = pytest.mark.gpu

# Rows and columns of more than 152 tiles of 128 x 128.
WIDE = {200: 9872, 300: 6601, 700: 3401, 1025: 2200, 2300: 1201}


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def runs(M, adapters, seed):
    """Long and short runs in turn, some without an adapter."""
    torch = torch_cuda()
    rng = np.random.default_rng(seed)
    ids = np.empty(M, np.int32)
    i = 0
    while i < M:
        n = int(rng.choice([1, 5, 40, 190, 192, 260, 520]))
        ids[i:i + n] = rng.integers(-1, adapters)
        i += n
    return torch.from_numpy(ids).cuda()


def plan(kind, M, adapters, seed):
    return runs(M, adapters, seed) if kind == "runs" else ids_of(kind, M, adapters, seed)


@pytest.mark.parametrize("M", sorted(WIDE))
@pytest.mark.parametrize("kind", ["one", "none", "requests", "any", "runs"])
@pytest.mark.parametrize("K,adapters,rank", [(64, 3, 8), (200, 12, 16), (104, 5, 24), (72, 4, 40),
                                             (136, 6, 64), (200, 3, 72), (96, 2, 256)])
def test_pairs_exact(tg, M, kind, K, adapters, rank):
    torch = torch_cuda()
    N = WIDE[M]
    gen = torch.Generator(device="cuda").manual_seed(M + rank)
    A, B, down, up = case(gen, quarters, M, N, K, adapters, rank)
    down[..., 64:] = 0          # few terms: the rank values fit two bf16 terms
    ids = plan(kind, M, adapters, M + rank)
    scales = 2.0 ** torch.randint(-2, 3, (adapters,), generator=gen, device="cuda").float()
    want, _, _ = definition(torch, A, B, ids, down, up, scales)
    got = tg.gemm_bf16_lora(A, B, ids, down, up, scales=scales)
    assert torch.equal(got.double(), want)
    bf = tg.gemm_bf16_lora(A, B, ids, down, up, scales=scales, out_dtype=torch.bfloat16)
    assert torch.equal(bf, got.to(torch.bfloat16))
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("M,N,rank", [(9, 300, 8), (130, 700, 24), (300, 6601, 16), (300, 6601, 40),
                                      (700, 3401, 8), (1100, 264, 128), (1100, 2201, 128)])
@pytest.mark.parametrize("kind", ["one", "requests", "any"])
def test_f32_keeps_every_bit_of_the_rank_values(tg, M, N, rank, kind):
    """Rank values of 20 significant bits, picked out one by one by `up`."""
    torch = torch_cuda()
    K, adapters = 8192, 4
    gen = torch.Generator(device="cuda").manual_seed(M)
    pos = lambda *s: (torch.randint(1, 17, s, generator=gen, device="cuda") / 4).bfloat16()  # noqa: E731
    A, down = pos(M, K), pos(adapters, rank, K)
    B = torch.zeros(N, K, device="cuda", dtype=torch.bfloat16)
    up = torch.zeros(adapters, N, rank, device="cuda", dtype=torch.bfloat16)
    n = torch.arange(N, device="cuda")
    for t in range(adapters):
        up[t, n, (n + t) % rank] = 1.0
    ids = ids_of(kind, M, adapters, M)
    want, _, _ = definition(torch, A, B, ids, down, up, None)
    assert float(want.abs().max()) * 16 > 2 ** 18
    assert torch.equal(tg.gemm_bf16_lora(A, B, ids, down, up).double(), want)


@pytest.mark.parametrize("M,N,K,adapters,rank", [(1000, 200, 1500, 20, 16), (5000, 300, 400, 9, 8),
                                                 (1600, 136, 900, 6, 128), (700, 3401, 800, 30, 32),
                                                 (2300, 1201, 6200, 5, 64)])
@pytest.mark.parametrize("kind", ["requests", "any", "runs"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_forms_normal(tg, M, N, K, adapters, rank, kind, out):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    A, B, down, up = case(gen, normal, M, N, K, adapters, rank)
    ids = plan(kind, M, adapters, M)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    got = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt)
    ref, mag, low = definition(torch, A, B, ids, down, up, None)
    if out == "f32":
        tol = F32_RTOL * (mag + 2 * low) + F32_ATOL
    else:
        tol = BF16_RTOL * (mag + low) + 2.0 ** -15 * low + BF16_ATOL
    assert float(((got.double() - ref).abs() / tol).max()) <= 1.0
    again = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt)
    assert torch.equal(again, got)
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("M", [300, 700, 2300])
@pytest.mark.parametrize("rank", [8, 24, 64, 136])
@pytest.mark.parametrize("kind", ["requests", "any", "runs"])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_pairs_broken_adapter_stays_with_its_rows(tg, M, rank, kind, bad):
    torch = torch_cuda()
    N, K, adapters = WIDE[M], 72, 4
    gen = torch.Generator(device="cuda").manual_seed(M)
    A, B, down, up = case(gen, normal, M, N, K, adapters, rank)
    ids = plan(kind, M, adapters, 1)
    other = ids != 2
    for dt in (torch.float32, torch.bfloat16):
        clean = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt)
        u2 = up.clone()
        u2[2, [5, N - 1], 7] = bad
        got = tg.gemm_bf16_lora(A, B, ids, down, u2, out_dtype=dt)
        hit = torch.zeros(N, dtype=torch.bool, device="cuda")
        hit[[5, N - 1]] = True
        assert torch.equal(got[other], clean[other])
        assert torch.equal(got[:, ~hit], clean[:, ~hit])
        assert not torch.isfinite(got[~other][:, hit]).any()
        d2 = down.clone()
        d2[2, rank - 1, 7] = bad
        got = tg.gemm_bf16_lora(A, B, ids, d2, up, out_dtype=dt)
        assert torch.equal(got[other], clean[other])
        assert not torch.isfinite(got[~other]).any()
    assert tg.tg_device_status()[0] == tg.TG_OK
