"""gemm_bf16_lora on prompts whose rank values take full waves of tiles and a
split last wave (more than one tile per SM, few left over).

Whole multiples of 1/4: products of 2048 of them are multiples of 1/16 below
2^8, the adapter term and the sum with the shared product multiples of 1/64
below 2^16, so every f32 sum is exact and the rank values fit two bf16 terms:
bit for bit.
"""
import pytest

from tests._gpu import torch_cuda
from tests.test_grouped_gpu import quarters
from tests.test_lora_forms_gpu import plan
from tests.test_lora_gpu import case, definition

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("M,rank", [(10000, 128), (10368, 64), (5000, 256), (20000, 64), (9729, 136),
                                    (20500, 32), (9800, 8)])
@pytest.mark.parametrize("kind", ["one", "requests", "runs"])
@pytest.mark.parametrize("N", [136, 520])
def test_split_tiles_after_full_waves(tg, M, rank, kind, N):
    torch = torch_cuda()
    K, adapters = 2048, 5
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    A, B, down, up = case(gen, quarters, M, N, K, adapters, rank)
    ids = plan(kind, M, adapters, M + rank)
    scales = torch.tensor([0.5, 2.0, 1.0, 0.25, 1.0], device="cuda")
    want, _, _ = definition(torch, A, B, ids, down, up, scales)
    assert float(want.abs().max()) < 2 ** 16
    got = tg.gemm_bf16_lora(A, B, ids, down, up, scales=scales)
    assert torch.equal(got.double(), want)
    bf = tg.gemm_bf16_lora(A, B, ids, down, up, scales=scales, out_dtype=torch.bfloat16)
    assert torch.equal(bf, got.to(torch.bfloat16))
    assert tg.tg_device_status()[0] == tg.TG_OK
