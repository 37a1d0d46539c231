"""Precision of gemm_bf16_lora's rank values where D is f32 and K is long.

The tensor cores truncate at every addition of 16 terms to an accumulator, up to
2^-23 of it.  Contractions are cut into chunks of 768 terms (48 additions) that
are added with rounding to nearest: at most 48 * 2^-24 on average, 2.9e-6, of the
sum; the adapter product adds three terms of the rank to that (12 additions at
rank 64, 0.7e-6).  So the adapter term alone (B is zero) is held to 4e-6 of its
norm, whatever K is.  In one accumulator 16384 terms are 1024 additions.
"""
import pytest

from tests._gpu import torch_cuda
from tests.test_grouped_gpu import normal
from tests.test_lora_forms_gpu import plan
from tests.test_lora_gpu import case, definition

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("M,rank,K,kind", [
    (4096, 64, 16384, "one"), (4096, 64, 16384, "runs"),     # tiles of 64 rows, tcgen05
    (12000, 16, 8192, "requests"),
    (2048, 16, 65536, "any"), (2000, 64, 65536, "any"),      # 8 rows a block, warp MMAs
    (300, 64, 16384, "any"),                                 # K over a cluster
])
def test_long_contractions_of_the_rank_values_keep_f32(tg, M, rank, K, kind):
    torch = torch_cuda()
    N, adapters = 136, 5
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    A, B, down, up = case(gen, normal, M, N, K, adapters, rank)
    B.zero_()
    ids = plan(kind, M, adapters, M)
    want, _, _ = definition(torch, A, B, ids, down, up, None)
    got = tg.gemm_bf16_lora(A, B, ids, down, up)
    off = float((got.double() - want).norm() / want.norm())
    print("relative error %.2g" % off)
    assert off <= 4e-6
    assert tg.tg_device_status()[0] == tg.TG_OK
