"""Rank values between bf16's largest number and f32's in gemm_bf16_lora: they
are finite, and so is what they give.

The rank value is 3.3895e38 + 1.2e36 = 3.4015e38 exactly up to f32's rounding,
above the 3.3962e38 from which bf16 rounds to infinity; times 2^-100 it is about
2.7e8.  Two bf16 terms hold it to 2^-16 of itself, bf16 D rounds to 2^-9, f32 D's
three terms and the products' truncation stay below 2^-20.
"""
import pytest

from tests._gpu import torch_cuda

pytestmark = pytest.mark.gpu


# Both kernels that compute rank values; single CTAs and pairs.
@pytest.mark.parametrize("M,N,rank", [(5, 264, 8), (100, 136, 24), (300, 6601, 16), (2100, 264, 72),
                                      (2300, 1201, 64)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rank_values_above_the_largest_bf16(M, N, rank, sign):
    torch = torch_cuda()
    import blackwell_tile_gemm_gb300 as tg
    K = 64
    A = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    A[:, 0], A[:, 1] = sign * 3.3895e38, sign * 1.2e36
    down = torch.zeros(2, rank, K, device="cuda", dtype=torch.bfloat16)
    down[..., :2] = 1
    up = torch.zeros(2, N, rank, device="cuda", dtype=torch.bfloat16)
    n = torch.arange(N, device="cuda")
    up[:, n, n % rank] = 2.0 ** -100
    ids = (torch.arange(M, device="cuda", dtype=torch.int32) // 7) % 3      # 2: no adapter
    B = torch.zeros(N, K, device="cuda", dtype=torch.bfloat16)
    h = float(A[0, 0]) + float(A[0, 1])
    assert abs(h) > 3.3962e38 and abs(h) < 3.4028e38
    want = torch.where(ids[:, None] < 2, h * 2.0 ** -100, 0.0).expand(M, N)
    for dt, tol in ((torch.float32, 2.0 ** -20), (torch.bfloat16, 2.0 ** -9 + 2.0 ** -16)):
        got = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt).double()
        assert torch.isfinite(got).all()
        assert float((got - want).abs().max()) <= tol * abs(h) * 2.0 ** -100
    assert tg.tg_device_status()[0] == tg.TG_OK
