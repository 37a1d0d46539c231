"""Gradients of rows whose target has nearly all of the probability: the target's dz is
w (p - 1), a small rest, and its digits are what such a row still learns from.

Tolerances, before anything ran.  A logit is off by 1e-6 of itself for each 1024 terms that
are summed without rounding to nearest, and no more terms are: the other columns' p by 4e-5
of itself (lse and the target's logit are below 23, the others below 12: 3.5e-5, and 5e-6 for
the exponential and the scaling), and the loss by 2e-5 of itself and 45 * 2^-24 (tests/test_xent_gpu.py).  With the loss given the target's
1 - p takes that on, and 2^-22 of itself (expm1f).  Without it, z and lse are two rounded numbers: 1e-6 of z
for the order of its sum, 2^-24 of both for their rounding, together below 1e-6 (|z| + |lse|)
and the same 2e-5 of the loss.  dz is rounded by 2^-8 of itself (two terms: 2^-16), the
products add 1e-5 of the sum of magnitudes, a bf16 result 2^-8 of itself.
"""
import pytest

from tests._gpu import torch_cuda
from tests.test_xent_gpu import rows, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def confident(seed, M, N, K):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B = rows(gen, N, K, scale=1.5 * K ** -0.5)
    t = torch.randperm(N, generator=gen, device="cuda")[:M].to(torch.int32)
    lean = torch.linspace(6.0, 8.5, M, device="cuda")[:, None]
    A = torch.randn(M, K, generator=gen, device="cuda") + lean * B[t.long()].float()
    ld = -(-K // 8) * 8
    a = torch.zeros(M, ld, device="cuda", dtype=torch.bfloat16)[:, :K]
    a.copy_(A)
    return a, B, t, torch.rand(M, generator=gen, device="cuda") + 0.5


def definition(A, B, t, grad, scale, given, terms):
    """(dA, dB, their tolerances) in 64 bits."""
    import torch
    a, b, w = A.double(), B.double(), grad.double() * scale
    row = torch.arange(len(t), device="cuda")
    z = scale * (a @ b.T)
    zt = z[row, t.long()]
    top = z.max(1).values
    lse = torch.logsumexp(z, 1)
    others = torch.exp(z - top[:, None])
    others[row, t.long()] = 0.0
    assert (zt == top).all() and float(lse.max()) < 23
    rest = others.sum(1)                            # (no difference of large numbers)
    loss, left = torch.log1p(rest), rest / (1 + rest)
    assert float(left.min()) < 5e-4 and float(left.max()) > 5e-3
    dz = others / (1 + rest)[:, None]
    dz[row, t.long()] = -left
    e = 4e-5 * dz.abs()
    e[row, t.long()] = 2e-5 * loss + (45 * 2.0 ** -24 + 2.0 ** -22 * left if given else
                                      1e-6 * (zt.abs() + lse.abs()))
    e += dz.abs() * (1e-5 + (2.0 ** -8 if terms == 1 else 2.0 ** -16))
    dz, e = dz * w[:, None], e * w[:, None]
    half = 2.0 ** -8 if terms == 1 else 2.0 ** -24
    out = [dz @ b, dz.T @ a]
    tol = [e @ b.abs(), e.T @ a.abs()]
    return out, [x + half * y.abs() + 1e-12 for x, y in zip(tol, out)]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,scale", [(100, 3000, 8192, 1.0), (300, 3000, 8192, 1.0),
                                         (300, 3000, 8192, 0.95), (100, 2999, 4099, 1.0)])
def test_the_rest_of_a_confident_row(tg, M, N, K, scale, f32, given):
    import torch
    A, B, t, grad = confident(M + K, M, N, K)
    loss, lse = tg.gemm_bf16_xent(A, B, t, scale=scale)
    extra = dict(loss=loss) if given else {}
    got = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, scale=scale, **extra,
                                 out_dtype=torch.float32 if f32 else torch.bfloat16)
    want, tol = definition(A, B, t, grad, scale, given, 2 if f32 else 1)
    for x, y, e in zip(got, want, tol):
        within(x, y, e)
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("M", [5, 200])
def test_a_loss_beside_rows_without_a_target(tg, M):
    """What the loss holds where nothing is learned reaches nothing; elsewhere the target's
    entry follows the given loss alone, and a loss of 0 or infinity is its limit."""
    import torch
    A, B, t, grad = confident(3, M, 700, 264)
    t[1::3] = -100
    outside = t < 0
    loss, lse = tg.gemm_bf16_xent(A, B, t)
    assert (loss[outside] == 0).all()
    odd = torch.where(outside, torch.full_like(loss, float("nan")), loss)
    for dtype in (torch.bfloat16, torch.float32):
        want = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, loss=loss, out_dtype=dtype)
        got = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, loss=odd, out_dtype=dtype)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert (got[0][outside] == 0).all()
    # lse far above every logit: p is 0, and dz the target's entry alone.
    far = torch.full_like(lse, 1e4)
    rows_ = torch.arange(M, device="cuda")[~outside]
    for value, entry in ((0.0, 0.0), (float("inf"), -1.0)):
        dA, _ = tg.gemm_bf16_xent_grad(A, B, t, far, None, loss=torch.full_like(loss, value),
                                       out_dtype=torch.float32)
        assert torch.equal(dA[rows_], entry * B[t[rows_].long()].float())


def test_captured_with_the_loss(tg):
    import torch
    A, B, t, grad = confident(7, 150, 2000, 520)
    # (Of the other pool: tests that want a stream without a workspace find one.)
    s = torch.cuda.Stream(priority=-1)
    tg.reserve_workspace(max(tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_XENT, 150, 2000, 520),
                             tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_XENT_GRAD, 150, 2000, 520,
                                                d_dtype=tg.TG_D_BF16)), stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        loss, lse = tg.gemm_bf16_xent(A, B, t)
        want = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, loss=loss)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        loss, lse = tg.gemm_bf16_xent(A, B, t)
        got = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, loss=loss)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
