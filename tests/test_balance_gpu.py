"""tg_balance_loss and its gradient against the definition in 64 bits.

p: an f32 exponential of a difference (2^-24 of a difference of at most 40 where p
counts: 3e-6) over a sum (1e-6): 5e-6 of itself.  The loss sums positive terms, at most
5e-6 and the roundings of f32 sums in a tree: 1e-5 of itself.  The gradient g p (share -
dot) has 1e-5 of g p (share + dot), and half a step of its type (bf16 2^-8).
"""
import pytest

from tests._gpu import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def inputs(seed, M, E, k, dtype, padding=0.1, pad=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = (2 * torch.randn(M, E + pad, generator=gen, device="cuda")).to(dtype)[:, :E]
    ids = torch.randint(0, E, (M, k), generator=gen, device="cuda", dtype=torch.int32)
    drop = torch.rand(M, k, generator=gen, device="cuda") < 0.1
    bad = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], device="cuda", dtype=torch.int32)
    ids = torch.where(drop, bad[torch.arange(k, device="cuda") % 4], ids)
    ids[torch.rand(M, generator=gen, device="cuda") < padding] = -1
    return z, ids


def reference(z, ids, g=1.0):
    import torch
    M, E = z.shape
    inside = (ids >= 0) & (ids < E)
    some = inside.any(1)
    counts = torch.bincount(ids[inside].long(), minlength=E)
    z = z.double()
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isneginf(top), torch.zeros_like(top), top))
    s = e.sum(1, keepdim=True)
    p = torch.where(s == 0, torch.zeros_like(e), e / s) * some[:, None]
    tokens = int(some.sum())
    shares = counts.double() * (E / (max(int(counts.sum()), 1) * max(tokens, 1)))
    dot = (p * shares).sum(1, keepdim=True)
    return dict(counts=counts.int(), shares=shares, loss=(shares * p.sum(0)).sum(),
                grad=g * p * (shares - dot), tol=1e-5 * abs(g) * p * (shares + dot), some=some)


def check(tg, z, ids, out_dtypes):
    import torch
    g = torch.tensor(-3.0, device="cuda")
    r = reference(z, ids, -3.0)
    loss, counts, shares = tg.balance_loss(z, ids)
    assert loss.shape == () and torch.equal(counts, r["counts"])
    assert ((shares.double() - r["shares"]).abs() <= 2.0 ** -23 * r["shares"]).all()
    assert abs(float(loss) - float(r["loss"])) <= 1e-5 * float(r["loss"])
    for dtype in out_dtypes:
        D = tg.balance_loss_grad(z, ids, shares, g, out_dtype=dtype)
        assert D.dtype == dtype
        half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
        assert ((D.double() - r["grad"]).abs() <= r["tol"] + half * r["grad"].abs() + 1e-37).all()
        assert (D[~r["some"]] == 0).all()
    again = tg.balance_loss(z, ids)
    assert torch.equal(again[0], loss) and torch.equal(again[2], shares)


@pytest.mark.parametrize("M,E,k", [
    (1, 1, 1), (1, 2, 1), (2, 3, 2), (500, 64, 8), (1000, 1, 3), (77, 5, 40), (33, 33, 1),
    (4097, 31, 4), (3000, 128, 2), (2000, 129, 8), (700, 256, 8), (900, 511, 3), (900, 512, 3),
    (300, 513, 4), (5, 1000, 70), (200, 4096, 8), (60000, 8, 2), (40000, 60, 6), (100000, 2, 1)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_loss_counts_and_gradient(tg, M, E, k, dtype):
    import torch
    z, ids = inputs(M + E + k, M, E, k, getattr(torch, dtype), pad=3 if M % 2 else 0)
    check(tg, z, ids, (torch.float32, torch.bfloat16))


def test_even_choices_give_one(tg):
    import torch
    z = torch.zeros(64, 16, device="cuda")
    ids = (torch.arange(128, device="cuda", dtype=torch.int32) % 16).view(64, 2)
    loss, counts, shares = tg.balance_loss(z, ids)
    assert float(loss) == 1.0 and (counts == 8).all() and (shares == 1 / 64).all()
    assert (tg.balance_loss_grad(z, ids, shares) == 0).all()


@pytest.mark.parametrize("E", [5, 64, 600])
def test_masked_logits(tg, E):
    """Experts at -inf, a row of nothing else, the type's lowest value, and padding
    rows of NaN and infinities."""
    import torch
    z, ids = inputs(E, 200, E, 2, torch.float32, padding=0.0)
    ids = ids.clamp(0, E - 1)
    z[::3, ::2] = -float("inf")
    z[5] = -float("inf")
    z[6] = torch.finfo(torch.float32).min
    z[7, 1:] = torch.finfo(torch.float32).min
    check(tg, z, ids, (torch.float32,))
    z2, ids2 = z.clone(), ids.clone()
    z2[50:60] = float("nan")
    z2[60:70] = float("inf")
    ids2[50:70] = -1
    keep = torch.cat([torch.arange(50), torch.arange(70, 200)]).cuda()
    loss, counts, shares = tg.balance_loss(z2, ids2)
    r = reference(z2[keep], ids2[keep])
    assert torch.equal(counts, r["counts"])
    assert abs(float(loss) - float(r["loss"])) <= 1e-5 * float(r["loss"])
    D = tg.balance_loss_grad(z2, ids2, shares)
    assert (D[50:70] == 0).all() and torch.isfinite(D).all()
    assert ((D[keep].double() - r["grad"]).abs() <= r["tol"] + 2.0 ** -24 * r["grad"].abs() + 1e-37).all()


def test_nothing_chosen_and_no_tokens(tg):
    import torch
    z = torch.randn(40, 12, device="cuda")
    for ids in (torch.full((40, 2), -1, device="cuda", dtype=torch.int32),
                torch.zeros(0, 2, device="cuda", dtype=torch.int32)):
        loss, counts, shares = tg.balance_loss(z[:len(ids)], ids)
        assert float(loss) == 0 and (counts == 0).all() and (shares == 0).all()
        D = tg.balance_loss_grad(z[:len(ids)], ids, shares)
        assert D.shape == (len(ids), 12) and (D == 0).all()


def test_gradient_agrees_with_differences(tg):
    import torch
    z, ids = inputs(9, 50, 24, 4, torch.float32)
    _, _, shares = tg.balance_loss(z, ids)
    D = tg.balance_loss_grad(z, ids, shares).double()
    zd, h = z.double(), 1e-5
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        u = torch.randn(zd.shape, generator=gen, device="cuda", dtype=torch.float64)
        slope = (reference(zd + h * u, ids)["loss"] - reference(zd - h * u, ids)["loss"]) / (2 * h)
        assert abs(float((D * u).sum() - slope)) <= 2e-5 * float((D * u).abs().sum())


def test_gradient_in_place_and_given_strides(tg):
    import torch
    z, ids = inputs(21, 300, 70, 3, torch.float32)
    _, _, shares = tg.balance_loss(z, ids)
    want = tg.balance_loss_grad(z, ids, shares)
    wide = torch.full((300, 91), 4.0, device="cuda")
    tg.balance_loss_grad(z, ids, shares, D=wide[:, 7:77])
    assert torch.equal(wide[:, 7:77], want)
    assert (wide[:, :7] == 4).all() and (wide[:, 77:] == 4).all()
    own = z.clone()
    assert torch.equal(tg.balance_loss_grad(own, ids, shares, D=own), want)


def test_captured_and_on_another_stream(tg):
    import torch
    z, ids = inputs(23, 3000, 96, 4, torch.bfloat16)
    loss, counts, shares = tg.balance_loss(z, ids)
    D = tg.balance_loss_grad(z, ids, shares)
    graphs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        tg.reserve_workspace(tg.workspace_bytes(tg.TG_CALL_BALANCE_LOSS, 3000, 96, 1), stream=s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = tg.balance_loss(z, ids)
            out = out + (tg.balance_loss_grad(z, ids, out[2]),)
        graphs.append((g, s, out))
    for _ in range(3):
        for g, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, (loss, counts, shares, D)))
