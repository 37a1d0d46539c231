"""embed_rows and embed_rows_grad.

The lookup rounds scale * w to 32 bits and once more to the result's type: its bits
are known.  The gradient sums c rows of one id in f32 and multiplies by scale: at most
c 2^-24 of the sum of magnitudes each, plus half a step of the result's type (bf16
2^-8), and with accumulate one more rounding in 32 bits of what was there.
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


def token_ids(gen, n, rows, kind):
    """`uneven`: frequent and rare ids; `one`: a single id; `spread`: mostly distinct."""
    import torch
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if kind == "uneven":
        ids = (3 * ((rows + 3) / 3) ** u - 3).long().clamp(0, rows - 1)
        ids = ids * 7919 % rows
    elif kind == "one":
        ids = torch.full((n,), rows // 2, device="cuda")
    else:
        ids = (u * rows).long()
    ids = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.05,
                      torch.tensor([-1, rows, 2 ** 31 - 1, -2 ** 31], device="cuda")
                      [torch.arange(n, device="cuda") % 4], ids)
    return ids.int()


def table(gen, m, k, dtype, pad=0):
    import torch
    t = torch.randn(m, -(-k // 8) * 8 + pad, generator=gen, device="cuda").to(dtype)
    return t[:, :k]


@pytest.mark.parametrize("n,rows,K,pad", [
    (1, 1, 1, 0), (1, 100, 8, 0), (5, 3, 7, 8), (33, 1000, 256, 0), (257, 50, 1001, 0),
    (1000, 5000, 2048, 16), (3, 4, 9000, 0), (0, 5, 16, 0), (4, 0, 16, 0)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_lookup_bits(tg, n, rows, K, pad, dtype):
    import torch
    dtype = getattr(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(n + rows + K)
    W = table(gen, rows, K, torch.bfloat16, pad)
    ids = token_ids(gen, n, max(rows, 1), "spread")
    D = tg.embed_rows(W, ids, scale=1.7, out_dtype=dtype)
    inside = (ids >= 0) & (ids < rows)
    want = torch.zeros(n, K, device="cuda")
    want[inside] = W[ids[inside].long()].float() * torch.tensor(1.7, device="cuda")
    assert torch.equal(D, want.to(dtype))
    # A given result with rows apart: what lies between stays.
    wide = torch.full((n, -(-K // 8) * 8 + 8), 9.0, device="cuda", dtype=dtype)
    tg.embed_rows(W, ids, wide[:, :K], scale=1.7)
    assert torch.equal(wide[:, :K], D) and (wide[:, K:] == 9).all()


def test_lookup_of_nan_and_infinite_rows(tg):
    import torch
    W = torch.ones(4, 16, device="cuda", dtype=torch.bfloat16)
    W[1], W[2] = float("nan"), float("inf")
    ids = torch.tensor([0, 1, 2, -1, 3], device="cuda", dtype=torch.int32)
    D = tg.embed_rows(W, ids, scale=0.5, out_dtype=torch.float32)
    assert (D[0] == 0.5).all() and D[1].isnan().all() and (D[2] == float("inf")).all()
    assert (D[3] == 0).all() and (D[4] == 0.5).all()


def sums(G, ids, rows, scale):
    """(gradient, sum of magnitudes, tokens) of each row in 64 bits."""
    import torch
    inside = (ids >= 0) & (ids < rows)
    at = ids[inside].long()
    g = G[inside].double()
    zero = torch.zeros(rows, G.shape[1], device="cuda", dtype=torch.float64)
    count = torch.zeros(rows, device="cuda", dtype=torch.float64)
    count.index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    s = float(torch.tensor(scale, dtype=torch.float32))
    return zero.index_add(0, at, g) * s, zero.index_add(0, at, g.abs()) * abs(s), count


def half(dtype):
    import torch
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


@pytest.mark.parametrize("n,rows,K", [
    (1, 1, 1), (1, 7, 8), (9, 5, 24), (100, 40, 1001), (2048, 512, 64), (2049, 513, 72),
    (5000, 100, 1032), (3000, 40000, 136), (20000, 300000, 40), (70000, 20, 16),
    (7, 262145, 8), (64, 1, 2056), (1024, 600, 1100), (1024, 600, 1025), (1030, 600, 200),
    (8192, 3000, 40), (8193, 3000, 40), (900, 524288, 16), (1500, 524287, 16), (1500, 524288, 16),
    (9217, 900, 40), (49152, 70000, 8), (49153, 70000, 8), (33333, 4194303, 8), (9000, 4194304, 8)])
@pytest.mark.parametrize("kind", ["uneven", "one", "spread"])
def test_gradient(tg, n, rows, K, kind):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(n + rows + K)
    ids = token_ids(gen, n, rows, kind)
    for given in (torch.bfloat16, torch.float32):
        G = table(gen, n, K, given, pad=8)
        want, mag, count = sums(G, ids, rows, -2.5)
        tol = (count + 2)[:, None] * 2.0 ** -24 * mag
        for out in (torch.bfloat16, torch.float32):
            D = tg.embed_rows_grad(G, ids, rows, scale=-2.5, out_dtype=out)
            assert D.dtype == out
            assert ((D.double() - want).abs() <= tol + half(out) * want.abs()).all()
            assert (D[count == 0] == 0).all()
            again = tg.embed_rows_grad(G, ids, rows, scale=-2.5, out_dtype=out)
            assert torch.equal(D, again)
            # Added to what is there; rows without tokens keep their bits.
            D0 = table(gen, rows, K, out, pad=8)
            D1 = D0.clone(memory_format=torch.preserve_format)
            wide = torch.full((rows, D0.stride(0) if rows > 1 else -(-K // 8) * 8), 5.0,
                              device="cuda", dtype=out)
            D1 = wide[:, :K]
            D1.copy_(D0)
            assert tg.embed_rows_grad(G, ids, rows, D1, scale=-2.5, accumulate=True) is D1
            both = D0.double() + want
            near = tol + half(out) * both.abs() + 2.0 ** -24 * (D0.double().abs() + mag)
            assert ((D1.double() - both).abs() <= near).all()
            assert torch.equal(D1[count == 0], D0[count == 0])
            assert (wide[:, K:] == 5).all()
    assert tg.tg_device_status()[0] == tg.TG_OK


def test_no_tokens_and_rows_without_an_id(tg):
    import torch
    none = torch.zeros(0, device="cuda", dtype=torch.int32)
    D = tg.embed_rows_grad(torch.zeros(0, 24, device="cuda"), none, 100)
    assert D.shape == (100, 24) and (D == 0).all()
    G = torch.full((50, 24), float("nan"), device="cuda")      # padding may hold anything
    out = torch.full((50,), -7, device="cuda", dtype=torch.int32)
    assert (tg.embed_rows_grad(G, out, 100) == 0).all()
    D = torch.ones(100, 24, device="cuda")
    tg.embed_rows_grad(G, out, 100, D, accumulate=True)
    tg.embed_rows_grad(G[:0], none, 100, D, accumulate=True)
    assert (D == 1).all()
    assert tg.embed_rows_grad(G, out, 0).shape == (0, 24)
    ids = torch.arange(50, device="cuda", dtype=torch.int32)
    ids[7] = 1000
    G = torch.ones(50, 24, device="cuda")
    G[7] = float("inf")
    D = tg.embed_rows_grad(G, ids, 100)
    assert (D[:7] == 1).all() and (D[7] == 0).all() and (D[8:50] == 1).all() and (D[50:] == 0).all()


def test_long_runs_join_in_order(tg):
    """Whole numbers: every order of f32 sums is exact, and none is lost or doubled."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(2)
    for n in (15, 16, 17, 97, 1023, 1024, 1025, 8191, 8192, 8193, 49152, 49153, 100000):
        G = torch.randint(-3, 4, (n, 40), generator=gen, device="cuda").float()
        ids = (torch.arange(n, device="cuda") * 3 // n).int()      # three runs
        D = tg.embed_rows_grad(G, ids, 5)
        want = torch.stack([G[ids == v].sum(0) for v in range(5)])
        assert torch.equal(D, want)


@pytest.mark.parametrize("accumulate", [False, True])
def test_captured_and_on_another_stream(tg, accumulate):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    n, rows, K = 5000, 30000, 136
    ids, G = token_ids(gen, n, rows, "uneven"), table(gen, n, K, torch.float32)
    want = tg.embed_rows_grad(G, ids, rows)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tg.reserve_workspace(tg.workspace_bytes(tg.TG_CALL_EMBED_ROWS_GRAD, n, rows, K), stream=s)
    count = tg.workspace_alloc_count()
    D = torch.zeros(rows, K, device="cuda")
    W = table(gen, rows, K, torch.bfloat16)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tg.embed_rows_grad(G, ids, rows, D, accumulate=accumulate)
        X = tg.embed_rows(W, ids)
    for i in range(1, 3):
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        if accumulate and i == 2:
            assert torch.equal(D, want + want)
        else:
            assert torch.equal(D, want)
    assert torch.equal(X, tg.embed_rows(W, ids))
    assert tg.workspace_alloc_count() == count
    t = torch.cuda.CUDAGraph()
    other = torch.cuda.Stream()
    code = None
    with torch.cuda.graph(t, stream=other):
        try:
            tg.embed_rows_grad(G, ids, rows, D)
        except tg.TgError as e:
            code = e.code
        D.add_(0)
    assert code == tg.TG_ERR_WORKSPACE


def test_more_than_2_31_elements(tg):
    import torch
    rows, K = 270000, 8192
    ids = torch.tensor([0, rows - 1, 5, rows - 1, rows // 2], device="cuda", dtype=torch.int32)
    W = torch.zeros(rows, K, device="cuda", dtype=torch.bfloat16)
    W[rows - 1] = 3.0
    W[rows // 2] = 2.0
    X = tg.embed_rows(W, ids)
    assert (X[1] == 3).all() and (X[4] == 2).all() and (X[[0, 2]] == 0).all()
    G = torch.arange(1, 6, device="cuda").float()[:, None].expand(5, K).contiguous()
    D = tg.embed_rows_grad(G, ids, rows, W)
    assert (D[rows - 1] == 6).all() and (D[rows // 2] == 5).all() and (D[0] == 1).all()
    assert float(D.float().abs().sum(1).count_nonzero()) == 4
