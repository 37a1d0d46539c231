"""embed_rows_grad where the ids are sorted digit by digit (more than 49152 tokens, or more
rows than the shorter sorts take): call after call on ids that change, against sums in 64
bits.  Whole numbers: every sum is exact."""
import pytest

from tests._gpu import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("n,rows", [(60000, 300), (131072, 50257), (70001, 300007),
                                    (5000, 5000011), (60000, (1 << 27) + 5)])
@pytest.mark.parametrize("captured", [False, True])
def test_digits_call_after_call(tg, n, rows, captured):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(n)
    K = 8
    G = torch.randint(-4, 5, (n, K), generator=gen, device="cuda").to(torch.bfloat16)
    # A few ids often, the others anywhere, some outside.
    draws = []
    for _ in range(6):
        v = torch.randint(0, rows, (n,), generator=gen, device="cuda", dtype=torch.int32)
        hot = torch.rand(n, generator=gen, device="cuda")
        v = torch.where(hot < 0.01, (v % 3) * (rows // 3), v)
        draws.append(torch.where(hot > 0.98, -1 - v, v))
    ids = draws[0].clone()
    D = torch.zeros(rows, K, device="cuda", dtype=torch.bfloat16)
    # (Of the other pool: tests that want a stream without a workspace find one.)
    s = torch.cuda.Stream(priority=-1)
    s.wait_stream(torch.cuda.current_stream())
    tg.reserve_workspace(tg.workspace_bytes(tg.TG_CALL_EMBED_ROWS_GRAD, n, rows, K), stream=s)
    out = []
    with torch.cuda.stream(s):
        if captured:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                tg.embed_rows_grad(G, ids, rows, D)
        for v in draws:
            ids.copy_(v)
            if captured:
                g.replay()
            else:
                tg.embed_rows_grad(G, ids, rows, D)
            # The rows that have a token, and how much there is in all.
            out.append((D[v.clamp(min=0).long()].clone(), D.float().abs().sum(dtype=torch.float64)))
    torch.cuda.synchronize()
    for v, (got, size) in zip(draws, out):
        inside = v >= 0
        used, at = torch.unique(v[inside], return_inverse=True)
        want = torch.zeros(len(used), K, device="cuda", dtype=torch.float64)
        want.index_add_(0, at, G[inside].double())
        # bf16 keeps whole numbers up to 256; larger sums are rounded once.
        want = want.to(torch.bfloat16)
        assert torch.equal(got[inside], want[at])
        assert float(size) == float(want.double().abs().sum())
