"""tg_balance_loss on streams that have what tg_workspace_bytes names and no more."""
import pytest

from tests._gpu import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("M", [0, 1, 9, 700])
@pytest.mark.parametrize("E", [3, 1000, 4096])
def test_what_the_call_names_is_enough(tg, M, E):
    """No token among them: nothing to read, and nothing to keep in between."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(M + E)
    logits = torch.randn(M, E, generator=gen, device="cuda")
    ids = torch.randint(0, E, (M, 2), generator=gen, device="cuda", dtype=torch.int32)
    # (Of the other pool: tests that want a stream without a workspace find one.)
    s = torch.cuda.Stream(priority=-1)
    s.wait_stream(torch.cuda.current_stream())
    tg.reserve_workspace(tg.workspace_bytes(tg.TG_CALL_BALANCE_LOSS, M, E, 1), stream=s)
    count = tg.workspace_alloc_count()
    with torch.cuda.stream(s):
        loss, counts, shares = tg.balance_loss(logits, ids)
    s.synchronize()
    assert tg.workspace_alloc_count() == count
    assert torch.equal(counts.cpu(), torch.bincount(ids.flatten().cpu(), minlength=E).int())
    want = (logits.double().softmax(1).sum(0) * shares.double()).sum()
    assert abs(float(loss) - float(want)) <= 1e-5 * float(want)
    if M == 0:
        assert float(loss) == 0 and (counts == 0).all() and (shares == 0).all()
