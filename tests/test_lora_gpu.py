"""GPU parity of gemm_bf16_lora with its definition in float64.

Quarter-integer inputs keep every partial sum exact (and the rank values
exact in two bf16 terms), so f32 results must equal the definition bit for
bit.  Normal inputs: |D - ref| <= rtol * (sum |a b| + s sum |h up|) + atol with
the product's rtol (tests/_gpu.py) plus 2^-15 of the adapter term, the
rounding of the rank values to two bf16 terms (2^-17 each way) and to f32.
"""
import numpy as np
import pytest

from tests._gpu import BF16_ATOL, BF16_RTOL, F32_ATOL, F32_RTOL, torch_cuda
from tests.test_grouped_gpu import normal, quarters

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def definition(torch, A, B, ids, down, up, scales):
    D = A.double() @ B.double().T
    mag = A.double().abs() @ B.double().abs().T
    low = torch.zeros_like(mag)
    for t in range(down.shape[0]):
        at = torch.nonzero(ids == t).flatten()
        if at.numel():
            s = 1.0 if scales is None else scales[t].double()
            h = (A[at].double() @ down[t].double().T) * s
            D[at] += h @ up[t].double().T
            low[at] += ((A[at].double().abs() @ down[t].double().abs().T) * s) @ up[t].double().abs().T
    return D, mag, low


def case(gen, make, M, N, K, adapters, rank):
    return make(gen, M, K), make(gen, N, K), make(gen, adapters, rank, K), make(gen, adapters, N, rank)


def ids_of(kind, M, adapters, seed):
    """Adapter per row: one for all, a request's rows together, or any; some
    rows without one."""
    torch = torch_cuda()
    rng = np.random.default_rng(seed)
    if kind == "one":
        ids = np.full(M, adapters - 1)
    elif kind == "none":
        ids = np.full(M, -1)
    elif kind == "requests":
        ids = np.sort(rng.integers(-1, adapters, M))
        ids = np.roll(ids, M // 3)
    else:
        ids = rng.integers(-2, adapters + 2, M)
    return torch.from_numpy(ids.astype(np.int32)).cuda()


@pytest.mark.parametrize("M", [1, 3, 8, 17, 64, 65, 128, 129, 300, 700])
@pytest.mark.parametrize("kind", ["one", "none", "requests", "any"])
@pytest.mark.parametrize("shape", [(128, 64, 3, 8), (257, 200, 5, 24), (520, 1001, 9, 72),
                                   (96, 72, 2, 136)])
def test_exact(tg, M, kind, shape):
    torch = torch_cuda()
    N, K, adapters, rank = shape
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    A, B, down, up = case(gen, quarters, M, N, K, adapters, rank)
    # The rank values keep 16 significant bits: with few non-zero entries of
    # `down` they are exact in them.
    down[..., ::7] = 0
    if K > 100:
        down[..., 64:] = 0
    ids = ids_of(kind, M, adapters, M + rank)
    scales = torch.tensor([0.5, 2.0, 1.0, 0.25, 4.0, 1.0, 1.0, 0.5, 1.0][:adapters], device="cuda")
    want, _, _ = definition(torch, A, B, ids, down, up, scales)
    got = tg.gemm_bf16_lora(A, B, ids, down, up, scales=scales)
    assert torch.equal(got.double(), want)
    bf = tg.gemm_bf16_lora(A, B, ids, down, up, scales=scales, out_dtype=torch.bfloat16)
    assert torch.equal(bf, got.to(torch.bfloat16))
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("M", [1, 40, 128, 200, 1000])
@pytest.mark.parametrize("kind", ["requests", "any"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1024, 2048, 7, 16), (1000, 1500, 4, 64), (300, 640, 3, 256)])
def test_normal(tg, M, kind, out, shape):
    torch = torch_cuda()
    N, K, adapters, rank = shape
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    A, B, down, up = case(gen, normal, M, N, K, adapters, rank)
    ids = ids_of(kind, M, adapters, M)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    got = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt, silu_affine=(2.0, 0.5))
    ref, mag, low = definition(torch, A, B, ids, down, up, None)
    # |silu'| <= 1.1; the output's own rounding is inside rtol * mag.
    y = ref * torch.sigmoid(ref) * 2.0 + 0.5
    rtol, atol = (F32_RTOL, F32_ATOL) if out == "f32" else (BF16_RTOL, BF16_ATOL)
    tol = 2.2 * (rtol * (mag + low) + 2.0 ** -15 * low) + atol
    if out == "f32":
        tol = tol + 2.0 ** -21 * y.abs()
    assert float(((got.double() - y).abs() / tol).max()) <= 1.0
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("M", [40, 100, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["down", "up"])
def test_a_broken_adapter_stays_with_its_rows(tg, M, bad, where):
    """Infinite or NaN weights of one adapter reach its own rows only."""
    torch = torch_cuda()
    N, K, adapters, rank = 264, 320, 4, 16
    gen = torch.Generator(device="cuda").manual_seed(M)
    A, B, down, up = case(gen, normal, M, N, K, adapters, rank)
    ids = ids_of("any", M, adapters, 1)
    for dt in (torch.float32, torch.bfloat16):
        clean = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt)
        d2, u2 = down.clone(), up.clone()
        (d2 if where == "down" else u2)[2, 5, 7] = bad
        got = tg.gemm_bf16_lora(A, B, ids, d2, u2, out_dtype=dt)
        other = ids != 2
        assert torch.equal(got[other], clean[other])
        if where == "up":
            hit = torch.zeros(N, dtype=torch.bool, device="cuda")
            hit[5] = True
            assert torch.equal(got[:, ~hit], clean[:, ~hit])
            assert not torch.isfinite(got[~other][:, 5]).any()
        else:
            assert not torch.isfinite(got[~other]).any()


def test_views_strides_and_an_output_of_the_callers(tg):
    torch = torch_cuda()
    M, N, K, adapters, rank = 150, 200, 256, 3, 16
    gen = torch.Generator(device="cuda").manual_seed(5)
    A, B, _, _ = case(gen, quarters, M, N, K, 1, 8)
    down = quarters(gen, 2 * adapters, rank + 8, K + 64)[::2, :rank, :K]
    up = quarters(gen, 2 * adapters, N + 3, 2 * rank)[::2, :N, rank:]
    down[..., 40:] = 0
    ids = ids_of("any", M, adapters, 2)
    want, _, _ = definition(torch, A, B, ids, down, up, None)
    for m in (100, M):
        D = torch.full((m, N + 8), 7.0, device="cuda")
        out = tg.gemm_bf16_lora(A[:m], B, ids[:m].contiguous(), down, up, D[:, :N])
        assert out.data_ptr() == D.data_ptr()
        assert torch.equal(D[:, :N].double(), want[:m]) and (D[:, N:] == 7.0).all()


@pytest.mark.parametrize("M", [1025, 1500, 5000])
@pytest.mark.parametrize("kind", ["one", "none", "requests", "any"])
@pytest.mark.parametrize("shape", [(136, 200, 5, 24), (264, 1001, 9, 72), (96, 520, 3, 136),
                                   (128, 1600, 70, 8)])
def test_many_rows_exact(tg, M, kind, shape):
    """Rows enough for the tiled computation of the rank values, split and
    unsplit, one and two tiles of the rank; tiles of one, two, many adapters."""
    torch = torch_cuda()
    N, K, adapters, rank = shape
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    A, B, down, up = case(gen, quarters, M, N, K, adapters, rank)
    down[..., 64:] = 0          # few terms: the rank values fit two bf16 terms
    ids = ids_of(kind, M, adapters, M + rank)
    scales = 2.0 ** torch.randint(-2, 3, (adapters,), generator=gen, device="cuda").float()
    want, _, _ = definition(torch, A, B, ids, down, up, scales)
    got = tg.gemm_bf16_lora(A, B, ids, down, up, scales=scales)
    assert torch.equal(got.double(), want)
    assert tg.tg_device_status()[0] == tg.TG_OK


def test_many_rows_normal_and_broken_adapter(tg):
    torch = torch_cuda()
    M, N, K, adapters, rank = 3000, 520, 2048, 6, 64
    gen = torch.Generator(device="cuda").manual_seed(9)
    A, B, down, up = case(gen, normal, M, N, K, adapters, rank)
    for kind in ("requests", "any"):
        ids = ids_of(kind, M, adapters, 4)
        ref, mag, low = definition(torch, A, B, ids, down, up, None)
        clean = tg.gemm_bf16_lora(A, B, ids, down, up)
        tol = F32_RTOL * (mag + low) + 2.0 ** -15 * low + F32_ATOL
        assert float(((clean.double() - ref).abs() / tol).max()) <= 1.0
        down2 = down.clone()
        down2[2, 5, 7] = float("nan")
        got = tg.gemm_bf16_lora(A, B, ids, down2, up)
        assert torch.equal(got[ids != 2], clean[ids != 2])
        assert torch.isnan(got[ids == 2]).all()


@pytest.mark.parametrize("M", [24, 200, 1444, 2300])
def test_same_bits_every_time(tg, M):
    """Also where a tile's contraction is split between units."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(M)
    A, B, down, up = case(gen, normal, M, 520, 7000, 5, 40)
    ids = ids_of("any", M, 5, M)
    for dt in (torch.float32, torch.bfloat16):
        first = tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt)
        for _ in range(3):
            assert torch.equal(tg.gemm_bf16_lora(A, B, ids, down, up, out_dtype=dt), first)


def test_streams_reservation_and_graphs(tg):
    torch = torch_cuda()
    N, K, adapters, rank = 264, 320, 4, 24
    gen = torch.Generator(device="cuda").manual_seed(3)
    s = torch.cuda.Stream()
    for M in (40, 300, 1200):
        A, B, down, up = case(gen, quarters, M, N, K, adapters, rank)
        down[..., 64:] = 0
        kinds = [ids_of(kind, M, adapters, 7) for kind in ("any", "requests", "one")]
        ids = kinds[0].clone()
        D = torch.empty(M, N, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            tg.reserve_workspace(tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_LORA, M, rank, 1))
            tg.gemm_bf16_lora(A, B, ids, down, up, D)
            s.synchronize()
            before = tg.workspace_alloc_count()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                tg.gemm_bf16_lora(A, B, ids, down, up, D)
            for now in kinds:
                ids.copy_(now)
                D.fill_(float("nan"))
                graph.replay()
                s.synchronize()
                assert torch.equal(D.double(), definition(torch, A, B, now, down, up, None)[0])
            assert tg.workspace_alloc_count() == before
    assert tg.tg_device_status()[0] == tg.TG_OK


def test_no_adapters_and_an_empty_contraction(tg):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(4)
    A, B, down, up = case(gen, quarters, 30, 40, 64, 2, 8)
    ids = ids_of("any", 30, 2, 1)
    none = tg.gemm_bf16_lora(A, B, ids, down[:0], up[:0])
    assert torch.equal(none.double(), A.double() @ B.double().T)
    got = tg.gemm_bf16_lora(A[:, :0], B[:, :0], ids, down[..., :0], up, epilogue_add=2.0)
    assert (got == 2.0).all()
    assert tg.gemm_bf16_lora(A[:0], B, ids[:0], down, up).shape == (0, 40)
