"""The grouped products where they can go wrong: values that no result may
depend on, rows picked by index, epilogues per group, strides and views, bad
offsets, lengths of zero, long contractions, streams and graphs; gradients
against differences of the product.

Tolerances as in test_grouped_gpu.py; the ones for long contractions and for
differences are derived where they are used.
"""
import numpy as np
import pytest

from tests._gpu import torch_cuda
from tests.test_grouped_gpu import forward64, normal, offsets_of, quarters, same, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    torch_cuda()
    import blackwell_tile_gemm_gb300 as m
    m.lib()
    return m


def gen_of(seed):
    torch = torch_cuda()
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.3895e38])
@pytest.mark.parametrize("sizes", [[70, 130, 5, 300], [3, 2, 1, 4] * 9])
def test_a_group_s_values_stay_with_it(tg, bad, sizes):
    """Rows, gradients and weights of one group reach its own results only."""
    torch = torch_cuda()
    N, K = 200, 328
    gen = gen_of(1)
    cut, off = offsets_of(sizes)
    M, groups = int(cut[-1]), len(sizes)
    A, G, B = quarters(gen, M, K), quarters(gen, M, N), quarters(gen, groups, N, K)
    D, dA, dB = (tg.gemm_bf16_grouped(A, B, off), tg.gemm_bf16_grouped_dgrad(G, B, off),
                 tg.gemm_bf16_grouped_wgrad(G, A, off))
    g = 1
    s = slice(int(cut[g]), int(cut[g + 1]))
    out = torch.ones(M, dtype=torch.bool, device="cuda")
    out[s] = False
    A[s], G[s], B[g] = bad, bad, bad
    assert torch.equal(tg.gemm_bf16_grouped(A, B, off)[out], D[out])
    assert torch.equal(tg.gemm_bf16_grouped_dgrad(G, B, off)[out], dA[out])
    dB2 = tg.gemm_bf16_grouped_wgrad(G, A, off)
    for h in range(groups):
        assert h == g or torch.equal(dB2[h], dB[h])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[40, 0, 300, 33], [1, 2, 0, 5]])
def test_rows_picked_by_index(tg, out, sizes):
    """Repeats, any order, and indices outside A, which give zero rows."""
    torch = torch_cuda()
    dt = torch.float32 if out == "f32" else torch.bfloat16
    N, K, a_rows = 136, 203, 90
    gen = gen_of(2)
    cut, off = offsets_of(sizes, 2)
    M, groups = int(cut[-1]) + 3, len(sizes)
    A, G, B = quarters(gen, a_rows, K), quarters(gen, M, N), quarters(gen, groups, N, K)
    idx = torch.randint(0, a_rows, (M,), generator=gen, device="cuda", dtype=torch.int32)
    idx[3], idx[4], idx[M - 4] = -1, a_rows, 2 ** 31 - 1
    inside = (idx >= 0) & (idx < a_rows)
    rows = torch.where(inside[:, None], A[idx.clamp(0, a_rows - 1).long()].float(), 0.0)
    rows = rows.to(torch.bfloat16)
    want, _ = forward64(torch, rows, B, cut)
    assert same(torch, tg.gemm_bf16_grouped(A, B, off, row_idx=idx, out_dtype=dt), want.to(dt))
    got = tg.gemm_bf16_grouped_wgrad(G, A, off, row_idx=idx, out_dtype=dt)
    for g in range(groups):
        s = slice(int(cut[g]), int(cut[g + 1]))
        assert same(torch, got[g], (G[s].double().T @ rows[s].double()).to(dt))


@pytest.mark.parametrize("sizes", [[40, 0, 300, 33], [1, 2, 0, 5]])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_epilogues(tg, sizes, out):
    """Each op, a bias of its own for each group; rows in no group stay zero."""
    torch = torch_cuda()
    dt = torch.float32 if out == "f32" else torch.bfloat16
    N, K = 137, 264
    gen = gen_of(3)
    cut, off = offsets_of(sizes, 1)
    M, groups = int(cut[-1]) + 2, len(sizes)
    A, B = normal(gen, M, K), normal(gen, groups, N, K)
    bias = torch.randn(groups, N, generator=gen, device="cuda")
    acc, mag = forward64(torch, A, B, cut)
    per_row = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    own = torch.zeros(M, 1, dtype=torch.bool, device="cuda")
    for g in range(groups):
        per_row[int(cut[g]):int(cut[g + 1])] = bias[g].double()
        own[int(cut[g]):int(cut[g + 1])] = True
    silu = lambda t: t * torch.sigmoid(t)  # noqa: E731
    ops = [(dict(epilogue_add=1.5), acc + 1.5, 1.0), (dict(affine=(-2.0, 0.25)), acc * -2 + 0.25, 2.0),
           (dict(silu_affine=(1.5, -0.5)), silu(acc) * 1.5 - 0.5, 1.65),
           (dict(bias=bias), acc + per_row, 1.0),
           (dict(bias=bias, bias_silu=True), silu(acc + per_row), 1.1)]
    for kw, ref, lip in ops:
        got = tg.gemm_bf16_grouped(A, B, off, out_dtype=dt, **kw)
        ref = torch.where(own, ref, 0.0)
        # The op's Lipschitz constant times the product's bound, and the
        # output's own rounding: 2^-8 (bf16), 2^-21 (f32 arithmetic and exp).
        extra = (2.0 ** -8 if out == "bf16" else 2.0 ** -21) * ref.abs()
        rtol = 8e-3 if out == "bf16" else 1e-5
        tol = lip * rtol * mag + extra + (1e-3 if out == "bf16" else 1e-6)
        assert float(((got.double() - ref).abs() / tol).max()) <= 1.0, kw
        assert (got[~own[:, 0]] == 0).all()


def test_views_and_results_of_the_caller(tg):
    """Strided operands; results in views whose surroundings keep their values."""
    torch = torch_cuda()
    N, K, groups = 100, 152, 3
    gen = gen_of(4)
    cut, off = offsets_of([130, 0, 77])
    M = int(cut[-1])
    A = quarters(gen, M, K + 24)[:, 8:8 + K]
    G = quarters(gen, 2 * M, N)[::2]
    B = quarters(gen, 2 * groups, N + 5, K + 8)[1::2, :N, :K]
    for dt, w in ((torch.float32, 4), (torch.bfloat16, 8)):
        D = torch.full((M + 2, N + 2 * w + 4), 7.0, device="cuda", dtype=dt)
        tg.gemm_bf16_grouped(A, B, off, D[1:M + 1, w:w + N])
        assert same(torch, D[1:M + 1, w:w + N], forward64(torch, A, B, cut)[0].to(dt))
        dA = torch.full((M, K + 2 * w), 7.0, device="cuda", dtype=dt)
        tg.gemm_bf16_grouped_dgrad(G, B, off, dA[:, w:w + K])
        assert same(torch, dA[:, w:w + K], forward64(torch, G, B.transpose(1, 2), cut)[0].to(dt))
        dB = torch.full((groups, N + 3, K + 2 * w), 7.0, device="cuda", dtype=dt)
        tg.gemm_bf16_grouped_wgrad(G, A, off, dB[:, 1:N + 1, w:w + K])
        for g in range(groups):
            s = slice(int(cut[g]), int(cut[g + 1]))
            assert same(torch, dB[g, 1:N + 1, w:w + K], (G[s].double().T @ A[s].double()).to(dt))
        D[1:M + 1, w:w + N] = 7
        dA[:, w:w + K] = 7
        dB[:, 1:N + 1, w:w + K] = 7
        assert (D == 7).all() and (dA == 7).all() and (dB == 7).all()


@pytest.mark.parametrize("raw", [[0, 50, 30, 100], [-5, 20, 60, 100], [0, 40, 200, 100],
                                 [90, 10, 20, 30], [0, 2 ** 31 - 1, -2 ** 31, 7]])
def test_bad_offsets_are_clamped_and_reported(tg, raw):
    """Each limit clamped to [0, M] and raised to the ones before it."""
    torch = torch_cuda()
    M, N, K = 100, 40, 64
    gen = gen_of(5)
    A, G, B = quarters(gen, M, K), quarters(gen, M, N), quarters(gen, 3, N, K)
    off = torch.tensor(raw, dtype=torch.int64).to(torch.int32).cuda()
    cut = np.maximum.accumulate(np.clip(np.array(raw), 0, M))
    tg.tg_device_status()
    for run in (lambda: tg.gemm_bf16_grouped(A, B, off), lambda: tg.gemm_bf16_grouped_dgrad(G, B, off),
                lambda: tg.gemm_bf16_grouped_wgrad(G, A, off)):
        got = run()
        assert tg.tg_device_status() == (tg.TG_ERR_INVALID_ARG, 40)
        assert tg.tg_device_status()[0] == tg.TG_OK
    assert same(torch, tg.gemm_bf16_grouped(A, B, off), forward64(torch, A, B, cut)[0])
    assert same(torch, got[1], G[cut[1]:cut[2]].double().T @ A[cut[1]:cut[2]].double())
    tg.tg_device_status()


def test_lengths_of_zero(tg):
    torch = torch_cuda()
    bf = torch.bfloat16
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    empty = lambda *shape: torch.empty(*shape, dtype=bf, device="cuda")  # noqa: E731
    B = torch.randn(3, 16, 24, device="cuda").to(bf)
    assert tg.gemm_bf16_grouped(empty(0, 24), B, zero).shape == (0, 16)
    assert tg.gemm_bf16_grouped_dgrad(empty(0, 16), B, zero).shape == (0, 24)
    D = torch.full((3, 16, 24), float("nan"), device="cuda")
    tg.gemm_bf16_grouped_wgrad(empty(0, 16), empty(0, 24), zero, D)
    assert (D == 0).all()
    # Rows, but none in a group.
    A, G = torch.randn(50, 24, device="cuda").to(bf), torch.randn(50, 16, device="cuda").to(bf)
    assert (tg.gemm_bf16_grouped(A, B, zero, epilogue_add=3.0) == 0).all()
    assert (tg.gemm_bf16_grouped_dgrad(G, B, zero + 50) == 0).all()
    assert (tg.gemm_bf16_grouped_wgrad(G, A, zero + 7) == 0).all()
    # An empty contraction: the epilogue of zero in groups, zero outside.
    off = torch.tensor([5, 5, 20, 40], dtype=torch.int32, device="cuda")
    bias = torch.randn(3, 16, device="cuda")
    got = tg.gemm_bf16_grouped(empty(50, 0), empty(3, 16, 0), off, bias=bias)
    want = torch.zeros(50, 16, device="cuda")
    want[5:20], want[20:40] = bias[1], bias[2]
    assert torch.equal(got, want)
    assert (tg.gemm_bf16_grouped_dgrad(empty(50, 0), empty(3, 0, 24), off) == 0).all()
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("sizes", [[9000], [20000, 3, 6500]])
def test_long_contractions_keep_f32(tg, sizes):
    """f32 results of long sums: with plain accumulation on the tensor cores the
    error grows with the length; chunks of 768 terms keep it below 4e-6 of
    sqrt(length), the root mean square of the sums of normal products (a sum
    of n terms rounds at most by n / 16 * 2^-23 of its size within a chunk)."""
    torch = torch_cuda()
    gen = gen_of(6)
    N, K = 130, 264
    cut, off = offsets_of(sizes)
    M = int(cut[-1])
    A, G = normal(gen, M, K), normal(gen, M, N)
    dB = tg.gemm_bf16_grouped_wgrad(G, A, off)
    for g, n in enumerate(sizes):
        s = slice(int(cut[g]), int(cut[g + 1]))
        ref = G[s].double().T @ A[s].double()
        assert float((dB[g].double() - ref).norm() / ref.norm()) <= 4e-6
    W = normal(gen, 2, 96, 8192)
    X = normal(gen, 700, 8192)
    off2 = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    ref, _ = forward64(torch, X, W, [0, 300, 700])
    D = tg.gemm_bf16_grouped(X, W, off2)
    assert float((D.double() - ref).norm() / ref.norm()) <= 4e-6


# Tiles for less than two waves and contractions long enough to be split: the
# pieces' sums are exact for quarter integers, and the same bits every time.
@pytest.mark.parametrize("sizes,N,K", [([7000], 300, 520), ([5000, 12000, 0, 9000], 256, 130),
                                       ([500, 900], 264, 6200), ([3, 1, 2], 128, 4096),
                                       ([17, 9], 2000, 2048)])
def test_split_contractions_exact_and_repeatable(tg, sizes, N, K):
    torch = torch_cuda()
    gen = gen_of(7)
    cut, off = offsets_of(sizes)
    M, groups = int(cut[-1]), len(sizes)
    A, G, B = quarters(gen, M, K), quarters(gen, M, N), quarters(gen, groups, N, K)
    D, dA, dB = (tg.gemm_bf16_grouped(A, B, off), tg.gemm_bf16_grouped_dgrad(G, B, off),
                 tg.gemm_bf16_grouped_wgrad(G, A, off))
    assert same(torch, D, forward64(torch, A, B, cut)[0])
    assert same(torch, dA, forward64(torch, G, B.transpose(1, 2), cut)[0])
    for g in range(groups):
        s = slice(int(cut[g]), int(cut[g + 1]))
        assert same(torch, dB[g], G[s].double().T @ A[s].double())
    for dt in (torch.float32, torch.bfloat16):
        X, W, Y = normal(gen, M, K), normal(gen, groups, N, K), normal(gen, M, N)
        first = (tg.gemm_bf16_grouped(X, W, off, out_dtype=dt),
                 tg.gemm_bf16_grouped_dgrad(Y, W, off, out_dtype=dt),
                 tg.gemm_bf16_grouped_wgrad(Y, X, off, out_dtype=dt))
        again = (tg.gemm_bf16_grouped(X, W, off, out_dtype=dt),
                 tg.gemm_bf16_grouped_dgrad(Y, W, off, out_dtype=dt),
                 tg.gemm_bf16_grouped_wgrad(Y, X, off, out_dtype=dt))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        ref, mag = forward64(torch, X, W, cut)
        assert within(torch, first[0], ref, mag)


def test_gradients_against_differences(tg):
    """loss = sum(C * product): its gradients with respect to one row and one
    weight are those of C through dgrad and wgrad.  The product is linear in
    each, so a difference of losses is the gradient times the step exactly, up
    to the rounding of f32 results: all values are quarter integers and the
    step is 1/4, so the equality is exact."""
    torch = torch_cuda()
    gen = gen_of(8)
    cut, off = offsets_of([30, 0, 41, 9])
    M, N, K, groups = int(cut[-1]), 48, 56, 4
    A, B, C = quarters(gen, M, K), quarters(gen, groups, N, K), quarters(gen, M, N)
    loss = lambda: (C.double() * tg.gemm_bf16_grouped(A, B, off).double()).sum()  # noqa: E731
    dA, dB = tg.gemm_bf16_grouped_dgrad(C, B, off), tg.gemm_bf16_grouped_wgrad(C, A, off)
    base = loss()
    for i, k in ((0, 0), (29, 55), (30, 7), (70, 20), (79, 31)):
        A[i, k] += 0.25
        assert float(loss() - base) == 0.25 * float(dA[i, k])
        A[i, k] -= 0.25
    for g, n, k in ((0, 0, 0), (1, 5, 5), (2, 47, 55), (3, 13, 2)):
        B[g, n, k] += 0.25
        assert float(loss() - base) == 0.25 * float(dB[g, n, k])
        B[g, n, k] -= 0.25


def test_streams_reservation_and_graphs(tg):
    """On a stream of its own, without allocating after a reservation, captured
    into a graph and replayed with other offsets."""
    torch = torch_cuda()
    gen = gen_of(9)
    M, N, K, groups = 600, 264, 520, 5
    A, B = quarters(gen, M, K), quarters(gen, groups, N, K)
    G = quarters(gen, M, N)
    idx = torch.randperm(M, generator=gen, device="cuda").int()
    cuts = [np.array([0, 100, 100, 350, 351, 600]), np.array([5, 5, 300, 300, 599, 600])]
    off = torch.from_numpy(cuts[0].astype(np.int32)).cuda()
    D, dB = torch.empty(M, N, device="cuda"), torch.empty(groups, N, K, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tg.reserve_workspace(tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_GATHER, M, N, K))
        run = lambda: (tg.gemm_bf16_grouped(A, B, off, D, row_idx=idx),  # noqa: E731
                       tg.gemm_bf16_grouped_wgrad(G, A, off, dB))
        run()
        s.synchronize()
        before = tg.workspace_alloc_count()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
        for cut in cuts:
            off.copy_(torch.from_numpy(cut.astype(np.int32)))
            D.fill_(float("nan"))
            graph.replay()
            s.synchronize()
            assert same(torch, D, forward64(torch, A, B, cut, idx)[0])
            for g in range(groups):
                t = slice(int(cut[g]), int(cut[g + 1]))
                assert same(torch, dB[g], G[t].double().T @ A[t].double())
        assert tg.workspace_alloc_count() == before
    assert tg.tg_device_status()[0] == tg.TG_OK


def test_the_widest_group_table(tg):
    torch = torch_cuda()
    gen = gen_of(10)
    groups, M, N, K = tg.TG_MAX_GROUPS, 3000, 8, 16
    sizes = np.random.default_rng(0).multinomial(M, np.ones(groups) / groups)
    cut, off = offsets_of(sizes)
    A, B = quarters(gen, M, K), quarters(gen, groups, N, K)
    g = torch.from_numpy(np.repeat(np.arange(groups), sizes)).cuda()
    want = torch.einsum("ik,ink->in", A.double(), B[g].double())
    assert same(torch, tg.gemm_bf16_grouped(A, B, off), want)
    dB = tg.gemm_bf16_grouped_wgrad(want.to(torch.bfloat16), A, off)
    full = torch.zeros(groups, N, K, dtype=torch.float64, device="cuda")
    full.index_add_(0, g, torch.einsum("in,ik->ink", want.to(torch.bfloat16).double(), A.double()))
    assert float((dB.double() - full).abs().max()) <= 1e-5 * float(full.abs().max())
