"""gemm_bf16_xent and gemm_bf16_xent_grad against the definition in 64 bits.

Tolerances, before anything ran.  A logit z = scale * sum a b in f32 is off by at
most ez = 1e-5 scale sum |a b| + 1e-6, the bound of every product here.  lse is a
weighted mean of such errors, plus the rounding of its own sum (2e-6 of it and of 1);
the loss has the target's error beside it.  dz = w (p - [target]): p = exp(z - lse) is
off by 2 ez + 4e-6 of itself, and the rounding of dz to bf16 by 2^-8 of itself (two
terms: 2^-16).  The products add 1e-5 of the sum of magnitudes, a bf16 result 2^-8 of
itself.
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


def rows(gen, m, k, pad=0, scale=1.0):
    """bf16 normal values, a row stride of a multiple of 8 and `pad` more columns."""
    import torch
    ld = -(-k // 8) * 8 + pad
    t = (torch.randn(m, ld, generator=gen, device="cuda") * scale).to(torch.bfloat16)
    return t[:, :k]


def inputs(seed, M, N, K, spread=1.5, ignored=0.1, pad=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    A, B = rows(gen, M, K, pad), rows(gen, N, K, pad, spread * max(K, 1) ** -0.5)
    t = torch.randint(0, max(N, 1), (M,), generator=gen, device="cuda", dtype=torch.int32)
    drop = torch.rand(M, generator=gen, device="cuda") < ignored
    bad = torch.tensor([-1, -100, N, 2 ** 31 - 1, -2 ** 31], device="cuda", dtype=torch.int32)
    t = torch.where(drop, bad[torch.arange(M, device="cuda") % 5], t)
    grad = torch.rand(M, generator=gen, device="cuda") + 0.5
    return A, B, t, grad


def reference(A, B, t, grad, scale):
    """Everything in 64 bits, with the tolerances of the module's text."""
    import torch
    a, b = A.double(), B.double()
    M, N = a.shape[0], b.shape[0]
    z = scale * (a @ b.T)
    ez = (1e-5 * scale * (a.abs() @ b.abs().T) + 1e-6).amax(1) if N else a.new_zeros(M)
    lse = torch.logsumexp(z, 1) if N else torch.full((M,), -float("inf"), device="cuda",
                                                     dtype=torch.float64)
    inside = (t >= 0) & (t < N)
    at = t.long().clamp(0, max(N - 1, 0))
    zt = z.gather(1, at[:, None])[:, 0] if N else lse
    zero = torch.zeros_like(lse)
    out = dict(lse=lse, loss=torch.where(inside, lse - zt, zero))
    out["lse_tol"] = ez + 2e-6 * (1 + lse.abs())
    out["loss_tol"] = 2 * ez + 2e-6 * (1 + out["loss"].abs())
    w = torch.where(inside, (grad.double() if grad is not None else zero + 1) * scale, zero)
    p = torch.exp(z - lse[:, None])
    dz = p.clone()
    dz[torch.arange(M, device="cuda"), at] -= 1.0
    dz *= w[:, None]
    out["dA"], out["dB"] = dz @ b, dz.T @ a
    ep = p * (w.abs() * (2 * ez + 4e-6))[:, None]
    for terms, half in ((1, 2.0 ** -8), (2, 0.0)):
        e = dz.abs() * (2.0 ** -8 if terms == 1 else 2.0 ** -16) + ep + 1e-5 * dz.abs()
        out[f"dA_tol{terms}"] = e @ b.abs() + half * out["dA"].abs() + 1e-12
        out[f"dB_tol{terms}"] = e.T @ a.abs() + half * out["dB"].abs() + 1e-12
    return out


def within(got, want, tol):
    import torch
    assert got.shape == want.shape
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    bad = off > tol
    assert not bad.any(), (int(bad.sum()), float((off / tol).max()))


def check(tg, A, B, t, grad, scale=1.0, dtypes=None):
    import torch
    r = reference(A, B, t, grad, scale)
    loss, lse = tg.gemm_bf16_xent(A, B, t, scale=scale)
    within(loss, r["loss"], r["loss_tol"])
    within(lse, r["lse"], r["lse_tol"])
    outside = (t < 0) | (t >= B.shape[0])
    assert (loss[outside] == 0).all()
    for dtype in dtypes or (torch.bfloat16, torch.float32):
        dA, dB = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, scale=scale, out_dtype=dtype)
        assert dA.dtype == dB.dtype == dtype
        terms = 1 if dtype == torch.bfloat16 else 2
        within(dA, r["dA"], r[f"dA_tol{terms}"])
        within(dB, r["dB"], r[f"dB_tol{terms}"])
        assert (dA[outside] == 0).all()
    assert tg.tg_device_status()[0] == tg.TG_OK


@pytest.mark.parametrize("M,N,K,pad", [
    (1, 1, 8, 0), (1, 2, 1, 0), (1, 33, 64, 0), (3, 50, 40, 8), (7, 300, 129, 0), (127, 1000, 72, 0),
    (128, 257, 128, 0), (129, 4097, 200, 24), (255, 31, 520, 0), (257, 5000, 136, 0),
    (300, 12345, 1001, 0), (130, 2999, 2600, 0), (64, 40000, 512, 0), (1, 65000, 1024, 0),
    (1000, 513, 4100, 0), (513, 777, 63, 0), (2049, 3000, 96, 0)])
def test_loss_and_gradients(tg, M, N, K, pad):
    check(tg, *inputs(M + 3 * N + 7 * K, M, N, K, pad=pad))


@pytest.mark.parametrize("M,N,K", [(9000, 20000, 72), (5000, 30000, 40)])
def test_several_pieces_of_the_vocabulary(tg, M, N, K):
    """More dz than the workspace holds at a time, for one term and for two."""
    check(tg, *inputs(M, M, N, K))


@pytest.mark.parametrize("scale", [0.05, 7.5])
@pytest.mark.parametrize("M,N", [(40, 900), (400, 900)])
def test_scale(tg, M, N, scale):
    A, B, t, grad = inputs(5, M, N, 200)
    check(tg, A, B, t, grad, scale=scale)
    check(tg, A, B, t, None, scale=scale)


def test_confident_rows_keep_their_digits(tg):
    """A target far above the others: the loss is a small rest of large logits.
    z is off by 1e-6 of itself at most (f32 sums), which the loss takes on times the
    distance of about 12 (2e-5 of it); a sum that begins with 1 is rounded by 2^-24 up
    to 32 times in a thread, 3 in a tile and 6 where the tiles join."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = 200, 3000, 4096
    B = rows(gen, N, K, scale=1.5 * K ** -0.5)
    t = torch.arange(M, device="cuda", dtype=torch.int32) * 7
    lean = torch.linspace(3.0, 8.0, M, device="cuda")[:, None]
    A = (torch.randn(M, K, generator=gen, device="cuda") + lean * B[t.long()].float()).bfloat16()
    z = A.double() @ B.double().T
    want = torch.logsumexp(z, 1) - z.gather(1, t.long()[:, None])[:, 0]
    loss, _ = tg.gemm_bf16_xent(A, B, t)
    off = (loss.double() - want).abs()
    assert (off <= 2e-5 * want + 45 * 2.0 ** -24).all(), float((off / want).max())


@pytest.mark.parametrize("rows_,weights", [(True, False), (False, True), (False, False)])
def test_one_gradient_alone_and_given_results(tg, rows_, weights):
    import torch
    A, B, t, grad = inputs(11, 150, 700, 90)
    _, lse = tg.gemm_bf16_xent(A, B, t)
    both = tg.gemm_bf16_xent_grad(A, B, t, lse, grad)
    dA, dB = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, rows=rows_, weights=weights)
    assert dA is None if not rows_ else torch.equal(dA, both[0])
    assert dB is None if not weights else torch.equal(dB, both[1])
    # Given results, their rows apart; what lies between stays.
    wide = torch.full((150, 104), 7.0, device="cuda", dtype=torch.bfloat16)
    tall = torch.full((700, 104), 7.0, device="cuda", dtype=torch.bfloat16)
    tg.gemm_bf16_xent_grad(A, B, t, lse, grad, wide[:, :90], tall[:, :90])
    assert torch.equal(wide[:, :90], both[0]) and torch.equal(tall[:, :90], both[1])
    assert (wide[:, 90:] == 7).all() and (tall[:, 90:] == 7).all()


def test_rows_without_a_target_may_hold_anything(tg):
    """Padding with NaN and infinities reaches nothing; without any target all is 0."""
    import torch
    A, B, t, grad = inputs(13, 300, 500, 100, ignored=0.3)
    outside = (t < 0) | (t >= 500)
    clean, dirty = (torch.zeros(300, 104, device="cuda", dtype=A.dtype)[:, :100] for _ in range(2))
    clean[~outside] = dirty[~outside] = A[~outside]
    dirty[outside] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38],
                                  device="cuda", dtype=A.dtype).repeat(25)
    odd = torch.where(outside, torch.full_like(grad, float("nan")), grad)
    for dtype in (torch.bfloat16, torch.float32):
        loss, lse = tg.gemm_bf16_xent(clean, B, t)
        want = tg.gemm_bf16_xent_grad(clean, B, t, lse, grad, out_dtype=dtype)
        loss2, lse2 = tg.gemm_bf16_xent(dirty, B, t)
        got = tg.gemm_bf16_xent_grad(dirty, B, t, lse2, odd, out_dtype=dtype)
        assert torch.equal(loss, loss2)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        none = torch.full_like(t, -1)
        loss, lse = tg.gemm_bf16_xent(dirty, B, none)
        got = tg.gemm_bf16_xent_grad(dirty, B, none, lse, odd, out_dtype=dtype)
        assert (loss == 0).all() and (got[0] == 0).all() and (got[1] == 0).all()


def test_infinite_and_nan_logits_stay_in_their_row(tg):
    import torch
    A, B, t, _ = inputs(17, 140, 600, 64, ignored=0.0)
    A[3] = float("nan")
    A[5] = 0.0
    A[5, 0] = float("inf")        # +-inf logits, whichever sign B has
    A[9] = 0.0                    # all logits equal
    loss, lse = tg.gemm_bf16_xent(A, B, t)
    assert torch.isnan(loss[3]) and torch.isnan(lse[3])
    assert lse[5] == float("inf")
    rest = torch.ones(140, device="cuda", dtype=torch.bool)
    rest[[3, 5]] = False
    r = reference(A[rest], B, t[rest], None, 1.0)
    within(loss[rest], r["loss"], r["loss_tol"])
    within(lse[rest], r["lse"], r["lse_tol"])
    # Logits of -inf (a vocabulary entry masked out) are as if they were not there.
    A2, B2 = A.clone(), B.clone()
    A2[:, 0] = 1.0
    A2[3] = A2[5] = 1.0
    B2[100:130] = 0.0
    B2[100:130, 0] = -float("inf")
    t2 = torch.where((t >= 100) & (t < 130), torch.zeros_like(t), t)
    keep = torch.cat([torch.arange(100), torch.arange(130, 600)]).cuda()
    t3 = torch.where(t2 >= 130, t2 - 30, t2)
    loss, lse = tg.gemm_bf16_xent(A2, B2, t2)
    r = reference(A2, B2[keep], t3, None, 1.0)
    within(loss, r["loss"], r["loss_tol"])
    within(lse, r["lse"], r["lse_tol"])


def test_far_apart_logits(tg):
    """Maxima of thousands on either side: neither overflow nor an empty sum."""
    import torch
    A, B, t, _ = inputs(19, 200, 1000, 64, ignored=0.0)
    A = A * 300
    r = reference(A, B, t, None, 1.0)
    loss, lse = tg.gemm_bf16_xent(A, B, t)
    within(loss, r["loss"], r["loss_tol"])
    within(lse, r["lse"], r["lse_tol"])
    A[:] = 0
    A[:, 0] = -5000.0
    B[:] = 0
    B[:, 0] = 1.0                 # every logit the same, about -5000
    loss, lse = tg.gemm_bf16_xent(A, B, t)
    want = torch.log(torch.tensor(1000.0, dtype=torch.float64))
    # (differences of equal logits are exact; lse is rounded at its own size)
    assert ((loss.double().cpu() - want).abs() <= 1e-6 + 2e-6 * want).all()
    assert ((lse.double().cpu() - (want + float(A[0, 0]))).abs() <= 5000 * 2.0 ** -22).all()


def test_empty_sizes(tg):
    import torch
    A, B, t, grad = inputs(23, 5, 9, 16, ignored=0.0)
    loss, lse = tg.gemm_bf16_xent(A[:0], B, t[:0])
    assert loss.shape == lse.shape == (0,)
    dA, dB = tg.gemm_bf16_xent_grad(A[:0], B, t[:0], lse, None)
    assert dA.shape == (0, 16) and dB.shape == (9, 16) and (dB == 0).all()
    loss, lse = tg.gemm_bf16_xent(A, B[:0], t)
    assert (loss == 0).all() and (lse == -float("inf")).all()
    dA, dB = tg.gemm_bf16_xent_grad(A, B[:0], t, lse, None, out_dtype=torch.float32)
    assert (dA == 0).all() and dB.shape == (0, 16)
    loss, lse = tg.gemm_bf16_xent(A[:, :0], B[:, :0], t)
    assert torch.allclose(lse.cpu(), torch.log(torch.full((5,), 9.0)), rtol=1e-6)
    assert torch.equal(loss, lse)
    dA, dB = tg.gemm_bf16_xent_grad(A[:, :0], B[:, :0], t, lse, None)
    assert dA.shape == (5, 0) and dB.shape == (9, 0)


def test_gradient_agrees_with_differences(tg):
    """Central differences of the 64-bit loss along random directions."""
    import torch
    A, B, t, grad = inputs(29, 60, 300, 48)
    _, lse = tg.gemm_bf16_xent(A, B, t, scale=2.0)
    dA, dB = tg.gemm_bf16_xent_grad(A, B, t, lse, grad, scale=2.0, out_dtype=torch.float32)
    inside = (t >= 0) & (t < 300)

    def total(a, b):
        z = 2.0 * a @ b.T
        own = z.gather(1, t.long().clamp(0, 299)[:, None])[:, 0]
        return ((torch.logsumexp(z, 1) - own) * grad.double() * inside).sum()

    a, b, h = A.double(), B.double(), 1e-5
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        u = torch.randn(a.shape, generator=gen, device="cuda", dtype=torch.float64)
        v = torch.randn(b.shape, generator=gen, device="cuda", dtype=torch.float64)
        slope = (total(a + h * u, b + h * v) - total(a - h * u, b - h * v)) / (2 * h)
        got = (dA.double() * u).sum() + (dB.double() * v).sum()
        # f32 gradients: 3e-5 of the sum of magnitudes, far above h^2.
        size = (dA.double() * u).abs().sum() + (dB.double() * v).abs().sum()
        assert abs(float(got - slope)) <= 3e-5 * float(size)


def test_same_bits_every_time_and_on_another_stream(tg):
    import torch
    A, B, t, grad = inputs(31, 700, 9000, 328)
    out = []
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side, side, torch.cuda.current_stream()):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            loss, lse = tg.gemm_bf16_xent(A, B, t)
            out.append((loss, lse) + tg.gemm_bf16_xent_grad(A, B, t, lse, grad))
        torch.cuda.synchronize()
    for o in out[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o, out[0]))


def test_captured_twice_on_two_streams(tg):
    """Reserved streams: two graphs, replayed at the same time, allocate nothing."""
    import torch
    sizes = (300, 20000, 256)
    need = max(tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_XENT, *sizes),
               tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_XENT_GRAD, *sizes, d_dtype=tg.TG_D_BF16),
               tg.workspace_bytes(tg.TG_CALL_GEMM_BF16_XENT_GRAD, *sizes, d_dtype=tg.TG_D_F32))
    graphs, results, wanted, data = [], [], [], []
    for seed in (1, 2):
        A, B, t, grad = inputs(seed, *sizes)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        tg.reserve_workspace(need, stream=s)
        count = tg.workspace_alloc_count()
        with torch.cuda.stream(s):
            loss, lse = tg.gemm_bf16_xent(A, B, t)
            wanted.append((loss, lse) + tg.gemm_bf16_xent_grad(A, B, t, lse, grad) +
                          tg.gemm_bf16_xent_grad(A, B, t, lse, grad, out_dtype=torch.float32))
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            loss, lse = tg.gemm_bf16_xent(A, B, t)
            results.append((loss, lse) + tg.gemm_bf16_xent_grad(A, B, t, lse, grad) +
                           tg.gemm_bf16_xent_grad(A, B, t, lse, grad, out_dtype=torch.float32))
        graphs.append((g, s))
        data.append((A, B, t, grad))
        assert tg.workspace_alloc_count() == count
    for _ in range(3):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for got, want in zip(results, wanted):
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    # Other values in the same buffers, and the graph gives theirs.
    A, B, t, grad = data[0]
    new = inputs(77, *sizes)
    for old, n in zip((A, B, t, grad), new):
        old.copy_(n)
    torch.cuda.synchronize()
    with torch.cuda.stream(graphs[0][1]):
        graphs[0][0].replay()
    torch.cuda.synchronize()
    r = reference(*new, 1.0)
    within(results[0][0], r["loss"], r["loss_tol"])
    within(results[0][2], r["dA"], r["dA_tol1"])
    within(results[0][5], r["dB"], r["dB_tol2"])


def test_captured_without_a_reservation_is_refused(tg):
    import torch
    A, B, t, grad = inputs(41, 300, 3000, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    codes = []
    with torch.cuda.graph(g, stream=s):
        for call in (lambda: tg.gemm_bf16_xent(A, B, t),
                     lambda: tg.gemm_bf16_xent_grad(A, B, t, grad, grad)):
            try:
                call()
            except tg.TgError as e:
                codes.append(e.code)
        grad.add_(0)
    assert codes == [tg.TG_ERR_WORKSPACE] * 2


def test_offsets_beyond_32_bits(tg):
    """More than 2^31 elements of B and dB: the last rows of a large vocabulary."""
    import torch
    M, N, K = 3, 270000, 8192
    A, B, t, grad = inputs(43, M, N, K, ignored=0.0)
    t[:] = torch.tensor([0, N - 1, N - 300], device="cuda", dtype=torch.int32)
    loss, lse = tg.gemm_bf16_xent(A, B, t)
    dA, dB = tg.gemm_bf16_xent_grad(A, B, t, lse, grad)
    a = A.double()
    z = torch.cat([a @ B[i:i + 30000].double().T for i in range(0, N, 30000)], 1)
    want = torch.logsumexp(z, 1)
    # 1e-5 of sum |a b|, about 1.5 * 0.64 * sqrt(K) here.
    tol = 1e-5 * 0.96 * K ** 0.5 + 2e-6 * 14
    assert ((lse.double() - want).abs() <= tol).all()
    assert ((loss.double() - (want - z.gather(1, t.long()[:, None])[:, 0])).abs() <= 2 * tol).all()
    dz = torch.exp(z - want[:, None])
    dz[torch.arange(M), t.long()] -= 1.0
    dz *= grad.double()[:, None]
    for lo in (0, N // 2, N - 1000):
        ref = dz[:, lo:lo + 1000].T @ a
        mag = dz[:, lo:lo + 1000].T.abs() @ a.abs()
        # dz: 2^-8 of rounding and 2 tol of p; the result 2^-8.
        within(dB[lo:lo + 1000], ref, (2.0 ** -8 + 2 * tol + 2e-5) * mag + 2.0 ** -8 * ref.abs() + 1e-12)
    ref, mag = 0, 0
    for i in range(0, N, 30000):
        b = B[i:i + 30000].double()
        ref = ref + dz[:, i:i + 30000] @ b
        mag = mag + dz[:, i:i + 30000].abs() @ b.abs()
    within(dA, ref, (2.0 ** -8 + 2 * tol + 2e-5) * mag + 2.0 ** -8 * ref.abs())
