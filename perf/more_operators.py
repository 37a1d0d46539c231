"""Workloads of the operators at both ends of a language model's training step, around its products:
the softmax cross entropy over a vocabulary and its gradient, the lookup of token rows and its
gradient, and the balance loss of a router with its gradient.

A case is a dict of plain sizes.  ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes
one pass: with ``own`` through this package's entry points, otherwise with elementary torch
operations in 32 bits, rounded once at the end.  ``exact`` evaluates the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

LOSS, STEP, LOOKUP, LOOKUP_GRAD, BALANCE = "loss", "step", "lookup", "lookup grad", "balance"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # Scoring one token of a request (its loss, no gradient): bound by reading the vocabulary.
        dict(name="loss: single token", op=LOSS, m=1, n=32000, k=4096),
        # Evaluation of a ragged batch, odd sizes, rows that end off a 16-byte boundary.
        dict(name="loss: ragged", op=LOSS, m=777, n=50257, k=1001),
        # Evaluation of 8192 tokens over a large vocabulary.
        dict(name="loss: batch", op=LOSS, m=8192, n=128000, k=4096),
        # Tuning on a few tokens: loss and both gradients, bound by the vocabulary's matrix.
        dict(name="step: few tokens", op=STEP, m=64, n=32000, k=2048, out="bf16"),
        # Odd sizes, gradients in 32 bits (kept for accumulation over small batches).
        dict(name="step: ragged", op=STEP, m=1000, n=50257, k=1001, out="f32"),
        # A training batch: loss and both gradients.
        dict(name="step: batch", op=STEP, m=4096, n=128000, k=4096, out="bf16"),
        # Decoding: one token for each of 16 requests.
        dict(name="lookup: decode", op=LOOKUP, m=16, n=32000, k=4096, out="bf16"),
        # A training batch, scaled rows in 32 bits.
        dict(name="lookup: batch", op=LOOKUP, m=32768, n=128000, k=4096, out="f32"),
        # Gradient of the table: a short ragged batch in 32 bits, and a training batch.
        dict(name="lookup grad: ragged", op=LOOKUP_GRAD, m=1000, n=5003, k=1001, given="f32",
             out="f32"),
        dict(name="lookup grad: batch", op=LOOKUP_GRAD, m=32768, n=128000, k=4096, given="bf16",
             out="bf16"),
        # Balance of 8 of 64 experts for 500 tokens, some of them padding; of 8 of 256 experts for
        # a training batch.
        dict(name="balance: short", op=BALANCE, m=500, n=64, k=8, given="f32"),
        dict(name="balance: batch", op=BALANCE, m=65536, n=256, k=8, given="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice([LOSS, STEP, STEP, LOOKUP, LOOKUP_GRAD, BALANCE])
    out, given = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32"])
    if op == BALANCE:
        n = _between(rng, 2, 512)
        return dict(op=op, m=_between(rng, 1, min(131072, 16_000_000 // n)), n=n,
                    k=rng.randint(1, min(8, n)), given=given)
    n, k = _between(rng, 1000, 128000), _between(rng, 128, 4096)
    if rng.random() < 0.5:                       # sizes as most models have them
        n, k = -(-n // 64) * 64, -(-k // 64) * 64
    if op in (LOSS, STEP):
        most = 8192 * 128000 * 4096 if op == LOSS else 4096 * 128000 * 4096
        case = dict(op=op, m=_between(rng, 1, min(8192, most // (n * k))), n=n, k=k)
        return case if op == LOSS else dict(case, out=out)
    case = dict(op=op, m=_between(rng, 1, 32768), n=n, k=k, out=out)
    return case if op == LOOKUP else dict(case, given=given, out=given)


def _rows(gen, shape, dtype=torch.bfloat16, scale=1.0):
    """Normal values whose rows start on 16-byte boundaries."""
    ld = -(-shape[-1] // 8) * 8
    t = torch.randn(*shape[:-1], ld, generator=gen, device="cuda", dtype=torch.float32) * scale
    return t.to(dtype)[..., :shape[-1]]


def _tokens(rng, m, n):
    """Token ids as texts have them: the r-th most frequent about 1 / (r + 3) of the time."""
    u = rng.random(m)
    rank = np.minimum((3.0 * ((n + 3.0) / 3.0) ** u - 3.0).astype(np.int64), n - 1)
    return (rank * 7919 + 13) % n if math.gcd(7919, n) == 1 else rank


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    gen, rng = torch.Generator(device="cuda").manual_seed(seed), np.random.default_rng(seed)
    s, (op, m, n, k) = dict(case), (case[x] for x in ("op", "m", "n", "k"))
    if op in (LOSS, STEP):
        target = _tokens(rng, m, n)
        s["B"] = _rows(gen, (n, k), scale=1.5 * k ** -0.5)
        # A trained model's rows lean towards their target: its logit is up to 14 above the others.
        lean = torch.from_numpy(rng.uniform(0.0, 14.0 / 2.25, m).astype(np.float32)).cuda()
        a = torch.randn(m, k, generator=gen, device="cuda")
        a += lean[:, None] * s["B"][torch.from_numpy(target).cuda()].float()
        s["A"] = torch.zeros(m, -(-k // 8) * 8, device="cuda", dtype=torch.bfloat16)[:, :k]
        s["A"].copy_(a)
        target[rng.random(m) < 0.05] = -100        # padding, and prompts that are not learned
        s["targets"] = _int32(target)
        s["grad"] = torch.from_numpy((rng.uniform(0.5, 1.5, m) / m).astype(np.float32)).cuda()
    elif op == BALANCE:
        # Some experts are more popular than others; a twentieth of the tokens is padding.
        logits = torch.randn(m, n, generator=gen, device="cuda")
        logits += 0.5 * torch.randn(n, generator=gen, device="cuda")
        s["logits"] = logits.to(TYPES[case["given"]])
        ids = s["logits"].float().topk(k, dim=1).indices.to(torch.int32)
        ids[torch.from_numpy(rng.random(m) < 0.05).cuda()] = -1
        s["ids"] = ids.contiguous()
        s["grad"] = torch.full((), 0.01, device="cuda")
    else:
        ids = _tokens(rng, m, n)
        ids[rng.random(m) < 0.02] = -1
        s["ids"], s["scale"] = _int32(ids), math.sqrt(k)
        if op == LOOKUP:
            s["W"] = _rows(gen, (n, k), scale=k ** -0.5)
        else:
            s["G"] = _rows(gen, (m, k), TYPES[case["given"]], 1e-3)
    return s


def _own(s):
    import blackwell_tile_gemm_gb300 as tg
    op, out = s["op"], TYPES.get(s.get("out"))
    if op in (LOSS, STEP):
        loss, lse = tg.gemm_bf16_xent(s["A"], s["B"], s["targets"])
        if op == LOSS:
            return loss, lse
        dA, dB = tg.gemm_bf16_xent_grad(s["A"], s["B"], s["targets"], lse, s["grad"],
                                        out_dtype=out)
        return loss, dA, dB
    if op == LOOKUP:
        return tg.embed_rows(s["W"], s["ids"], scale=s["scale"], out_dtype=out)
    if op == LOOKUP_GRAD:
        return tg.embed_rows_grad(s["G"], s["ids"], s["n"], scale=s["scale"], out_dtype=out)
    loss, counts, shares = tg.balance_loss(s["logits"], s["ids"])
    return loss, counts, tg.balance_loss_grad(s["logits"], s["ids"], shares, s["grad"])


def _plain(s):
    op, m, n, out = s["op"], s["m"], s["n"], TYPES.get(s.get("out"))
    if op in (LOSS, STEP):
        a, b, t = s["A"].float(), s["B"].float(), s["targets"].long()
        inside = (t >= 0) & (t < n)
        at = t.clamp(0, n - 1)
        z = a @ b.T
        top = z.max(dim=1).values
        e = torch.exp(z - top[:, None])
        total = e.sum(dim=1)
        lse = top + torch.log(total)
        loss = torch.where(inside, lse - z.gather(1, at[:, None])[:, 0], lse.new_zeros(()))
        if op == LOSS:
            return loss, lse
        p = e / total[:, None]
        p[torch.arange(m, device=p.device), at] -= 1.0
        dz = p * torch.where(inside, s["grad"], s["grad"].new_zeros(()))[:, None]
        return loss, (dz @ b).to(out), (dz.T @ a).to(out)
    ids = s["ids"].long()
    inside = (ids >= 0) & (ids < n)
    if op == LOOKUP:
        rows = s["W"][ids.clamp(0, n - 1)].float() * s["scale"]
        return torch.where(inside[:, None], rows, rows.new_zeros(())).to(out)
    if op == LOOKUP_GRAD:
        g = torch.where(inside[:, None], s["G"].float() * s["scale"], 0.0)
        dw = torch.zeros(n, s["k"], device=g.device)
        return dw.index_add_(0, ids.clamp(0, n - 1), g).to(out)
    z = s["logits"].float()
    some = inside.any(dim=1)
    counts = torch.bincount(torch.where(inside, ids, n).flatten(), minlength=n + 1)[:n]
    e = torch.exp(z - z.max(dim=1, keepdim=True).values)
    p = torch.where(some[:, None], e / e.sum(dim=1, keepdim=True), e.new_zeros(()))
    share = counts.float() / counts.sum().clamp(min=1) * n / some.sum().clamp(min=1)
    loss = (share * p.sum(dim=0)).sum()
    dz = s["grad"] * p * (share - (p * share).sum(dim=1, keepdim=True))
    return loss, counts.to(torch.int32), dz.to(s["logits"].dtype)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, m, n, k = (case[x] for x in ("op", "m", "n", "k"))
    size = 2 if case.get("out") == "bf16" else 4
    given = 2 if case.get("given") == "bf16" else 4
    if op == LOSS:
        return {"bytes": 2 * k * (m + n) + 12 * m, "flops": 2 * m * n * k}
    if op == STEP:      # the product once, and one for each gradient
        return {"bytes": (2 + size) * k * (m + n) + 12 * m, "flops": 6 * m * n * k}
    if op == LOOKUP:    # distinct rows of the table: at most all of it
        return {"bytes": 2 * k * min(m, n) + size * m * k + 4 * m, "flops": m * k}
    if op == LOOKUP_GRAD:
        return {"bytes": given * m * k + size * n * k + 4 * m, "flops": 2 * m * k}
    return {"bytes": 2 * given * m * n + 4 * m * k + 4 * n, "flops": 10 * m * n}


def _exact_loss(s, case):
    """The definition for blocks of 512 rows, every logit at once in 64 bits."""
    b, targets, n = s["B"].double(), s["targets"].cpu().numpy(), case["n"]
    f64 = dict(dtype=torch.float64, device="cuda")
    losses, lses = [], []
    da, db = torch.empty(case["m"], case["k"], **f64), torch.zeros(n, case["k"], **f64)
    for lo in range(0, case["m"], 512):
        x = s["A"][lo:lo + 512].double()
        z = torch.mm(x, b.t())
        lse = torch.logsumexp(z, dim=1)
        here = targets[lo:lo + 512]
        rows = torch.from_numpy(np.flatnonzero((here >= 0) & (here < n))).cuda()
        cols = s["targets"][lo:lo + 512][rows].long()
        loss = torch.zeros(len(here), **f64)
        loss[rows] = lse[rows] - z[rows, cols]
        losses.append(loss)
        lses.append(lse)
        if case["op"] == STEP:
            weight = torch.zeros(len(here), **f64)
            weight[rows] = s["grad"][lo:lo + 512][rows].double()
            z.sub_(lse[:, None]).exp_()
            z[rows, cols] -= 1.0
            z.mul_(weight[:, None])
            da[lo:lo + 512] = torch.mm(z, b)
            db += torch.mm(z.t(), x)
    if case["op"] == LOSS:
        return torch.cat(losses), torch.cat(lses)
    return torch.cat(losses), da, db


def exact(case, seed):
    s = prepare(case, seed)
    op, m, n, k = (case[x] for x in ("op", "m", "n", "k"))
    if op in (LOSS, STEP):
        return _exact_loss(s, case)
    ids = s["ids"].cpu().numpy()
    if op == LOOKUP:
        d = torch.zeros(m, k, dtype=torch.float64, device="cuda")
        rows = torch.from_numpy(np.flatnonzero((ids >= 0) & (ids < n))).cuda()
        d[rows] = torch.index_select(s["W"], 0, s["ids"][rows].long()).double() * s["scale"]
        return d
    if op == LOOKUP_GRAD:
        # Rows in the order of their ids, each run of one id summed on its own.
        d = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        there = np.flatnonzero((ids >= 0) & (ids < n))
        order = there[np.argsort(ids[there], kind="stable")]
        used, first = np.unique(ids[order], return_index=True)
        g = s["G"][torch.from_numpy(order).cuda()].double()
        lengths = torch.from_numpy(np.diff(np.append(first, len(order)))).cuda()
        if len(used):
            d[torch.from_numpy(used).cuda().long()] = s["scale"] * torch.segment_reduce(
                g, "sum", lengths=lengths)
        return d
    inside = (ids >= 0) & (ids < n)
    counts = np.zeros(n, np.int64)
    np.add.at(counts, ids[inside], 1)
    some = torch.from_numpy(inside.any(axis=1)).cuda()
    p = torch.softmax(s["logits"].double(), dim=1) * some[:, None]
    tokens = max(int(some.sum()), 1)
    f = torch.from_numpy(counts / max(counts.sum(), 1)).cuda()
    mean = p.sum(dim=0) / tokens
    loss = n * torch.dot(f, mean)
    dz = s["grad"].double() * n / tokens * p * (f - (p @ f)[:, None])
    return loss, torch.from_numpy(counts.astype(np.int32)).cuda(), dz
