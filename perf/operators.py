"""Workloads of the grouped operators: rows grouped by id, products grouped by expert (forward and
both gradients) and a shared projection with a low-rank adapter per row.

A case is a dict of plain sizes.  ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes
one pass: with ``own`` through this package's entry points, otherwise with elementary torch
operations in 32 bits, rounded once at the end.  ``exact`` evaluates the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

ROWS, GROUPED, DGRAD, WGRAD, LORA = "rows", "grouped", "dgrad", "wgrad", "lora"


def listed():
    return [
        # The routing plan of one decoding step: 32 tokens, 8 experts each.
        dict(name="rows: decode", op=ROWS, n=256, groups=64, dropped=0.0),
        # The plan of a long training batch: 32768 tokens, 8 of 256 experts each, some dropped.
        dict(name="rows: long", op=ROWS, n=262144, groups=256, dropped=0.02),
        # Serving, 4 requests decode one token each, 8 of 64 experts: about one row per expert,
        # bound by reading the weights of the experts that are hit.
        dict(name="grouped: single tokens", op=GROUPED, m=32, groups=64, n=2048, k=4096, out="bf16",
             epi="none", gather=0, outside=0),
        # Odd sizes: few groups of uneven length, an empty one, rows in no group, row strides that
        # are multiples of 16 bytes only, a bias and an activation per group, f32 output.
        dict(name="grouped: ragged", op=GROUPED, m=3001, groups=7, n=1000, k=1001, out="f32",
             epi="bias_silu", gather=0, outside=37),
        # A prompt of 4096 tokens, 8 of 64 experts each, rows gathered from the token matrix.
        dict(name="grouped: prompt", op=GROUPED, m=32768, groups=64, n=2048, k=4096, out="bf16",
             epi="none", gather=4096, outside=0),
        # Gradient of the inputs: a small ragged batch, and a training batch.
        dict(name="dgrad: ragged", op=DGRAD, m=2000, groups=13, n=1000, k=760, out="f32",
             gather=0, outside=11),
        dict(name="dgrad: batch", op=DGRAD, m=32768, groups=64, n=2048, k=4096, out="bf16",
             gather=0, outside=0),
        # Gradient of the weights: a small ragged batch, and a training batch with f32 gradients.
        dict(name="wgrad: ragged", op=WGRAD, m=1500, groups=13, n=1000, k=760, out="bf16",
             gather=0, outside=11),
        dict(name="wgrad: batch", op=WGRAD, m=32768, groups=32, n=2048, k=4096, out="f32",
             gather=4096, outside=0),
        # Serving with adapters: 4 requests decode one token each; 64 requests over 48 adapters;
        # prompts of 16 requests.
        dict(name="lora: single tokens", op=LORA, m=4, requests=4, adapters=32, rank=16, n=4096,
             k=4096, out="bf16"),
        dict(name="lora: decode", op=LORA, m=64, requests=64, adapters=48, rank=16, n=8192, k=8192,
             out="bf16"),
        dict(name="lora: prompts", op=LORA, m=8000, requests=16, adapters=32, rank=64, n=8192,
             k=4096, out="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice([ROWS, GROUPED, GROUPED, DGRAD, WGRAD, LORA, LORA])
    out = rng.choice(["bf16", "bf16", "f32"])
    if op == ROWS:
        return dict(op=op, n=_between(rng, 1, 262144), groups=_between(rng, 1, 256),
                    dropped=rng.choice([0.0, 0.02]))
    if op == LORA:
        requests = _between(rng, 1, 128)
        # Half of the calls decode one token for each request.
        m = requests if rng.random() < 0.5 else _between(rng, requests, 8000)
        n, k = _between(rng, 500, 8192), _between(rng, 500, 8192)
        m = max(requests, min(m, 260_000_000_000 // (n * k)))
        return dict(op=op, m=m, requests=requests, adapters=_between(rng, 1, 64),
                    rank=8 * rng.choice([1, 2, 4, 8, 16]), n=n, k=k, out=out)
    n, k = _between(rng, 200, 4096), _between(rng, 200, 4096)
    if rng.random() < 0.5:                       # sizes as most models have them
        n, k = -(-n // 128) * 128, -(-k // 128) * 128
    m = _between(rng, 1, min(32768, 270_000_000_000 // (n * k)))
    groups = _between(rng, 1, 64)
    case = dict(op=op, m=m, groups=groups, n=n, k=k, out=out)
    if op == GROUPED:
        case["epi"] = rng.choice(["none", "bias_silu"])
    case["gather"] = rng.choice([0, max(1, m // 8)]) if op != DGRAD else 0
    case["outside"] = rng.choice([0, m // 50])
    return case


def _generators(seed):
    return torch.Generator(device="cuda").manual_seed(seed), np.random.default_rng(seed)


def _rows(gen, shape, scale=1.0):
    """bf16 normal values whose rows start on 16-byte boundaries."""
    ld = -(-shape[-1] // 8) * 8
    t = torch.randn(*shape[:-1], ld, generator=gen, device="cuda", dtype=torch.float32) * scale
    return t.to(torch.bfloat16)[..., :shape[-1]]


def _popularity(rng, groups):
    """Uneven shares: a few groups get several times the mean, some next to nothing."""
    p = np.exp(0.7 * rng.standard_normal(groups))
    return p / p.sum()


def prepare(case, seed):
    gen, rng = _generators(seed)
    s = dict(case)
    if case["op"] == ROWS:
        ids = rng.choice(case["groups"], size=case["n"], p=_popularity(rng, case["groups"]))
        ids[rng.random(case["n"]) < case["dropped"]] = -1
        s["ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["type"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    if case["op"] == LORA:
        # A request's tokens stand together; every tenth request has no adapter.
        cuts = np.sort(rng.choice(np.arange(1, m), case["requests"] - 1, replace=False)) if m > 1 else []
        lengths = np.diff(np.concatenate([[0], cuts, [m]])).astype(np.int64)
        of = rng.integers(0, case["adapters"], case["requests"])
        of[rng.random(case["requests"]) < 0.1] = -1
        s["ids"] = torch.from_numpy(np.repeat(of, lengths).astype(np.int32)).cuda()
        s["A"] = _rows(gen, (m, k))
        s["B"] = _rows(gen, (n, k), k ** -0.5)
        s["down"] = _rows(gen, (case["adapters"], case["rank"], k), k ** -0.5)
        s["up"] = _rows(gen, (case["adapters"], n, case["rank"]), case["rank"] ** -0.5)
        s["scales"] = torch.from_numpy(rng.uniform(0.25, 1.0, case["adapters"]).astype(np.float32)).cuda()
        return s
    inside = m - case["outside"]
    sizes = rng.multinomial(inside, _popularity(rng, case["groups"]))
    if case["groups"] > 2 and m > 1000 and case["groups"] < 32:   # an empty group among long ones
        sizes[0] += sizes[1]
        sizes[1] = 0
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    s["offsets"] = torch.from_numpy(offsets.astype(np.int32)).cuda()
    s["longest"] = int(sizes.max())
    a_rows = case["gather"] or m
    s["row_idx"] = None
    if case["gather"]:
        s["row_idx"] = torch.from_numpy(rng.integers(0, a_rows, m).astype(np.int32)).cuda()
    if case["op"] != DGRAD:
        s["A"] = _rows(gen, (a_rows, k))
    if case["op"] != WGRAD:
        s["B"] = _rows(gen, (case["groups"], n, k), (k if case["op"] == GROUPED else n) ** -0.5)
    if case["op"] != GROUPED:
        s["G"] = _rows(gen, (m, n))
    s["bias"] = None
    if case.get("epi") == "bias_silu":
        s["bias"] = torch.randn(case["groups"], n, generator=gen, device="cuda")
    return s


def _own(s):
    import blackwell_tile_gemm_gb300 as tg
    op = s["op"]
    if op == ROWS:
        return tg.group_rows(s["ids"], s["groups"])
    if op == GROUPED:
        return tg.gemm_bf16_grouped(s["A"], s["B"], s["offsets"], row_idx=s["row_idx"],
                                    bias=s["bias"], bias_silu=s["bias"] is not None,
                                    out_dtype=s["type"])
    if op == DGRAD:
        return tg.gemm_bf16_grouped_dgrad(s["G"], s["B"], s["offsets"], out_dtype=s["type"])
    if op == WGRAD:
        return tg.gemm_bf16_grouped_wgrad(s["G"], s["A"], s["offsets"], row_idx=s["row_idx"],
                                          out_dtype=s["type"])
    return tg.gemm_bf16_lora(s["A"], s["B"], s["ids"], s["down"], s["up"], scales=s["scales"],
                             out_dtype=s["type"])


def _plain_rows(s):
    ids, groups = s["ids"], s["groups"]
    key = torch.where((ids >= 0) & (ids < groups), ids, groups)
    ordered, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(groups + 1, device=ids.device,
                                                       dtype=ids.dtype), out_int32=True)
    slot = torch.empty_like(ids)
    slot[order] = torch.arange(ids.numel(), device=ids.device, dtype=ids.dtype)
    return offsets, order.to(torch.int32), slot


def _padded(s, x):
    """[groups, longest, width] f32 of x's rows by group, zeros past each group's end."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(max(1, s["longest"]), device=x.device)
    there = at < off[1:, None]
    rows = x[at.clamp(max=x.shape[0] - 1)].float()
    return torch.where(there[..., None], rows, rows.new_zeros(()))


def _unpadded(s, y):
    """[m, width]: row i of its group's block in y, zeros for rows of no group."""
    off = s["offsets"].long()
    i = torch.arange(s["m"], device=y.device)
    g = torch.searchsorted(off[1:], i, right=True)
    inside = g < s["groups"]
    g = g.clamp(max=s["groups"] - 1)
    at = (i - off[g]).clamp(0, y.shape[1] - 1)
    return torch.where(inside[:, None], y[g, at], y.new_zeros(()))


def _plain(s):
    op = s["op"]
    if op == ROWS:
        return _plain_rows(s)
    if op == LORA:
        m, adapters, rank = s["m"], s["adapters"], s["rank"]
        a = s["A"].float()
        h = (a @ s["down"].float().reshape(adapters * rank, -1).T).view(m, adapters, rank)
        mine = s["ids"][:, None] == torch.arange(adapters, device=a.device)
        h = torch.where(mine[..., None], h * s["scales"][:, None], h.new_zeros(()))
        up = s["up"].float().permute(0, 2, 1).reshape(adapters * rank, -1)
        return (a @ s["B"].float().T + h.view(m, -1) @ up).to(s["type"])
    if op == GROUPED:
        a = s["A"] if s["row_idx"] is None else s["A"][s["row_idx"].long()]
        y = torch.bmm(_padded(s, a), s["B"].float().transpose(1, 2))
        if s["bias"] is not None:
            y = y + s["bias"][:, None]
            y = y / (1 + torch.exp(-y))
        return _unpadded(s, y).to(s["type"])
    if op == DGRAD:
        return _unpadded(s, torch.bmm(_padded(s, s["G"]), s["B"].float())).to(s["type"])
    a = s["A"] if s["row_idx"] is None else s["A"][s["row_idx"].long()]
    return torch.bmm(_padded(s, s["G"]).transpose(1, 2), _padded(s, a)).to(s["type"])


def run(state):
    return _own(state) if own else _plain(state)


def _groups_hit(case):
    """Groups that get a row, for evenly spread rows (the weights that have to be read)."""
    return case["groups"] * (1 - (1 - 1 / case["groups"]) ** (case["m"] - case["outside"]))


def work(case):
    if case["op"] == ROWS:
        return {"bytes": 12 * case["n"] + 4 * (case["groups"] + 1), "flops": 0}
    m, n, k = case["m"], case["n"], case["k"]
    size = 2 if case["out"] == "bf16" else 4
    if case["op"] == LORA:
        of = min(case["adapters"], case["requests"])
        rank = case["rank"]
        return {"bytes": 2 * (m * k + n * k + of * rank * (n + k)) + size * m * n + 4 * m,
                "flops": 2 * m * n * k + 2 * m * rank * (n + k)}
    rows = min(case["gather"] or m, m)
    inside = m - case["outside"]
    hit = _groups_hit(case)
    moved = {GROUPED: 2 * (rows * k + hit * n * k) + size * m * n,
             DGRAD: 2 * (m * n + hit * n * k) + size * m * k,
             WGRAD: 2 * (m * n + rows * k) + size * case["groups"] * n * k}[case["op"]]
    if case["gather"]:
        moved += 4 * m
    if case.get("epi") == "bias_silu":
        moved += 4 * hit * n
    return {"bytes": moved + 4 * (case["groups"] + 1), "flops": 2 * inside * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == ROWS:
        # Whole numbers, counted one by one on the host.
        ids, groups = s["ids"].cpu().numpy(), case["groups"]
        lists = [np.flatnonzero(ids == g) for g in range(groups)]
        rest = np.flatnonzero((ids < 0) | (ids >= groups))
        order = np.concatenate(lists + [rest]).astype(np.int32)
        offsets = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
        slot = np.empty_like(order)
        slot[order] = np.arange(len(order), dtype=np.int32)
        return offsets, order, slot
    if op == LORA:
        a = s["A"].double()
        d = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
        for r0 in range(0, case["n"], 1024):
            d[:, r0:r0 + 1024] = torch.mm(a, s["B"][r0:r0 + 1024].double().t())
        ids = s["ids"].cpu().numpy()
        for t in np.unique(ids[(ids >= 0) & (ids < case["adapters"])]):
            at = torch.from_numpy(np.flatnonzero(ids == t)).cuda()
            low = torch.mm(a[at], s["down"][int(t)].double().t()) * s["scales"][int(t)].double()
            d[at] += torch.mm(low, s["up"][int(t)].double().t())
        return d
    cut = s["offsets"].cpu().numpy()
    a = s.get("A")
    if s["row_idx"] is not None:
        a = torch.index_select(a, 0, s["row_idx"].long())
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == WGRAD:
        d = torch.zeros(case["groups"], case["n"], case["k"], **f64)
    else:
        d = torch.zeros(case["m"], case["n"] if op == GROUPED else case["k"], **f64)
    for g in range(case["groups"]):
        lo, hi = int(cut[g]), int(cut[g + 1])
        if lo == hi:
            continue
        if op == WGRAD:
            d[g] = torch.mm(s["G"][lo:hi].double().t(), a[lo:hi].double())
        elif op == DGRAD:
            d[lo:hi] = torch.mm(s["G"][lo:hi].double(), s["B"][g].double())
        else:
            y = torch.mm(a[lo:hi].double(), s["B"][g].double().t())
            if s["bias"] is not None:
                y += s["bias"][g].double()
                y = y * torch.sigmoid(y)
            d[lo:hi] = y
    return d
