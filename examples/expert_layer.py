"""A mixture-of-experts layer with an adapter per request, on the grouped calls.

    python examples/expert_layer.py

serve() is what a serving program runs for a batch of tokens: the experts'
choices are grouped (group_rows), both expert products read their rows by
group (gemm_bf16_grouped), and a shared output projection adds each request's
low-rank adapter (gemm_bf16_lora).  train() is the expert part of a training
step: the same products and, through gemm_bf16_grouped_dgrad and _wgrad, the
gradients of the tokens and of both weights.  step() is the training step of a
small model around that layer: token rows (embed_rows), the router's balance
(balance_loss), the loss over a vocabulary that is also the table of the token
rows (gemm_bf16_xent), and every gradient, the table's from both of its uses.
Sizes of groups never leave the device, so nothing here synchronises.  main()
runs all of it on random data and compares it with plain torch operations in 64
bits.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blackwell_tile_gemm_gb300 as tg  # noqa: E402


def route(logits, k):
    """(weights [tokens, k], experts [tokens, k], plan): the k best experts of each token."""
    best, expert = logits.topk(k, dim=1)
    expert = expert.int()
    return best.softmax(dim=1), expert, tg.group_rows(expert.flatten(), logits.shape[1])


def serve(x, logits, k, w_in, w_out, w_proj, adapter, down, up, scales):
    """[tokens, model] bf16: experts (w_in, SiLU, w_out), combined, projected.

    x: bf16 [tokens, model]; w_in: [experts, hidden, model]; w_out: [experts,
    model, hidden]; w_proj: [model, model]; adapter: int32 [tokens], -1 for none.
    """
    weights, _, (offsets, order, slot) = route(logits, k)
    rows = torch.div(order, k, rounding_mode="floor").int()     # the token of each grouped row
    h = tg.gemm_bf16_grouped(x, w_in, offsets, row_idx=rows, silu_affine=(1.0, 0.0),
                             out_dtype=torch.bfloat16)
    y = tg.gemm_bf16_grouped(h, w_out, offsets, out_dtype=torch.bfloat16)
    y = (y[slot.view(-1, k)].float() * weights[..., None]).sum(1).to(torch.bfloat16)
    return tg.gemm_bf16_lora(y, w_proj, adapter, down, up, scales=scales, out_dtype=torch.bfloat16)


def experts(x, weights, plan, k, w_in, w_out):
    """(output f32 [tokens, model], what experts_back needs of it)."""
    offsets, order, slot = plan
    rows = torch.div(order, k, rounding_mode="floor").int()
    pre = tg.gemm_bf16_grouped(x, w_in, offsets, row_idx=rows)
    h = torch.nn.functional.silu(pre).to(torch.bfloat16)
    y = tg.gemm_bf16_grouped(h, w_out, offsets)[slot.view(-1, k)]
    return (y * weights[..., None]).sum(1), (rows, pre, h, y)


def experts_back(x, weights, plan, k, w_in, w_out, kept, grad):
    """Gradients of the tokens, the weights [tokens, k], w_in and w_out."""
    offsets, order, slot = plan
    rows, pre, h, y = kept
    # Each grouped row's share of its token's gradient.
    share = weights.flatten()[order.long()]
    g_y = (grad[rows.long()] * share[:, None]).to(torch.bfloat16)
    g_out = tg.gemm_bf16_grouped_wgrad(g_y, h, offsets)
    g_h = tg.gemm_bf16_grouped_dgrad(g_y, w_out, offsets)
    s = torch.sigmoid(pre)
    g_pre = (g_h * (s * (1 + pre * (1 - s)))).to(torch.bfloat16)
    g_in = tg.gemm_bf16_grouped_wgrad(g_pre, x, offsets, row_idx=rows)
    g_x = tg.gemm_bf16_grouped_dgrad(g_pre, w_in, offsets)[slot.view(-1, k)].sum(1)
    return g_x, (y * grad[:, None]).sum(2), g_in, g_out


def train(x, logits, k, w_in, w_out, grad):
    """(output, gradient of x, of w_in, of w_out) of sum(grad * experts(x))."""
    weights, _, plan = route(logits, k)
    out, kept = experts(x, weights, plan, k, w_in, w_out)
    g_x, _, g_in, g_out = experts_back(x, weights, plan, k, w_in, w_out, kept, grad)
    return out, g_x, g_in, g_out


def step(ids, targets, table, w_router, w_in, w_out, k, balance=0.01):
    """(loss, experts [tokens, k], counts, gradients) of one training step.

    ids, targets: int32 [tokens], targets outside the vocabulary are not learned;
    table: bf16 [vocabulary, model], the tokens' rows and the vocabulary of the loss;
    w_router: [experts, model].  The gradients (f32): of table, w_router, w_in, w_out.
    """
    vocabulary, model = table.shape
    scale = math.sqrt(model)
    one = len(ids) * torch.arange(2, device=table.device, dtype=torch.int32)   # a single group
    x = tg.embed_rows(table, ids, scale=scale)
    logits = tg.gemm_bf16_grouped(x, w_router[None], one)   # (rows on 16 bytes, as many experts as like)
    weights, expert, plan = route(logits, k)
    uneven, counts, shares = tg.balance_loss(logits, expert)
    out, kept = experts(x, weights, plan, k, w_in, w_out)
    h = (x + out).to(torch.bfloat16)
    losses, lse = tg.gemm_bf16_xent(h, table, targets)
    learned = ((targets >= 0) & (targets < vocabulary)).float()
    learned /= learned.sum().clamp(min=1)
    loss = (losses * learned).sum() + balance * uneven
    # Back.
    g_h, g_table = tg.gemm_bf16_xent_grad(h, table, targets, lse, learned, loss=losses,
                                          out_dtype=torch.float32)
    g_x, g_weights, g_in, g_out = experts_back(x, weights, plan, k, w_in, w_out, kept, g_h)
    g_best = weights * (g_weights - (weights * g_weights).sum(1, keepdim=True))
    g_uneven = tg.balance_loss_grad(logits, expert, shares, torch.full_like(uneven, balance))
    wide = -(-logits.shape[1] // 8) * 8                      # rows of bf16 on 16 bytes
    g_logits = torch.empty(len(ids), wide, device=x.device, dtype=x.dtype)[:, :logits.shape[1]]
    g_logits.copy_(g_uneven.scatter_add(1, expert.long(), g_best))
    g_router = tg.gemm_bf16_grouped_wgrad(g_logits, x, one)[0]
    g_x += g_h + tg.gemm_bf16_grouped_dgrad(g_logits, w_router[None], one)
    tg.embed_rows_grad(g_x, ids, vocabulary, g_table, scale=scale, accumulate=True)
    return loss, expert, counts, (g_table, g_router, g_in, g_out)


def plain_step(ids, targets, table, w_router, w_in, w_out, expert, balance):
    """step's loss in 64 bits, for the experts that it chose."""
    x = table[ids.long()] * math.sqrt(table.shape[1])
    logits = x @ w_router.T
    share = torch.zeros_like(logits).scatter(1, expert, logits.gather(1, expert).softmax(dim=1))
    inner = torch.nn.functional.silu(torch.einsum("tm,ehm->eth", x, w_in))
    h = x + torch.einsum("eth,emh,te->tm", inner, w_out, share)
    chosen = torch.bincount(expert.flatten(), minlength=logits.shape[1]) / expert.numel()
    uneven = logits.shape[1] * (chosen * logits.softmax(dim=1).mean(dim=0)).sum()
    inside = (targets >= 0) & (targets < len(table))
    return torch.nn.functional.cross_entropy((h @ table.T)[inside],
                                             targets[inside].long()) + balance * uneven


def plain_experts(x, logits, k, w_in, w_out):
    """The experts' part in 64 bits, every expert on every token."""
    best, expert = logits.double().topk(k, dim=1)
    share = torch.zeros_like(logits, dtype=torch.float64).scatter(1, expert, best.softmax(dim=1))
    h = torch.nn.functional.silu(torch.einsum("tm,ehm->eth", x, w_in))
    return torch.einsum("eth,emh,te->tm", h, w_out, share)


def main(tokens=300, model=256, hidden=384, experts=8, k=2, adapters=5, rank=16):
    gen = torch.Generator(device="cuda").manual_seed(0)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    bf16 = lambda t: t.to(torch.bfloat16)  # noqa: E731
    x, logits = bf16(normal(tokens, model)), normal(tokens, experts)
    w_in = bf16(normal(experts, hidden, model) * model ** -0.5)
    w_out = bf16(normal(experts, model, hidden) * hidden ** -0.5)
    w_proj = bf16(normal(model, model) * model ** -0.5)
    down = bf16(normal(adapters, rank, model) * model ** -0.5)
    up = bf16(normal(adapters, model, rank) * rank ** -0.5)
    scales = torch.full((adapters,), 0.5, device="cuda")
    adapter = torch.randint(-1, adapters, (tokens,), generator=gen, device="cuda",
                            dtype=torch.int32)

    got = serve(x, logits, k, w_in, w_out, w_proj, adapter, down, up, scales)
    mid = plain_experts(x.double(), logits, k, w_in.double(), w_out.double())
    want = mid @ w_proj.double().T
    low = torch.einsum("tm,arm->tar", mid, down.double()) * scales.double()[:, None]
    own = adapter[:, None] == torch.arange(adapters, device="cuda")
    want = want + torch.einsum("tar,anr,ta->tn", low, up.double(), own.double())
    off = [float((got.double() - want).norm() / want.norm())]

    grad = normal(tokens, model)
    got = train(x, logits, k, w_in, w_out, grad)
    leaves = [t.double().requires_grad_() for t in (x, w_in, w_out)]
    out = plain_experts(leaves[0], logits, k, leaves[1], leaves[2])
    out.backward(grad.double())
    want = [out.detach()] + [t.grad for t in leaves]
    off += [float((a.double() - b).norm() / b.norm()) for a, b in zip(got, want)]
    assert tg.tg_device_status()[0] == tg.TG_OK
    for name, e in zip(("serving output", "training output", "gradient of x", "gradient of w_in",
                        "gradient of w_out"), off):
        print(f"{name:20s} relative error {e:.2g}")
    return off


def main_step(tokens=300, model=256, hidden=384, experts=8, k=2, vocabulary=5000, balance=0.01):
    """step() against plain torch: relative errors of the loss and of the gradients."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    weight = lambda *shape: (torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
                             * shape[-1] ** -0.5).to(torch.bfloat16)
    table, w_router = weight(vocabulary, model), weight(experts, model)
    w_in, w_out = weight(experts, hidden, model), weight(experts, model, hidden)
    ids, targets = (torch.randint(0, vocabulary, (tokens,), generator=gen, device="cuda",
                                  dtype=torch.int32) for _ in range(2))
    targets[::7] = -100
    loss, expert, counts, got = step(ids, targets, table, w_router, w_in, w_out, k, balance)
    assert int(counts.sum()) == tokens * k
    leaves = [t.double().requires_grad_() for t in (table, w_router, w_in, w_out)]
    want = plain_step(ids, targets, *leaves, expert.long(), balance)
    want.backward()
    off = [float(abs(loss.double() - want.detach()) / want.detach())]
    off += [float((a.double() - t.grad).norm() / t.grad.norm()) for a, t in zip(got, leaves)]
    assert tg.tg_device_status()[0] == tg.TG_OK
    for name, e in zip(("loss of the step", "gradient of table", "gradient of w_router",
                        "gradient of w_in", "gradient of w_out"), off):
        print(f"{name:20s} relative error {e:.2g}")
    return off


if __name__ == "__main__":
    main()
    main_step()
