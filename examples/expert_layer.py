"""A mixture-of-experts layer with an adapter per request, on the grouped calls.

    python examples/expert_layer.py

serve() is what a serving program runs for a batch of tokens: the experts'
choices are grouped (group_rows), both expert products read their rows by
group (gemm_bf16_grouped), and a shared output projection adds each request's
low-rank adapter (gemm_bf16_lora).  train() is the expert part of a training
step: the same products and, through gemm_bf16_grouped_dgrad and _wgrad, the
gradients of the tokens and of both weights.  Sizes of groups never leave the
device, so nothing here synchronises.  main() runs both on random data and
compares them with plain torch operations in 64 bits.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blackwell_tile_gemm_gb300 as tg  # noqa: E402


def route(logits, k):
    """(weights [tokens, k], plan): the k best experts of each token."""
    best, expert = logits.topk(k, dim=1)
    plan = tg.group_rows(expert.flatten().int(), logits.shape[1])
    return best.softmax(dim=1), plan


def serve(x, logits, k, w_in, w_out, w_proj, adapter, down, up, scales):
    """[tokens, model] bf16: experts (w_in, SiLU, w_out), combined, projected.

    x: bf16 [tokens, model]; w_in: [experts, hidden, model]; w_out: [experts,
    model, hidden]; w_proj: [model, model]; adapter: int32 [tokens], -1 for none.
    """
    weights, (offsets, order, slot) = route(logits, k)
    rows = torch.div(order, k, rounding_mode="floor").int()     # the token of each grouped row
    h = tg.gemm_bf16_grouped(x, w_in, offsets, row_idx=rows, silu_affine=(1.0, 0.0),
                             out_dtype=torch.bfloat16)
    y = tg.gemm_bf16_grouped(h, w_out, offsets, out_dtype=torch.bfloat16)
    y = (y[slot.view(-1, k)].float() * weights[..., None]).sum(1).to(torch.bfloat16)
    return tg.gemm_bf16_lora(y, w_proj, adapter, down, up, scales=scales, out_dtype=torch.bfloat16)


def train(x, logits, k, w_in, w_out, grad):
    """(output, gradient of x, of w_in, of w_out) of sum(grad * experts(x))."""
    weights, (offsets, order, slot) = route(logits, k)
    rows = torch.div(order, k, rounding_mode="floor").int()
    pre = tg.gemm_bf16_grouped(x, w_in, offsets, row_idx=rows)
    h = torch.nn.functional.silu(pre).to(torch.bfloat16)
    y = tg.gemm_bf16_grouped(h, w_out, offsets)
    out = (y[slot.view(-1, k)] * weights[..., None]).sum(1)
    # Back: each grouped row's share of its token's gradient.
    share = weights.flatten()[order.long()]
    g_y = (grad[rows.long()] * share[:, None]).to(torch.bfloat16)
    g_out = tg.gemm_bf16_grouped_wgrad(g_y, h, offsets)
    g_h = tg.gemm_bf16_grouped_dgrad(g_y, w_out, offsets)
    s = torch.sigmoid(pre)
    g_pre = (g_h * (s * (1 + pre * (1 - s)))).to(torch.bfloat16)
    g_in = tg.gemm_bf16_grouped_wgrad(g_pre, x, offsets, row_idx=rows)
    g_rows = tg.gemm_bf16_grouped_dgrad(g_pre, w_in, offsets)
    g_x = g_rows[slot.view(-1, k)].sum(1)
    return out, g_x, g_in, g_out


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


if __name__ == "__main__":
    main()
