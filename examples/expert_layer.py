"""An expert layer over offset-delimited segments, trained for a few steps and
then served with per-request adapters.

    python examples/expert_layer.py [--tokens 4096] [--steps 5]

Training: every token goes to its two highest-scoring experts.  Sorted by
expert, the rows of an expert are a segment, so the layer is two
``segment_matmul`` calls (forward; their backward is ``seg_matmul`` and
``seg_matmul_grad_w``), and the weighted sum back to the tokens is the
deterministic ``scatter``.

Serving: requests of different lengths share an output projection, each with
its own low-rank adapter (``seg_lora``), first as prompts, then one token each.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import segmented_reduction_csr_gb300 as sr  # noqa: E402


def route(scores, top: int):
    """(expert-sorted row order, token of each row, its weight, offsets of the experts)."""
    tokens, experts = scores.shape
    weight, expert = torch.topk(torch.softmax(scores.float(), dim=-1), top, dim=-1)
    weight = weight / weight.sum(dim=-1, keepdim=True)
    order = torch.argsort(expert.reshape(-1), stable=True)
    token = torch.div(order, top, rounding_mode="floor")
    counts = torch.bincount(expert.reshape(-1), minlength=experts)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    return token, weight.reshape(-1)[order], offsets


class CombineRows(torch.autograd.Function):
    """out[t] = sum of the rows of token t (their order is fixed, so the sum repeats bit for bit)."""

    @staticmethod
    def forward(ctx, rows, token, tokens):
        ctx.save_for_backward(token)
        return sr.scatter(rows.contiguous(), token, tokens, "sum", deterministic=True)

    @staticmethod
    def backward(ctx, dout):
        token, = ctx.saved_tensors
        return dout[token], None, None


class ExpertLayer(torch.nn.Module):
    def __init__(self, width: int, hidden: int, experts: int, top: int = 2, dtype=torch.bfloat16):
        super().__init__()
        self.top = top
        self.router = torch.nn.Parameter(torch.randn(width, experts, device="cuda", dtype=dtype) * width ** -0.5)
        self.up = torch.nn.Parameter(torch.randn(experts, width, hidden, device="cuda", dtype=dtype) * width ** -0.5)
        self.down = torch.nn.Parameter(torch.randn(experts, hidden, width, device="cuda", dtype=dtype) * hidden ** -0.5)

    def forward(self, x):
        token, weight, offsets = route(x @ self.router, self.top)
        h = torch.relu(sr.segment_matmul(x[token], self.up, offsets))
        y = sr.segment_matmul(h, self.down, offsets)
        return CombineRows.apply(y.float() * weight[:, None], token, x.shape[0]).to(x.dtype)


def train(tokens: int = 4096, width: int = 512, hidden: int = 1024, experts: int = 16, steps: int = 5, seed: int = 0):
    """Losses of a few steps that fit the layer to a fixed random map."""
    torch.manual_seed(seed)
    layer = ExpertLayer(width, hidden, experts)
    x = torch.randn(tokens, width, device="cuda", dtype=torch.bfloat16)
    want = torch.relu(x @ (torch.randn(width, width, device="cuda", dtype=torch.bfloat16) * width ** -0.5))
    opt = torch.optim.SGD(layer.parameters(), lr=0.2)
    losses = []
    for _ in range(steps):
        loss = (layer(x).float() - want.float()).square().mean() * 100
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


def serve(lengths=(700, 3, 1, 1290, 64), width: int = 1024, out: int = 2048, rank: int = 16, adapters: int = 3, seed: int = 0):
    """(prompt outputs, one-token outputs) of requests with adapters; the last request has none."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(torch.bfloat16)

    w = normal(out, width, scale=width ** -0.5)
    a, b = normal(adapters, rank, width, scale=width ** -0.5), normal(adapters, out, rank, scale=rank ** -0.5)
    scale = torch.full((adapters,), 2.0, device="cuda")
    ids = torch.arange(len(lengths), device="cuda", dtype=torch.int32) % adapters
    ids[-1] = -1
    offsets = torch.tensor([0, *lengths], device="cuda").cumsum(0)
    x = normal(int(sum(lengths)), width)
    prompts = sr.seg_lora(x, w, a, b, offsets, ids, scale)
    # one more token of every request: the last row of each prompt again
    one = torch.arange(len(lengths) + 1, device="cuda")
    tokens = sr.seg_lora(x[offsets[1:] - 1], w, a, b, one, ids, scale)
    return prompts, tokens, offsets


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=5)
    args = ap.parse_args()
    losses = train(tokens=args.tokens, steps=args.steps)
    print("training losses:", " ".join(f"{v:.4f}" for v in losses))
    prompts, tokens, offsets = serve()
    gap = (prompts[offsets[1:] - 1].float() - tokens.float()).abs().max().item()
    print(f"served {prompts.shape[0]} prompt rows and {tokens.shape[0]} single tokens; "
          f"largest difference of a row in both: {gap:.2g}")


if __name__ == "__main__":
    main()
