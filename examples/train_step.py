"""Training a small model of recurrent and expert layers: the library's calls
inside torch's autograd.

``Recurrence`` and ``Experts`` wrap ``gated_scan`` and the experts' sort,
dispatch and return with their gradients; documents are packed behind each
other, so that no token is padding.  The matrix products are torch's.  After
the backward pass ``clip_grad_norm`` scales all gradients at once, and the step
reads nothing back to the host but the loss it prints.

    python examples/train_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stream_compaction_device_gb300 as ds  # noqa: E402


class Recurrence(torch.autograd.Function):
    """h_t = s(gate) h_{t-1} + (1 - s(gate)) x within each document."""

    @staticmethod
    def forward(ctx, x, gate, starts):
        h, _ = ds.gated_scan(x, gate, starts=starts, kind="sigmoid")
        ctx.save_for_backward(x, gate, h, starts)
        return h

    @staticmethod
    def backward(ctx, grad):
        x, gate, h, starts = ctx.saved_tensors
        dx, dgate, _ = ds.gated_scan_backward(grad.contiguous(), x, gate, h, starts=starts, kind="sigmoid")
        return dx, dgate, None


class Dispatch(torch.autograd.Function):
    """Tokens' rows to their places among the experts'."""

    @staticmethod
    def forward(ctx, x, places, order):
        ctx.save_for_backward(places)
        out = torch.zeros(order.numel(), x.shape[1], dtype=x.dtype, device=x.device)
        return ds.expert_dispatch(x, places, order, out=out)

    @staticmethod
    def backward(ctx, grad):
        return ds.expert_combine(grad.contiguous(), *ctx.saved_tensors), None, None


class Combine(torch.autograd.Function):
    """The experts' rows back to the tokens, with weights."""

    @staticmethod
    def forward(ctx, y, weights, places, order):
        ctx.save_for_backward(y, weights, places, order)
        return ds.expert_combine(y, places, weights)

    @staticmethod
    def backward(ctx, grad):
        y, weights, places, order = ctx.saved_tensors
        dy, dweights = ds.expert_combine_backward(grad.contiguous(), y, places, weights, order, grad_y=torch.zeros_like(y))
        return dy, dweights, None, None


class Model(torch.nn.Module):
    """A recurrent layer and an expert layer, each added to what comes in."""

    def __init__(self, vocab: int, width: int, experts: int, choices: int, rows: int):
        super().__init__()
        self.experts, self.choices, self.rows = experts, choices, rows   # rows of an expert's product
        p = lambda *s: torch.nn.Parameter(torch.randn(*s) / s[-2] ** 0.5)  # noqa: E731
        self.embedding, self.head = p(vocab, width), p(width, vocab)
        self.into, self.router = p(width, 2 * width), p(width, experts)
        self.up, self.down = p(experts, width, 2 * width), p(experts, 2 * width, width)

    def forward(self, tokens: torch.Tensor, starts: torch.Tensor) -> torch.Tensor:
        x = self.embedding[tokens] * self.embedding.shape[0] ** 0.5
        both = x @ self.into
        width = x.shape[1]
        x = x + Recurrence.apply(both[:, :width], both[:, width:] + 2, starts)
        top, ids = (x @ self.router).topk(self.choices, dim=1)
        # every expert's product has the same number of rows, so that one batched product has them all; one
        # without tokens has no rows of its own, and takes a row of zeros behind the others
        first, counts, order, places = ds.expert_sort(ids, self.experts, align=self.rows, rows=self.experts * self.rows)
        xs = Dispatch.apply(x, places, order)
        xs = torch.cat([xs, xs.new_zeros(1, width)])
        at = torch.where(counts[:, None] > 0, first[:-1, None].long() + torch.arange(self.rows, device=x.device), len(xs) - 1)
        ys = torch.bmm(torch.relu(torch.bmm(xs[at], self.up)), self.down)
        back = torch.zeros_like(xs).index_copy(0, at.reshape(-1), ys.reshape(-1, width))[:-1]
        x = x + Combine.apply(back, torch.softmax(top, 1), places, order)
        return x @ self.head


def train(steps: int, seed: int = 1, device: str = "cuda") -> list[float]:
    torch.manual_seed(seed)
    vocab, width, experts, choices, tokens = 64, 32, 4, 2, 240
    model = Model(vocab, width, experts, choices, rows=tokens * choices).to(device)
    starts = torch.tensor([0, 50, 51, 130, 240], dtype=torch.int32, device=device)
    text = torch.randint(0, vocab, (tokens,), device=device)
    losses = []
    for _ in range(steps):
        loss = torch.nn.functional.cross_entropy(model(text, starts), text.roll(-1))
        grads = torch.autograd.grad(loss, list(model.parameters()))
        _, grads = ds.clip_grad_norm([g.contiguous() for g in grads], 1.0)
        with torch.no_grad():
            for p, g in zip(model.parameters(), grads):
                p -= 0.2 * g
        losses.append(loss.detach())
    return [v.item() for v in losses]


def main() -> None:
    for i, loss in enumerate(train(40)):
        if i % 10 == 9:
            print(f"step {i}: loss {loss:.3f}")
    assert ds.device_status() == 0


if __name__ == "__main__":
    main()
