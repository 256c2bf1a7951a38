"""The training example's model where its router leaves experts without tokens."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(p, tokens, starts, choices):
    """The model's logits from its parameters, in 64 bits, token by token."""
    x = p["embedding"][tokens] * p["embedding"].shape[0] ** 0.5
    both, width = x @ p["into"], x.shape[1]
    a, h = torch.sigmoid(both[:, width:] + 2), []
    b = torch.sigmoid(-both[:, width:] - 2) * both[:, :width]
    for t in range(len(x)):
        h.append(b[t] if t in starts else a[t] * h[-1] + b[t])
    x = x + torch.stack(h)
    top, ids = (x @ p["router"]).topk(choices, dim=1)
    weights = torch.softmax(top, 1)
    y = torch.stack([sum(weights[t, k] * (torch.relu(x[t] @ p["up"][ids[t, k]]) @ p["down"][ids[t, k]]) for k in range(choices))
                     for t in range(len(x))])
    return (x + y) @ p["head"], ids


@pytest.mark.parametrize("empty", [0, 1, 2])
def test_an_expert_without_tokens(example, empty):
    """Logits and all gradients against autograd in 64 bits.  The router's columns
    are v, -v and 0: the last is never the largest.  Rooms as for the training
    step's test: at most 800 roundings of 2^-24 on ten times the largest value."""
    torch.manual_seed(4)
    vocab, width, tokens = 16, 12, 40
    model = example.Model(vocab, width, 3, 1, rows=tokens).cuda()
    with torch.no_grad():
        model.router[:, (empty + 1) % 3] = -model.router[:, (empty + 2) % 3]
        model.router[:, empty] = 0
    text = torch.randint(0, vocab, (tokens,), device="cuda")
    grad = torch.randn(tokens, vocab, device="cuda")
    wide = {k: v.detach().double().requires_grad_() for k, v in model.named_parameters()}
    want, ids = plain(wide, text, [0, 11], 1)
    assert set(ids.reshape(-1).tolist()) == {0, 1, 2} - {empty}
    starts = torch.tensor([0, 11, tokens], dtype=torch.int32, device="cuda")
    got = model(text, starts)
    names = list(wide)
    mine = torch.autograd.grad((got * grad).sum(), [dict(model.named_parameters())[k] for k in names])
    theirs = torch.autograd.grad((want * grad.double()).sum(), [wide[k] for k in names])
    for name, u, v in zip(["logits", *names], [got, *mine], [want, *theirs]):
        assert (u.double() - v).abs().max() <= 8000 * 2 ** -24 * v.abs().max(), name
