"""The serving loop of examples/decode_loop.py: every request's tokens are
what the plain draw gives on the same logits and noise, no page is ever held
twice, and all pages come back."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import serving_ref as ref
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_loop", os.path.join(ROOT, "examples", "decode_loop.py"))
    m = sys.modules[spec.name] = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("pages", [40, 14])      # room for all rows; a pool that runs out
def test_decode_loop(example, pages):
    vocab, page, rows = 700, 4, 6
    loop = example.DecodeLoop(example.ToyModel(vocab, 16, 3), rows=rows, pages=pages, page=page, width=8,
                              step_tokens=24)
    kinds = [{"temperature": 0.0}, {"top_k": 30, "top_p": 0.9, "temperature": 0.8}, {"min_p": 0.1}, {"top_p": 0.7}]
    waiting = [example.Request([(11 * i + j) % vocab for j in range(1 + 3 * i % 11)], 1 + i % 6, **kinds[i % 4])
               for i in range(15)]
    total, ended, steps = len(waiting), [], 0
    seen = {}
    model = loop.model.logits
    loop.model.logits = lambda *a: seen.setdefault("logits", model(*a))
    g = torch.Generator(device="cuda").manual_seed(4)
    while (waiting or any(r is not None for r in loop.running)) and steps < 200:
        loop.admit(waiting)
        before = [(r, len(r.tokens)) if r is not None else None for r in loop.running]
        noise = torch.empty(rows, vocab, device="cuda").exponential_(generator=g).clamp_(min=1e-30)
        seen.clear()
        ended += loop.step(noise)
        x, q = seen["logits"].cpu().numpy(), noise.cpu().numpy()
        for i, was in enumerate(before):
            if was is not None and len(was[0].tokens) > was[1]:
                r = was[0]
                f = lambda v: float(np.float32(v))  # noqa: E731
                good, logprob = ref.draw(x[i], q[i], f(r.temperature), r.top_k, f(r.top_p), f(r.min_p))
                assert r.tokens[-1] in good
                value, room = logprob(r.tokens[-1])
                assert abs(r.logprobs[-1] - value) <= room
        cached, table = loop.cached.tolist(), loop.table.tolist()
        held = [p for i in range(rows) for p in table[i][: ref.blocks(cached[i], page)]]
        spare = loop.pages[: loop.free.item()].tolist()
        assert sorted(held + spare) == list(range(pages))
        steps += 1
    assert len(ended) == total and steps < 200
    assert loop.free.item() == pages
    assert all(1 <= len(r.tokens) <= r.max_new for r in ended)
