"""The serving loop of examples/decode_loop.py when its pool and its step are
too small for the requests that wait: what a step brings fits the step, every
request ends, all pages come back, and what can never be served is refused.  On
the CPU the library's calls are the plain ones of serving_ref; on a GPU, its own."""
import importlib.util
import os
import sys
import types

import numpy as np
import pytest
import torch

import serving_ref as ref
from conftest import ROOT


def load_example():
    spec = importlib.util.spec_from_file_location("decode_loop_admission",
                                                  os.path.join(ROOT, "examples", "decode_loop.py"))
    m = sys.modules[spec.name] = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_calls():
    """The calls that the loop makes, on CPU tensors."""
    def extend(table, cached, fresh, pages, free, page, left):
        granted, height = ref.extend(table.numpy(), cached, fresh, pages.numpy(), free.item(), page)
        left.fill_(height)
        return torch.from_numpy(granted), left

    def slots(table, cached, fresh, page, tokens, granted):
        got = ref.slots(table.numpy(), cached, fresh, page, tokens, granted.numpy())
        return tuple(torch.from_numpy(a) for a in got)

    def release(table, cached, done, pages, free, page, left):
        return left.fill_(ref.release(table.numpy(), cached, done, pages.numpy(), free.item(), page))

    def sample(logits, noise, **settings):
        kept = torch.softmax(logits, 1)
        tokens = (kept / noise).argmax(1)
        return tokens.to(torch.int32), kept.log().gather(1, tokens[:, None])[:, 0]

    def compact(values, flags):
        kept = values[flags != 0]
        return torch.cat([kept, values[: values.numel() - kept.numel()]]), torch.tensor(kept.numel())

    return types.SimpleNamespace(block_table_extend=extend, slot_map=slots, block_table_release=release,
                                 sample_tokens=sample, compact=compact)


# rows, page, width, pages, tokens per step, (prompt, most new tokens) of each request
CASES = [(3, 4, 8, 6, 12, [(12, 6), (11, 3), (10, 3)]),        # two prompts wait for pages and come together
         (3, 4, 8, 6, 24, [(7, 9), (7, 9), (7, 9)]),           # rows that grow until no page is left
         (2, 1, 16, 16, 16, [(8, 9), (8, 9), (8, 9)]),
         (4, 16, 2, 5, 40, [(1, 32), (16, 17), (30, 3), (31, 2), (3, 1)]),
         (1, 4, 4, 4, 16, [(16, 1), (1, 16), (9, 8)]),
         (2, 4, 8, 12, 5, [(20, 4), (9, 9), (1, 20), (32, 1)]),   # prompts longer than a step
         (5, 3, 9, 13, 3, [(2 + 3 * i % 9, 1 + 5 * i % 17) for i in range(9)]),   # more rows than a step has tokens
         (8, 8, 6, 17, 48, [(1 + 5 * i % 13, 1 + 7 * i % 23) for i in range(20)])]


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
@pytest.mark.parametrize("case", CASES)
def test_every_request_ends(case, device):
    rows, page, width, pages, step_tokens, requests = case
    m = load_example()
    if device == "cpu":
        m.ds = plain_calls()
    vocab = 50
    loop = m.DecodeLoop(m.ToyModel(vocab, 8, 1, device), rows=rows, pages=pages, page=page, width=width,
                        step_tokens=step_tokens)
    brought, slot_map = [], m.ds.slot_map
    waiting = [m.Request([1 + (3 * i + j) % (vocab - 1) for j in range(n)], most) for i, (n, most) in enumerate(requests)]
    everyone = list(waiting)

    def watched(table, cached, fresh, p, tokens, granted):
        brought.append(int((fresh * granted).sum()))
        assert brought[-1] <= tokens == step_tokens
        return slot_map(table, cached, fresh, p, tokens, granted=granted)

    m.ds = types.SimpleNamespace(**{**{k: getattr(m.ds, k) for k in ("block_table_extend", "block_table_release",
                                                                    "sample_tokens", "compact")}, "slot_map": watched})
    rng = np.random.default_rng(2)
    ended, steps = [], 0
    while waiting or any(r is not None for r in loop.running):
        loop.admit(waiting)
        noise = rng.exponential(1.0, (rows, vocab)).astype(np.float32) + np.float32(1e-30)
        noise[:, 0] = 1e30                                   # the token that ends a row: hardly ever
        ended += loop.step(torch.from_numpy(noise).to(device))
        cached, table = loop.cached.tolist(), loop.table.tolist()
        held = [p for i in range(rows) for p in table[i][: ref.blocks(cached[i], page)]]
        assert sorted(held + loop.pages[: loop.free.item()].tolist()) == list(range(pages))
        steps += 1
        assert steps < 2000
    assert sorted(map(id, ended)) == sorted(map(id, everyone))
    assert all(len(r.tokens) == len(r.logprobs) == r.max_new for r in everyone)
    assert loop.free.item() == pages


@pytest.mark.parametrize("request_", [(17, 1), (10, 8), (1, 17), (0, 3)])
@pytest.mark.parametrize("shape", [(4, 4, 9), (4, 9, 4)])
def test_what_never_fits_is_refused(request_, shape):
    """17 tokens against 16 of a row and of the pool, and no prompt at all."""
    page, width, pages = shape
    m = load_example()
    m.ds = plain_calls()
    loop = m.DecodeLoop(m.ToyModel(20, 4, 1, "cpu"), rows=2, pages=pages, page=page, width=width, step_tokens=8)
    with pytest.raises(ValueError):
        loop.admit([m.Request([1] * request_[0], request_[1])])
    assert loop.running == [None, None]
