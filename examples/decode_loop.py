"""A serving loop over a paged cache: requests come in with prompts, share one
pool of pages, draw a token per step with settings of their own, and give
their pages back when they end.

Each step makes the library's calls in the order of a server:
``block_table_extend`` opens pages for the new tokens, ``slot_map`` says where
these go, the model writes its cache there and computes logits,
``sample_tokens`` draws, ``compact`` lists the rows that ended, and
``block_table_release`` returns their pages.  The model is a toy (its cache
holds token vectors, its state is their mean), so that the loop is about the
calls.  The batch has a fixed number of rows and of tokens per step; a prompt
that is longer than what the step has left comes in parts.  Tables, lengths and
the pool's height are on the device.  The host knows each row's tokens and
length, and reads per step which rows were granted, the tokens and
log-probabilities, and which rows ended.  Where no row gets the pages that it
needs, the youngest gives its own back and waits, with the tokens drawn so far.

    python examples/decode_loop.py
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass, field

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stream_compaction_device_gb300 as ds  # noqa: E402


@dataclass
class Request:
    prompt: list[int]
    max_new: int
    temperature: float = 1.0
    top_k: int = 0
    top_p: float = 1.0
    min_p: float = 0.0
    tokens: list[int] = field(default_factory=list)
    logprobs: list[float] = field(default_factory=list)


class ToyModel:
    """Vectors per token; the next token's logits from the mean of the row's
    cached vectors."""

    def __init__(self, vocab: int, width: int, seed: int, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.embedding = torch.randn(vocab, width, generator=g).to(device)
        self.head = (torch.randn(width, vocab, generator=g) * 2).to(device)

    def logits(self, cache: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor, page: int) -> torch.Tensor:
        at = torch.arange(table.shape[1] * page, device=cache.device)
        slots = table[:, at // page].clamp(min=0).long() * page + at % page
        held = (at < lengths[:, None]).to(cache.dtype)
        mean = (cache[slots] * held[..., None]).sum(1) / lengths.clamp(min=1)[:, None]
        return mean @ self.head


class DecodeLoop:
    def __init__(self, model: ToyModel, rows: int, pages: int, page: int, width: int, step_tokens: int):
        self.model, self.rows, self.page, self.step_tokens = model, rows, page, step_tokens
        dev = model.embedding.device
        i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=dev)  # noqa: E731
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
        self.cache = torch.zeros(pages * page, model.embedding.shape[1], device=dev)
        self.pages = torch.arange(pages, dtype=torch.int32, device=dev)
        # The pool's height, in two words that the calls read and write in turn.
        self.free, self.left = torch.full((1,), pages, dtype=torch.int32, device=dev), i32(1)
        self.cached = i32(rows)
        self.settings = {"temperature": torch.ones(rows, device=dev), "top_k": i32(rows),
                         "top_p": torch.ones(rows, device=dev), "min_p": torch.zeros(rows, device=dev)}
        self.row_ids = torch.arange(rows, dtype=torch.int32, device=dev)
        self.running: list[Request | None] = [None] * rows
        self.pending: list[list[int]] = [[] for _ in range(rows)]   # a row's tokens that are not in the cache
        self.lengths = [0] * rows                                   # and how many are
        self.order: list[int] = []                                  # rows, oldest first
        self.evicted: list[Request] = []

    def pages_of(self, tokens: int) -> int:
        return -(-tokens // self.page)

    def admit(self, waiting: list[Request]) -> None:
        """Fill empty rows while the pool has pages for all that the rows bring.
        A request that no row or pool could ever hold is a ValueError."""
        waiting[:0], self.evicted = self.evicted, []
        pages, width = self.pages.numel(), self.table.shape[1]
        spare = pages - sum(self.pages_of(n + len(p)) for n, p in zip(self.lengths, self.pending))
        for i in range(self.rows):
            if self.running[i] is not None or not waiting:
                continue
            request = waiting[0]
            if not request.prompt or self.pages_of(len(request.prompt) + request.max_new - 1) > min(width, pages):
                raise ValueError("a request needs a prompt, and its tokens must fit in a row and in the pool")
            tokens = request.prompt + request.tokens
            if self.pages_of(len(tokens)) > spare:
                break
            spare -= self.pages_of(len(tokens))
            self.running[i], self.pending[i] = waiting.pop(0), tokens
            self.order.append(i)
            for name, values in self.settings.items():
                values[i] = getattr(request, name)

    def step(self, noise: torch.Tensor) -> list[Request]:
        """One step of the running rows; returns the requests that ended."""
        dev, brought, room = self.cache.device, [0] * self.rows, self.step_tokens
        for i in self.order:
            brought[i] = min(len(self.pending[i]), room)
            room -= brought[i]
        fresh = torch.tensor(brought, dtype=torch.int32, device=dev)
        granted, _ = ds.block_table_extend(self.table, self.cached, fresh, self.pages, self.free, self.page,
                                           left=self.left)
        self.free, self.left = self.left, self.free
        _, slots, _, _ = ds.slot_map(self.table, self.cached, fresh, self.page, self.step_tokens, granted=granted)
        # The step's tokens, packed as the slots are.
        ran = [n if g else 0 for n, g in zip(brought, granted.tolist())]
        packed = [t for n, tokens in zip(ran, self.pending) for t in tokens[:n]]
        ids = torch.tensor(packed, dtype=torch.long, device=dev)
        self.cache[slots[: len(packed)]] = self.model.embedding[ids]
        self.cached += fresh * granted
        logits = self.model.logits(self.cache, self.table, self.cached, self.page)
        tokens, logprobs = ds.sample_tokens(logits, noise, **self.settings)

        done = [0] * self.rows
        for i, (token, logprob) in enumerate(zip(tokens.tolist(), logprobs.tolist())):
            request = self.running[i]
            self.lengths[i] += ran[i]
            self.pending[i] = self.pending[i][ran[i]:]
            if request is None or self.pending[i]:
                continue                      # empty, or with a part of its prompt still to come
            request.tokens.append(token)
            request.logprobs.append(logprob)
            self.pending[i] = [token]
            done[i] = len(request.tokens) >= request.max_new or token == 0
        waits = self.order[-1] if self.order and not any(ran) else None
        if waits is not None:
            done[waits] = 1
        done = torch.tensor(done, dtype=torch.uint8, device=dev)
        ended, count = ds.compact(self.row_ids, done)
        ds.block_table_release(self.table, self.cached, done, self.pages, self.free, self.page, left=self.left)
        self.free, self.left = self.left, self.free
        self.cached *= 1 - done
        out = []
        for i in ended[: int(count)].tolist():
            (self.evicted if i == waits else out).append(self.running[i])
            self.running[i], self.pending[i], self.lengths[i] = None, [], 0
            self.order.remove(i)
        return out


def main() -> None:
    vocab, g = 4000, torch.Generator(device="cuda").manual_seed(2)
    loop = DecodeLoop(ToyModel(vocab, 32, 1), rows=8, pages=40, page=16, width=8, step_tokens=64)
    kinds = [{"temperature": 0.0}, {"top_k": 40, "top_p": 0.95, "temperature": 0.8}, {"min_p": 0.05}, {}]
    waiting = [Request([(7 * i + j) % vocab for j in range(3 + 5 * i % 30)], 4 + i % 9, **kinds[i % 4])
               for i in range(24)]
    steps = 0
    while waiting or any(r is not None for r in loop.running):
        loop.admit(waiting)
        noise = torch.empty(loop.rows, vocab, device="cuda").exponential_(generator=g).clamp_(min=1e-30)
        for request in loop.step(noise):
            print(f"step {steps}: {len(request.prompt)} + {len(request.tokens)} tokens, "
                  f"mean logprob {sum(request.logprobs) / len(request.logprobs):.2f}: {request.tokens}")
        steps += 1
    assert loop.free.item() == 40 and ds.device_status() == 0
    print(f"{steps} steps, all pages back")


if __name__ == "__main__":
    main()
