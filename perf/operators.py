"""The serving step's operators as measured cases: drawing each row's next
token from its logits, and the bookkeeping of a paged key/value cache (block
tables grown and given back, slot maps of the new tokens).

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits) or, where ``own`` is true, by the calls a user makes of this
package.  ``exact`` computes the token draw from its definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# What the rows of a mixed batch ask for, in turn: requests of one serving
# batch each bring their own settings (temperature, top-k, top-p, min-p).
MIXED = (
    (0.0, 0, 1.0, 0.0),      # greedy
    (0.8, 50, 1.0, 0.0),     # top-k
    (0.7, 40, 0.95, 0.0),    # top-k, then top-p
    (0.9, 0, 0.9, 0.0),      # top-p over the whole vocabulary
    (1.0, 0, 1.0, 0.05),     # min-p
    (1.0, 0, 1.0, 0.0),      # temperature only
    (0.6, 20, 0.9, 0.02),    # all of them
    (1.1, 200, 0.98, 0.0),   # a wide top-k with top-p
)
SETTINGS = {"top_k_p": (0.8, 50, 0.9, 0.0), "top_p": (0.9, 0, 0.92, 0.0), "min_p": (1.0, 0, 1.0, 0.04),
            "plain": (1.0, 0, 1.0, 0.0)}


def listed():
    return [
        # One user's decode step: latency of a single row.
        {"name": "sample 1 x 32768 bf16 top-k and top-p", "op": "sample", "rows": 1, "vocab": 32768, "dtype": "bf16",
         "ask": "top_k_p"},
        # A small batch in fp32 that truncates by probability mass alone.
        {"name": "sample 16 x 65536 f32 top-p", "op": "sample", "rows": 16, "vocab": 65536, "dtype": "f32",
         "ask": "top_p"},
        # An odd vocabulary: rows that start at every alignment.
        {"name": "sample 37 x 100003 f16 min-p", "op": "sample", "rows": 37, "vocab": 100003, "dtype": "f16",
         "ask": "min_p"},
        # Roll-outs for training: the untruncated distribution, all of the noise is read.
        {"name": "sample 256 x 131072 f32 temperature", "op": "sample", "rows": 256, "vocab": 131072, "dtype": "f32",
         "ask": "plain"},
        # A full serving batch whose requests differ in their settings.
        {"name": "sample 512 x 131072 bf16 mixed", "op": "sample", "rows": 512, "vocab": 131072, "dtype": "bf16",
         "ask": "mixed"},
        # A decode step: one token per request, a page for every sixteenth.
        {"name": "extend 64 rows decode", "op": "extend", "rows": 64, "width": 2048, "page": 16, "kind": "decode"},
        # Decode rows beside chunks of prompts.
        {"name": "extend 1000 rows mixed", "op": "extend", "rows": 1000, "width": 1024, "page": 64, "kind": "mixed"},
        # Long prompts arriving together: millions of pages handed out.
        {"name": "extend 4096 rows prompts", "op": "extend", "rows": 4096, "width": 2048, "page": 16,
         "kind": "prompts"},
        # A decode step's slots: one new token per request.
        {"name": "slots 256 rows decode", "op": "slots", "rows": 256, "width": 2048, "page": 16, "kind": "decode"},
        # Prompts of very different lengths packed into one pass of 2.7 million tokens.
        {"name": "slots 1000 rows prompts", "op": "slots", "rows": 1000, "width": 512, "page": 16, "kind": "prompts"},
        # A few requests of a decode batch end.
        {"name": "release 256 rows", "op": "release", "rows": 256, "width": 2048, "page": 16, "kind": "decode"},
        # A large batch is torn down: half of its rows end at once.
        {"name": "release 4096 rows", "op": "release", "rows": 4096, "width": 2048, "page": 16, "kind": "prompts"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("sample", "sample", "extend", "slots", "release"))
    if op == "sample":
        ask = rng.choice(("top_k_p", "top_p", "min_p", "plain", "mixed"))
        vocab = _spread(rng, 2000, 131072)
        rows = _spread(rng, 1, min(512, (1 << 25 if ask == "plain" else 1 << 26) // vocab))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": rng.choice(("f32", "f16", "bf16")), "ask": ask}
    page = rng.choice((16, 32, 64, 24))
    rows = _spread(rng, 1, 4096)
    width = _spread(rng, 64, 2048)
    kind = rng.choice(("decode", "mixed", "prompts"))
    if op == "slots" and kind != "decode":
        width = max(1, min(width, (1 << 13) * 1000 // (rows * page)))
    return {"op": op, "rows": rows, "width": width, "page": page, "kind": kind}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _asked(case):
    if case["ask"] == "mixed":
        return [MIXED[i % len(MIXED)] for i in range(case["rows"])]
    return [SETTINGS[case["ask"]]] * case["rows"]


def _logits(case, seed):
    """Logits as a language model gives them: a bell-shaped bulk and some
    tokens far above it, row by row from nearly decided to nearly flat."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn(rows, vocab, generator=g, device="cuda")
    x *= 1.5 + torch.rand(rows, 1, generator=g, device="cuda")
    few = min(64, vocab)
    at = torch.randint(0, vocab, (rows, few), generator=g, device="cuda")
    lift = torch.empty(rows, few, device="cuda").exponential_(1.0, generator=g)
    lift *= 8.0 * torch.rand(rows, 1, generator=g, device="cuda")
    x.scatter_add_(1, at, lift)
    noise = torch.empty(rows, vocab, device="cuda").exponential_(1.0, generator=g)
    noise.clamp_(min=1e-30)
    return x.to(DTYPES[case["dtype"]]), noise


def _budget(case):
    """The tokens that one pass takes up: what the batch is padded to."""
    rows, limit = case["rows"], case["width"] * case["page"]
    if case["kind"] == "decode":
        return rows
    return max(1, rows + rows * min(limit // 2, 1024) // 5 if case["kind"] == "mixed" else rows * limit // 3)


def _lengths(case, seed):
    """(cached, new) tokens per row, host arrays; their pages fit the table."""
    rng = np.random.default_rng(seed)
    rows, limit = case["rows"], case["width"] * case["page"]
    kind = case["kind"]
    if case["op"] == "release":
        cached = rng.integers(0, limit + 1, rows)
        return cached.astype(np.int32), np.zeros(rows, np.int32)
    if kind == "decode":
        cached = rng.integers(0, limit, rows)
        new = np.ones(rows, np.int64)
    elif kind == "mixed":
        cached = rng.integers(0, limit, rows)
        new = np.where(rng.random(rows) < 0.8, 1, np.minimum(limit - cached, rng.integers(1, 2049, rows)))
        new[rng.random(rows) < 0.05] = 0      # idle slots of the batch
    else:
        cached = np.zeros(rows, np.int64)
        new = np.maximum(1, (limit * rng.random(rows) ** 2).astype(np.int64))
    # What the budget does not cover waits: the row that crosses it comes in
    # part, those after it not at all.
    before = np.cumsum(new) - new
    new = np.clip(_budget(case) - before, 0, new)
    return cached.astype(np.int32), new.astype(np.int32)


def _paged(case, seed):
    rows, width, page = case["rows"], case["width"], case["page"]
    cached, new = _lengths(case, seed)
    have = -(-cached.astype(np.int64) // page)
    want = -(-(cached.astype(np.int64) + new) // page)
    held = want if case["op"] == "slots" else have
    pool = rows * width + 1024
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    ids = torch.randperm(pool, generator=g, device="cuda", dtype=torch.int32)
    d = {"op": case["op"], "page": page,
         "cached": torch.from_numpy(cached).cuda(), "new": torch.from_numpy(new).cuda()}
    # The rows' pages: the first `held` entries of each row, taken from the pool in row order.
    held_t = torch.from_numpy(held).cuda()
    first = torch.cumsum(held_t, 0) - held_t
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j).clamp_(max=pool - 1)
    d["table"] = torch.where(j < held_t[:, None], ids[at], torch.full((), -1, device="cuda", dtype=torch.int32))
    del at
    used = int(held.sum())
    d["pages"] = torch.full((pool,), -1, device="cuda", dtype=torch.int32)
    d["pages"][: pool - used] = ids[used:]
    d["free"] = torch.tensor([pool - used], device="cuda", dtype=torch.int32)
    if case["op"] == "extend":
        d["granted"] = torch.empty(rows, device="cuda", dtype=torch.uint8)
        d["left"] = torch.empty(1, device="cuda", dtype=torch.int32)
    elif case["op"] == "slots":
        d["tokens"] = _budget(case) + 5       # a padded batch: the last places stay empty
        d["out"] = (torch.empty(rows + 1, device="cuda", dtype=torch.int32),
                    torch.empty(d["tokens"], device="cuda", dtype=torch.int64),
                    torch.empty(d["tokens"], device="cuda", dtype=torch.int32),
                    torch.empty(d["tokens"], device="cuda", dtype=torch.int32))
    else:
        share = 0.1 if case["kind"] == "decode" else 0.5
        d["done"] = (torch.rand(rows, generator=g, device="cuda") < share).to(torch.uint8)
        d["left"] = torch.empty(1, device="cuda", dtype=torch.int32)
    return d


def prepare(case, seed):
    if case["op"] != "sample":
        return _paged(case, seed)
    logits, noise = _logits(case, seed)
    t, k, p, m = (list(c) for c in zip(*_asked(case)))
    rows = case["rows"]
    return {"op": "sample", "logits": logits, "noise": noise,
            "temperature": torch.tensor(t, device="cuda", dtype=torch.float32),
            "top_k": torch.tensor(k, device="cuda", dtype=torch.int32),
            "top_p": torch.tensor(p, device="cuda", dtype=torch.float32),
            "min_p": torch.tensor(m, device="cuda", dtype=torch.float32),
            "tokens": torch.empty(rows, device="cuda", dtype=torch.int32),
            "logprobs": torch.empty(rows, device="cuda", dtype=torch.float32)}


# ---------------------------------------------------------------------------
# The plain forms.
# ---------------------------------------------------------------------------
def _plain_sample(s):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -torch.inf, x)
    vocab = x.shape[1]
    t, k = s["temperature"][:, None], s["top_k"][:, None]
    greedy = ~(t > 0)
    t = torch.where(greedy, 1.0, t)
    k = torch.where(k > 0, k, vocab)
    x, order = torch.sort(x, dim=1, descending=True, stable=True)   # ties: the lowest index first
    top = x[:, :1]
    d = torch.where(x == top, 0.0, (x - top) / t)
    w = torch.where(x > -torch.inf, torch.exp(d), 0.0)
    rank = torch.arange(vocab, device=x.device)
    keep = (rank < k) & (w > 0)
    inside = torch.where(keep, w, 0.0)
    upto = torch.cumsum(inside, 1)
    ahead = torch.cat([torch.zeros_like(top), upto[:, :-1]], 1)
    p = s["top_p"][:, None]
    keep &= (p >= 1) | (ahead < p * inside.sum(1, keepdim=True))
    keep &= w >= s["min_p"][:, None]
    keep &= ~greedy
    keep |= rank == 0
    score = torch.where(keep, w / s["noise"].gather(1, order), -1.0)
    score = torch.empty_like(score).scatter_(1, order, score)
    token = score.argmax(1, keepdim=True)
    d = torch.empty_like(d).scatter_(1, order, d).gather(1, token)
    rest = torch.where(keep & (rank > 0), w, 0.0).sum(1, keepdim=True)   # the first one's weight is 1
    logprob = d - torch.log1p(rest)
    empty = top == -torch.inf
    return [torch.where(empty, -1, token).to(torch.int32)[:, 0], torch.where(empty, -torch.inf, logprob)[:, 0]]


def _blocks(length, page):
    return (length + (page - 1)) // page


def _plain_extend(s):
    table, page = s["table"], s["page"]
    width = table.shape[1]
    cached, new = s["cached"].long(), s["new"].long()
    have, want = _blocks(cached, page), _blocks(cached + new, page)
    valid = (cached >= 0) & (new >= 0) & (want <= width)
    need = torch.where(valid, want - have, 0)
    end = torch.cumsum(need, 0)
    granted = valid & ((need == 0) | (end <= s["free"]))
    j = torch.arange(width, device=table.device)
    fresh = (j >= have[:, None]) & (j < want[:, None]) & granted[:, None]
    at = s["free"].long() - 1 - ((end - need - have)[:, None] + j)
    table.copy_(torch.where(fresh, s["pages"][at.clamp(0, s["pages"].numel() - 1)], table))
    taken = torch.where(granted, need, 0).sum()
    return [table, granted.to(torch.uint8), (s["free"] - taken).to(torch.int32)]


def _plain_slots(s):
    table, page, tokens = s["table"], s["page"], s["tokens"]
    rows = table.shape[0]
    new = s["new"].long()
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=table.device), torch.cumsum(new, 0)])
    t = torch.arange(tokens, device=table.device)
    row = torch.searchsorted(starts[1:], t, right=True)
    real = row < rows
    row = row.clamp(max=rows - 1)
    position = s["cached"].long()[row] + t - starts[row]
    block = torch.div(position, page, rounding_mode="floor")
    inside = real & (block < table.shape[1])
    entry = table[row, block.clamp(max=table.shape[1] - 1)].long()
    slot = torch.where(inside & (entry >= 0), entry * page + position % page, -1)
    return [starts.to(torch.int32), slot, torch.where(real, position, -1).to(torch.int32),
            torch.where(real, row, -1).to(torch.int32)]


def _plain_release(s):
    table, pages, page = s["table"], s["pages"], s["page"]
    width = table.shape[1]
    count = torch.where(s["done"] != 0, _blocks(s["cached"].long(), page), 0)
    end = torch.cumsum(count, 0)
    j = torch.arange(width, device=table.device)
    given = j < count[:, None]
    at = s["free"].long() + (end - count)[:, None] + j
    pages[at[given]] = table[given]
    return [pages, (s["free"] + end[-1:]).to(torch.int32)]


def run(state):
    s = state
    if not own:
        return {"sample": _plain_sample, "extend": _plain_extend, "slots": _plain_slots,
                "release": _plain_release}[s["op"]](s)
    import stream_compaction_device_gb300 as ds
    if s["op"] == "sample":
        tokens, logprobs = ds.sample_tokens(s["logits"], s["noise"], temperature=s["temperature"], top_k=s["top_k"],
                                            top_p=s["top_p"], min_p=s["min_p"], out=s["tokens"],
                                            logprobs=s["logprobs"])
        return [tokens, logprobs]
    if s["op"] == "extend":
        granted, left = ds.block_table_extend(s["table"], s["cached"], s["new"], s["pages"], s["free"], s["page"],
                                              granted=s["granted"], left=s["left"])
        return [s["table"], granted, left]
    if s["op"] == "slots":
        return list(ds.slot_map(s["table"], s["cached"], s["new"], s["page"], s["tokens"], out=s["out"]))
    left = ds.block_table_release(s["table"], s["cached"], s["done"], s["pages"], s["free"], s["page"],
                                  left=s["left"])
    return [s["pages"], left]


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    rows = case["rows"]
    if case["op"] == "sample":
        vocab, size = case["vocab"], 4 if case["dtype"] == "f32" else 2
        read = rows * (vocab * size + 16)
        flops = rows * vocab
        for t, k, p, m in _asked(case):
            if t > 0 and k == 0 and p >= 1 and m == 0:
                read += vocab * 4             # every token races: all of the row's noise
                flops += 3 * vocab            # exp, quotient, sum
            elif t > 0:
                read += 4 * max(1, k)
                flops += 2 * vocab if k == 0 and p < 1 else 0
        return {"bytes": read + 8 * rows, "flops": flops}
    width, page = case["width"], case["page"]
    if case["op"] == "release":               # half the table per ended row, on average
        moved = rows * (0.1 if case["kind"] == "decode" else 0.5) * width / 2
        return {"bytes": 8 * moved + 5 * rows + 8, "flops": moved}
    new = _budget(case)
    if case["op"] == "extend":
        return {"bytes": 8 * new / page + 9 * rows + 8, "flops": new / page}
    return {"bytes": 16 * new + 4 * new / page + 12 * rows, "flops": new}


# ---------------------------------------------------------------------------
# The token draw from its definition, in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] != "sample":
        return None                           # whole numbers throughout
    logits, noise = _logits(case, seed)
    settings = _asked(case)
    tokens, logprobs = [], []
    for r in range(case["rows"]):
        t, k, p, m = (float(np.float32(v)) for v in settings[r])
        x = logits[r].double().cpu().numpy()
        alive = np.flatnonzero(~np.isnan(x) & (x > -np.inf))
        if alive.size == 0:
            tokens.append(-1)
            logprobs.append(-math.inf)
            continue
        best = alive[np.argmax(x[alive])]
        if not t > 0:
            tokens.append(int(best))
            logprobs.append(0.0)
            continue
        weight = np.exp((x[alive] - x[best]) / t)
        by = None
        if 0 < k < alive.size or p < 1:
            by = np.lexsort((alive, -x[alive]))     # largest first, ties by index
            if 0 < k < alive.size:
                by = by[: int(k)]
            if p < 1:
                mass = np.cumsum(weight[by])
                by = by[: max(1, int(np.searchsorted(mass, p * mass[-1], side="left")) + 1)]
            alive, weight = alive[by], weight[by]
        stay = (weight >= m) | (alive == best)
        alive, weight = alive[stay], weight[stay]
        score = weight / noise[r].double().cpu().numpy()[alive]
        token = int(alive[np.argmax(score)])
        tokens.append(token)
        logprobs.append(float((x[token] - x[best]) / t - math.log1p(weight[alive != best].sum())))
    return [None, torch.tensor(logprobs, dtype=torch.float64)]
