"""What a model of recurrent and expert layers does outside its matrix
products, as measured cases: the gated recurrence over long, packed and
single-token rows and its gradient; tokens sorted by expert, and back with
weights and their gradient; the norm over all gradients, and clipping.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, long sums in 64) or, where ``own`` is true, by the calls a user
makes of this package.  ``exact`` computes the same from the definitions in 64
bits, one token after the other.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6                                # of the clipping coefficient


def listed():
    return [
        # One long document through a recurrent layer.
        {"name": "scan 1 x 65536 x 2048 bf16 log", "op": "scan", "rows": 1, "tokens": 65536, "channels": 2048,
         "dtype": "bf16", "gate": "bf16", "kind": "log", "packed": False, "carry": False},
        # Chunks of prompts packed into one serving pass, each row with its state; an odd width, a padded end.
        {"name": "scan packed 24 rows 8191 x 1000 f32 decay", "op": "scan", "rows": 24, "tokens": 8191,
         "channels": 1000, "dtype": "f32", "gate": "f32", "kind": "decay", "packed": True, "carry": True},
        # The training step of a wide layer: a batch of sequences, all gradients.
        {"name": "backward 8 x 4096 x 4096 bf16 sigmoid", "op": "backward", "rows": 8, "tokens": 4096,
         "channels": 4096, "dtype": "bf16", "gate": "bf16", "kind": "sigmoid", "packed": False, "carry": False},
        # Documents packed into one training row, decays kept in 32 bits.
        {"name": "backward packed 37 rows 5000 x 1024 f16 log", "op": "backward", "rows": 37, "tokens": 5000,
         "channels": 1024, "dtype": "f16", "gate": "f32", "kind": "log", "packed": True, "carry": False},
        # One user's decode step: latency.
        {"name": "step 1 row x 2048 bf16 log", "op": "step", "rows": 1, "tokens": 1, "channels": 2048,
         "dtype": "bf16", "gate": "bf16", "kind": "log", "packed": False, "carry": True},
        # The decode step of a full serving batch.
        {"name": "step 512 rows x 4096 bf16 sigmoid", "op": "step", "rows": 512, "tokens": 1, "channels": 4096,
         "dtype": "bf16", "gate": "bf16", "kind": "sigmoid", "packed": False, "carry": True},
        # The decode step of an expert layer: a small batch, two of its tokens padding.
        {"name": "experts in 16 x 8 of 64, 2048 bf16", "op": "in", "tokens": 16, "choices": 8, "experts": 64,
         "width": 2048, "dtype": "bf16", "ids": "i32", "align": 1, "pad": 2},
        # Its training step: segments rounded up to the tiles of the experts' products.
        {"name": "experts in 16384 x 8 of 256, 2048 bf16", "op": "in", "tokens": 16384, "choices": 8,
         "experts": 256, "width": 2048, "dtype": "bf16", "ids": "i64", "align": 128, "pad": 0},
        # The way back of a decode batch.
        {"name": "experts out 64 x 4 of 32, 4096 f16", "op": "out", "tokens": 64, "choices": 4, "experts": 32,
         "width": 4096, "dtype": "f16", "ids": "i32", "align": 1, "pad": 3, "gradient": False},
        # The way back of a training step with the gradients of rows and weights; an odd number of tokens.
        {"name": "experts out 8191 x 6 of 160, 2048 bf16 gradient", "op": "out", "tokens": 8191, "choices": 6,
         "experts": 160, "width": 2048, "dtype": "bf16", "ids": "i64", "align": 16, "pad": 0, "gradient": True},
        # A small model's gradients: matrices and vectors of odd sizes, one after the other in one buffer.
        {"name": "clip 40 tensors 1.3 M f32", "op": "clip", "tensors": 40, "elements": 1300000, "dtype": "f32",
         "close": True},
        # A large model's gradients in 16 bits, vectors in 32.
        {"name": "clip 300 tensors 1.5 G mixed", "op": "clip", "tensors": 300, "elements": 1500000000,
         "dtype": "mixed", "close": False},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("scan", "scan", "backward", "backward", "step", "in", "out", "clip"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op in ("scan", "backward", "step"):
        channels = _spread(rng, 64, 4096)
        case = {"op": op, "channels": channels, "dtype": dtype, "gate": rng.choice((dtype, "f32")),
                "kind": rng.choice(("decay", "log", "sigmoid"))}
        if op == "step":
            return {**case, "rows": _spread(rng, 1, 1024), "tokens": 1, "packed": False, "carry": True}
        most = (1 << 26) // channels
        packed = rng.random() < 0.5
        rows = _spread(rng, 1, 64)
        tokens = _spread(rng, 64, min(32768, most if packed else max(64, most // rows)))
        return {**case, "rows": rows, "tokens": tokens, "packed": packed, "carry": rng.random() < 0.5}
    if op in ("in", "out"):
        experts = _spread(rng, 4, 512)
        choices = rng.randint(1, min(8, experts))
        width = _spread(rng, 128, 8192)
        tokens = _spread(rng, 1, min(32768, (1 << 28) // (width * choices)))
        case = {"op": op, "tokens": tokens, "choices": choices, "experts": experts, "width": width, "dtype": dtype,
                "ids": rng.choice(("i32", "i64")), "align": rng.choice((1, 16, 128)),
                "pad": rng.choice((0, 0, 1, 5))}
        return {**case, "gradient": rng.random() < 0.6} if op == "out" else case
    return {"op": op, "tensors": _spread(rng, 1, 400), "elements": _spread(rng, 100000, 500000000),
            "dtype": rng.choice(("f32", "f16", "bf16", "mixed")), "close": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _starts(case, seed):
    """Where the packed rows begin: lengths from nothing to a large share,
    and a few tokens of padding behind the last row."""
    rng = np.random.default_rng(seed)
    rows, tokens = case["rows"], case["tokens"]
    used = tokens - min(tokens // 50, 100)
    cuts = np.sort(rng.integers(0, used + 1, rows - 1))
    if rows > 4:
        cuts[rows // 2] = cuts[rows // 2 - 1]         # a row without tokens
    return np.concatenate([[0], cuts, [used]]).astype(np.int32)


def _recurrence(case, seed):
    """Inputs of a recurrent layer: each channel with a memory of its own,
    from a few tokens to thousands, moved by the token."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, tokens, channels = case["rows"], case["tokens"], case["channels"]
    shape = (tokens, channels) if case["packed"] else (rows, tokens, channels)
    dtype, gate_dtype = DTYPES[case["dtype"]], DTYPES[case["gate"]]
    s = {"op": case["op"], "kind": case["kind"], "starts": None, "initial": None, "slots": None,
         "x": torch.randn(shape, generator=g, device="cuda").to(dtype)}
    slow = torch.exp(torch.rand(channels, generator=g, device="cuda") * 7.6 - 8.0)     # exp(-8) .. exp(-0.4)
    token = torch.randn(shape, generator=g, device="cuda")
    if case["kind"] == "sigmoid":
        gate = token - torch.log(slow)
    else:
        gate = token.sigmoid_().mul_(-2 * slow)
        gate = gate.exp_() if case["kind"] == "decay" else gate
    s["gate"] = gate.to(gate_dtype)
    del token, gate
    if case["packed"]:
        s["starts"] = torch.from_numpy(_starts(case, seed)).cuda()
    if case["carry"]:
        pool = rows
        if case["op"] != "backward" and (case["packed"] or case["op"] == "step"):
            pool = rows + 3 + rows // 8               # the rows' states lie in a larger pool
            s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:rows].to(torch.int32)
        s["initial"] = torch.randn(pool, channels, generator=g, device="cuda")
    if case["op"] != "backward":
        s["out"] = torch.zeros(shape, dtype=dtype, device="cuda")
        s["final"] = torch.zeros(rows if s["initial"] is None else len(s["initial"]), channels, device="cuda")
        return s
    s["y"] = _plain_scan({**s, "out": s["x"], "final": torch.empty(rows, channels, device="cuda")})[0]
    s["grad"] = torch.randn(shape, generator=g, device="cuda").to(dtype)
    s["grad_final"] = torch.randn(rows, channels, generator=g, device="cuda") if case["carry"] else None
    return s


def _placed(case):
    """Rows of the sorted buffer: what the pairs can need at most."""
    pairs = case["tokens"] * case["choices"]
    return pairs + min(case["experts"], pairs) * (case["align"] - 1)


def _expert_rows(case, seed):
    """A router's choice: experts of unequal favour, the last tokens of a
    padded batch without any."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens, choices, experts, width = (case[k] for k in ("tokens", "choices", "experts", "width"))
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    logits += torch.randn(experts, generator=g, device="cuda") * 0.7
    top, ids = logits.topk(choices, dim=1)
    weights = torch.softmax(top, 1)
    if case["pad"]:
        ids[max(0, tokens - case["pad"]):] = -1
    ids = ids.to(torch.int32) if case["ids"] == "i32" else ids
    s = {"op": case["op"], "ids": ids, "experts": experts, "align": case["align"], "rows": _placed(case)}
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "in":
        s["x"] = torch.randn(tokens, width, generator=g, device="cuda").to(dtype)
        s["out"] = torch.zeros(s["rows"], width, dtype=dtype, device="cuda")
        return s
    s["starts"], s["counts"], s["order"], s["places"] = _plain_sort(s)
    s["weights"], s["gradient"] = weights, case["gradient"]
    s["y"] = torch.randn(s["rows"], width, generator=g, device="cuda").to(dtype)
    if case["gradient"]:
        s["grad"] = torch.randn(tokens, width, generator=g, device="cuda").to(dtype)
        s["grad_y"] = torch.zeros_like(s["y"])
    return s


def _tensors(case):
    """(elements, type) of each tensor: matrices that hold nearly all, and
    vectors between them."""
    rng = random.Random(case["tensors"] * 1000003 + case["elements"])
    count, left = case["tensors"], case["elements"]
    parts = []
    for i in range(count):
        vector = i % 3 == 2 and count > 3
        even = left / max(1, count - i)
        n = rng.randint(1, 8192) if vector else even * rng.uniform(0.5, 1.5) if i + 1 < count else left
        n = max(1, min(int(n), left - (count - i - 1)))
        left -= n
        parts.append((n, ("f32" if vector else "bf16") if case["dtype"] == "mixed" else case["dtype"]))
    return parts


def _gradients(case, seed):
    """Gradients in one buffer per type; where they do not lie close, each
    begins on 16 bytes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    parts, size, at = _tensors(case), {}, []
    for n, dtype in parts:
        begin = size.get(dtype, 0)
        size[dtype] = begin + n if case["close"] else -(-(begin + n) // 8) * 8
        at.append(begin)
    s = {"op": "clip", "max_norm": 1.0}
    flat, out = {}, {}
    for dtype, n in size.items():
        flat[dtype] = torch.empty(n, dtype=DTYPES[dtype], device="cuda")
        for i in range(0, n, 1 << 28):
            flat[dtype][i:i + (1 << 28)].normal_(0.0, 0.01, generator=g)
        out[dtype] = torch.zeros_like(flat[dtype])
    s["grads"] = [flat[d][b:b + n] for b, (n, d) in zip(at, parts)]
    s["out"] = [out[d][b:b + n] for b, (n, d) in zip(at, parts)]
    s["flat"] = out
    return s


def prepare(case, seed):
    return {"clip": _gradients, "in": _expert_rows, "out": _expert_rows}.get(case["op"], _recurrence)(case, seed)


# ---------------------------------------------------------------------------
# The plain forms.
# ---------------------------------------------------------------------------
def _coefficients(s):
    """(a, 1 - a or None) of the gate's kind.  A decay next to 1 acts thousands
    of times, and with it the bias that an exponential in 32 bits has there, so
    it is computed in 64 and rounded once."""
    if s["kind"] == "decay":
        return s["gate"].to(torch.float32, copy=True), None
    gate = s["gate"].double()
    if s["kind"] == "log":
        return torch.exp(gate).float(), None
    return torch.sigmoid(gate).float(), torch.sigmoid(-gate).float()


def _row_of(s):
    """Per packed token: its row (rows: none), whether it is the row's first,
    whether its last."""
    starts, tokens = s["starts"].long(), s["x"].shape[0]
    t = torch.arange(tokens, device=starts.device)
    row = torch.searchsorted(starts[1:], t, right=True)
    inside = row.clamp(max=starts.numel() - 2)
    real = row < starts.numel() - 1
    return row, real, real & (starts[inside] == t), real & (starts[inside + 1] == t + 1)


def _doubling(a, b):
    """b[t] += a[t] b[t - 1], over the second dimension from the last, by
    composing ever longer steps."""
    step = 1
    while step < b.shape[-2]:
        b[..., step:, :] += a[..., step:, :] * b[..., :-step, :]
        a[..., step:, :] *= a[..., :-step, :].clone()
        step *= 2
    return b


def _plain_scan(s):
    a, rest = _coefficients(s)
    b = s["x"].float() * rest if rest is not None else s["x"].to(torch.float32, copy=True)
    state, final = s["initial"], s["final"]
    if s["starts"] is None:
        h0 = 0.0 if state is None else state if s["slots"] is None else state[s["slots"].long()]
        b[:, 0] += a[:, 0] * h0
        a[:, 0] = 0
        h = _doubling(a, b)
        if s["slots"] is None:
            final.copy_(h[:, -1])
        else:
            final[s["slots"].long()] = h[:, -1]
        return [h.to(s["x"].dtype), final]
    row, real, first, last = _row_of(s)
    rows = s["starts"].numel() - 1
    slot = torch.arange(rows, device=a.device) if s["slots"] is None else s["slots"].long()
    b *= real[:, None]
    if state is not None:
        b[first] += a[first] * state[slot[row[first]]]
    a *= (real & ~first)[:, None]
    h = _doubling(a, b)
    empty = s["starts"][1:] == s["starts"][:-1]
    final[slot[empty]] = 0.0 if state is None else state[slot[empty]]
    final[slot[row[last]]] = h[last]
    return [h.to(s["x"].dtype), final]


def _plain_backward(s):
    a, rest = _coefficients(s)
    y, grad = s["y"].float(), s["grad"].to(torch.float32, copy=True)
    before = torch.zeros_like(y)
    after = torch.zeros_like(a)
    before[..., 1:, :] = y[..., :-1, :]
    after[..., :-1, :] = a[..., 1:, :]
    if s["starts"] is None:
        before[:, 0] = 0.0 if s["initial"] is None else s["initial"]
        if s["grad_final"] is not None:
            grad[:, -1] += s["grad_final"]
    else:
        row, real, first, last = _row_of(s)
        before[first] = 0.0 if s["initial"] is None else s["initial"][row[first]]
        after *= ~last[:, None]
        grad *= real[:, None]
        after *= real[:, None]
        if s["grad_final"] is not None:
            grad[last] += s["grad_final"][row[last]]
    weight = _doubling(after.flip(-2), grad.flip(-2)).flip(-2)
    grad_initial = None
    if s["initial"] is not None:
        if s["starts"] is None:
            grad_initial = a[:, 0] * weight[:, 0]
        else:
            grad_initial = torch.zeros_like(s["initial"]) if s["grad_final"] is None else s["grad_final"].clone()
            grad_initial[row[first]] = a[first] * weight[first]
    if s["kind"] == "sigmoid":
        grad_gate, grad_x = weight * (before - s["x"].float()) * (a * rest), weight * rest
    else:
        grad_gate, grad_x = weight * before if s["kind"] == "decay" else weight * before * a, weight
    if s["starts"] is not None:
        grad_gate *= real[:, None]
    outputs = [grad_x.to(s["x"].dtype), grad_gate.to(s["gate"].dtype)]
    return outputs if grad_initial is None else outputs + [grad_initial]


def _plain_sort(s):
    ids, experts, align, rows = s["ids"].long().reshape(-1), s["experts"], s["align"], s["rows"]
    good = (ids >= 0) & (ids < experts)
    key = torch.where(good, ids, experts)
    by = torch.argsort(key, stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.long, device=ids.device)
    counts = counts.index_add_(0, key, torch.ones_like(key))[:-1]
    room = torch.div(counts + align - 1, align, rounding_mode="floor") * align
    zero = counts.new_zeros(1)
    starts = torch.cat([zero, torch.cumsum(room, 0)])
    ahead = torch.cat([zero, torch.cumsum(counts, 0)])
    rank = torch.arange(ids.numel(), device=ids.device) - ahead[key[by]]
    at = torch.where(good[by], starts[key[by]] + rank, -1)
    places = torch.empty_like(ids).scatter_(0, by, at)
    order = torch.where(torch.arange(rows, device=ids.device) < starts[-1], -1, -2)
    order[at[good[by]]] = by[good[by]]
    i32 = torch.int32
    return [starts.to(i32), counts.to(i32), order.to(i32), places.to(i32).reshape(s["ids"].shape)]


def _plain_in(s):
    starts, counts, order, places = _plain_sort(s)
    token = torch.div(order.long(), s["ids"].shape[1], rounding_mode="floor")
    rows = torch.where((order >= 0)[:, None], s["x"][token.clamp(min=0)], torch.zeros_like(s["x"][:1]))
    out = torch.where((order > -2)[:, None], rows, s["out"])
    return [starts, counts, order, places, out]


def _plain_out(s):
    places, weights = s["places"].long(), s["weights"]
    live = places >= 0
    weights = torch.where(live, weights, 0.0)
    y = s["y"].float()[places.clamp(min=0)]
    out = (weights[..., None] * y).sum(1).to(s["y"].dtype)
    if not s["gradient"]:
        return [out]
    grad = s["grad"].float()
    grad_weights = torch.where(live, (grad[:, None] * y).sum(2), 0.0)
    grad_y = torch.where((s["order"] > -2)[:, None], torch.zeros_like(s["grad_y"]), s["grad_y"])
    grad_y[places[live]] = (weights[..., None] * grad[:, None]).to(grad_y.dtype)[live]
    return [out, grad_y, grad_weights]


def _plain_clip(s):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = total.sqrt()
    scale = (s["max_norm"] / (norm + EPS)).clamp(max=1.0).float()
    for g, out in zip(s["grads"], s["out"]):
        out.copy_(g.float() * scale)
    return [norm.float(), s["flat"]]


def run(state):
    s = state
    if not own:
        return {"scan": _plain_scan, "step": _plain_scan, "backward": _plain_backward, "in": _plain_in,
                "out": _plain_out, "clip": _plain_clip}[s["op"]](s)
    import stream_compaction_device_gb300 as ds
    if s["op"] in ("scan", "step"):
        return list(ds.gated_scan(s["x"], s["gate"], starts=s["starts"], initial=s["initial"], slots=s["slots"],
                                  kind=s["kind"], out=s["out"], final=s["final"]))
    if s["op"] == "backward":
        grads = ds.gated_scan_backward(s["grad"], s["x"], s["gate"], s["y"], starts=s["starts"],
                                       initial=s["initial"], grad_final=s["grad_final"], kind=s["kind"])
        return [g for g in grads if g is not None]
    if s["op"] == "in":
        starts, counts, order, places = ds.expert_sort(s["ids"], s["experts"], align=s["align"], rows=s["rows"])
        return [starts, counts, order, places, ds.expert_dispatch(s["x"], places, order, out=s["out"])]
    if s["op"] == "out":
        out = ds.expert_combine(s["y"], s["places"], s["weights"])
        if not s["gradient"]:
            return [out]
        return [out, *ds.expert_combine_backward(s["grad"], s["y"], s["places"], s["weights"], s["order"],
                                                 grad_y=s["grad_y"])]
    return [ds.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])[0], s["flat"]]


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("scan", "step", "backward"):
        size, gate = SIZES[case["dtype"]], SIZES[case["gate"]]
        rows, states = case["rows"], case["rows"] * case["channels"] * 4
        n = case["tokens"] * case["channels"] * (1 if case["packed"] else rows)
        more = 4 * (rows + 1) if case["packed"] else 0
        if op != "backward":
            return {"bytes": n * (2 * size + gate) + states * (2 if case["carry"] else 1) + more, "flops": 4 * n}
        values = 3 if case["kind"] != "sigmoid" else 4
        return {"bytes": n * (values * size + 2 * gate) + states * (3 if case["carry"] else 0) + more,
                "flops": 8 * n}
    if op in ("in", "out"):
        size, width, tokens = SIZES[case["dtype"]], case["width"], case["tokens"]
        real = tokens - min(tokens, case["pad"])
        pairs = tokens * case["choices"]
        moved = real * case["choices"] * width * size
        if op == "in":
            ids = 4 if case["ids"] == "i32" else 8
            return {"bytes": moved + real * width * size + pairs * (ids + 8) + 8 * case["experts"], "flops": pairs}
        once = tokens * width * size
        if not case["gradient"]:
            return {"bytes": moved + once + 8 * pairs, "flops": 2 * pairs * width}
        return {"bytes": 2 * moved + 2 * once + 12 * pairs, "flops": 5 * pairs * width}
    return {"bytes": sum(2 * n * SIZES[d] for n, d in _tensors(case)), "flops": 3 * case["elements"]}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits.
# ---------------------------------------------------------------------------
def _exact_gate(s):
    g = s["gate"].double()
    if s["kind"] == "decay":
        return g, torch.ones_like(g)
    if s["kind"] == "log":
        return torch.exp(g), torch.ones_like(g)
    return 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))


def _spans(s):
    """Each row's tokens: (row or all rows, first, end)."""
    if s["starts"] is None:
        return [(None, 0, s["x"].shape[1])]
    at = s["starts"].tolist()
    return [(r, at[r], at[r + 1]) for r in range(len(at) - 1)]


def _exact_scan(s):
    a, part = _exact_gate(s)
    b = part * s["x"].double()
    out, final = torch.zeros_like(b), torch.zeros(s["final"].shape, dtype=torch.float64, device="cuda")
    slots = None if s["slots"] is None else s["slots"].long()
    for r, t0, t1 in _spans(s):
        where = (slice(None) if r is None else r) if slots is None else slots if r is None else slots[r]
        h = s["initial"].double()[where] if s["initial"] is not None else final[where]
        get = (lambda v, t: v[:, t]) if r is None else (lambda v, t: v[t])
        for t in range(t0, t1):
            h = get(a, t) * h + get(b, t)
            get(out, t).copy_(h)
        final[where] = h
    return [out, final]


def _exact_backward(s):
    a, part = _exact_gate(s)
    x, y, grad = s["x"].double(), s["y"].double(), s["grad"].double()
    grad_x, grad_gate = torch.zeros_like(x), torch.zeros_like(x)
    rows, channels = s["grad_rows"], x.shape[-1]
    zero = torch.zeros(rows, channels, dtype=torch.float64, device="cuda")
    first = s["initial"].double() if s["initial"] is not None else zero
    grad_initial = s["grad_final"].double().clone() if s["grad_final"] is not None else zero.clone()
    for r, t0, t1 in _spans(s):
        where = slice(None) if r is None else r
        get = (lambda v, t: v[:, t]) if r is None else (lambda v, t: v[t])
        flow = grad_initial[where].clone()
        for t in range(t1 - 1, t0 - 1, -1):
            flow = flow + get(grad, t)
            ahead = get(y, t - 1) if t > t0 else first[where]
            d = ahead - get(x, t) if s["kind"] == "sigmoid" else ahead
            if s["kind"] == "log":
                d = d * get(a, t)
            elif s["kind"] == "sigmoid":
                d = d * get(a, t) * get(part, t)
            get(grad_gate, t).copy_(flow * d)
            get(grad_x, t).copy_(flow * get(part, t))
            flow = flow * get(a, t)
        grad_initial[where] = flow
    return [grad_x, grad_gate] + ([grad_initial] if s["initial"] is not None else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("scan", "step"):
        return _exact_scan(s)
    if case["op"] == "backward":
        return _exact_backward({**s, "grad_rows": case["rows"]})
    if case["op"] == "in":
        return None                           # whole numbers, and copies of rows
    if case["op"] == "out":
        tokens, choices = s["places"].shape
        out = torch.zeros(tokens, case["width"], dtype=torch.float64, device="cuda")
        grad_weights = torch.zeros(tokens, choices, dtype=torch.float64, device="cuda")
        grad_y = s["grad_y"].double() if case["gradient"] else None
        for k in range(choices):
            at = s["places"][:, k].long()
            token = torch.nonzero(at >= 0)[:, 0]
            y, w = s["y"][at[token]].double(), s["weights"][token, k].double()
            out[token] += w[:, None] * y
            if case["gradient"]:
                g = s["grad"][token].double()
                grad_weights[token, k] = torch.einsum("th,th->t", g, y)
                grad_y[at[token]] = w[:, None] * g
        return [out, grad_y, grad_weights] if case["gradient"] else [out]
    norm = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in s["grads"]))
    scale, sizes = min(1.0, s["max_norm"] / (norm + EPS)), {d: v.double() for d, v in s["flat"].items()}
    place = dict.fromkeys(sizes, 0)
    for (n, d), g in zip(_tensors(case), s["grads"]):
        sizes[d][place[d]:place[d] + n] = g.double() * scale
        place[d] += n if case["close"] else -(-n // 8) * 8
    return [torch.tensor(norm, dtype=torch.float64), sizes]
