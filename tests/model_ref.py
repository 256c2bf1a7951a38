"""Plain implementations in 64 bits for the tests of the gated recurrence, the
experts' sort and return, and the gradient norm, each with the room that the
library's arithmetic in 32 bits has (derived here, before any run)."""
import numpy as np
import torch

U = 2.0 ** -24                                    # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half the last denormal's


def as64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def decays(gate, kind):
    """(a, its relative room, what x is multiplied by, its relative room).

    log: within 1/16 of 0, 1 + s is rounded once (u, or 2u above 1) from an s of
    at most 0.065 with four roundings (a quarter u) and a series off by 2^-26 (a
    quarter u): below 4u.
    Elsewhere the hardware's exponential, off by 2 + 1.173 |g| units in the last
    place at most (2^-23 each).
    sigmoid: u = exp(-g) has that error; 1 + u another half unit, the reciprocal
    one: 1 / (1 + u) and r = u / (1 + u), a rounding more, are within (2 + 1.173
    |g| + 2) 2^-23; where u <= 1, a = 1 - r has r's error in absolute terms, less
    than that relative to a, which is not the smaller, and a rounding."""
    g = gate
    if kind == "decay":
        return g, np.zeros_like(g), np.ones_like(g), np.zeros_like(g)
    with np.errstate(over="ignore", invalid="ignore"):
        hard = (3 + 1.2 * np.minimum(np.abs(g), 1e3)) * 2 * U
        if kind == "log":
            return np.exp(g), hard + 4 * U, np.ones_like(g), np.zeros_like(g)
        room = hard + 6 * U
        return 1 / (1 + np.exp(-g)), room, 1 / (1 + np.exp(g)), room


def rows_of(starts, tokens, rows):
    """Token ranges of the rows of [rows, tokens] flattened, or packed."""
    if starts is None:
        return [(r * tokens, (r + 1) * tokens) for r in range(rows)]
    at = [min(max(int(s), 0), tokens) for s in starts]
    return list(zip(at[:-1], at[1:]))


def scan(x, gate, kind, spans, initial=None):
    """Forward over flat [n, channels] arrays in 64 bits, rows at `spans`.
    Returns (h, room of h, final, room of final).

    Room: however the maps are composed, each term a_t ... a_{s+1} b_s of h_t is
    reached through at most two roundings per token on its way (a product and a
    sum) and the decays' own errors, and through at most 40 more where warps,
    blocks and rounds are joined.  With G the same recurrence on absolute
    values, E_t = |a_t| E_{t-1} + (room of a_t + 2u) |a_t| G_{t-1} bounds the first."""
    a, ra, m, rm = decays(gate, kind)
    h, room = np.zeros_like(x), np.zeros_like(x)
    final = np.zeros((len(spans), x.shape[1]))
    final_room = np.zeros_like(final)
    for r, (t0, t1) in enumerate(spans):
        v = np.zeros(x.shape[1]) if initial is None else initial[r].copy()
        g, e = np.abs(v), np.zeros_like(v)
        first = initial is None
        for t in range(t0, t1):
            at = np.zeros_like(v) if first else a[t]
            first = False
            b = m[t] * x[t]
            e = np.abs(at) * e + (ra[t] + 2 * U) * np.abs(at) * g + (rm[t] + 2 * U) * np.abs(b)
            v = b if not np.any(at) else at * v + b
            g = np.abs(at) * g + np.abs(b)
            h[t], room[t] = v, e + 40 * U * g + 2.0 ** -120
        final[r], final_room[r] = v, (room[t1 - 1] if t1 > t0 else 0.0)
    return h, room, final, final_room


def scan_backward(grad, x, gate, y, kind, spans, initial=None, grad_final=None):
    """Backward in 64 bits: dict of (value, room) for x, gate and initial."""
    a, ra, m, rm = decays(gate, kind)
    channels = grad.shape[1]
    out = {k: (np.zeros_like(grad), np.zeros_like(grad)) for k in ("x", "gate")}
    gi = (np.zeros((len(spans), channels)), np.zeros((len(spans), channels)))
    for r, (t0, t1) in enumerate(spans):
        f = np.zeros(channels) if grad_final is None else grad_final[r].copy()
        g, e = np.abs(f), np.zeros(channels)
        for t in range(t1 - 1, t0 - 1, -1):
            w, gw = f + grad[t], g + np.abs(grad[t])
            ew = e + 2 * U * gw
            rw = ew + 40 * U * gw + 2.0 ** -120
            before = y[t - 1] if t > t0 else np.zeros(channels) if initial is None else initial[r]
            if kind == "decay":
                k, rk = before, np.zeros(channels)
            elif kind == "log":
                k, rk = before * a[t], np.abs(before * a[t]) * (ra[t] + 2 * U)
            else:
                k = (before - x[t]) * a[t] * m[t]
                rk = np.abs(k) * (ra[t] + rm[t] + 4 * U)
            out["x"][0][t], out["x"][1][t] = w * m[t], rw * m[t] + np.abs(w * m[t]) * (rm[t] + 2 * U)
            out["gate"][0][t], out["gate"][1][t] = w * k, rw * np.abs(k) + (np.abs(w) + rw) * rk + 2 * U * np.abs(w * k)
            f, g, e = a[t] * w, np.abs(a[t]) * gw, np.abs(a[t]) * (ew + (ra[t] + 2 * U) * gw)
        gi[0][r], gi[1][r] = f, e + 40 * U * g + 2.0 ** -120
    return {**out, "initial": gi}


def close(got, want, room, what=""):
    """got (a tensor of its type) is want within room and one rounding to its
    type; infinities and NaN where want has them."""
    v = got.detach().cpu().double().numpy()
    half, tiny = HALF[got.dtype], TINY[got.dtype]
    with np.errstate(invalid="ignore", over="ignore"):
        limit = room * (1 + half) + half * np.abs(want) + tiny
        top = torch.finfo(got.dtype).max
        bad = ~(np.abs(v - want) <= limit)
        bad &= ~(np.isnan(v) & np.isnan(want))
        bad &= ~(np.isinf(v) & (np.sign(v) == np.sign(want)) & (np.abs(want) + limit >= top))
    at = np.argwhere(bad)
    assert at.size == 0, (f"{what}: {len(at)} of {v.size} outside; first at {tuple(at[0])}: got {v[tuple(at[0])]!r}, "
                          f"want {want[tuple(at[0])]!r}, room {limit[tuple(at[0])]!r}")


def sort(ids, experts, align, rows):
    """(starts, counts, order, places) of a loop over the pairs."""
    flat = [int(i) for i in np.asarray(ids).reshape(-1)]
    of = [[i for i, e in enumerate(flat) if e == k] for k in range(experts)]
    starts = [0]
    for pairs in of:
        starts.append(starts[-1] + -(-len(pairs) // align) * align)
    order, places = np.full(rows, -2, np.int64), np.full(len(flat), -1, np.int64)
    order[: starts[-1]] = -1
    for e, pairs in enumerate(of):
        for j, i in enumerate(pairs):
            if starts[e] + j < rows:
                order[starts[e] + j], places[i] = i, starts[e] + j
    return np.array(starts), np.array([len(p) for p in of]), order, places


def combine(y, places, weights):
    """(out, room): sums of at most `choices` products in fp32."""
    tokens, choices = places.shape
    out, size = np.zeros((tokens, y.shape[1])), np.zeros((tokens, y.shape[1]))
    for t in range(tokens):
        for k in range(choices):
            if 0 <= places[t, k] < len(y):
                term = y[places[t, k]] * (1.0 if weights is None else weights[t, k])
                out[t] += term
                size[t] += np.abs(term)
    return out, (choices + 1) * U * size + 2.0 ** -149 * choices


def combine_backward(grad, y, places, weights, grad_y):
    """(grad_y with what stays of it, grad_weights, room of those): a lane adds
    at most width / 128 + 8 products, then seven sums."""
    tokens, choices = places.shape
    grad_y, gw, size = grad_y.copy(), np.zeros((tokens, choices)), np.zeros((tokens, choices))
    for t in range(tokens):
        for k in range(choices):
            p = places[t, k]
            if 0 <= p < len(y):
                grad_y[p] = grad[t] * (1.0 if weights is None else weights[t, k])
                gw[t, k] = grad[t] @ y[p]
                size[t, k] = np.abs(grad[t]) @ np.abs(y[p])
    return grad_y, gw, (grad.shape[1] / 128 + 24) * U * size + 2.0 ** -149 * grad.shape[1]


def norm(tensors):
    """A share of 64 values at most is added in fp32 (33 roundings on two
    paths and a sum), all else in fp64: the relative room of the sum is 34u, of
    its root half of it, and a rounding."""
    value = float(np.sqrt(sum(float((as64(t) ** 2).sum()) for t in tensors)))
    return value, value * 20 * U
