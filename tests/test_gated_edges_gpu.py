"""The gated recurrence where a call's arguments are at an edge: rows that begin
in front of the tokens, first gates that do not count, arrays side by side."""
import numpy as np
import pytest
import torch

import model_ref as ref
from test_gated_scan_gpu import BF16, F16, F32, KINDS, check, cuda, ds, flat, gates  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("starts,tokens", [([-50, 7, 20, 30], 30), ([-5, -3, -1, 40, 64], 70), ([-1, 300], 300), ([-9, 0, 0, 250], 300),
                                           ([-50, 7000, *range(7001, 7060)], 7060), ([-7, *range(1, 60), 6000], 6000)],
                         ids=lambda v: str(v)[:12])
def test_rows_that_begin_in_front(ds, starts, tokens, kind):  # noqa: F811
    """Such a row's first token is the first that there is: with its state or without, forward and back."""
    rng = np.random.default_rng(tokens)
    for dtype, channels in ((F32, 40), (BF16, 64), (F16, 33)):
        for carry in (False, True):
            check(ds, rng, len(starts) - 1, tokens, channels, dtype, dtype, kind, starts=starts, carry=carry)


@pytest.mark.parametrize("kind", ["decay", "log"])
def test_first_gates_in_front(ds, kind):  # noqa: F811
    """The first gate of a row that begins in front does not count without a state."""
    x, gate = torch.randn(30, 64, device="cuda"), -torch.rand(30, 64, device="cuda")
    where = torch.tensor([-4, 9, 30], dtype=torch.int32, device="cuda")
    want, last = ds.gated_scan(x, gate, starts=where, kind=kind)
    gate[[0, 9]] = float("nan")
    out, final = ds.gated_scan(x, gate, starts=where, kind=kind)
    assert out.isfinite().all() and torch.equal(out, want) and torch.equal(final, last)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 200.0])
@pytest.mark.parametrize("kind", ["decay", "log"])
@pytest.mark.parametrize("dtype,channels", [(F32, 40), (BF16, 64), (BF16, 33)])
def test_gradients_of_first_gates(ds, dtype, channels, kind, bad):  # noqa: F811
    """What does not count has no gradient, whatever it holds: the first gates of
    rows without a state, of equal rows and of packed ones."""
    rng = np.random.default_rng(3)
    for starts in (None, [0, 1, 1, 60, 100]):
        shape = (3, 100, channels) if starts is None else (110, channels)
        x, gate = cuda(rng.standard_normal(shape), dtype), cuda(gates(rng, shape, kind), dtype)
        grad = cuda(rng.standard_normal(shape), dtype)
        where = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
        first = (slice(None), 0) if starts is None else ([0, 1, 60],)
        y = ds.gated_scan(x, gate, starts=where, kind=kind)[0]
        want = ds.gated_scan_backward(grad, None, gate, y, starts=where, kind=kind)
        assert not want[1][first].any()
        gate[first] = bad
        assert torch.equal(ds.gated_scan(x, gate, starts=where, kind=kind)[0], y)
        got = ds.gated_scan_backward(grad, None, gate, y, starts=where, kind=kind)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        grad[first] = float("inf")
        got = ds.gated_scan_backward(grad, None, gate, y, starts=where, kind=kind)
        assert torch.equal(got[1], want[1])


def test_time_major_arrays_side_by_side(ds):  # noqa: F811
    """Parts of one time-major projection, [tokens, rows, parts x channels], as
    x, gate and outputs: the same strides, side by side in each token."""
    rng = np.random.default_rng(5)
    for tokens, rows, c in ((40, 3, 16), (5, 4, 24), (200, 2, 8)):
        buffer = cuda(rng.standard_normal((tokens, rows, 5 * c)), BF16)
        parts = [buffer[..., c * i:c * i + c].transpose(0, 1) for i in range(5)]
        x, gate = parts[0].contiguous(), parts[2].contiguous()
        want, _ = ds.gated_scan(x, gate, kind="sigmoid")
        out, _ = ds.gated_scan(parts[0], parts[2], kind="sigmoid", out=parts[1])
        assert torch.equal(out, want) and torch.equal(parts[0], x) and torch.equal(parts[2], gate)
        back = ds.gated_scan_backward(x, x, gate, want, kind="sigmoid")
        ds.gated_scan_backward(parts[0], parts[0], parts[2], parts[1], kind="sigmoid", grad_x=parts[4], grad_gate=parts[3])
        assert torch.equal(parts[4], back[0]) and torch.equal(parts[3], back[1]) and torch.equal(parts[1], want)
        for shift in (c // 2, c + c // 2, 4 * c + c // 2):      # across a neighbour, and into the next row's
            if shift + c <= 5 * c:
                with pytest.raises(ds.DevscanError):
                    ds.gated_scan(parts[0], parts[2], kind="sigmoid", out=buffer[..., shift:shift + c].transpose(0, 1))
        wide = buffer.reshape(tokens, -1)                       # the last part shifted into the next row's first
        across = wide[:, 4 * c + c // 2:].as_strided((rows - 1, tokens, c), (5 * c, rows * 5 * c, 1))
        x, gate = x[:-1], gate[:-1]
        if rows > 2:
            with pytest.raises(ds.DevscanError):
                ds.gated_scan(parts[0][:-1], parts[2][:-1], kind="sigmoid", out=across)
        else:                                                   # one row, and the next one's part is not given
            want, _ = ds.gated_scan(x, gate, kind="sigmoid")
            assert torch.equal(ds.gated_scan(parts[0][:-1], parts[2][:-1], kind="sigmoid", out=across)[0], want)


def test_errors_do_not_lean(ds):  # noqa: F811
    """60,000 tokens through decays next to 1, all terms positive.  Errors that
    are as often up as down: with memories of M tokens the state's relative error
    is a sum of M / 2 tokens' worth of independent roundings, of the decay (next
    to 1 from below: at most 2^-25, variance 2^-50 / 3) and of the running value
    (at most 2^-24: 2^-48 / 3), a standard deviation of 2^-24 sqrt(5 M / 24).
    Five of those; log: M = 2,000, and for its series four roundings of values of
    10^-3 at most, M / 2 of them; sigmoid: M = 1,740, and the hardware's
    exponential, which may lean by (3 + 1.2 |g|) 2^-23 in b and as much, times
    M (1 - a), in a.  A decay off to one side by a tenth of 2^-24 is 1.2e-5 and
    1.0e-5 off."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n, c = 60000, 64
    x = torch.randn(1, n, c, generator=g, device="cuda").abs_()
    for kind, memory, lean in (("log", 2000, 1000 * 4 * 1e-3 * 2.0 ** -24), ("sigmoid", 1740, 2 * (3 + 1.2 * 8) * 2.0 ** -23)):
        gate = torch.rand(1, n, c, generator=g, device="cuda")
        gate = -gate * 1e-3 if kind == "log" else 7 + gate
        final = ds.gated_scan(x, gate, kind=kind)[1]
        a = torch.exp(gate.double()) if kind == "log" else torch.sigmoid(gate.double())
        b = x.double() * (1 if kind == "log" else torch.sigmoid(-gate.double()))
        h = torch.zeros(c, dtype=torch.float64, device="cuda")
        for t in range(n):
            h = a[0, t] * h + b[0, t]
        error = (final[0].double() - h) / h
        limit = 5 * 2.0 ** -24 * (5 * memory / 24) ** 0.5 + lean
        assert error.abs().max().item() < limit < 1e-5, (kind, error.abs().max().item(), limit)


def test_what_rounded_outputs_cost_the_gates(ds):  # noqa: F811
    """The backward call takes h as it was rounded to the output's type.  Where x
    moves slowly h' - x is small beside h', and the gate's gradient is then off
    by at most |w| a (1 - a) half |h'| from that of the recurrence that is not
    rounded: more than its own rounding in 16 bits, nothing to speak of in 32."""
    rng = np.random.default_rng(8)
    rows, tokens, channels = 1, 400, 32
    shape = (rows, tokens, channels)
    slow = 1 + 0.02 * np.sin(np.arange(tokens) / 40)[None, :, None] + 0.002 * rng.standard_normal(shape)
    shares = {}
    for dtype in (F32, F16, BF16):
        x, gate, grad = cuda(slow, dtype), cuda(rng.standard_normal(shape) + 1, F32), cuda(rng.standard_normal(shape), dtype)
        spans = ref.rows_of(None, tokens, rows)
        initial = torch.ones(1, channels, device="cuda")
        y = ds.gated_scan(x, gate, initial=initial, kind="sigmoid")[0]
        got = ds.gated_scan_backward(grad, x, gate, y, initial=initial, kind="sigmoid")[1]
        h, h_room, _, _ = ref.scan(flat(x), flat(gate), "sigmoid", spans, np.ones((1, channels)))
        value, room = ref.scan_backward(flat(grad), flat(x), flat(gate), h, "sigmoid", spans, np.ones((1, channels)))["gate"]
        a = 1 / (1 + np.exp(-flat(gate)))
        w = np.abs(ref.scan_backward(flat(grad), flat(x), flat(gate), h, "sigmoid", spans)["x"][0]) / (1 - a)
        before = np.vstack([np.zeros((1, channels)), ref.HALF[dtype] * np.abs(h[:-1]) + h_room[:-1] * 2])   # the state is fp32
        cost = w * a * (1 - a) * before
        ref.close(got.reshape(-1, channels), value, room + cost, f"{dtype}")
        error = np.abs(ref.as64(got)[0] - value)
        shares[dtype] = np.linalg.norm(error) / np.linalg.norm(value)
    assert shares[F32] < 1e-4 < shares[BF16], shares


@pytest.mark.parametrize("dtype,gate_dtype,sign", [(F32, F32, "plus"), (F32, F32, "minus"), (F32, F32, "in turn"), (F16, F16, "plus"),
                                                   (F16, F16, "minus"), (F16, F16, "in turn"), (BF16, BF16, "plus"),
                                                   (BF16, BF16, "minus"), (BF16, F32, "plus")])
@pytest.mark.parametrize("how", ["shared", "drawn"])
def test_decays_that_repeat(ds, how, dtype, gate_dtype, sign):  # noqa: F811
    """Decays next to 1 that all tokens share, or that 16 bits leave few of: what
    is rounded alike in every run of tokens does not add up.  A run (24 tokens
    forward, 16 backward, of long rows) leaves one rounding of its product, and the
    product of the runs one more, each of variance 2^-50 / 3 over the channels,
    which have decays of their own; a channel's memory of M <= 4,900 tokens adds
    M / 24 (16) of them, all alike: the error's norm over the channels is at most
    that of the longest memory, beside which independent roundings (2^-24 sqrt(5 M
    / 24) as in test_errors_do_not_lean, of which the runs' sums have a part) are
    small; both are in the limit.  Multiplied up token by token, (1 - 2^-11)^24
    alone is 4 times 2^-24 off."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, c = 20000, 256
    slow = torch.exp(torch.rand(c, generator=g, device="cuda") * 5 - 8.5)
    noise = torch.ones(1, n, c, device="cuda") if how == "shared" else 2 * torch.rand(1, n, c, generator=g, device="cuda")
    gate = torch.exp(-slow * noise)
    if sign != "plus":
        gate[:, ::1 if sign == "minus" else 2] *= -1
    gate = gate.to(gate_dtype)
    x = torch.rand(1, n, c, generator=g, device="cuda").to(dtype)
    y, final = ds.gated_scan(x, gate)
    state = torch.zeros(1, c, device="cuda")
    back = ds.gated_scan_backward(x, None, gate, y, initial=state)[2]
    a, b = gate[0].double(), x[0].double()
    h, f = torch.zeros(c, dtype=torch.float64, device="cuda"), torch.zeros(c, dtype=torch.float64, device="cuda")
    for t in range(n):
        h = a[t] * h + b[t]
        f = a[n - 1 - t] * (f + b[n - 1 - t])
    for got, want, run in ((final[0], h, 24), (back[0], f, 16)):
        limit = 4900 / run * (2 / 3) ** 0.5 * 2.0 ** -25 + 2.0 ** -24 * (5 * 4900 / 24) ** 0.5 / 4
        error = ((got.double() - want).norm() / want.norm()).item()
        assert error < limit, (how, dtype, sign, run, error, limit)
