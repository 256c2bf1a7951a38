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
