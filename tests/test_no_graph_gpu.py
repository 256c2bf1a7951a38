"""The calls are no autograd functions, and say so where a gradient is lost."""
import warnings

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def test_lost_gradients_are_told(ds):
    x, gate = torch.randn(1, 20, 8, device="cuda"), torch.rand(1, 20, 8, device="cuda")
    state, leaf = torch.randn(1, 8, device="cuda"), lambda t: t.clone().requires_grad_()
    y, _ = ds.gated_scan(x, gate)
    _, _, order, places = ds.expert_sort(torch.zeros(20, 1, dtype=torch.int32, device="cuda"), 2)
    tokens, weights = torch.randn(20, 8, device="cuda"), torch.rand(20, 1, device="cuda")
    lost = [lambda: ds.gated_scan(leaf(x), gate), lambda: ds.gated_scan(x, leaf(gate)), lambda: ds.gated_scan(x, gate, initial=leaf(state)),
            lambda: ds.gated_scan_backward(leaf(x), None, gate, y), lambda: ds.expert_dispatch(leaf(tokens), places, order),
            lambda: ds.expert_combine(leaf(tokens), places, weights), lambda: ds.expert_combine(tokens, places, leaf(weights)),
            lambda: ds.expert_combine_backward(leaf(tokens), tokens, places, weights, order)]
    for call in lost:
        with pytest.warns(UserWarning, match="autograd"):
            call()
        with warnings.catch_warnings(), torch.no_grad():
            warnings.simplefilter("error")
            call()

    class Inside(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gate):
            h, _ = ds.gated_scan(x, gate)
            ctx.save_for_backward(gate, h)
            return h

        @staticmethod
        def backward(ctx, grad):
            return ds.gated_scan_backward(grad.contiguous(), None, *ctx.saved_tensors)[:2]

    with warnings.catch_warnings():
        warnings.simplefilter("error")
        ds.gated_scan(x, gate, initial=state)
        Inside.apply(leaf(x), leaf(gate)).sum().backward()
