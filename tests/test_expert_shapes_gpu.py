"""Weights of the experts' rows have the shape of their places."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def test_weights_shapes(ds):
    """[choices, tokens] in place of [tokens, choices] is refused, not taken in
    another order; weights in the places' order are taken flat, too."""
    ids = torch.arange(8, dtype=torch.int32, device="cuda").reshape(4, 2) % 3
    _, _, order, places = ds.expert_sort(ids, 3)
    y, grad = torch.randn(8, 16, device="cuda"), torch.randn(4, 16, device="cuda")
    w = torch.rand(4, 2, device="cuda")
    want = ds.expert_combine(y, places, w)
    back = ds.expert_combine_backward(grad, y, places, w, order)
    for same in (w.reshape(-1), w.reshape(1, 8), w[..., None], w[None]):
        assert torch.equal(ds.expert_combine(y, places, same), want)
        got = ds.expert_combine_backward(grad, y, places, same, order, grad_weights=torch.empty_like(same))
        assert torch.equal(got[0], back[0]) and torch.equal(got[1].reshape(4, 2), back[1])
    for other in (w.t().contiguous(), w.reshape(1, 8, 1)[:, :, 0].reshape(2, 2, 2), w.reshape(8)[:4].reshape(4, 1)):
        for call in (lambda: ds.expert_combine(y, places, other), lambda: ds.expert_combine_backward(grad, y, places, other, order),
                     lambda: ds.expert_combine_backward(grad, y, places, w, order, grad_weights=torch.empty_like(other))):
            with pytest.raises(ValueError):
                call()
    one = places[:, :1].contiguous()                              # one choice, one token: the order is one
    assert torch.equal(ds.expert_combine(y, one, w[:, :1].reshape(1, 4).contiguous()), ds.expert_combine(y, one, w[:, :1].contiguous()))
