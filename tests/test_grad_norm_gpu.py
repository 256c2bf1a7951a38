"""The norm over many tensors, and clipping, on the GPU against 64 bits."""
import math

import numpy as np
import pytest
import torch

import model_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def check(ds, tensors, max_norm=1.0):
    want, room = ref.norm(tensors)
    norm = ds.grad_norm(tensors)
    ref.close(norm, np.array([want]), np.array([room]), "norm")
    scale = min(1.0, max_norm / (want + 1e-6))
    near = [(ref.as64(t) * scale, np.abs(ref.as64(t)) * scale * 24 * ref.U) for t in tensors]
    out = [torch.full_like(t, 7) for t in tensors]
    again, got = ds.clip_grad_norm(tensors, max_norm, out=out)
    assert torch.equal(again, norm) and got[0] is out[0]
    for t, (value, r) in zip(out, near):
        ref.close(t, value, r, "clipped")
    into = [t.clone() for t in tensors]
    ds.clip_grad_norm(into, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(into, out))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("n", [1, 3, 7, 8, 9, 31, 4096, 16384, 16385, 100003, 1 << 20])
def test_sizes(ds, dtype, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    check(ds, [torch.randn(n, generator=g, device="cuda").to(dtype)], 0.5)
    check(ds, [torch.randn(n, generator=g, device="cuda").to(dtype)], 1e9)      # nothing to clip


def test_mixed_tensors_at_every_alignment(ds):
    g = torch.Generator(device="cuda").manual_seed(1)
    tensors = []
    for i, n in enumerate([5, 1000, 0, 64, 70001, 1, 16, 40000, 9, 33333]):
        dtype = (F32, F16, BF16)[i % 3]
        tensors.append(torch.randn(n + 8, generator=g, device="cuda").to(dtype)[i % 8:i % 8 + n])
    check(ds, tensors, 3.0)
    check(ds, [t.reshape(-1, 1, 1) for t in tensors], 3.0)


def test_outputs_of_other_alignment(ds):
    g = torch.Generator(device="cuda").manual_seed(2)
    for dtype in (F32, BF16):
        t = torch.randn(50001, generator=g, device="cuda").to(dtype)
        want = ds.clip_grad_norm([t], 1.0, out=[torch.empty_like(t)])[1][0]
        for shift in (1, 3):
            out = torch.full((50011,), 7.0, device="cuda").to(dtype)
            ds.clip_grad_norm([t], 1.0, out=[out[shift:shift + 50001]])
            assert torch.equal(out[shift:shift + 50001], want) and (out[:shift] == 7).all() and (out[shift + 50001:] == 7).all()


def test_many_tensors(ds):
    """More than one launch's table, empty ones among them."""
    g = torch.Generator(device="cuda").manual_seed(3)
    flat = torch.randn(400000, generator=g, device="cuda")
    for count in (511, 512, 513, 1300):
        cuts = torch.sort(torch.randint(0, 400000, (count - 1,), generator=torch.Generator().manual_seed(count)))[0].tolist()
        tensors = [flat[a:b] for a, b in zip([0, *cuts], [*cuts, 400000])]
        check(ds, tensors, 2.0)


def test_range(ds):
    """Values whose squares overflow or vanish in fp32, beside each other."""
    for values in ([3e38, 1e38], [1e-30, 2e-30], [1e-45, 3e-42], [1e25, 1e-30, 1.0], [0.0, 0.0]):
        for n in (1, 5000):
            t = torch.tensor(values * n, device="cuda")
            norm = ds.grad_norm([t, t[:1]])
            want, room = ref.norm([t, t[:1]])
            ref.close(norm, np.array([want]), np.array([room]), f"{values}")
    t = torch.full((3000,), 1e30, device="cuda")
    assert torch.allclose(ds.clip_grad_norm([t], 1.0)[1][0], torch.full_like(t, 1 / math.sqrt(3000)), rtol=1e-6)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("at", [0, 5, 40001])
def test_not_finite(ds, bad, at):
    """Such a norm is reported and clips nothing, in place or not."""
    t = torch.randn(40003, device="cuda")
    t[at] = bad
    other = torch.randn(100, device="cuda").to(BF16)
    norm = ds.grad_norm([other, t])
    assert torch.isnan(norm) if math.isnan(bad) else torch.isposinf(norm)
    keep = t.clone()
    ds.clip_grad_norm([other, t], 1.0)
    assert torch.equal(t.nan_to_num(5.0), keep.nan_to_num(5.0))
    out = ds.clip_grad_norm([t], 1.0, out=[torch.zeros_like(t)])[1][0]
    assert torch.equal(out.nan_to_num(5.0), keep.nan_to_num(5.0))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_range_in_whole_vectors(ds, dtype):
    """Shares of a thread whose squares leave fp32, next to ordinary ones, at every size of value."""
    exponents = range(-24, 16, 3) if dtype == F16 else range(-149, 128, 5) if dtype == F32 else range(-133, 128, 5)
    for e in exponents:
        t = torch.full((5000,), 2.0 ** e, dtype=torch.float64).to(dtype).cuda()
        t[::3] *= -1
        t[::7] = 0
        for tensors in ([t], [t, torch.ones(4096, dtype=dtype, device="cuda")]):
            want, room = ref.norm(tensors)
            ref.close(ds.grad_norm(tensors), np.array([want]), np.array([room]), f"2^{e}")


def test_norm_past_fp32(ds):
    """A norm of finite values that fp32 does not hold is given as infinite, and clips nothing."""
    for n, whole in ((1, True), (300, False)):
        t = torch.full((n,), 3e38, device="cuda")
        keep = t.clone()
        norm, _ = ds.clip_grad_norm([t], 1.0)
        assert torch.isfinite(norm).item() is whole
        assert torch.allclose(t, torch.ones_like(t)) if whole else torch.equal(t, keep)


def test_nothing(ds):
    assert ds.grad_norm([]).item() == 0
    norm, out = ds.clip_grad_norm([torch.empty(0, device="cuda")], 1.0)
    assert norm.item() == 0 and out[0].numel() == 0
    t = torch.zeros(100, device="cuda")
    assert ds.clip_grad_norm([t], 0.0)[0].item() == 0 and not t.any()
    t += 3
    ds.clip_grad_norm([t], 0.0)
    assert not t.any()


def test_same_bits_streams_and_graphs(ds):
    g = torch.Generator(device="cuda").manual_seed(4)
    tensors = [torch.randn(n, generator=g, device="cuda").to(d) for n, d in ((300000, F32), (77, BF16), (1 << 20, BF16))]
    want = ds.clip_grad_norm(tensors, 1.0, out=[torch.empty_like(t) for t in tensors])
    torch.cuda.synchronize()
    graphs, results, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:                       # two graphs at once do not share scratch
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            results.append(ds.clip_grad_norm(tensors, 1.0, out=[torch.empty_like(t) for t in tensors]))
        graphs.append(graph)
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for norm, out in results:
        assert torch.equal(norm, want[0]) and all(torch.equal(a, b) for a, b in zip(out, want[1]))
    for s in (streams[1], streams[1].cuda_stream):
        norm = torch.zeros((), device="cuda")
        torch.cuda.synchronize()
        ds.grad_norm(tensors, norm=norm, stream=s)
        streams[1].synchronize()
        assert torch.equal(norm, want[0])


def test_scratch_belongs_to_the_calls_stream(ds, monkeypatch):
    """The call's own scratch is memory of the stream that it runs on, whichever is current."""
    side, made, empty = torch.cuda.Stream(), [], torch.empty
    t, norm = torch.ones(100, device="cuda"), torch.zeros((), device="cuda")
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (made.append(torch.cuda.current_stream().cuda_stream), empty(*a, **k))[1])
    for stream, want in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (None, torch.cuda.current_stream().cuda_stream)):
        made.clear()
        ds.grad_norm([t], norm=norm, stream=stream)
        torch.cuda.synchronize()
        assert made == [want] and norm.item() == 10


def test_large(ds):
    """Elements behind 2^32 bytes."""
    t = torch.zeros((1 << 31) + 5, dtype=BF16, device="cuda")
    t[-3:] = 2.0
    t[:2] = 1.0
    norm, out = ds.clip_grad_norm([t], 1.0)
    assert abs(norm.item() - math.sqrt(14)) < 1e-5
    assert abs(out[0][-1].item() - 2 / math.sqrt(14)) < 2e-3 and out[0][5:-3].count_nonzero().item() == 0


def test_refusals(ds):
    t = torch.ones(10, device="cuda")
    work = torch.empty(100, dtype=torch.uint8, device="cuda")
    bad = [(TypeError, lambda: ds.grad_norm([t.double()])), (ValueError, lambda: ds.grad_norm([t[::2]])),
           (ValueError, lambda: ds.grad_norm([t.cpu()])), (ValueError, lambda: ds.clip_grad_norm([t], -1.0)),
           (ValueError, lambda: ds.clip_grad_norm([t], float("nan"))), (ValueError, lambda: ds.clip_grad_norm([t], 1.0, out=[])),
           (ValueError, lambda: ds.clip_grad_norm([t], 1.0, out=[t[:9]])),
           (ValueError, lambda: ds.clip_grad_norm([t], 1.0, out=[t.half()])),
           (ValueError, lambda: ds.grad_norm([t], work=work)), (TypeError, lambda: ds.grad_norm([t], norm=t[:1].half())),
           (ds.DevscanError, lambda: ds.grad_norm([t], norm=t[3:4])), (ValueError, lambda: ds.clip_grad_norm([t, t], 1.0)),
           (ds.DevscanError, lambda: ds.clip_grad_norm([t[:9]], 1.0, out=[t[1:]]))]
    for error, call in bad:
        with pytest.raises(error):
            call()
    assert (t == 1).all()
