"""Tokens sorted by expert, and back, on the GPU against loops in 64 bits."""
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


def ids_of(rng, tokens, choices, experts, stray=0.05, dtype=np.int32):
    p = rng.dirichlet(np.full(experts, 0.5))
    ids = rng.choice(experts, (tokens, choices), p=p)
    return np.where(rng.random(ids.shape) < stray, rng.choice([-1, experts, -2**31, 2**31 - 1], ids.shape), ids).astype(dtype)


def check_sort(ds, ids, experts, align, rows=None):
    got = ds.expert_sort(torch.from_numpy(ids).cuda(), experts, align=align, rows=rows)
    m = got[2].numel()
    starts, counts, order, places = ref.sort(ids, experts, align, m)
    for name, g, w in zip(("starts", "counts", "order", "places"), got, (starts, counts, order, places)):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy().reshape(-1), w), name
    assert got[3].shape == ids.shape
    return got


@pytest.mark.parametrize("tokens,choices,experts", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (16, 8, 64), (33, 1, 2),
                                                    (100, 3, 1024), (511, 2, 7), (1025, 4, 40), (2050, 2, 129),
                                                    (4099, 4, 256), (9001, 6, 33), (20011, 2, 1)])
@pytest.mark.parametrize("align", [1, 16, 100])
def test_sort(ds, tokens, choices, experts, align):
    rng = np.random.default_rng(tokens)
    check_sort(ds, ids_of(rng, tokens, choices, experts), experts, align)


def test_sort_of_wide_ids_and_few_rows(ds):
    rng = np.random.default_rng(1)
    ids = ids_of(rng, 700, 3, 20, dtype=np.int64)
    ids[0, 0], ids[5, 1] = 2**40 + 3, -2**40      # whose low words look valid
    check_sort(ds, ids, 20, 8)
    for rows in (0, 1, 37, 1000, 5000):           # fewer rows than pairs, and more
        check_sort(ds, ids, 20, 8, rows)


def test_sort_without_tokens_or_matches(ds):
    starts, counts, order, places = ds.expert_sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4, rows=6)
    assert not starts.any() and not counts.any() and (order == -2).all() and places.shape == (0, 2)
    check_sort(ds, np.full((50, 2), -1, np.int32), 4, 16, 10)
    check_sort(ds, np.full((5000, 2), 3, np.int32), 4, 16)      # all to one


@pytest.mark.parametrize("dtype", [F32, F16, BF16, torch.uint8, torch.float64])
@pytest.mark.parametrize("width", [1, 7, 64, 100, 1000, 2056])
def test_dispatch(ds, dtype, width):
    rng = np.random.default_rng(width)
    tokens, choices, experts, align = 70, 3, 9, 16
    ids = ids_of(rng, tokens, choices, experts, 0.1)
    ids[-2:] = -1                                  # a padded batch
    _, _, order, places = ds.expert_sort(torch.from_numpy(ids).cuda(), experts, align=align)
    x = (torch.rand(tokens, width, device="cuda") * 200 + 1).to(dtype)
    x[-2:] = 0
    out = torch.full((order.numel(), width), 77, dtype=dtype, device="cuda")
    got = ds.expert_dispatch(x, places, order, out=out)
    assert got is out
    o = order.cpu().numpy()
    want = torch.full_like(out, 77)
    for r, pair in enumerate(o):
        want[r] = x[pair // choices] if pair >= 0 else 0 if pair == -1 else 77
    assert torch.equal(out, want)
    wide = torch.full((order.numel(), width + 5), 77, dtype=dtype, device="cuda")     # strided rows
    ds.expert_dispatch(torch.cat([x, x], 1)[:, width:], places, order, out=wide[:, 3:3 + width])
    assert torch.equal(wide[:, 3:3 + width], want) and (wide[:, :3] == 77).all() and (wide[:, 3 + width:] == 77).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("tokens,choices,width", [(1, 1, 8), (5, 8, 64), (70, 3, 100), (33, 9, 2048), (8, 20, 515),
                                                  (300, 2, 1), (64, 4, 4096), (2, 33, 72)])
def test_combine_and_gradient(ds, dtype, tokens, choices, width):
    rng = np.random.default_rng(tokens + width)
    experts = 7
    ids = ids_of(rng, tokens, choices, experts, 0.15)
    ids[tokens // 2] = -1                          # a token without any expert
    _, _, order, places = ds.expert_sort(torch.from_numpy(ids).cuda(), experts, align=8)
    y = torch.randn(order.numel(), width, device="cuda").to(dtype)
    y[order < 0] = float("nan")                    # rows of no pair are not looked at
    w = torch.randn(tokens, choices, device="cuda")
    grad = torch.randn(tokens, width, device="cuda").to(dtype)
    p = places.cpu().numpy()
    for weights in (w, None):
        w64 = ref.as64(weights)
        want, room = ref.combine(ref.as64(y), p, w64)
        out = ds.expert_combine(y, places, weights)
        ref.close(out, want, room, "out")
        assert not out[tokens // 2].any()
        keep = torch.full_like(y, 5)
        gy, gw = ds.expert_combine_backward(grad, y, places, weights, order, grad_y=keep,
                                            grad_weights=torch.full_like(w, 3))
        base = np.where((order.cpu().numpy() == -1)[:, None], 0.0, np.full(y.shape, 5.0))
        wy, ww, wroom = ref.combine_backward(ref.as64(grad), ref.as64(y), p, w64, base)
        ref.close(gy, wy, ref.U * np.abs(wy), "grad_y")
        ref.close(gw, ww, wroom, "grad_weights")
        assert not gw[tokens // 2].any()
    gy, gw = ds.expert_combine_backward(grad, y, places, None, order, grad_y=torch.full_like(y, 5))
    assert gw is None
    ref.close(gy, wy, 0 * wy, "grad_y alone")
    # the gradient of dispatch is combine
    x = torch.randn(tokens, width, device="cuda").to(dtype)
    gx = ds.expert_combine(gy, places)
    assert gx.shape == x.shape


def test_strided_rows(ds):
    rng = np.random.default_rng(3)
    ids = ids_of(rng, 40, 2, 5)
    _, _, order, places = ds.expert_sort(torch.from_numpy(ids).cuda(), 5)
    y, w = torch.randn(order.numel(), 64, device="cuda"), torch.rand(40, 2, device="cuda")
    y[order < 0] = 0
    wide = torch.randn(order.numel(), 200, device="cuda")
    wide[:, 33:97] = y
    out = torch.zeros(40, 130, device="cuda")
    want = ds.expert_combine(y, places, w)
    assert torch.equal(ds.expert_combine(wide[:, 33:97], places, w, out=out[:, 1:65]), want) and not out[:, 65:].any()
    grad = torch.randn(40, 64, device="cuda")
    a = ds.expert_combine_backward(grad, y, places, w, order, grad_y=torch.zeros_like(y))
    b = ds.expert_combine_backward(grad, wide[:, 33:97], places, w, order, grad_y=torch.zeros_like(wide)[:, 33:97])
    assert torch.equal(a[0], b[0])
    size = np.abs(ref.as64(grad))[:, None] * np.abs(ref.as64(y)[places.clamp(min=0).cpu().numpy()])
    assert ((a[1] - b[1]).abs().cpu().numpy() <= 2 * (64 / 128 + 24) * ref.U * size.sum(-1)).all()


def test_bad_places_touch_nothing(ds):
    """Places outside the rows count as none, whatever they are."""
    x = torch.randn(4, 32, device="cuda")
    places = torch.tensor([[0, 5], [-7, 2**31 - 1], [-2**31, 6], [4, 3]], dtype=torch.int32, device="cuda")
    order = torch.full((5,), -2, dtype=torch.int32, device="cuda")
    big = torch.full((9, 32), 7.0, device="cuda")
    ds.expert_dispatch(x, places, order, out=big[2:7])
    want = torch.full((9, 32), 7.0, device="cuda")
    want[2], want[6], want[5] = x[0], x[3], x[3]
    assert torch.equal(big, want)
    got = ds.expert_combine(big[2:7], places)
    assert torch.equal(got, torch.stack([x[0], x[0] * 0, x[0] * 0, x[3] + x[3]]))
    gy, gw = ds.expert_combine_backward(x, big[2:7], places, torch.ones(4, 2, device="cuda"), order, grad_y=big[2:7] * 0 + 7)
    assert torch.equal(gy, want[2:7]) and not gw[1:3].any() and gw[0, 1] == 0


def test_large(ds):
    """More pairs than one block sorts, rows behind 2^32 bytes; against sorted and gathered rows."""
    g = torch.Generator(device="cuda").manual_seed(2)
    tokens, choices, experts, width = 150000, 8, 300, 2048
    ids = torch.randint(-1, experts, (tokens, choices), generator=g, device="cuda")
    starts, counts, order, places = ds.expert_sort(ids, experts, align=4)
    key = torch.where(ids.reshape(-1) < 0, experts, ids.reshape(-1))
    by = torch.argsort(key, stable=True)
    n = torch.bincount(key, minlength=experts + 1)[:experts]
    assert torch.equal(counts.long(), n)
    assert torch.equal(starts.long(), torch.cat([n[:1] * 0, ((n + 3) // 4 * 4).cumsum(0)]))
    live = order[order >= 0].long()
    assert torch.equal(live, by[: live.numel()])
    assert torch.equal(order[places.reshape(-1)[live].long()].long(), live)
    assert ((places < 0) == (ids < 0)).all()
    x = torch.randn(tokens, width, generator=g, device="cuda").to(BF16)
    xs = ds.expert_dispatch(x, places, order)
    for r0 in range(0, order.numel(), 100000):
        o = order[r0:r0 + 100000].long()
        rows = xs[r0:r0 + 100000]
        assert torch.equal(rows[o >= 0], x[o[o >= 0] // choices]) and not rows[o == -1].any()
    back = ds.expert_combine(xs, places)
    assert torch.equal(back, (x.float() * (places >= 0).sum(1, keepdim=True)).to(BF16))    # sums of equal rows are exact


def test_same_bits_streams_and_graphs(ds):
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, 64, (3000, 4), generator=g, device="cuda")
    x, w = torch.randn(3000, 256, generator=g, device="cuda").to(BF16), torch.rand(3000, 4, generator=g, device="cuda")

    def run():
        starts, counts, order, places = ds.expert_sort(ids, 64, align=8)
        xs = ds.expert_dispatch(x, places, order, out=torch.zeros(order.numel(), 256, dtype=BF16, device="cuda"))
        out = ds.expert_combine(xs, places, w)
        return (starts, counts, order, places, xs, out,
                *ds.expert_combine_backward(out, xs, places, w, order, grad_y=torch.zeros_like(xs)))

    want = run()
    torch.cuda.synchronize()
    graphs, results, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            results.append(run())
        graphs.append(graph)
    for _ in range(3):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for got in results:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(ds):
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    starts, counts, order, places = ds.expert_sort(ids, 3)
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(4, 2, device="cuda")
    y = ds.expert_dispatch(x, places, order)
    bad = [(TypeError, lambda: ds.expert_sort(ids.float(), 3)), (ValueError, lambda: ds.expert_sort(ids, 0)),
           (ds.DevscanError, lambda: ds.expert_sort(ids, 1025)), (ValueError, lambda: ds.expert_sort(ids, 3, align=0)),
           (ValueError, lambda: ds.expert_sort(ids[:, 0], 3)), (ValueError, lambda: ds.expert_sort(ids, 3, rows=-1)),
           (ValueError, lambda: ds.expert_sort(ids, 3, rows=4, order=order)),
           (ds.DevscanError, lambda: ds.expert_sort(ids, 3, places=ids)),
           (ds.DevscanError, lambda: ds.expert_sort(ids, 3, align=2**31 - 1, rows=8)),
           (ValueError, lambda: ds.expert_dispatch(x[:3], places, order)),
           (ValueError, lambda: ds.expert_dispatch(x, places.long(), order)),
           (TypeError, lambda: ds.expert_dispatch(x, places, order.long())),
           (ds.DevscanError, lambda: ds.expert_dispatch(y[:4], places, order, out=y)),
           (TypeError, lambda: ds.expert_combine(y.double(), places)),
           (TypeError, lambda: ds.expert_combine(y, places, w.half())),
           (ValueError, lambda: ds.expert_combine(y, places, w[:3])),
           (TypeError, lambda: ds.expert_combine(y, places, out=x.half())),
           (ValueError, lambda: ds.expert_combine(y.t(), places)),
           (ValueError, lambda: ds.expert_combine_backward(x[:, :7], y, places, w, order)),
           (ds.DevscanError, lambda: ds.expert_combine_backward(x, y, places, w, order, grad_y=y)),
           (ValueError, lambda: ds.expert_combine(y.cpu(), places))]
    for error, call in bad:
        with pytest.raises(error):
            call()
