"""The calls as a model uses them, together: a training step of a recurrent
layer and an expert layer behind each other, with all gradients and their
clipping, against the same step in 64 bits; and the serving of the same layers,
prompts in parts and token by token, against one call over whole sequences."""
import numpy as np
import pytest
import torch

import model_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def experts_forward(x, w1, starts, counts):
    """Each expert's rows times its matrix."""
    out = torch.zeros_like(x)
    for e in range(len(counts)):
        a, n = int(starts[e]), int(counts[e])
        out[a:a + n] = x[a:a + n] @ w1[e]
    return out


def plain_step(x, gate, starts, w, router, choices, target):
    """The step with autograd in 64 bits."""
    leaves = {k: v.double().requires_grad_() for k, v in (("x", x), ("gate", gate), ("w", w), ("router", router))}
    a = torch.sigmoid(leaves["gate"])
    b = torch.sigmoid(-leaves["gate"]) * leaves["x"]
    h = []
    for t0, t1 in zip(starts[:-1], starts[1:]):
        v = torch.zeros_like(b[0])
        for t in range(t0, t1):
            v = b[t] if t == t0 else a[t] * v + b[t]
            h.append(v)
    h = torch.stack(h)
    top, ids = (h @ leaves["router"]).topk(choices, dim=1)
    weights = torch.softmax(top, 1)
    y = torch.stack([sum(weights[t, k] * (h[t] @ leaves["w"][ids[t, k]]) for k in range(choices)) for t in range(len(h))])
    loss = ((y - target.double()) ** 2).sum()
    loss.backward()
    return loss.detach(), ids, {k: v.grad for k, v in leaves.items()}


def test_training_step(ds):
    """The library's step in fp32 against autograd in 64 bits.  Tolerance: the
    longest path goes through three products of 24 terms, sums of 90 tokens and
    decays below 0.9: fewer than 400 roundings of 2^-24 on the largest values of
    each gradient, and as many again from torch's products."""
    g = torch.Generator().manual_seed(5)
    tokens, width, experts, choices, starts = 90, 24, 6, 2, [0, 40, 41, 90]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, gate, w, router, target = r(tokens, width), r(tokens, width), r(experts, width, width) / 5, r(width, experts), r(tokens, width)
    loss, ids, want = plain_step(x, gate, starts, w, router, choices, target)
    x, gate, w, router, target = (v.cuda() for v in (x, gate, w, router, target))
    where = torch.tensor(starts, dtype=torch.int32, device="cuda")

    h, _ = ds.gated_scan(x, gate, starts=where, kind="sigmoid")
    top, chosen = (h @ router).topk(choices, dim=1)
    assert torch.equal(chosen.cpu(), ids)                     # no two logits are near each other
    weights = torch.softmax(top, 1)
    first, counts, order, places = ds.expert_sort(chosen, experts, align=4)
    xs = ds.expert_dispatch(h, places, order)
    ys = experts_forward(xs, w, first, counts)
    y = ds.expert_combine(ys, places, weights)
    dy = 2 * (y - target)
    assert abs(((y - target) ** 2).sum().item() - loss.item()) < 400 * 2 ** -24 * loss.item()

    dys, dweights = ds.expert_combine_backward(dy, ys, places, weights, order)
    dw, dxs = torch.zeros_like(w), torch.zeros_like(xs)
    for e in range(experts):
        a, n = int(first[e]), int(counts[e])
        dw[e] = xs[a:a + n].t() @ dys[a:a + n]
        dxs[a:a + n] = dys[a:a + n] @ w[e].t()
    dh = ds.expert_combine(dxs, places)                       # the gradient of dispatch
    dtop = weights * (dweights - (dweights * weights).sum(1, keepdim=True))
    dlogits = torch.zeros(tokens, experts, device="cuda").scatter_(1, chosen, dtop)
    drouter = h.t() @ dlogits
    dh = dh + dlogits @ router.t()
    dx, dgate, _ = ds.gated_scan_backward(dh, x, gate, h, starts=where, kind="sigmoid")
    got = {"x": dx, "gate": dgate, "w": dw, "router": drouter}
    for k, v in got.items():
        error = (v.cpu().double() - want[k]).abs().max().item()
        assert error <= 800 * 2 ** -24 * want[k].abs().max().item() * 10, (k, error)

    grads = list(got.values())
    norm = sum(float((v ** 2).sum()) for v in want.values()) ** 0.5
    keep = [v.clone() for v in grads]
    told, clipped = ds.clip_grad_norm(grads, 1.0)
    assert abs(told.item() - norm) < 1e-4 * norm and clipped[0] is grads[0]
    for v, k in zip(grads, keep):
        assert torch.allclose(v, k / (told + 1e-6), rtol=4 * 2 ** -24, atol=0)
    assert abs(ds.grad_norm(grads).item() - 1) < 1e-5


@pytest.mark.parametrize("dtype,kind", [(F32, "log"), (BF16, "sigmoid")])
def test_serving_in_parts(ds, dtype, kind):
    """Prompts that come in parts, packed by slot_map beside single tokens, and
    the last tokens one by one leave the states and outputs of one call."""
    rng = np.random.default_rng(7)
    rows, channels, lengths = 5, 48, [37, 1, 80, 12, 64]
    x = [torch.from_numpy(rng.standard_normal((n, channels))).to(dtype).cuda() for n in lengths]
    gate = [-torch.rand(n, channels, device="cuda").to(dtype) if kind == "log" else
            torch.randn(n, channels, device="cuda").to(dtype) for n in lengths]
    states = torch.full((9, channels), 5.0, device="cuda")     # a pool: what it holds at first is cleared below
    slots = torch.tensor([3, 8, 0, 5, 1], dtype=torch.int32, device="cuda")
    states[slots.long()] = 0
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros(rows, 8, dtype=torch.int32, device="cuda")
    done, got, budget = [0] * rows, [[] for _ in range(rows)], 60
    while any(d < n for d, n in zip(done, lengths)):
        room, fresh = budget, []
        for d, n in zip(done, lengths):
            fresh.append(min(n - d, room, 25 if n - d > 6 else 1))
            room -= fresh[-1]
        starts = ds.slot_map(table, i32(done), i32(fresh), 16, budget)[0]
        packed = lambda v: torch.cat([v[r][done[r]:done[r] + f] for r, f in enumerate(fresh)] +  # noqa: E731
                                     [torch.full((room, channels), float("nan"), dtype=dtype, device="cuda")])
        if sum(fresh) == rows and max(fresh) == 1:            # a decode step
            out, _ = ds.gated_scan(torch.stack([v[d] for v, d in zip(x, done)])[:, None],
                                   torch.stack([v[d] for v, d in zip(gate, done)])[:, None], initial=states, slots=slots, kind=kind)
            out = out[:, 0]
        else:
            out, _ = ds.gated_scan(packed(x), packed(gate), starts=starts, initial=states, slots=slots, kind=kind)
            assert not out[budget - room:].any()
        at = 0
        for r, f in enumerate(fresh):
            got[r].append(out[at:at + f])
            at, done[r] = at + f, done[r] + f
    for r in range(rows):
        # a first state of zeros and none are the same
        h, h_room, last, last_room = ref.scan(ref.as64(x[r]), ref.as64(gate[r]), kind, [(0, lengths[r])], np.zeros((1, channels)))
        ref.close(torch.cat(got[r]), h, h_room, f"row {r}")
        ref.close(states[slots[r].long()], last[0], last_room[0], f"state {r}")
    assert (states[[2, 4, 6, 7]] == 5).all()


def test_captured_step_beside_eager_calls(ds):
    """A whole step in a graph, replayed on new inputs while eager calls run."""
    g = torch.Generator(device="cuda").manual_seed(9)
    tokens, width, experts = 600, 128, 16
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    x, gate, grad = r(tokens, width), r(tokens, width), r(tokens, width)
    ids = torch.randint(0, experts, (tokens, 2), generator=g, device="cuda")
    weights = torch.rand(tokens, 2, generator=g, device="cuda")

    def step():
        h, _ = ds.gated_scan(x, gate, kind="sigmoid")
        _, _, order, places = ds.expert_sort(ids, experts, align=8)
        ys = ds.expert_dispatch(h, places, order, out=torch.zeros(order.numel(), width, dtype=BF16, device="cuda"))
        y = ds.expert_combine(ys, places, weights)
        dys, dweights = ds.expert_combine_backward(grad, ys, places, weights, order, grad_y=torch.zeros_like(ys))
        dh = ds.expert_combine(dys, places)
        dx, dgate, _ = ds.gated_scan_backward(dh, x, gate, h, kind="sigmoid")
        norm, clipped = ds.clip_grad_norm([dx, dgate, dweights], 1.0, out=[torch.empty_like(v) for v in (dx, dgate, dweights)])
        return [y, norm, *clipped]

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    for _ in range(4):
        for v in (x, gate, grad):
            v.copy_(r(tokens, width))
        ids.copy_(torch.randint(0, experts, (tokens, 2), generator=g, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))


def test_threads(ds):
    """Calls from several threads on one stream and on streams of their own."""
    import threading
    g = torch.Generator(device="cuda").manual_seed(3)
    x, gate = torch.randn(2, 700, 64, generator=g, device="cuda"), torch.randn(2, 700, 64, generator=g, device="cuda")
    ids = torch.randint(0, 8, (900, 3), generator=g, device="cuda")
    want = [ds.gated_scan(x, gate, kind="sigmoid")[0], *ds.expert_sort(ids, 8), ds.grad_norm([x, gate])]
    torch.cuda.synchronize()
    wrong = []

    def work(stream):
        with torch.cuda.stream(stream):
            for _ in range(30):
                got = [ds.gated_scan(x, gate, kind="sigmoid")[0], *ds.expert_sort(ids, 8), ds.grad_norm([x, gate])]
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    wrong.append(stream)

    shared = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(s,)) for s in (shared, shared, torch.cuda.Stream(), torch.cuda.Stream())]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_example_gradients(ds):
    """The example's autograd functions against autograd through plain formulas
    in 64 bits (rooms as in test_training_step), and that it runs."""
    import importlib.util
    import os

    from conftest import ROOT
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    g = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, gate, grad = r(30, 12), r(30, 12), r(30, 12)
    starts = torch.tensor([0, 11, 30], dtype=torch.int32, device="cuda")
    leaves = [x.requires_grad_(), gate.requires_grad_()]
    got = torch.autograd.grad((m.Recurrence.apply(*leaves, starts) * grad).sum(), leaves)
    wide = [v.detach().double().requires_grad_() for v in leaves]
    a, b, h = torch.sigmoid(wide[1]), torch.sigmoid(-wide[1]) * wide[0], []
    for t in range(30):
        h.append(b[t] if t in (0, 11) else a[t] * h[-1] + b[t])
    want = torch.autograd.grad((torch.stack(h) * grad.double()).sum(), wide)
    for u, v in zip(got, want):
        assert (u.double() - v).abs().max() <= 400 * 2 ** -24 * v.abs().max()

    ids = torch.randint(0, 4, (30, 2), generator=g, device="cuda")
    _, _, order, places = ds.expert_sort(ids, 4, align=4)
    weights = torch.rand(30, 2, generator=g, device="cuda").requires_grad_()
    leaves = [x, weights]
    scale = r(order.numel(), 1)
    y = m.Combine.apply(m.Dispatch.apply(x, places, order) * scale, weights, places, order)
    got = torch.autograd.grad((y * grad).sum(), leaves)
    wide = [v.detach().double().requires_grad_() for v in leaves]
    at = places.long()
    plain = (wide[1][..., None] * wide[0][:, None] * scale.double()[at]).sum(1)
    want = torch.autograd.grad((plain * grad.double()).sum(), wide)
    for u, v in zip(got, want):
        assert (u.double() - v).abs().max() <= 400 * 2 ** -24 * v.abs().max()
    losses = m.train(3)
    assert all(np.isfinite(losses))
