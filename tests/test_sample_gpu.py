"""The token draw against its definition in 64 bits: types, sizes from one
token up, every truncation alone and together, ties, masked and non-finite
logits, strides and offsets, streams, and the arguments it refuses."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def peaked(rows, vocab, seed):
    """Logits with a bell-shaped bulk and some tokens far above it."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, vocab)) * 2.0
    for r in range(rows):
        at = rng.integers(0, vocab, min(24, vocab))
        x[r, at] += rng.exponential(1.0, at.size) * 3.0 * (r % 4)
    q = rng.exponential(1.0, (rows, vocab)).astype(np.float32) + np.float32(1e-30)
    return torch.from_numpy(x.astype(np.float32)), torch.from_numpy(q)


def check(x, noise, tokens, logprobs, asks):
    """x, noise: host tensors as the kernel saw them."""
    tokens, logprobs = tokens.cpu().numpy(), logprobs.cpu().numpy().astype(np.float64)
    x = x.float().cpu().numpy()
    for r, (t, k, p, m) in enumerate(asks):
        t, p, m = (float(np.float32(v)) for v in (t, p, m))
        q = None if noise is None else noise[r].cpu().numpy()
        good, logprob = ref.draw(x[r], q, t, k, p, m)
        assert int(tokens[r]) in good, (r, (t, k, p, m), int(tokens[r]), good)
        value, room = logprob(int(tokens[r]))
        if math.isinf(value):
            assert logprobs[r] == value, (r, logprobs[r], value)
        else:
            assert abs(logprobs[r] - value) <= room, (r, (t, k, p, m), logprobs[r], value, room)


def asked(asks):
    t, k, p, m = zip(*asks)
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    return {"temperature": f(t), "top_k": torch.tensor(k, dtype=torch.int32, device="cuda"), "top_p": f(p),
            "min_p": f(m)}


def run(ds, x, noise, asks, dtype=torch.float32):
    x = x.to(dtype)
    tokens, logprobs = ds.sample_tokens(x.cuda(), None if noise is None else noise.cuda(), **asked(asks))
    check(x, noise, tokens, logprobs, asks)
    return tokens


ASKS = [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.8, 5, 1.0, 0.0), (0.8, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.1),
        (0.7, 40, 0.95, 0.02), (1.3, 1, 1.0, 0.0), (1.0, 300, 0.5, 0.0), (2.0, 0, 0.999, 0.0), (0.9, 2000, 0.99, 0.0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 257, 1000, 4097, 8192, 32771, 65536])
def test_sizes_and_settings(ds, dtype, vocab):
    x, q = peaked(len(ASKS), vocab, vocab)
    run(ds, x, q, ASKS, DTYPES[dtype])


@pytest.mark.parametrize("dtype", DTYPES)
def test_largest_vocabulary(ds, dtype):
    vocab = 1 << 18
    asks = [ASKS[1], ASKS[3], ASKS[5], ASKS[9], (1.0, 5000, 0.9, 0.0)]
    x, q = peaked(len(asks), vocab, 5)
    run(ds, x, q, asks, DTYPES[dtype])


@pytest.mark.parametrize("rows", [1, 7, 40, 153, 400])
def test_many_rows(ds, rows):
    asks = [ASKS[r % len(ASKS)] for r in range(rows)]
    x, q = peaked(rows, 5000, rows)
    run(ds, x, q, asks, torch.bfloat16)


@pytest.mark.parametrize("vocab", [9, 1500, 40000])
@pytest.mark.parametrize("ask", [(1.0, 7, 1.0, 0.0), (1.0, 1200, 1.0, 0.0), (1.0, 0, 0.3, 0.0), (1.0, 0, 0.9, 0.0),
                                 (1.0, 0, 1.0, 1.0), (1.0, 6, 0.5, 0.0), (1.0, 0, 1.0, 0.0)])
def test_ties_go_to_the_lowest_index(ds, vocab, ask):
    """All logits equal, two values, and four: the kept set ends inside a tie."""
    rng = np.random.default_rng(3)
    x = torch.stack([torch.zeros(vocab), torch.from_numpy(rng.integers(0, 2, vocab).astype(np.float32)),
                     torch.from_numpy(rng.integers(-2, 2, vocab).astype(np.float32)) * 0.5])
    x[2][x[2] == 0] = -0.0 * torch.ones(())     # zeros of both signs tie
    x[2][::3][x[2][::3] == 0] = 0.0
    q = torch.from_numpy(rng.exponential(1.0, (3, vocab)).astype(np.float32) + np.float32(1e-30))
    run(ds, x, q, [ask] * 3)


def test_equal_scores_take_the_lowest_index(ds):
    x, q = torch.zeros(2, 3000), torch.ones(2, 3000)
    tokens, logprobs = ds.sample_tokens(x.cuda(), q.cuda(), **asked([(1.0, 0, 1.0, 0.0), (1.0, 50, 1.0, 0.0)]))
    assert tokens.tolist() == [0, 0]
    assert abs(logprobs[0].item() + math.log(3000)) < 1e-4 and abs(logprobs[1].item() + math.log(50)) < 1e-5
    tokens, logprobs = ds.sample_tokens(x.cuda(), None)
    assert tokens.tolist() == [0, 0] and logprobs.tolist() == [0.0, 0.0]


@pytest.mark.parametrize("vocab", [5, 1030, 20000])
def test_masked_and_non_finite_logits(ds, vocab):
    x, q = peaked(10, vocab, 11)
    low = torch.finfo(torch.float32).min
    x[0] = -INF                                   # nothing left
    x[1] = math.nan
    x[2] = -INF
    x[2, vocab // 2] = -3.5                       # one token left
    x[3, ::2] = -INF
    x[4, ::2] = low                               # masked by the type's lowest value
    x[5] = low
    x[6, 1::2] = math.nan
    x[7, vocab // 3] = INF
    x[7, vocab - 1] = INF
    x[8, 0] = torch.finfo(torch.float32).max
    x[8, 1] = low
    x[9, : vocab - 1] = -INF
    x[9, vocab - 1] = low
    for ask in [(1.0, 0, 1.0, 0.0), (0.7, 3, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.3), (0.9, 4, 0.8, 0.1),
                (0.0, 0, 1.0, 0.0), (1.0, 1100, 0.9, 0.0)]:
        run(ds, x, q, [ask] * 10)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_lowest_value_masks_in_sixteen_bits(ds, dtype):
    x, q = peaked(4, 6000, 12)
    x = x.to(DTYPES[dtype])
    x[0, ::2] = torch.finfo(x.dtype).min
    x[1, 100:] = -INF
    x[2] = torch.finfo(x.dtype).min
    x[3, 5] = INF
    for ask in [(1.0, 0, 1.0, 0.0), (0.8, 30, 0.9, 0.0), (1.0, 0, 0.95, 0.0), (1.0, 3500, 1.0, 0.0)]:
        run(ds, x, q, [ask] * 4, x.dtype)


def test_extreme_settings(ds):
    asks = [(1e-6, 0, 1.0, 0.0), (1e6, 0, 1.0, 0.0), (INF, 0, 1.0, 0.0), (math.nan, 0, 1.0, 0.0), (-1.0, 0, 1.0, 0.0),
            (1.0, -3, 1.0, 0.0), (1.0, 10**9, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, -1.0, 0.0), (1.0, 0, 1e-7, 0.0),
            (1.0, 0, 1.0, 1.0), (1.0, 0, 1.0, 5.0), (1.0, 3999, 1.0, 0.0), (1.0, 4000, 1.0, 0.0), (1.0, 0, 2.0, -1.0),
            (50.0, 0, 0.5, 0.0), (50.0, 2500, 0.5, 0.0), (INF, 100, 0.5, 0.0)]
    x, q = peaked(len(asks), 4000, 13)
    run(ds, x, q, asks)


def test_settings_left_out(ds):
    x, q = peaked(6, 3001, 14)
    xd, qd = x.cuda(), q.cuda()
    for only, at in (("temperature", 0), ("top_k", 1), ("top_p", 2), ("min_p", 3)):
        ask = [1.0, 0, 1.0, 0.0]
        ask[at] = (0.5, 9, 0.8, 0.2)[at]
        kw = {only: asked([tuple(ask)] * 6)[only]}
        tokens, logprobs = ds.sample_tokens(xd, qd, **kw)
        check(x, q, tokens, logprobs, [tuple(ask)] * 6)
    tokens, logprobs = ds.sample_tokens(xd, None, **asked([(0.7, 0, 0.9, 0.0)] * 6))
    check(x, None, tokens, logprobs, [(0.7, 0, 0.9, 0.0)] * 6)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (3, 5), (8, 8), (5, 1)])
def test_strides_and_offsets(ds, dtype, offset, pad):
    rows, vocab = 5, 4099
    x, q = peaked(rows, vocab, 15)
    x = x.to(DTYPES[dtype])
    wide = torch.full((rows * (vocab + pad) + offset + 16,), 99.0, dtype=x.dtype, device="cuda")   # larger than any logit
    noisy = torch.full((rows * (vocab + pad) + offset + 16,), 1e-30, device="cuda")
    view = lambda t: t[offset: offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]  # noqa: E731
    view(wide).copy_(x)
    view(noisy).copy_(q)
    for ask in ASKS[1:7]:
        tokens, logprobs = ds.sample_tokens(view(wide), view(noisy), **asked([ask] * rows))
        check(x, q, tokens, logprobs, [ask] * rows)


def test_other_stream_and_given_outputs(ds):
    x, q = peaked(9, 20000, 16)
    asks = [ASKS[r % len(ASKS)] for r in range(9)]
    kw = asked(asks)
    xd, qd = x.cuda(), q.cuda()
    out = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    logprobs = torch.zeros(9, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ds.sample_tokens(xd, qd, **kw, out=out, logprobs=logprobs, stream=s)
    s.synchronize()
    assert got[0] is out and got[1] is logprobs
    check(x, q, out, logprobs, asks)
    ds.stream_release(s)


def test_repeats_are_equal_bit_for_bit(ds):
    x, q = peaked(64, 30000, 17)
    asks = [ASKS[r % len(ASKS)] for r in range(64)]
    kw, xd, qd = asked(asks), x.cuda(), q.cuda()
    first = [t.clone() for t in ds.sample_tokens(xd, qd, **kw)]
    for _ in range(5):
        again = ds.sample_tokens(xd, qd, **kw)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_draws_follow_the_distribution(ds):
    """20,000 draws of one truncated row: every kept token's share is within
    five standard deviations, and nothing else is drawn."""
    rows = 20000
    rng = np.random.default_rng(18)
    row = torch.from_numpy((rng.standard_normal(200) * 2).astype(np.float32))
    x = row.expand(rows, 200).contiguous().cuda()
    q = torch.from_numpy(rng.exponential(1.0, (rows, 200)).astype(np.float32) + np.float32(1e-30)).cuda()
    kw = {k: v.expand(rows).contiguous() for k, v in asked([(0.9, 12, 0.9, 0.0)]).items()}
    tokens, _ = ds.sample_tokens(x, q, **kw)
    counts = np.bincount(tokens.cpu().numpy(), minlength=200)
    v = row.double().numpy()
    order = np.argsort(-v, kind="stable")[:12]
    w = np.exp((v[order] - v[order[0]]) / float(np.float32(0.9)))
    keep = np.concatenate([[0.0], np.cumsum(w)[:-1]]) < float(np.float32(0.9)) * w.sum()
    order, w = order[keep], w[keep] / w[keep].sum()
    assert counts.sum() == counts[order].sum() == rows
    assert np.all(np.abs(counts[order] - rows * w) <= 5 * np.sqrt(rows * w * (1 - w)) + 1)


def test_graph_replay(ds):
    x, q = peaked(12, 9000, 19)
    asks = [ASKS[r % len(ASKS)] for r in range(12)]
    kw, xd, qd = asked(asks), x.cuda(), q.cuda()
    out, logprobs = torch.empty(12, dtype=torch.int32, device="cuda"), torch.empty(12, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ds.sample_tokens(xd, qd, **kw, out=out, logprobs=logprobs)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ds.sample_tokens(xd, qd, **kw, out=out, logprobs=logprobs)
    x2, q2 = peaked(12, 9000, 20)
    xd.copy_(x2)
    qd.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    check(x2, q2, out, logprobs, asks)
    ds.stream_release(s)


def test_rows_left_to_a_second_launch(ds):
    """More rows than fit at once with their slices: flat rows whose cut needs
    histograms beside peaked ones and races of all tokens, again and again on
    one stream and in a graph."""
    rows, vocab = 330, 40000
    kinds = [(1.0, 0, 0.9, 0.0), (0.8, 50, 0.9, 0.0), (1.0, 0, 1.0, 0.0), (1.0, 3000, 0.95, 0.0), (0.0, 0, 1.0, 0.0),
             (1.0, 2000, 1.0, 0.001), (3.0, 0, 0.5, 0.0)]
    asks = [kinds[r % len(kinds)] for r in range(rows)]
    kw = asked(asks)
    for seed, dtype in ((21, torch.float32), (22, torch.bfloat16)):
        x, q = peaked(rows, vocab, seed)
        x = x.to(dtype)
        xd, qd = x.cuda(), q.cuda()
        first = [t.clone() for t in ds.sample_tokens(xd, qd, **kw)]
        check(x, q, *first, asks)
        for _ in range(4):
            assert all(torch.equal(a, b) for a, b in zip(first, ds.sample_tokens(xd, qd, **kw)))
        assert ds.device_status() == 0
        out, logprobs = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ds.sample_tokens(xd, qd, **kw, out=out, logprobs=logprobs)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(2):
                ds.sample_tokens(xd, qd, **kw, out=out, logprobs=logprobs)
        out.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(logprobs, first[1])
        assert ds.device_status(s) == 0
        ds.stream_release(s)


@pytest.mark.parametrize("rows", [2, 330])
def test_wide_cuts(ds, rows):
    """Cuts far down the order, in rows of ties and of masked tokens."""
    vocab = 36001
    rng = np.random.default_rng(23)
    x, q = peaked(rows, vocab, 24)
    x[0] = torch.from_numpy(rng.integers(-3, 3, vocab).astype(np.float32))
    x[1, rng.random(vocab) < 0.7] = -INF
    for ask in [(1.0, 20000, 1.0, 0.0), (1.0, 5000, 0.99, 0.0), (0.5, 0, 0.9999, 0.0), (1e-3, 0, 0.9, 0.0),
                (30.0, 0, 0.97, 0.0), (1.0, 9999, 0.3, 0.01), (1.0, 36000, 0.999, 0.0), (1e-30, 30000, 0.9, 0.0)]:
        tokens, logprobs = ds.sample_tokens(x.cuda(), q.cuda(), **asked([ask] * rows))
        check(x[:8], q[:8], tokens[:8], logprobs[:8], [ask] * min(rows, 8))


def test_refusals(ds):
    x, q = torch.zeros(4, 64, device="cuda"), torch.ones(4, 64, device="cuda")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        ds.sample_tokens(x.cpu(), q)
    with pytest.raises(ValueError):
        ds.sample_tokens(x[0], q[0])
    with pytest.raises(ValueError):
        ds.sample_tokens(x.t(), q.t())
    with pytest.raises(TypeError):
        ds.sample_tokens(x.double(), q)
    with pytest.raises(TypeError):
        ds.sample_tokens(x, q.half())
    with pytest.raises(ValueError):
        ds.sample_tokens(x, q[:, :32])
    with pytest.raises(ValueError):
        ds.sample_tokens(x, q, temperature=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError):
        ds.sample_tokens(x, q, top_k=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        ds.sample_tokens(x, q, out=i32(5))
    with pytest.raises(ValueError):
        ds.sample_tokens(x[:1].expand(4, 64), q)
    with pytest.raises(ds.DevscanError):
        ds.sample_tokens(x, q, out=x.view(torch.int32)[0, :4])            # output inside the input
    with pytest.raises(ds.DevscanError):
        ds.sample_tokens(torch.zeros(1, (1 << 18) + 1, device="cuda"))    # vocabulary over the limit
    tokens, logprobs = ds.sample_tokens(x[:0], q[:0])
    assert tokens.numel() == 0 and logprobs.numel() == 0
