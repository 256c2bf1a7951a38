"""The gated recurrence and its gradient on the GPU against loops over tokens
in 64 bits (tests/model_ref.py has their room): types, kinds, rows, packed
rows, states in pools, strides, and values that must stay where they are."""
import numpy as np
import pytest
import torch

import model_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [(F32, F32), (F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)]
KINDS = ["decay", "log", "sigmoid"]


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def gates(rng, shape, kind):
    slow = np.exp(rng.uniform(-7, 0, shape[-1]))
    token = rng.standard_normal(shape)
    if kind == "sigmoid":
        return token * 2 - np.log(slow)
    g = -slow / (1 + np.exp(-token)) * 3
    return g if kind == "log" else np.exp(g) * np.where(rng.random(shape) < 0.1, -1, 1)


def cuda(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def flat(t):
    return ref.as64(t.reshape(-1, t.shape[-1]))


def check(ds, rng, rows, tokens, channels, dtype=F32, gate_dtype=F32, kind="decay", starts=None, carry=False,
          backward=True):
    shape = (tokens, channels) if starts is not None else (rows, tokens, channels)
    x, gate = cuda(rng.standard_normal(shape), dtype), cuda(gates(rng, shape, kind), gate_dtype)
    initial = cuda(rng.standard_normal((rows, channels))) if carry else None
    where = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    spans = ref.rows_of(starts, tokens, rows)
    out, final = ds.gated_scan(x, gate, starts=where, initial=initial, kind=kind)
    h, room, last, last_room = ref.scan(flat(x), flat(gate), kind, spans, ref.as64(initial))
    assert out.dtype == dtype and out.shape == x.shape and final.shape == (rows, channels)
    ref.close(out.reshape(-1, channels), h, room, "out")
    ref.close(final, last, last_room, "final")
    if not backward:
        return
    grad = cuda(rng.standard_normal(shape), dtype)
    grad_final = cuda(rng.standard_normal((rows, channels))) if carry else None
    got = ds.gated_scan_backward(grad, x, gate, out, starts=where, initial=initial, grad_final=grad_final, kind=kind)
    want = ref.scan_backward(flat(grad), flat(x), flat(gate), flat(out), kind, spans, ref.as64(initial),
                             ref.as64(grad_final))
    assert got[0].dtype == dtype and got[1].dtype == gate_dtype
    ref.close(got[0].reshape(-1, channels), *want["x"], "grad_x")
    ref.close(got[1].reshape(-1, channels), *want["gate"], "grad_gate")
    assert (got[2] is None) == (initial is None)
    if carry:
        ref.close(got[2], *want["initial"], "grad_initial")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
def test_types_and_kinds(ds, dtype, gate_dtype, kind):
    rng = np.random.default_rng(1)
    check(ds, rng, 2, 150, 70, dtype, gate_dtype, kind, carry=True)      # pairs of channels
    check(ds, rng, 1, 67, 33, dtype, gate_dtype, kind)                   # single ones
    check(ds, rng, 5, 90, 64, dtype, gate_dtype, kind, starts=[0, 1, 1, 17, 80, 88], carry=True)


@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 511, 512, 513, 1025, 2100])
def test_lengths(ds, tokens):
    rng = np.random.default_rng(tokens)
    check(ds, rng, 1, tokens, 5, carry=True)                             # spread over a cluster's blocks
    check(ds, rng, 3, tokens, 66, BF16, BF16, "log")
    check(ds, rng, 1, tokens, 8, F16, F16, "sigmoid", starts=[0, tokens])


@pytest.mark.parametrize("channels", [1, 2, 31, 32, 33, 63, 64, 65, 128, 1000])
def test_channels(ds, channels):
    rng = np.random.default_rng(channels)
    check(ds, rng, 2, 140, channels, F32, F32, "sigmoid", carry=True)
    check(ds, rng, 2, 140, channels, BF16, F32, "log")


@pytest.mark.parametrize("rows,tokens,channels", [(400, 3, 40), (700, 1, 17), (64, 20, 300), (1, 5000, 130),
                                                  (9, 700, 2050)])
def test_shapes(ds, rows, tokens, channels):
    """Many short rows (several in a warp's tokens), few long ones, many channels."""
    rng = np.random.default_rng(rows)
    check(ds, rng, rows, tokens, channels, BF16, BF16, "log", carry=True)
    check(ds, rng, rows, tokens, channels, F32, F32, "sigmoid")


PACKED = [[0, 0], [0, 300], [0, 0, 0, 300], [0, 1, 2, 3, 4, 300], [0, 128, 256, 300], [0, 127, 129, 300],
          [0, 290], [5, 20, 20, 200, 295], [0, 100, 100, 100, 400, 500], [300, 300, 300], [299, 300, 300],
          [0, *range(1, 301)], [0, 16, 32, 48, 299, 300]]


@pytest.mark.parametrize("starts", PACKED, ids=lambda s: "-".join(map(str, s[:6])))
@pytest.mark.parametrize("carry", [False, True])
def test_packed_rows(ds, starts, carry):
    """Rows that begin anywhere, empty ones, tokens in front and behind, rows that go on past the tokens."""
    rng = np.random.default_rng(len(starts))
    check(ds, rng, len(starts) - 1, 300, 40, F32, F32, "decay", starts=starts, carry=carry)
    check(ds, rng, len(starts) - 1, 300, 64, BF16, BF16, "sigmoid", starts=starts, carry=carry)


def test_many_packed_rows(ds):
    """Spans of rows begin where rows do."""
    rng = np.random.default_rng(5)
    starts = np.concatenate([[0], np.sort(rng.integers(0, 6001, 99)), [6001]]).tolist()
    check(ds, rng, 100, 6050, 36, F32, F32, "log", starts=starts, carry=True)
    check(ds, rng, 100, 6050, 36, F16, F16, "log", starts=starts)
    one_long = [0, *range(1, 50), 5900, *range(5950, 6000)]
    check(ds, rng, len(one_long) - 1, 6000, 70, BF16, F32, "decay", starts=one_long, carry=True)


@pytest.mark.parametrize("dtype,channels", [(F32, 36), (BF16, 33), (BF16, 64)])
@pytest.mark.parametrize("real", [0, 50, 3000, 11999])
def test_padded_batches(ds, real, dtype, channels):
    """Tokens behind all rows get 0, whatever they hold and however many of them there are."""
    rng = np.random.default_rng(real)
    cuts = np.sort(rng.integers(0, real + 1, 59)).tolist()
    starts = [0, *cuts, real]
    check(ds, rng, 60, 12000, channels, dtype, dtype, "log", starts=starts, carry=True)
    nan = float("nan")
    x, gate = cuda(rng.standard_normal((12000, channels)), dtype), cuda(rng.standard_normal((12000, channels)), dtype)
    x[real:], gate[real:] = nan, nan
    where = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out, final = ds.gated_scan(x, gate, starts=where, kind="sigmoid", out=torch.full_like(x, nan))
    assert out.isfinite().all() and final.isfinite().all() and not out[real:].any()
    out[real:] = nan
    gx, gg, _ = ds.gated_scan_backward(x, x, gate, out, starts=where, kind="sigmoid", grad_x=torch.full_like(x, nan),
                                       grad_gate=torch.full_like(x, nan))
    assert gx.isfinite().all() and gg.isfinite().all() and not gx[real:].any() and not gg[real:].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
def test_few_tokens(ds, dtype, gate_dtype, kind):
    """Rows of a few tokens, whose threads go through them: one row and many, whole vectors and not."""
    rng = np.random.default_rng(17)
    for rows, tokens, channels in ((1, 2, 136), (3, 3, 24), (70, 5, 1000), (130, 8, 64), (130, 9, 1024), (9, 32, 1030), (40, 33, 256),
                                   (600, 4, 3)):
        check(ds, rng, rows, tokens, channels, dtype, gate_dtype, kind, carry=rows % 2 == 0, backward=False)


def test_few_tokens_in_place(ds):
    """Over x, from and into a pool; a first gate without a state does not count; other tokens stay."""
    rng = np.random.default_rng(18)
    x, gate = cuda(rng.standard_normal((6, 12, 200)), BF16), cuda(rng.standard_normal((6, 12, 200)), BF16)
    states, slots = cuda(rng.standard_normal((9, 200))), torch.tensor([3, -1, 8, 0, 9, 5], dtype=torch.int32, device="cuda")
    gate[[1, 4], 5] = float("nan")
    before, keep = states.clone(), x.clone()
    at = x[:, 5:11]
    out, final = ds.gated_scan(at, gate[:, 5:11], initial=states, slots=slots, kind="sigmoid", out=at)
    assert final is states and torch.equal(x[:, :5], keep[:, :5]) and torch.equal(x[:, 11:], keep[:, 11:])
    # without a state the first token's b = (1 - a) x has its own gate in it
    assert out[[1, 4], 0].isnan().all()
    rows, used = [0, 2, 3, 5], [3, 8, 0, 5]
    spans = ref.rows_of(None, 6, 4)
    h, room, last, last_room = ref.scan(flat(keep[rows, 5:11]), flat(gate[rows, 5:11]), "sigmoid", spans, ref.as64(before)[used])
    ref.close(out[rows].reshape(-1, 200), h, room, "out")
    ref.close(states[used], last, last_room, "states")
    assert torch.equal(states[[1, 2, 4, 6, 7]], before[[1, 2, 4, 6, 7]])
    gate[:, 5] = float("nan")
    free = ds.gated_scan(keep[:, 5:11], gate[:, 5:11], kind="decay")[0]
    assert torch.equal(free[:, 0], keep[:, 5]) and free.isfinite().all()


@pytest.mark.parametrize("at", [0, 30, 59])
@pytest.mark.parametrize("dtype,channels,kind", [(BF16, 640, "sigmoid"), (F32, 333, "decay"), (F16, 333, "log")])
def test_one_long_row(ds, dtype, channels, kind, at):
    """A row longer than all others, before, between and behind them; empty rows and a padded end beside it."""
    rng = np.random.default_rng(at)
    lengths = rng.integers(0, 4, 60)
    lengths[at] = 6000
    starts = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    check(ds, rng, 60, starts[-1], channels, dtype, dtype, kind, starts=starts, carry=True)
    lengths[at] = 3100                                                  # just more than half, and just not
    lengths[(at + 7) % 60] = 3050 - (lengths.sum() - lengths[(at + 7) % 60] - 3100)
    for more in (0, 200):
        lengths[(at + 7) % 60] += more
        starts = np.concatenate([[0], np.cumsum(lengths)]).tolist()
        check(ds, rng, 60, starts[-1] + 500, channels, dtype, dtype, kind, starts=starts, carry=at == 0)


def test_one_long_row_within_a_share(ds):
    """A row longer than half of all that ends inside the first share of a padded batch, in place."""
    rng = np.random.default_rng(19)
    for starts, n, channels in (([0, 200, 4200, 4300, 4400, 4900, 5000], 36000, 640), ([0, 10, 910, 1000], 60000, 640),
                                ([0, 5000, 5100], 30000, 256)):
        rows = len(starts) - 1
        x, gate = cuda(rng.standard_normal((n, channels)), BF16), cuda(rng.standard_normal((n, channels)), BF16)
        states, where = cuda(rng.standard_normal((rows, channels))), torch.tensor(starts, dtype=torch.int32, device="cuda")
        h, room, last, last_room = ref.scan(flat(x), flat(gate), "sigmoid", ref.rows_of(starts, n, rows), ref.as64(states))
        for _ in range(3):
            into, pool = x.clone(), states.clone()
            ds.gated_scan(into, gate, starts=where, initial=pool, kind="sigmoid", out=into, final=pool)
            ref.close(into, h, room, "out")
            ref.close(pool, last, last_room, "states")


def test_one_long_row_that_is_cut(ds):
    """Rows that begin in front of the tokens or go on behind them."""
    rng = np.random.default_rng(15)
    for starts in ([-50, 7000, *range(7001, 7060)], [*range(59), 9000], [*range(59), 8000, 9000], [1000, *range(1001, 1060), 9000]):
        x, gate = cuda(rng.standard_normal((8000, 640)), BF16), cuda(rng.standard_normal((8000, 640)), BF16)
        where = torch.tensor(starts, dtype=torch.int32, device="cuda")
        out, final = ds.gated_scan(x, gate, starts=where, kind="sigmoid")
        kept = [min(max(s, 0), 8000) for s in starts]
        h, room, last, last_room = ref.scan(flat(x), flat(gate), "sigmoid", ref.rows_of(kept, 8000, len(kept) - 1))
        ref.close(out, h, room, "out")
        ref.close(final, last, last_room, "final")


def test_long_row_streams_and_graphs(ds):
    """Both launches stay in their stream's order, eager and captured."""
    rng = np.random.default_rng(16)
    starts = torch.tensor([*range(60), 9000], dtype=torch.int32, device="cuda")
    x, gate = cuda(rng.standard_normal((9000, 640)), BF16), cuda(rng.standard_normal((9000, 640)), BF16)
    want, last = ds.gated_scan(x, gate, starts=starts, kind="sigmoid")
    once, _ = ds.gated_scan(want, gate, starts=starts, kind="sigmoid")
    back = ds.gated_scan_backward(once, x, gate, want, starts=starts, kind="sigmoid")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def steps():
        out, final = ds.gated_scan(x, gate, starts=starts, kind="sigmoid")
        twice, _ = ds.gated_scan(out, gate, starts=starts, kind="sigmoid")
        return (out, final, twice, *ds.gated_scan_backward(twice, x, gate, out, starts=starts, kind="sigmoid")[:2])

    with torch.cuda.graph(graph, stream=side):
        captured = steps()
    for _ in range(3):
        for t in captured:
            t.fill_(7)
        graph.replay()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            eager = steps()
        torch.cuda.synchronize()
        for got in (captured, eager):
            assert all(torch.equal(a, b) for a, b in zip(got, (want, last, once, *back[:2])))


@pytest.mark.parametrize("tokens", [1, 5, 200])
def test_states_in_a_pool(ds, tokens):
    """Slots of a larger pool, in place; a row without a state; other states stay."""
    rng = np.random.default_rng(3)
    rows, channels, pool = 6, 48, 11
    slots = [4, 10, -1, 0, 99, 7]
    x, gate = cuda(rng.standard_normal((rows, tokens, channels)), BF16), cuda(rng.standard_normal((rows, tokens, channels)), BF16)
    states = cuda(rng.standard_normal((pool, channels)))
    before = states.clone()
    where = torch.tensor(slots, dtype=torch.int32, device="cuda")
    out, final = ds.gated_scan(x, gate, initial=states, slots=where, kind="sigmoid")
    assert final is states
    start = np.stack([ref.as64(before)[s] if 0 <= s < pool else np.zeros(channels) for s in slots])
    h, room, last, last_room = ref.scan(flat(x), flat(gate), "sigmoid", ref.rows_of(None, tokens, rows), start)
    ref.close(out.reshape(-1, channels), h, room, "out")
    used = [r for r, s in enumerate(slots) if 0 <= s < pool]
    ref.close(states[[slots[r] for r in used]], last[used], last_room[used], "states")
    others = [s for s in range(pool) if s not in slots]
    assert torch.equal(states[others], before[others])


def test_states_of_packed_rows(ds):
    """A step of a server: packed rows with slots, one of them without tokens, a padded end."""
    rng = np.random.default_rng(8)
    starts, slots, channels = [0, 1, 1, 140, 141, 300], [3, 2, 6, 0, 5], 32
    x, gate = cuda(rng.standard_normal((310, channels))), cuda(gates(rng, (310, channels), "log"))
    states, final = cuda(rng.standard_normal((7, channels))), torch.full((7, channels), 9.0, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x[300:] = float("nan")
    out, _ = ds.gated_scan(x, gate, starts=i32(starts), initial=states, slots=i32(slots), kind="log", final=final)
    h, room, last, last_room = ref.scan(flat(x), flat(gate), "log", ref.rows_of(starts, 310, 5), ref.as64(states)[slots])
    ref.close(out[:300], h[:300], room[:300], "out")
    assert not out[300:].any()
    ref.close(final[slots], last, last_room, "final")
    assert torch.equal(final[2], states[2]) and (final[[1, 4]] == 9).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(ds, dtype):
    """Halves of one projection, time-major arrays, a slice of time, a gate that all tokens share."""
    rng = np.random.default_rng(4)
    both = cuda(rng.standard_normal((2, 200, 128)), dtype)
    gate, x = both[..., :64].abs_().neg_(), both[..., 64:]
    want, _ = ds.gated_scan(x.contiguous(), gate.contiguous(), kind="log")
    grads = torch.zeros_like(both)
    out, _ = ds.gated_scan(x, gate, kind="log", out=torch.zeros_like(both)[..., 10:74])
    assert torch.equal(out, want)
    gx, gg, _ = ds.gated_scan_backward(x, None, gate, out, kind="log", grad_x=grads[..., 64:], grad_gate=grads[..., :64])
    wx, wg, _ = ds.gated_scan_backward(x.contiguous(), None, gate.contiguous(), want, kind="log")
    assert torch.equal(gx, wx) and torch.equal(gg, wg) and torch.equal(grads[..., 64:], wx)
    turned = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    assert torch.equal(ds.gated_scan(turned(x), turned(gate), kind="log", out=turned(torch.zeros_like(x)))[0], want)
    assert torch.equal(ds.gated_scan(x[:, 50:111], gate[:, 50:111], kind="log")[0],
                       ds.gated_scan(x[:, 50:111].contiguous(), gate[:, 50:111].contiguous(), kind="log")[0])
    shared = gate[:1, :1].expand(2, 200, 64)
    assert torch.equal(ds.gated_scan(x, shared, kind="log")[0], ds.gated_scan(x, shared.contiguous(), kind="log")[0])
    odd = torch.zeros(2, 200, 131, dtype=dtype, device="cuda")[..., 1:65]      # tokens at odd addresses
    assert torch.equal(ds.gated_scan(x, gate, kind="log", out=odd)[0], want)
    into = x.clone()
    assert ds.gated_scan(into, gate, kind="log", out=into)[0] is into and torch.equal(into, want)


@pytest.mark.parametrize("tokens", [1, 200])
def test_wide_gates_at_any_address(ds, tokens):
    """fp32 gates and their gradients on 4 bytes beside pairs of 16-bit values, and 4-byte-aligned rows."""
    rng = np.random.default_rng(9)
    x = cuda(rng.standard_normal((3, tokens, 70)), BF16)
    gate = cuda(rng.standard_normal((3, tokens, 75)))
    at = gate[..., 1:71]
    spans = ref.rows_of(None, tokens, 3)
    out, final = ds.gated_scan(x, at, kind="sigmoid")
    h, room, last, last_room = ref.scan(flat(x), flat(at), "sigmoid", spans)
    ref.close(out.reshape(-1, 70), h, room, "out")
    ref.close(final, last, last_room, "final")
    wide = torch.zeros(3, tokens, 76, device="cuda")
    gx, _, _ = ds.gated_scan_backward(x, x, at, out, kind="sigmoid", grad_gate=wide[..., 3:73])
    want = ref.scan_backward(flat(x), flat(x), flat(at), flat(out), "sigmoid", spans)
    ref.close(gx.reshape(-1, 70), *want["x"], "grad_x")
    ref.close(wide[..., 3:73].reshape(-1, 70), *want["gate"], "grad_gate")
    assert not wide[..., :3].any() and not wide[..., 73:].any()


def test_what_is_not_a_number_stays_in_its_row(ds):
    """Rows after one that ends in infinity or NaN are what they are without it, forward and back."""
    rng = np.random.default_rng(6)
    for starts in ([0, 100, 300, 700], [0, 3, 5, 700], [0, 650, 651, 700]):
        x, gate = cuda(rng.standard_normal((700, 64)), BF16), cuda(rng.standard_normal((700, 64)), BF16)
        where = torch.tensor(starts, dtype=torch.int32, device="cuda")
        clean = ds.gated_scan(x, gate, starts=where, kind="sigmoid")[0]
        grad = cuda(rng.standard_normal((700, 64)), BF16)
        want = ds.gated_scan_backward(grad, x, gate, clean, starts=where, kind="sigmoid")
        for r, bad in ((0, float("nan")), (1, float("inf"))):
            a, b = starts[r], starts[r + 1]
            x2, grad2 = x.clone(), grad.clone()
            x2[a], grad2[b - 1] = bad, bad
            got = ds.gated_scan(x2, gate, starts=where, kind="sigmoid")[0]
            keep = [t for t in range(700) if not a <= t < b]
            assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[a]).any()
            back = ds.gated_scan_backward(grad2, x, gate, clean, starts=where, kind="sigmoid")
            assert torch.equal(back[0][keep], want[0][keep]) and torch.equal(back[1][keep], want[1][keep])


def test_first_gates_do_not_count_without_a_state(ds):
    x, gate = torch.ones(2, 40, 8, device="cuda"), torch.full((2, 40, 8), 0.5, device="cuda")
    want, last = ds.gated_scan(x, gate)
    gate[:, 0] = float("nan")
    out, final = ds.gated_scan(x, gate)
    assert torch.equal(out, want) and torch.equal(final, last)
    assert torch.equal(ds.gated_scan(x[:, :1], gate[:, :1])[0], x[:, :1])


def test_extreme_gates(ds):
    """Gates whose decay is 0 or 1: forgetting and holding are exact."""
    inf = float("inf")
    x = torch.randn(1, 300, 64, device="cuda")
    assert torch.equal(ds.gated_scan(x, torch.full_like(x, -inf), kind="log")[0], x)
    assert torch.equal(ds.gated_scan(x, torch.full_like(x, -200.0), kind="sigmoid")[0], x)
    state = torch.randn(1, 64, device="cuda")
    held, final = ds.gated_scan(x, torch.full_like(x, inf), initial=state, kind="sigmoid")
    assert torch.equal(held, state[:, None].expand_as(held)) and torch.equal(final, state)
    assert torch.equal(ds.gated_scan(torch.zeros_like(x), torch.zeros_like(x), initial=state, kind="log")[1], state)


def test_long_memory(ds):
    """60,000 tokens through decays next to 1: errors do not lean to one side.
    Against 64 bits on the GPU; the room is that of test_lengths with memories of
    3,000 tokens: 3,000 * (4u + 2u) as a bound, of which independent roundings
    use about a 50th."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n, c = 60000, 64
    x = torch.randn(1, n, c, generator=g, device="cuda").abs_()
    for kind in ("log", "sigmoid"):
        gate = torch.rand(1, n, c, generator=g, device="cuda") * 1e-3
        gate = -gate if kind == "log" else 7 + 1e3 * gate
        out, final = ds.gated_scan(x, gate, kind=kind)
        a = torch.exp(gate.double()) if kind == "log" else torch.sigmoid(gate.double())
        b = x.double() * (1 if kind == "log" else torch.sigmoid(-gate.double()))
        h, size = torch.zeros(c, dtype=torch.float64, device="cuda"), 0.0
        for t in range(n):
            h = a[0, t] * h + b[0, t]
        err = ((final[0].double() - h).abs() / h).max().item()
        assert err < 3000 * 6 * 2.0 ** -24 / 50, (kind, err)


def test_empty_calls(ds):
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    out, final = ds.gated_scan(e(3, 0, 8), e(3, 0, 8))
    assert out.shape == (3, 0, 8) and not final.any()
    state = torch.randn(3, 8, device="cuda")
    assert torch.equal(ds.gated_scan(e(3, 0, 8), e(3, 0, 8), initial=state)[1], state)
    assert ds.gated_scan(e(0, 5, 8), e(0, 5, 8))[0].shape == (0, 5, 8)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert not ds.gated_scan(torch.ones(5, 8, device="cuda"), torch.ones(5, 8, device="cuda"), starts=none)[0].any()
    _, _, gi = ds.gated_scan_backward(e(3, 0, 8), None, e(3, 0, 8), e(3, 0, 8), initial=state, grad_final=state * 2)
    assert torch.equal(gi, state * 2)


def test_same_bits_and_streams(ds):
    """Calls repeat their bits, on other streams and in captured graphs at once."""
    rng = np.random.default_rng(12)
    x, gate = cuda(rng.standard_normal((2, 3000, 256)), BF16), cuda(rng.standard_normal((2, 3000, 256)), BF16)
    want, last = ds.gated_scan(x, gate, kind="sigmoid")
    back = ds.gated_scan_backward(x, x, gate, want, kind="sigmoid")
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, results = [], []
    torch.cuda.synchronize()
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out, final = ds.gated_scan(x, gate, kind="sigmoid")
            results.append((out, final, *ds.gated_scan_backward(x, x, gate, out, kind="sigmoid")[:2]))
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got in results:
        assert all(torch.equal(a, b) for a, b in zip(got, (want, last, *back[:2])))
    out = torch.empty_like(x)
    ds.gated_scan(x, gate, kind="sigmoid", out=out, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("tokens", [1, 2])
def test_arrays_side_by_side(ds, tokens):
    """Inputs and outputs in one buffer, next to each other in every token: of a step, too."""
    rng = np.random.default_rng(14)
    buffer = cuda(rng.standard_normal((5, tokens, 5 * 16)), BF16)
    parts = [buffer[..., 16 * i:16 * i + 16] for i in range(5)]
    x, gate = parts[0].clone(), parts[2].clone()
    want, _ = ds.gated_scan(x, gate, kind="sigmoid")
    out, _ = ds.gated_scan(parts[0], parts[2], kind="sigmoid", out=parts[1])
    assert torch.equal(out, want) and torch.equal(parts[0], x) and torch.equal(parts[2], gate)
    back = ds.gated_scan_backward(x, x, gate, want, kind="sigmoid")
    ds.gated_scan_backward(parts[0], parts[0], parts[2], parts[1], kind="sigmoid", grad_x=parts[4], grad_gate=parts[3])
    assert torch.equal(parts[4], back[0]) and torch.equal(parts[3], back[1]) and torch.equal(parts[1], want)
    for shift in (8, 24):
        with pytest.raises(ds.DevscanError):
            ds.gated_scan(parts[0], parts[2], kind="sigmoid", out=buffer[..., shift:shift + 16])


def test_far_offsets(ds):
    """Elements behind 2^32 bytes and 2^31 elements."""
    wide = torch.zeros(40, 1 << 26, dtype=BF16, device="cuda")
    x = wide[:, -64:]
    x.copy_(torch.randn(40, 64, device="cuda"))
    gate = torch.rand(40, 64, device="cuda").to(BF16)
    out = wide[:, :64]
    assert torch.equal(ds.gated_scan(x, gate, out=out)[0], ds.gated_scan(x.contiguous(), gate)[0])


def test_most_tokens(ds):
    """2^31 - 2 tokens in one row and in two: h = 2 - 2^-t exactly, from inputs that repeat themselves."""
    n = 2**31 - 2
    one, half = torch.ones(1, 1, device="cuda").expand(n, 1), torch.full((1, 1), 0.5, device="cuda").expand(n, 1)
    out = torch.empty(n, 1, device="cuda")
    starts = torch.tensor([0, 2**30 + 1, n], dtype=torch.int32, device="cuda")
    for where, begins in ((None, [0]), (starts, [0, 2**30 + 1])):
        out.zero_()
        _, final = ds.gated_scan(one, half, starts=where, out=out)
        assert (final == 2).all() and final.shape == (len(begins), 1)
        for b in begins:
            assert out[b:b + 4, 0].tolist() == [1.0, 1.5, 1.75, 1.875]
        assert (out[-5:] == 2).all() and (out < 2).sum().item() == 24 * len(begins)


def test_refusals(ds):
    x, g = torch.ones(2, 10, 8, device="cuda"), torch.ones(2, 10, 8, device="cuda")
    state, i32 = torch.ones(2, 8, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [(ValueError, lambda: ds.gated_scan(x, g[:, :9])), (TypeError, lambda: ds.gated_scan(x, g.half())),
           (TypeError, lambda: ds.gated_scan(x.double(), g)), (ValueError, lambda: ds.gated_scan(x, g, kind="tanh")),
           (ValueError, lambda: ds.gated_scan(x, g, starts=i32)), (ValueError, lambda: ds.gated_scan(x.transpose(1, 2), g)),
           (ValueError, lambda: ds.gated_scan(x, g, initial=state[:1])),
           (ValueError, lambda: ds.gated_scan(x, g, final=state[:1])),
           (ValueError, lambda: ds.gated_scan(x, g, slots=i32[:2])),
           (ValueError, lambda: ds.gated_scan(x, g, initial=state, slots=i32)),
           (TypeError, lambda: ds.gated_scan(x, g, initial=state.half())),
           (ds.DevscanError, lambda: ds.gated_scan(x, g, out=g)),
           (ds.DevscanError, lambda: ds.gated_scan(x[:, :5], g[:, :5], out=x[:, 1:6])),
           (ds.DevscanError, lambda: ds.gated_scan(x, g, out=x[:, :1].expand(2, 10, 8))),
           (ValueError, lambda: ds.gated_scan_backward(x, None, g, x.clone(), kind="sigmoid")),
           (ds.DevscanError, lambda: ds.gated_scan_backward(x, x, g, x.clone(), grad_x=x)),
           (ValueError, lambda: ds.gated_scan(x.cpu(), g))]
    for error, call in bad:
        with pytest.raises(error):
            call()
