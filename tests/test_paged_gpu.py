"""Block tables and slot maps against loops over the rows: sizes from no row
to more than one launch covers, pages of any size, pools that run out, rows
that cannot be served, strides, streams, and the arguments they refuse."""
import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def batch(rows, width, page, seed, most=None):
    """A batch whose rows hold pages for `cached` tokens, and the stack of the
    rest, lengths at and around the pages' ends among them."""
    rng = np.random.default_rng(seed)
    limit = width * page
    cached = rng.integers(0, limit + 1, rows)
    edge = rng.random(rows) < 0.5
    cached[edge] = np.clip(cached[edge] // page * page + rng.integers(-1, 2, edge.sum()), 0, limit)
    cached[rng.random(rows) < 0.2] = 0
    fresh = np.where(rng.random(rows) < 0.5, 1, rng.integers(0, (most or limit) + 1, rows))
    fresh = np.minimum(fresh, limit - cached)
    have = -(-cached // page)
    pool = int((-(-(cached + fresh) // page)).sum()) + 7
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((rows, width), -1, np.int32)
    at = 0
    for r in range(rows):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    stack = np.full(pool, -1, np.int32)
    stack[:pool - at] = ids[at:]
    return table, cached.astype(np.int32), fresh.astype(np.int32), stack, pool - at


SHAPES = [(1, 1, 1), (1, 300, 16), (3, 40, 16), (64, 33, 5), (511, 20, 16), (513, 9, 64), (4096, 3, 1), (2000, 70, 24),
          (4097, 4, 16), (8192, 4, 16), (8193, 4, 16), (20001, 3, 7)]


@pytest.mark.parametrize("rows,width,page", SHAPES)
@pytest.mark.parametrize("share", [1.0, 0.6, 0.0])
def test_extend(ds, rows, width, page, share):
    table, cached, fresh, stack, free = batch(rows, width, page, rows + width)
    free = int(free * share)                       # a pool that runs out
    want = table.copy()
    granted, left = ref.extend(want, cached, fresh, stack, free, page)
    t, f = dev(table), dev([free])
    for _ in range(2):                             # the second call repeats the first
        got, height = ds.block_table_extend(t, dev(cached), dev(fresh), dev(stack), f, page)
        assert np.array_equal(got.cpu().numpy(), granted)
        assert height.item() == left
        assert np.array_equal(t.cpu().numpy(), want)
    assert f.item() == free


def test_extend_rows_that_cannot_be_served(ds):
    table = np.full((7, 4), -1, np.int32)
    cached = np.array([0, -1, 3, 60, 0, 2**31 - 1, 5])
    fresh = np.array([17, 1, -2, 5, 64, 2**31 - 1, 65])
    stack, free = np.arange(100, 120).astype(np.int32), 20
    want = table.copy()
    granted, left = ref.extend(want, cached, fresh, stack, free, 16)
    t = dev(table)
    got, height = ds.block_table_extend(t, dev(cached), dev(fresh), dev(stack), dev([free]), 16)
    assert got.cpu().tolist() == granted.tolist() == [1, 0, 0, 0, 1, 0, 0]
    assert height.item() == left == 20 - 2 - 4
    assert np.array_equal(t.cpu().numpy(), want)


@pytest.mark.parametrize("free", [-5, 0, 3, 50])
def test_heights_outside_the_pool(ds, free):
    table = np.full((4, 4), -1, np.int32)
    cached, fresh, stack = np.zeros(4), np.full(4, 20), np.arange(6).astype(np.int32)
    want = table.copy()
    granted, left = ref.extend(want, cached, fresh, stack, free, 16)
    t = dev(table)
    got, height = ds.block_table_extend(t, dev(cached), dev(fresh), dev(stack), dev([free]), 16)
    assert np.array_equal(got.cpu().numpy(), granted) and height.item() == left
    assert np.array_equal(t.cpu().numpy(), want)
    full = np.arange(16).reshape(4, 4).astype(np.int32)
    pages, back = stack.copy(), dev(stack)
    left = ref.release(full, np.full(4, 20), np.array([1, 0, 1, 1]), pages, free, 16)
    height = ds.block_table_release(dev(full), dev(np.full(4, 20)), dev([1, 0, 1, 1], np.uint8), back, dev([free]), 16)
    assert height.item() == left and np.array_equal(back.cpu().numpy(), pages)


@pytest.mark.parametrize("rows,width,page", SHAPES)
@pytest.mark.parametrize("pad", [0, 13, -3])
def test_slot_map(ds, rows, width, page, pad):
    table, cached, fresh, _, _ = batch(rows, width, page, rows * 3 + width, most=200)
    rng = np.random.default_rng(rows)
    granted = (rng.random(rows) < 0.7).astype(np.uint8)
    for flags in (None, granted):
        total = int(fresh.sum() if flags is None else fresh[flags != 0].sum())
        tokens = max(0, total + pad)
        want = ref.slots(table, cached, fresh, page, tokens, flags)
        got = ds.slot_map(dev(table), dev(cached), dev(fresh), page, tokens,
                          granted=None if flags is None else dev(flags, np.uint8))
        for g, w, dtype in zip(got, want, (torch.int32, torch.int64, torch.int32, torch.int32)):
            assert g.dtype == dtype
            assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("offset", [0, 1])
def test_slot_map_of_many_tokens(ds, offset):
    """A million tokens in rows from none up to thousands, and outputs that do
    not start on 16 bytes."""
    rng = np.random.default_rng(77)
    rows, width, page = 500, 300, 24
    fresh = rng.integers(0, 4500, rows)
    fresh[rng.random(rows) < 0.3] = rng.integers(0, 3, (rng.random(rows) < 0.3).sum())[0]
    cached = rng.integers(0, width * page - 4500, rows)
    table = rng.permutation(rows * width).reshape(rows, width).astype(np.int32)
    table[::7, 5] = -1
    tokens = int(fresh.sum()) + 3
    assert tokens > 700_000
    out = [torch.zeros(rows + 1, dtype=torch.int32, device="cuda")] + [
        torch.zeros(tokens + offset, dtype=d, device="cuda")[offset:] for d in (torch.int64, torch.int32, torch.int32)]
    ds.slot_map(dev(table), dev(cached), dev(fresh), page, tokens, out=out)
    starts = np.concatenate([[0], np.cumsum(fresh)])
    row = np.repeat(np.arange(rows), fresh)
    pos = cached[row] + np.arange(len(row)) - starts[row]
    entry = table[row, pos // page].astype(np.int64)
    pad = np.full(3, -1)
    assert np.array_equal(out[0].cpu().numpy(), starts)
    assert np.array_equal(out[1].cpu().numpy(), np.concatenate([np.where(entry < 0, -1, entry * page + pos % page), pad]))
    assert np.array_equal(out[2].cpu().numpy(), np.concatenate([pos, pad]))
    assert np.array_equal(out[3].cpu().numpy(), np.concatenate([row, pad]))


def test_slots_past_32_bits(ds):
    """Pages whose slots pass 2^31 and 2^32, and lengths whose sums do."""
    table = np.array([[2**31 - 1, 2**30], [7, -1]], np.int32)
    cached, fresh = np.array([15, 14]), np.array([3, 4])
    want = ref.slots(table, cached, fresh, 16, 9)
    got = ds.slot_map(dev(table), dev(cached), dev(fresh), 16, 9)
    assert got[1][0].item() == (2**31 - 1) * 16 + 15
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    big = np.array([2**31 - 1, 2**31 - 1, 5])
    table, cached = np.zeros((3, 1), np.int32), np.array([2**31 - 3, 0, 0])
    got = ds.slot_map(dev(table), dev(cached), dev(big), 1 << 20, 10)
    starts, _, positions, ids = (g.cpu().numpy() for g in got)
    assert starts.tolist() == [0, 2**31 - 1, 2**31 - 1, 2**31 - 1]
    assert positions.tolist() == [2**31 - 3, 2**31 - 2, 2**31 - 1] + [-1] * 7 and ids.tolist() == [0] * 10


def test_slot_map_of_negative_lengths(ds):
    table = np.array([[4, 5], [6, 7], [8, 9]], np.int32)
    cached, fresh = np.array([-2, 3, 0]), np.array([4, -1, 2])
    want = ref.slots(table, cached, fresh, 4, 8)
    for g, w in zip(ds.slot_map(dev(table), dev(cached), dev(fresh), 4, 8), want):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("rows,width,page", SHAPES)
@pytest.mark.parametrize("share,room", [(1.0, 0), (0.3, 0), (0.5, -3), (0.0, 0)])
def test_release(ds, rows, width, page, share, room):
    table, cached, _, stack, free = batch(rows, width, page, rows + 5)
    rng = np.random.default_rng(rows)
    done = (rng.random(rows) < share).astype(np.uint8) * 255
    if room < 0:                                   # a pool that the last rows' pages do not fit
        count = int((-(-cached[done != 0] // page)).sum())
        stack = np.ascontiguousarray(stack[:max(0, free + count + room)])
        free = min(free, len(stack))
    want = stack.copy()
    left = ref.release(table, cached, done, want, free, page)
    pages = dev(stack)
    height = ds.block_table_release(dev(table), dev(cached), dev(done, np.uint8), pages, dev([free]), page)
    assert height.item() == left
    assert np.array_equal(pages.cpu().numpy(), want)


def test_release_then_extend_returns_the_same_pages(ds):
    table, cached, fresh, stack, free = batch(50, 12, 16, 9)
    t, pages = dev(table), dev(stack)
    done = np.zeros(50, np.uint8)
    done[::3] = 1
    left = ds.block_table_release(t, dev(cached), dev(done, np.uint8), pages, dev([free]), 16)
    lengths = np.where(done != 0, 0, cached)
    again = np.where(done != 0, cached, 0)
    granted, height = ds.block_table_extend(t, dev(lengths), dev(again), pages, left, 16)
    assert granted.cpu().numpy().all() and height.item() == free
    held = [x for r in range(50) for x in t[r, : ref.blocks(cached[r], 16)].tolist()]
    assert len(set(held)) == len(held) and sorted(held) == sorted(x for x in table[table >= 0].tolist())


def test_strided_table_and_other_stream(ds):
    table, cached, fresh, stack, free = batch(100, 9, 16, 21)
    wide = np.full((100, 16), 12345, np.int32)
    wide[:, 3:12] = table
    w = dev(wide)
    t = w[:, 3:12]
    want = table.copy()
    granted, left = ref.extend(want, cached, fresh, stack, free, 16)
    args = dev(cached), dev(fresh), dev(stack), dev([free])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, height = ds.block_table_extend(t, *args, 16, stream=s)
    tokens = int(fresh.sum())
    mapped = ds.slot_map(t, args[0], args[1], 16, tokens, granted=got, stream=s)
    s.synchronize()
    assert np.array_equal(got.cpu().numpy(), granted) and height.item() == left
    after = w.cpu().numpy()
    assert np.array_equal(after[:, 3:12], want)
    assert (after[:, :3] == 12345).all() and (after[:, 12:] == 12345).all()
    for g, x in zip(mapped, ref.slots(want, cached, fresh, 16, tokens, granted)):
        assert np.array_equal(g.cpu().numpy(), x)
    ds.stream_release(s)


@pytest.mark.parametrize("width", [0, 5])
def test_no_rows(ds, width):
    t = torch.zeros(0, width, dtype=torch.int32, device="cuda")
    none, pages = dev([]), dev(np.arange(6))
    granted, left = ds.block_table_extend(t, none, none, pages, dev([4]), 16)
    assert granted.numel() == 0 and left.item() == 4
    starts, slots, positions, rows = ds.slot_map(t, none, none, 16, 3)
    assert starts.tolist() == [0] and slots.tolist() == positions.tolist() == rows.tolist() == [-1] * 3
    assert ds.block_table_release(t, none, dev([], np.uint8), pages, dev([4]), 16).item() == 4


def test_graph_replay(ds):
    table, cached, fresh, stack, free = batch(200, 10, 16, 31, most=20)
    t, c, n, p, f = dev(table), dev(cached), dev(fresh), dev(stack), dev([free])
    tokens = int(fresh.sum())
    granted, left = torch.empty(200, dtype=torch.uint8, device="cuda"), dev([0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ds.block_table_extend(t, c, n, p, f, 16, granted=granted, left=left)
        out = ds.slot_map(t, c, n, 16, tokens, granted=granted)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ds.block_table_extend(t, c, n, p, f, 16, granted=granted, left=left)
        ds.slot_map(t, c, n, 16, tokens, granted=granted, out=out)
    table, cached, fresh, stack2, free = batch(200, 10, 16, 32, most=20)
    size = min(len(stack), len(stack2))
    p[:size].copy_(dev(stack2)[:size])
    free = min(free, size)
    t.copy_(dev(table)), c.copy_(dev(cached)), n.copy_(dev(fresh)), f.fill_(free)
    graph.replay()
    torch.cuda.synchronize()
    want = table.copy()
    flags, height = ref.extend(want, cached, fresh, p.cpu().numpy(), free, 16)
    assert np.array_equal(granted.cpu().numpy(), flags) and left.item() == height
    assert np.array_equal(t.cpu().numpy(), want)
    for g, x in zip(out, ref.slots(want, cached, fresh, 16, tokens, flags)):
        assert np.array_equal(g.cpu().numpy(), x)
    ds.stream_release(s)


def test_refusals(ds):
    t, one, four = dev(np.zeros((4, 8))), dev([3]), dev(np.zeros(4))
    pages, flags = dev(np.arange(9)), torch.zeros(4, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        ds.block_table_extend(t.cpu(), four, four, pages, one, 16)
    with pytest.raises(TypeError):
        ds.block_table_extend(t.float(), four, four, pages, one, 16)
    with pytest.raises(ValueError):
        ds.block_table_extend(t, four[:3], four, pages, one, 16)
    with pytest.raises(TypeError):
        ds.block_table_extend(t, four, four.long(), pages, one, 16)
    with pytest.raises(ValueError):
        ds.block_table_extend(t, four, four, pages, four, 16)
    with pytest.raises(ValueError):
        ds.block_table_extend(t, four, four, pages, one, 0)
    with pytest.raises(ValueError):
        ds.block_table_extend(t.t(), four, four, pages, one, 16)
    with pytest.raises(ds.DevscanError):
        ds.block_table_extend(t, four, four, pages, one, 16, left=one)               # height in place
    with pytest.raises(ds.DevscanError):
        ds.block_table_extend(t, four, four, t.view(-1)[:9], one, 16)                # the stack inside the table
    with pytest.raises(ValueError):
        ds.slot_map(t, four, four, 16, -1)
    with pytest.raises(ValueError):
        ds.slot_map(t, four, four, 16, 5, granted=flags[:2])
    with pytest.raises(ValueError):
        ds.slot_map(t, four, four, 16, 5, out=(four, four, four, four))
    with pytest.raises(TypeError):
        ds.block_table_release(t, four, four, pages, one, 16)                        # done must be uint8
    with pytest.raises(ds.DevscanError):
        ds.block_table_release(t, four, flags, pages, pages[:1], 16)                 # height inside the stack
