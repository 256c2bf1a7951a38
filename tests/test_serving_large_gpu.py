"""The serving operators at the ends of their ranges: token and page counts
whose last index is next to 2^31, and as many rows.  Expected values are worked
out on the device, a part at a time."""
import pytest
import torch

pytestmark = pytest.mark.gpu

PART = 1 << 27


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


@pytest.fixture
def room(ds):
    """Asks for free device memory; afterwards gives back what was cached."""
    def ask(gib):
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < gib << 30:
            pytest.skip(f"needs {gib} GiB of free device memory")
    yield ask
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def parts(n):
    for at in range(0, n, PART):
        yield at, min(n, at + PART)


def test_slots_of_2_31_tokens(ds, room):
    """Two rows of about 2^30 tokens, 200 of one token, a few places left."""
    room(60)
    width, page, tokens = 1024, 1 << 20, 2**31 - 1
    fresh = torch.ones(202, dtype=torch.int32, device="cuda")
    fresh[0], fresh[1] = 2**30, 2**30 - 301
    cached = torch.zeros_like(fresh)
    cached[2:] = torch.arange(200, dtype=torch.int32, device="cuda") * 1001
    table = torch.randperm(202 * width, device="cuda").to(torch.int32).view(202, width)
    total = int(fresh.sum(dtype=torch.int64))
    assert tokens - 110 < total < tokens
    starts, slots, positions, rows = ds.slot_map(table, cached, fresh, page, tokens)
    want = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), fresh.cumsum(0, dtype=torch.int64)])
    assert torch.equal(starts.long(), want)
    for lo, hi in parts(tokens):
        g = torch.arange(lo, min(hi, total), device="cuda")
        row = torch.searchsorted(want[1:], g, right=True)
        pos = cached.long()[row] + g - want[row]
        place = table.long()[row, pos // page] * page + pos % page
        n = len(g)
        assert torch.equal(rows[lo:lo + n].long(), row)
        assert torch.equal(positions[lo:lo + n].long(), pos)
        assert torch.equal(slots[lo:lo + n], place)
        for out in (slots, positions, rows):
            assert bool((out[lo + n:hi] == -1).all())


def test_2_31_pages(ds, room):
    """The largest pool, opened by one call and given back by another."""
    room(40)
    width, pool = 2**30 - 1, 2**31 - 2
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    pages = torch.arange(pool, dtype=torch.int32, device="cuda")
    none, full = i32(0, 0), i32(width, width)
    granted, left = ds.block_table_extend(table, none, full, pages, i32(pool), 1)
    assert granted.tolist() == [1, 1] and left.item() == 0
    flat = table.view(-1)
    for lo, hi in parts(pool):
        assert torch.equal(flat[lo:hi], pool - 1 - torch.arange(lo, hi, dtype=torch.int32, device="cuda"))
    pages.fill_(-1)
    done = torch.ones(2, dtype=torch.uint8, device="cuda")
    height = ds.block_table_release(table, full, done, pages, left, 1)
    assert height.item() == pool
    for lo, hi in parts(pool):
        assert torch.equal(pages[lo:hi], flat[lo:hi])


def test_2_31_rows(ds, room):
    """Nearly all rows idle; those that are not at the ends and past 2^30."""
    room(75)
    rows = 2**31 - 2
    busy = torch.tensor([0, 1, 4095, 4096, 2**30 - 1, 2**30, 2**30 + 77, rows - 4097, rows - 2, rows - 1], device="cuda")
    n = len(busy)
    table = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    idle = torch.zeros(rows, dtype=torch.int32, device="cuda")
    fresh = torch.zeros(rows, dtype=torch.int32, device="cuda")
    fresh[busy] = 3
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        granted, left = ds.block_table_extend(table, idle, fresh, torch.arange(100, 100 + n, dtype=torch.int32, device="cuda"),
                                              i32(n), 4)
        assert left.item() == 0 and bool(granted.all())
        assert table[busy, 0].tolist() == list(range(100 + n - 1, 99, -1))
        assert int(sum((table[lo:hi, 0] != -1).sum() for lo, hi in parts(rows))) == n
        del granted
        starts, slots, positions, ids = ds.slot_map(table, idle, fresh, 4, 3 * n + 2)
        assert ids.tolist() == [r for r in busy.tolist() for _ in range(3)] + [-1, -1]
        assert positions.tolist() == [0, 1, 2] * n + [-1, -1]
        assert slots.tolist() == [4 * (100 + n - 1 - k) + j for k in range(n) for j in range(3)] + [-1, -1]
        assert starts[0].item() == 0 and starts[rows].item() == 3 * n
        for lo, hi in parts(rows):
            assert torch.equal(starts[lo + 1:hi + 1] - starts[lo:hi], fresh[lo:hi])
        del starts
        done = torch.zeros(rows, dtype=torch.uint8, device="cuda")
        done[busy] = 1
        done[17] = 1                                 # ended without a page
        pages = torch.full((n + 3,), -1, dtype=torch.int32, device="cuda")
        height = ds.block_table_release(table, fresh, done, pages, i32(2), 4)
        assert height.item() == n + 2
        assert pages.tolist() == [-1, -1] + list(range(100 + n - 1, 99, -1)) + [-1]
    s.synchronize()
    ds.stream_release(s)


def test_draw_of_2_28_rows(ds, room):
    room(20)
    rows = 2**28 + 3
    logits = torch.empty(rows, 3, dtype=torch.bfloat16, device="cuda")
    for lo, hi in parts(rows):
        logits[lo:hi] = torch.randint(-3, 4, (hi - lo, 3), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    tokens, logprobs = ds.sample_tokens(logits)
    for lo, hi in parts(rows):
        x = logits[lo:hi]
        top = x.amax(1)
        want = torch.where(x[:, 0] == top, 0, torch.where(x[:, 1] == top, 1, 2))
        assert torch.equal(tokens[lo:hi].long(), want)
    assert not bool(logprobs.any())


def test_sizes_that_do_not_fit_in_int32_are_refused(ds):
    four, one = i32(0, 0, 0, 0), i32(0)
    table, pages = torch.zeros(4, 8, dtype=torch.int32, device="cuda"), i32(1, 2, 3)
    flags = torch.zeros(4, dtype=torch.uint8, device="cuda")
    wide = torch.zeros(0, 2**32 + 8, dtype=torch.int32, device="cuda")
    none = i32()
    for t, lengths, done, page in ((table, four, flags, 2**32 + 16), (wide, none, flags[:0], 16)):
        with pytest.raises(ValueError):
            ds.block_table_extend(t, lengths, lengths, pages, one, page)
        with pytest.raises(ValueError):
            ds.slot_map(t, lengths, lengths, page, 5)
        with pytest.raises(ValueError):
            ds.block_table_release(t, lengths, done, pages, one, page)
