"""Calls of several launches from several host threads on one stream: each
call's launches hand rows to each other through the stream's workspace, and must
get their own.  And the same calls on several streams at once."""
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


@pytest.fixture(autouse=True)
def short_turns():
    """Threads take turns between nearly all instructions."""
    was = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    yield
    sys.setswitchinterval(was)


def together(works, repeats, streams=None):
    """Runs work(stream) of each in a thread of its own, `repeats` times, all
    starting together; works return lists of tensors."""
    streams = streams or [torch.cuda.current_stream()] * len(works)
    start, got, failed = threading.Barrier(len(works)), [None] * len(works), []

    def body(i):
        try:
            start.wait()
            got[i] = [works[i](streams[i]) for _ in range(repeats)]
        except BaseException as e:   # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(len(works))]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    return got


def draw(ds, rows, vocab, seed, dtype):
    """A batch whose rows are partly left to the second launch: flat ones with
    top-p and wide top-k beside short lists and races of all tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 1.5).to(dtype)
    q = torch.empty(rows, vocab, device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    kinds = [(0, 0.9), (50, 1.0), (3000, 1.0), (0, 1.0), (0, 0.5)]
    k = torch.tensor([kinds[(r + seed) % 5][0] for r in range(rows)], dtype=torch.int32, device="cuda")
    p = torch.tensor([kinds[(r + seed) % 5][1] for r in range(rows)], device="cuda")
    out = iter([(torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda"))
                for _ in range(64)])

    def work(stream):
        tokens, logprobs = next(out)
        return list(ds.sample_tokens(x, q, top_k=k, top_p=p, out=tokens, logprobs=logprobs, stream=stream))
    return work


def tables(ds, rows, seed):
    """A step's tables, slots and release of more rows than one launch takes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width, page = 6, 8
    i32 = lambda hi: torch.randint(0, hi, (rows,), generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    cached, fresh = i32(page * 3), i32(page * 3)
    done = (i32(4) == 0).to(torch.uint8)
    pool = rows * width
    stack = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    height = torch.tensor([pool - rows], dtype=torch.int32, device="cuda")
    tokens = int(fresh.sum()) + 3
    new = lambda n, dtype: torch.full((n,), -7, dtype=dtype, device="cuda")  # noqa: E731
    sets = iter([{"table": torch.full((rows, width), -1, dtype=torch.int32, device="cuda"), "stack": stack.clone(),
                  "granted": new(rows, torch.uint8), "left": new(1, torch.int32), "back": new(1, torch.int32),
                  "out": (new(rows + 1, torch.int32), new(tokens, torch.int64), new(tokens, torch.int32),
                          new(tokens, torch.int32))} for _ in range(40)])

    def work(stream):
        s = next(sets)
        ds.block_table_extend(s["table"], cached, fresh, s["stack"], height, page, granted=s["granted"],
                              left=s["left"], stream=stream)
        ds.slot_map(s["table"], cached, fresh, page, tokens, granted=s["granted"], out=s["out"], stream=stream)
        ds.block_table_release(s["table"], cached, done, s["stack"], s["left"], page, left=s["back"], stream=stream)
        return [s["table"], s["granted"], s["left"], *s["out"], s["stack"], s["back"]]
    return work


def same(got, want):
    return len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def batches(ds, kind):
    if kind == "draw":
        return [draw(ds, rows, 40000, seed, dtype)
                for rows, seed, dtype in ((310, 1, torch.float32), (500, 2, torch.bfloat16), (410, 3, torch.float16))]
    if kind == "tables":
        return [tables(ds, rows, seed) for rows, seed in ((5000, 4), (20001, 5), (9000, 6))]
    return [draw(ds, 330, 40000, 7, torch.bfloat16), tables(ds, 7000, 8), draw(ds, 450, 40000, 9, torch.float32),
            tables(ds, 15000, 10)]


@pytest.mark.parametrize("kind", ["draw", "tables", "both"])
def test_threads_on_one_stream(ds, kind):
    works = batches(ds, kind)
    want = [[t.clone() for t in work(None)] for work in works]
    for runs, first in zip(together(works, 20), want):
        assert all(same(run, first) for run in runs)
    assert ds.device_status() == 0


@pytest.mark.parametrize("kind", ["draw", "both"])
def test_threads_on_streams_of_their_own(ds, kind):
    works = batches(ds, kind)
    want = [[t.clone() for t in work(None)] for work in works]
    streams = [torch.cuda.Stream() for _ in works]
    for runs, first in zip(together(works, 12, streams), want):
        assert all(same(run, first) for run in runs)
    for s in streams:
        assert ds.device_status(s) == 0
        ds.stream_release(s)


def test_one_thread_and_two_streams(ds):
    """Second launches of two streams beside each other's first ones."""
    a, b = batches(ds, "draw")[:2]
    want = [[t.clone() for t in work(None)] for work in (a, b)]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(a(streams[0]), b(streams[1])) for _ in range(20)]
    torch.cuda.synchronize()
    for ran in got:
        assert same(ran[0], want[0]) and same(ran[1], want[1])
    for s in streams:
        ds.stream_release(s)


def test_release_beside_calls(ds):
    """A workspace released by one thread while another's calls use the stream."""
    work = draw(ds, 320, 40000, 11, torch.bfloat16)
    want = [t.clone() for t in work(None)]
    stream = torch.cuda.Stream()
    got = together([work, lambda s: ds.stream_release(s)], 40, [stream, stream])[0]
    assert all(same(run, want) for run in got)
    ds.stream_release(stream)
