"""What a call makes for itself (outputs that it was not given, scratch) is
memory of the stream that the call runs on: the current stream's allocator hands
out blocks whose last owner may still run there."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def calls(ds):
    """(name, call with a stream) of every entry point, without the tensors that it can make itself."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, gate, state = r(2, 100, 64), r(2, 100, 64), r(2, 64)
    y, _ = ds.gated_scan(x, gate, initial=state, kind="sigmoid")
    ids = torch.randint(0, 8, (50, 2), generator=g, device="cuda")
    _, _, order, places = ds.expert_sort(ids, 8)
    tokens, weights = r(50, 64), torch.rand(50, 2, generator=g, device="cuda")
    rows = ds.expert_dispatch(tokens, places, order, out=torch.zeros(order.numel(), 64, device="cuda"))
    n = torch.randint(-1000, 1000, (5000,), generator=g, device="cuda").to(torch.int32)
    heads = (torch.rand(5000, generator=g, device="cuda") < 0.01).to(torch.uint8)
    assert (order > -2).all()                                 # every row is written
    table, cached, fresh = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), i32(3, 0, 17), i32(1, 20, 4)
    pages, free, done = torch.arange(16, dtype=torch.int32, device="cuda"), i32(16), torch.tensor([0, 1, 1], dtype=torch.uint8, device="cuda")
    logits, noise = r(4, 1000), torch.rand(4, 1000, generator=g, device="cuda") + 0.1
    clipped = [torch.zeros_like(x), torch.zeros_like(gate)]
    host = torch.arange(1000, dtype=torch.int32).pin_memory()
    return [
        ("gated_scan", lambda s: ds.gated_scan(x, gate, initial=state, kind="sigmoid", stream=s)),
        ("gated_scan_backward", lambda s: ds.gated_scan_backward(x, x, gate, y, initial=state, kind="sigmoid", stream=s)),
        ("expert_sort", lambda s: ds.expert_sort(ids, 8, stream=s)),
        ("expert_dispatch", lambda s: ds.expert_dispatch(tokens, places, order, stream=s)),
        ("expert_combine", lambda s: ds.expert_combine(rows, places, weights, stream=s)),
        ("expert_combine_backward", lambda s: ds.expert_combine_backward(tokens, rows, places, weights, order, stream=s)),
        ("grad_norm", lambda s: ds.grad_norm([x, gate], stream=s)),
        ("clip_grad_norm", lambda s: ds.clip_grad_norm([x, gate], 1.0, out=clipped, stream=s)[0]),
        ("scan_inclusive", lambda s: ds.scan_inclusive(n, stream=s)),
        ("scan_exclusive_carry", lambda s: ds.scan_exclusive_carry(n, n[:1], stream=s)),
        ("reduce", lambda s: ds.reduce(n, stream=s)),
        ("sharded_scan", lambda s: ds.sharded_scan(n, stream=s)),
        ("sharded_compact", lambda s: ds.sharded_compact(n, threshold=0, stream=s)),
        ("segmented_scan_inclusive", lambda s: ds.segmented_scan_inclusive(n, heads, stream=s)),
        ("compact", lambda s: ds.compact(n, heads, stream=s)),
        ("compact_greater", lambda s: ds.compact_greater(n, 0, stream=s)),
        ("bracket_scan", lambda s: ds.bracket_scan(n, stream=s)),
        ("split_bit", lambda s: ds.split_bit(n, 3, stream=s)),
        ("radix_sort", lambda s: ds.radix_sort(n, stream=s)),
        ("radix_sort_digits", lambda s: ds.radix_sort_digits(n, stream=s)),
        ("block_table_extend", lambda s: ds.block_table_extend(table, cached, fresh, pages, free, 16, stream=s)),
        ("slot_map", lambda s: ds.slot_map(table, cached, fresh, 16, 30, stream=s)),
        ("block_table_release", lambda s: ds.block_table_release(table, cached, done, pages, free, 16, stream=s)),
        ("sample_tokens", lambda s: ds.sample_tokens(logits, noise, stream=s)),
        ("scan_host", lambda s: ds.scan_host(host, stream=s)),
    ]


def tensors(name, result):
    """What of a call's results is defined."""
    got = [v for v in (result if isinstance(result, (list, tuple)) else [result]) if v is not None]
    if "compact" in name:
        got[0] = got[0][: int(got[1])]
    return got


def test_made_on_the_calls_stream(ds, monkeypatch):
    """Every tensor that a call makes, on a stream object and on a handle; on the current stream without."""
    made, empty, like = [], torch.empty, torch.empty_like
    side = torch.cuda.Stream()

    def seen(make):
        def wrapped(*a, **k):
            t = make(*a, **k)
            if t.is_cuda:
                made.append(torch.cuda.current_stream().cuda_stream)
            return t
        return wrapped

    todo = calls(ds)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", seen(empty))
    monkeypatch.setattr(torch, "empty_like", seen(like))
    here = torch.cuda.current_stream().cuda_stream
    for name, call in todo:
        for stream, want in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (None, here), (torch.cuda.current_stream(), here)):
            if isinstance(stream, int) and name == "scan_host":
                continue                                       # takes a Stream
            made.clear()
            got = call(stream)
            torch.cuda.synchronize()
            assert made and set(made) == {want}, (name, stream)
            del got
    for handle in (0, 1):                                      # the legacy default stream's
        ds.grad_norm([torch.ones(100, device="cuda")], stream=handle)
        torch.cuda.synchronize()


def test_a_block_that_the_current_stream_still_writes(ds):
    """Blocks freed on the current stream while it has yet to write them: a call
    on another stream, whose inputs are long ready, keeps its result."""
    side = torch.cuda.Stream()
    for name, call in calls(ds):
        result = call(None)
        torch.cuda.synchronize()
        sizes = [(v.shape, v.dtype) for v in result] if isinstance(result, (list, tuple)) else [(result.shape, result.dtype)]
        want = [v.clone() for v in tensors(name, result)]
        del result
        torch.cuda.synchronize()
        # the shapes that the call will ask for, to be written late
        torch.cuda._sleep(200_000_000)
        late = [torch.empty(size, dtype=dtype, device="cuda") for size, dtype in sizes for _ in range(2)]
        for v in late:
            v.fill_(77)
        del late, v
        got = call(side)
        torch.cuda.synchronize()
        for a, b in zip(tensors(name, got), want):
            assert torch.equal(a, b), name
