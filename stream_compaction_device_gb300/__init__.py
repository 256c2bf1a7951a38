"""devscan for GB300: device-wide prefix scan, stream compaction and the
radix one-bit split as hand-written sm_103a CUDA kernels behind a C ABI.

The functions below take CUDA tensors (PyTorch is used for device memory
and streams only), pass their device pointers and the current CUDA stream
to ``libdevscan.so`` and return.  All work is asynchronous on that stream, or
on the one that ``stream`` names (an object or a handle).  What a call makes for
itself, outputs that it was not given among it, is memory of the stream that it
runs on; that the tensors which it was given are ready there, and that what it
returns is ready where it is used, the caller sees to, as with any torch
operation on two streams.  No call is an autograd function: results carry no
graph, and the calls of a model's layers warn where a gradient is lost with that.
``scan_host`` is the host-buffer entry: the library copies a pinned host
array to the device, scans it and copies the result back.
"""
from __future__ import annotations

import array
import contextlib
import functools
import operator
import warnings

import torch

from . import _lib
from ._lib import DevscanError, OPS, load

__all__ = ["scan_inclusive", "scan_exclusive", "scan_inclusive_carry", "scan_exclusive_carry", "reduce",
           "sharded_scan", "exchange_totals", "compact", "split_bit", "radix_sort", "radix_sort_digits", "scan_host",
           "compact_greater", "bracket_scan", "segmented_scan_inclusive", "segmented_scan_exclusive",
           "sample_tokens", "block_table_extend", "slot_map", "block_table_release",
           "gated_scan", "gated_scan_backward", "expert_sort", "expert_dispatch", "expert_combine",
           "expert_combine_backward", "grad_norm", "clip_grad_norm",
           "device_status", "set_carry_mode", "stream_release", "selftest_stalled_wait", "DevscanError",
           "load"]

_SUFFIX = {torch.int32: "i32", torch.float32: "f32"}
if hasattr(torch, "uint32"):
    _SUFFIX[torch.uint32] = "u32"


_INT32_MAX = 2**31 - 1
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream) -> int:
    if stream is None:
        # The current device's current stream without a Stream object: the
        # object takes longer to make than a small call's launch.
        if _RAW_STREAM is not None:
            return _RAW_STREAM(torch._C._cuda_getDevice())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream):
    """Context in which torch works on that stream (None: on the current one)."""
    if stream is None or _stream_handle(stream) == _stream_handle(None):
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)                 # 0 and 1 are the legacy default stream
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _made_on(stream, make, *args, **kwargs) -> torch.Tensor:
    """``make(*args, **kwargs)`` in the memory of that stream.  A block of the
    current stream's may still be in use there by kernels of its last owner, and
    goes to its next one as soon as it is freed, while the call runs on another."""
    with _on(stream):
        return make(*args, **kwargs)


def _empty_on(stream):
    """``torch.empty`` for what a call on that stream makes."""
    return functools.partial(_made_on, stream, torch.empty)


def _check_cuda(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _scan(direction: str, x: torch.Tensor, out, op: str, stream, dtype_override=None):
    _check_cuda(x, "x")
    suffix = dtype_override or _SUFFIX.get(x.dtype)
    if suffix is None:
        raise TypeError(f"unsupported dtype {x.dtype} (int32, uint32, float32)")
    if out is None:
        out = torch.empty_like(x) if stream is None else _made_on(stream, torch.empty_like, x)
    _check_cuda(out, "out")
    if out.numel() != x.numel() or out.dtype != x.dtype:
        raise ValueError("out must match x in size and dtype")
    fn = getattr(load(), f"scan_{direction}_{suffix}")
    _lib.check(fn(x.data_ptr(), out.data_ptr(), x.numel(), OPS[op], _stream_handle(stream)),
               f"scan_{direction}_{suffix}")
    return out


def scan_inclusive(x: torch.Tensor, out: torch.Tensor | None = None, op: str = "add", stream=None,
                   as_uint32: bool = False) -> torch.Tensor:
    """y[i] = x[0] op ... op x[i].  ``as_uint32`` treats an int32 tensor's
    bits as uint32 (unsigned max)."""
    return _scan("inclusive", x, out, op, stream, "u32" if as_uint32 else None)


def scan_exclusive(x: torch.Tensor, out: torch.Tensor | None = None, op: str = "add", stream=None,
                   as_uint32: bool = False) -> torch.Tensor:
    """z[i] = x[0] op ... op x[i-1]; z[0] = identity of op."""
    return _scan("exclusive", x, out, op, stream, "u32" if as_uint32 else None)


def _carry_scan(direction: str, x: torch.Tensor, carry: torch.Tensor | None, out, op: str, stream,
                dtype_override=None):
    _check_cuda(x, "x")
    suffix = dtype_override or _SUFFIX.get(x.dtype)
    if suffix is None:
        raise TypeError(f"unsupported dtype {x.dtype} (int32, uint32, float32)")
    if carry is not None:
        _check_cuda(carry, "carry")
        if carry.dtype != x.dtype or carry.numel() < 1:
            raise ValueError("carry must be a device tensor of x's dtype holding one element")
    if out is None:
        out = torch.empty_like(x) if stream is None else _made_on(stream, torch.empty_like, x)
    _check_cuda(out, "out")
    if out.numel() != x.numel() or out.dtype != x.dtype:
        raise ValueError("out must match x in size and dtype")
    name = f"scan_{direction}_carry_{suffix}"
    _lib.check(getattr(load(), name)(x.data_ptr(), out.data_ptr(), x.numel(), OPS[op],
                                     None if carry is None else carry.data_ptr(), _stream_handle(stream)), name)
    return out


def scan_inclusive_carry(x: torch.Tensor, carry: torch.Tensor | None, out: torch.Tensor | None = None,
                         op: str = "add", stream=None, as_uint32: bool = False) -> torch.Tensor:
    """y[i] = carry op x[0] op ... op x[i], ``carry`` a one-element device
    tensor (None: the identity)."""
    return _carry_scan("inclusive", x, carry, out, op, stream, "u32" if as_uint32 else None)


def scan_exclusive_carry(x: torch.Tensor, carry: torch.Tensor | None, out: torch.Tensor | None = None,
                         op: str = "add", stream=None, as_uint32: bool = False) -> torch.Tensor:
    """z[i] = carry op x[0] op ... op x[i-1]; z[0] = carry."""
    return _carry_scan("exclusive", x, carry, out, op, stream, "u32" if as_uint32 else None)


def reduce(x: torch.Tensor, op: str = "add", out: torch.Tensor | None = None, stream=None,
           as_uint32: bool = False) -> torch.Tensor:
    """Fold of all of ``x`` under ``op`` into a one-element device tensor
    (the identity for an empty ``x``)."""
    _check_cuda(x, "x")
    suffix = "u32" if as_uint32 else _SUFFIX.get(x.dtype)
    if suffix is None:
        raise TypeError(f"unsupported dtype {x.dtype} (int32, uint32, float32)")
    empty = torch.empty if stream is None else _empty_on(stream)
    if out is None:
        out = empty(1, dtype=x.dtype, device=x.device)
    _check_cuda(out, "out")
    if out.dtype != x.dtype or out.numel() < 1:
        raise ValueError("out must hold one element of x's dtype")
    name = f"reduce_{suffix}"
    _lib.check(getattr(load(), name)(x.data_ptr() if x.numel() else None, x.numel(), OPS[op], out.data_ptr(),
                                     _stream_handle(stream)), name)
    return out


def exchange_totals(total: torch.Tensor, group=None) -> torch.Tensor:
    """All-gather of one total per rank: returns a tensor of ``world_size``
    elements on ``total``'s device, element r from rank r (the one exchange
    step of a sharded scan; NCCL for device tensors, gloo for host
    tensors).  A single process returns ``total`` itself."""
    import torch.distributed as dist
    if not (dist.is_available() and dist.is_initialized()):
        return total.reshape(1)
    world = dist.get_world_size(group)
    totals = torch.empty(world, dtype=total.dtype, device=total.device)
    dist.all_gather_into_tensor(totals, total.reshape(1).contiguous(), group=group)
    return totals


def sharded_scan(shard: torch.Tensor, out: torch.Tensor | None = None, inclusive: bool = False, op: str = "add",
                 group=None, stream=None, as_uint32: bool = False) -> torch.Tensor:
    """This rank's part of the scan of an array split into contiguous shards,
    shard r on rank r of ``group`` (in rank order).  The library folds this
    shard's total, the ranks exchange their totals (one all-gather of one
    element each), the library folds the totals of the ranks before this
    one into a carry and scans the shard from it.  Every rank calls it; the
    ranks' outputs, concatenated in rank order, are the scan of the whole
    array."""
    import torch.distributed as dist
    rank = dist.get_rank(group) if dist.is_available() and dist.is_initialized() else 0
    total = reduce(shard, op, stream=stream, as_uint32=as_uint32)
    with _on(stream):
        totals = exchange_totals(total, group)
    carry = reduce(totals[:rank], op, stream=stream, as_uint32=as_uint32)
    fn = scan_inclusive_carry if inclusive else scan_exclusive_carry
    return fn(shard, carry, out, op=op, stream=stream, as_uint32=as_uint32)


def sharded_compact(values: torch.Tensor, flags: torch.Tensor | None = None, threshold: int | None = None,
                    out: torch.Tensor | None = None, group=None, stream=None):
    """This rank's part of the order-preserving compaction of an array split
    into contiguous shards, shard r on rank r of ``group`` (in rank order).
    The library compacts the shard (the values whose flag is nonzero, or the
    values greater than ``threshold``), the ranks exchange their kept counts
    (one all-gather of one count each), and the library folds the counts of
    the ranks before this one into this rank's output offset and all of them
    into the total.  Returns (out, count, offset, total), all on the device:
    the first ``count`` elements of ``out`` are this rank's kept values,
    elements offset .. offset + count - 1 of the whole compaction."""
    import torch.distributed as dist
    if (flags is None) == (threshold is None):
        raise ValueError("give either flags or a threshold")
    rank = dist.get_rank(group) if dist.is_available() and dist.is_initialized() else 0
    if threshold is None:
        out, count = compact(values, flags, out, stream=stream)
    else:
        out, count = compact_greater(values, threshold, out, stream=stream)
    with _on(stream):
        counts = exchange_totals(count, group)
    offset = reduce(counts[:rank], "add", stream=stream)
    total = reduce(counts, "add", stream=stream)
    return out, count, offset, total


def _segscan(direction: str, x: torch.Tensor, heads: torch.Tensor, out, op: str, stream, dtype_override=None):
    _check_cuda(x, "x")
    _check_cuda(heads, "heads")
    suffix = dtype_override or _SUFFIX.get(x.dtype)
    if suffix is None:
        raise TypeError(f"unsupported dtype {x.dtype} (int32, uint32, float32)")
    if heads.dtype != torch.uint8 or heads.numel() != x.numel():
        raise ValueError("heads must be a uint8 tensor of x's length")
    if out is None:
        out = torch.empty_like(x) if stream is None else _made_on(stream, torch.empty_like, x)
    _check_cuda(out, "out")
    if out.numel() != x.numel() or out.dtype != x.dtype:
        raise ValueError("out must match x in size and dtype")
    name = f"segmented_scan_{direction}_{suffix}"
    _lib.check(getattr(load(), name)(x.data_ptr(), heads.data_ptr(), out.data_ptr(), x.numel(), OPS[op],
                                     _stream_handle(stream)), name)
    return out


def segmented_scan_inclusive(x: torch.Tensor, heads: torch.Tensor, out: torch.Tensor | None = None,
                             op: str = "add", stream=None, as_uint32: bool = False) -> torch.Tensor:
    """Inclusive scan restarted at every nonzero ``heads[i]`` (element 0
    always starts a segment)."""
    return _segscan("inclusive", x, heads, out, op, stream, "u32" if as_uint32 else None)


def segmented_scan_exclusive(x: torch.Tensor, heads: torch.Tensor, out: torch.Tensor | None = None,
                             op: str = "add", stream=None, as_uint32: bool = False) -> torch.Tensor:
    """Exclusive scan restarted at every nonzero ``heads[i]``: the identity
    at each segment start."""
    return _segscan("exclusive", x, heads, out, op, stream, "u32" if as_uint32 else None)


def compact(values: torch.Tensor, flags: torch.Tensor, out: torch.Tensor | None = None,
            count: torch.Tensor | None = None, stream=None):
    """Order-preserving compaction.  Returns (out, count): the first
    ``count`` elements of ``out`` are the values whose flag is nonzero.
    Both stay on the device; nothing synchronises."""
    _check_cuda(values, "values")
    _check_cuda(flags, "flags")
    if values.dtype != torch.int32 or flags.dtype != torch.uint8:
        raise TypeError("values must be int32 and flags uint8")
    if values.numel() != flags.numel():
        raise ValueError("values and flags differ in length")
    if out is None:
        out = torch.empty_like(values) if stream is None else _made_on(stream, torch.empty_like, values)
    empty = torch.empty if stream is None else _empty_on(stream)
    if count is None:
        count = empty(1, dtype=torch.int32, device=values.device)
    _check_cuda(out, "out")
    _check_cuda(count, "count")
    _lib.check(load().compact_i32(values.data_ptr(), flags.data_ptr(), out.data_ptr(), count.data_ptr(),
                                  values.numel(), _stream_handle(stream)), "compact_i32")
    return out, count


def compact_greater(values: torch.Tensor, threshold: int, out: torch.Tensor | None = None,
                    count: torch.Tensor | None = None, stream=None):
    """Order-preserving compaction of the int32 values greater than
    ``threshold`` (signed), the predicate evaluated on the device.  Returns
    (out, count) as :func:`compact`."""
    _check_cuda(values, "values")
    if values.dtype != torch.int32:
        raise TypeError("values must be int32")
    if out is None:
        out = torch.empty_like(values) if stream is None else _made_on(stream, torch.empty_like, values)
    empty = torch.empty if stream is None else _empty_on(stream)
    if count is None:
        count = empty(1, dtype=torch.int32, device=values.device)
    _check_cuda(out, "out")
    _check_cuda(count, "count")
    _lib.check(load().compact_gt_i32(values.data_ptr(), int(threshold), out.data_ptr(), count.data_ptr(),
                                     values.numel(), _stream_handle(stream)), "compact_gt_i32")
    return out, count


def bracket_scan(weights: torch.Tensor, out: torch.Tensor | None = None, result: torch.Tensor | None = None,
                 store: bool = True, stream=None):
    """Inclusive int32 add-scan of +1/-1 bracket weights with the bracket
    check in the same pass.  Returns (out or None, result): result[0] is 1
    when some running sum is negative, result[1] the final sum.  With
    ``store=False`` the scan is not written (the check alone)."""
    _check_cuda(weights, "weights")
    if weights.dtype != torch.int32:
        raise TypeError("weights must be int32")
    if store and out is None:
        out = torch.empty_like(weights) if stream is None else _made_on(stream, torch.empty_like, weights)
    if not store:
        out = None
    empty = torch.empty if stream is None else _empty_on(stream)
    if result is None:
        result = empty(2, dtype=torch.int32, device=weights.device)
    _check_cuda(result, "result")
    if out is not None:
        _check_cuda(out, "out")
    _lib.check(load().bracket_scan_i32(weights.data_ptr(), None if out is None else out.data_ptr(),
                                       result.data_ptr(), weights.numel(), _stream_handle(stream)),
               "bracket_scan_i32")
    return out, result


def split_bit(keys: torch.Tensor, bit: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Stable partition of 32-bit keys by bit ``bit``: zeros first."""
    _check_cuda(keys, "keys")
    if keys.element_size() != 4 or keys.is_floating_point():
        raise TypeError("keys must be a 32-bit integer tensor (bits read as uint32)")
    if out is None:
        out = torch.empty_like(keys) if stream is None else _made_on(stream, torch.empty_like, keys)
    _check_cuda(out, "out")
    _lib.check(load().split_bit_u32(keys.data_ptr(), out.data_ptr(), int(bit), keys.numel(),
                                    _stream_handle(stream)), "split_bit_u32")
    return out


def radix_sort(keys: torch.Tensor, tmp: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """In-place ascending sort of 32-bit keys (bits read as uint32) by 32
    one-bit splits; ``tmp`` is a same-size scratch tensor."""
    _check_cuda(keys, "keys")
    if keys.element_size() != 4 or keys.is_floating_point():
        raise TypeError("keys must be a 32-bit integer tensor (bits read as uint32)")
    if tmp is None:
        tmp = torch.empty_like(keys) if stream is None else _made_on(stream, torch.empty_like, keys)
    _check_cuda(tmp, "tmp")
    _lib.check(load().radix_sort_u32(keys.data_ptr(), tmp.data_ptr(), keys.numel(), _stream_handle(stream)),
               "radix_sort_u32")
    return keys


def radix_sort_digits(keys: torch.Tensor, tmp: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """In-place ascending sort of 32-bit keys (bits read as uint32) by 4
    passes of 8-bit digits; ``tmp`` is a same-size scratch tensor."""
    _check_cuda(keys, "keys")
    if keys.element_size() != 4 or keys.is_floating_point():
        raise TypeError("keys must be a 32-bit integer tensor (bits read as uint32)")
    if tmp is None:
        tmp = torch.empty_like(keys) if stream is None else _made_on(stream, torch.empty_like, keys)
    _check_cuda(tmp, "tmp")
    _lib.check(load().radix_sort_digits_u32(keys.data_ptr(), tmp.data_ptr(), keys.numel(),
                                            _stream_handle(stream)), "radix_sort_digits_u32")
    return keys


def _check_vector(t: torch.Tensor, name: str, dtype: torch.dtype, size: int) -> int:
    """A contiguous CUDA tensor of that type and size; returns its address."""
    if t.is_cuda and t.dtype is dtype and t.numel() == size and t.is_contiguous():
        return t.data_ptr()
    _check_cuda(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    raise ValueError(f"{name} must hold {size} elements")


def _check_matrix(t: torch.Tensor, name: str) -> int:
    """A 2-d CUDA tensor whose rows are contiguous; returns its row stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    rows, width = t.shape
    stride, step = t.stride()
    if width > 1 and step != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    if rows <= 1 or width == 0:
        return max(width, 1)
    if stride < width:
        raise ValueError(f"{name}'s rows must not overlap")
    return stride


def _check_table(table: torch.Tensor, page_size: int) -> int:
    stride = _check_matrix(table, "table")
    if table.dtype != torch.int32:
        raise TypeError("table must be int32")
    if not 1 <= page_size <= _INT32_MAX:
        raise ValueError("page_size must be positive and fit in int32")
    if table.shape[1] > _INT32_MAX:
        raise ValueError("table's rows must have at most INT32_MAX entries")
    return stride


def block_table_extend(table: torch.Tensor, cached: torch.Tensor, fresh: torch.Tensor, pages: torch.Tensor,
                       free: torch.Tensor, page_size: int, granted: torch.Tensor | None = None,
                       left: torch.Tensor | None = None, stream=None):
    """Open the pages that each row's ``fresh`` new tokens need beyond its
    ``cached`` ones: they are taken from the top of the stack ``pages[:free]``
    in row order, while it lasts, and written into the rows of ``table`` (int32,
    in place).  Returns (granted, left): uint8 per row, 1 where the row's
    tokens have their pages, and the stack's height afterwards (one int32,
    another tensor than ``free``)."""
    stride = _check_table(table, page_size)
    rows, width = table.shape
    pool = pages.numel()
    empty = torch.empty if stream is None else _empty_on(stream)
    if granted is None:
        granted = empty(rows, dtype=torch.uint8, device=table.device)
    if left is None:
        left = empty(1, dtype=torch.int32, device=table.device)
    status = load().block_table_extend_i32(
        table.data_ptr(), stride, rows, width, _check_vector(cached, "cached", torch.int32, rows),
        _check_vector(fresh, "fresh", torch.int32, rows), int(page_size),
        _check_vector(pages, "pages", torch.int32, pool), pool, _check_vector(free, "free", torch.int32, 1),
        _check_vector(granted, "granted", torch.uint8, rows), _check_vector(left, "left", torch.int32, 1),
        _stream_handle(stream))
    if status:
        _lib.check(status, "block_table_extend_i32")
    return granted, left


def slot_map(table: torch.Tensor, cached: torch.Tensor, fresh: torch.Tensor, page_size: int, tokens: int,
             granted: torch.Tensor | None = None, out=None, stream=None):
    """Places of the new tokens, packed in row order and padded with -1 to
    ``tokens``.  Returns (starts, slots, positions, rows): int32 starts of
    every row and the total, and for each token its int64 slot in the paged
    cache, its int32 position in its row, and its row.  ``granted`` (uint8)
    leaves out the rows whose flag is 0; ``out`` passes the four tensors."""
    stride = _check_table(table, page_size)
    rows, width = table.shape
    tokens = int(tokens)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    empty = torch.empty if stream is None else _empty_on(stream)
    if out is None:
        new = lambda n, dtype: empty(n, dtype=dtype, device=table.device)  # noqa: E731
        out = (new(rows + 1, torch.int32), new(tokens, torch.int64), new(tokens, torch.int32),
               new(tokens, torch.int32))
    starts, slots, positions, row_ids = out
    status = load().slot_map_i32(
        table.data_ptr(), stride, rows, width, _check_vector(cached, "cached", torch.int32, rows),
        _check_vector(fresh, "fresh", torch.int32, rows),
        None if granted is None else _check_vector(granted, "granted", torch.uint8, rows), int(page_size), tokens,
        _check_vector(starts, "starts", torch.int32, rows + 1), _check_vector(slots, "slots", torch.int64, tokens),
        _check_vector(positions, "positions", torch.int32, tokens), _check_vector(row_ids, "rows", torch.int32, tokens),
        _stream_handle(stream))
    if status:
        _lib.check(status, "slot_map_i32")
    return starts, slots, positions, row_ids


def block_table_release(table: torch.Tensor, cached: torch.Tensor, done: torch.Tensor, pages: torch.Tensor,
                        free: torch.Tensor, page_size: int, left: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Give the pages of the rows with a nonzero ``done`` (uint8) back: their
    entries go on top of the stack ``pages[:free]`` in row order.  Returns the
    stack's height afterwards (one int32, another tensor than ``free``).  The
    table is not changed; the caller sets the ended rows' lengths to 0."""
    stride = _check_table(table, page_size)
    rows, width = table.shape
    pool = pages.numel()
    empty = torch.empty if stream is None else _empty_on(stream)
    if left is None:
        left = empty(1, dtype=torch.int32, device=table.device)
    status = load().block_table_release_i32(
        table.data_ptr(), stride, rows, width, _check_vector(cached, "cached", torch.int32, rows),
        _check_vector(done, "done", torch.uint8, rows), int(page_size),
        _check_vector(pages, "pages", torch.int32, pool), pool, _check_vector(free, "free", torch.int32, 1),
        _check_vector(left, "left", torch.int32, 1), _stream_handle(stream))
    if status:
        _lib.check(status, "block_table_release_i32")
    return left


_SAMPLE_SYMBOL = {torch.float32: "sample_tokens_f32", torch.float16: "sample_tokens_f16",
                  torch.bfloat16: "sample_tokens_bf16"}


def sample_tokens(logits: torch.Tensor, noise: torch.Tensor | None = None, temperature: torch.Tensor | None = None,
                  top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                  min_p: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  logprobs: torch.Tensor | None = None, stream=None):
    """Draw one token from each row of ``logits`` (fp32, fp16 or bf16, rows
    contiguous) with that row's ``temperature``, ``top_k`` (int32), ``top_p``
    and ``min_p`` (fp32, each optional), by an exponential race with the given
    ``noise`` (fp32 of the logits' shape, positive, Exp(1)).  Without noise, or
    where the temperature is 0, the largest logit is taken.  Returns (tokens,
    logprobs): int32 per row (-1 for a row with nothing above -inf) and fp32
    log-probabilities under the truncated distribution."""
    stride = _check_matrix(logits, "logits")
    rows, vocab = logits.shape
    if logits.dtype not in _SAMPLE_SYMBOL:
        raise TypeError(f"unsupported dtype {logits.dtype} (float32, float16, bfloat16)")
    noise_stride = vocab
    if noise is not None:
        noise_stride = _check_matrix(noise, "noise")
        if noise.dtype != torch.float32:
            raise TypeError("noise must be float32")
        if noise.shape != logits.shape:
            raise ValueError("noise must have the logits' shape")
    empty = torch.empty if stream is None else _empty_on(stream)
    if out is None:
        out = empty(rows, dtype=torch.int32, device=logits.device)
    if logprobs is None:
        logprobs = empty(rows, dtype=torch.float32, device=logits.device)
    f32, i32 = torch.float32, torch.int32
    status = getattr(load(), _SAMPLE_SYMBOL[logits.dtype])(
        logits.data_ptr(), rows, vocab, stride, None if noise is None else noise.data_ptr(), noise_stride,
        None if temperature is None else _check_vector(temperature, "temperature", f32, rows),
        None if top_k is None else _check_vector(top_k, "top_k", i32, rows),
        None if top_p is None else _check_vector(top_p, "top_p", f32, rows),
        None if min_p is None else _check_vector(min_p, "min_p", f32, rows),
        _check_vector(out, "out", i32, rows), _check_vector(logprobs, "logprobs", f32, rows), _stream_handle(stream))
    if status:
        _lib.check(status, _SAMPLE_SYMBOL[logits.dtype])
    return out, logprobs


_VALUES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
_F32, _I32 = torch.float32, torch.int32
_GATES = _lib.GATES


def _value_suffix(t: torch.Tensor) -> str:
    suffix = _VALUES.get(t.dtype)
    if suffix is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32, float16, bfloat16)")
    return suffix


def _no_graph(name: str, *tensors) -> None:
    """Tells of a gradient that is lost: the calls are no autograd functions."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                warnings.warn(f"{name} has no autograd graph: its result does not lead back to tensors that require a "
                              "gradient (call it in the forward and backward of a torch.autograd.Function, or under "
                              "torch.no_grad)", stacklevel=3)
                return


def _device_of(t: torch.Tensor, name: str) -> int:
    """The device of a call that begins with that tensor: the current one,
    whose stream it takes."""
    here = t.get_device()
    if here < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if here != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current device")
    return here


def _vector(t, name: str, dtype: torch.dtype, size: int, here: int):
    """Address of a contiguous tensor of that type, size and device; None for
    None."""
    if t is None:
        return None
    if t.get_device() == here and t.dtype is dtype and t.numel() == size and t.is_contiguous():
        return t.data_ptr()
    _device_of(t, name)
    _check_vector(t, name, dtype, size)
    raise ValueError(f"{name} must be on the current device")


def _token_array(t: torch.Tensor, name: str, shape, dtype, here: int):
    """(address, row stride, token stride) of a tensor [rows, tokens, channels]
    or [tokens, channels] with neighbouring channels."""
    strides = t.stride()
    if t.get_device() == here and t.dtype is dtype and t.shape == shape and (strides[-1] == 1 or shape[-1] == 1):
        return t.data_ptr(), strides[0] if len(strides) == 3 else 0, strides[-2]
    if t.get_device() != here:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    raise ValueError(f"{name}'s channels must be contiguous")


def _gated_rows(x: torch.Tensor, gate: torch.Tensor, starts, kind: str):
    """(rows, tokens, channels, the kind's number, whether the gates are fp32
    beside 16 bits)."""
    number = _GATES.get(kind)
    if number is None:
        raise ValueError(f"unknown kind {kind!r} (decay, log, sigmoid)")
    dtype = gate.dtype
    wide = dtype is not x.dtype
    if wide and dtype is not _F32:
        raise TypeError("gate must be float32 or of x's type")
    shape = x.shape
    if len(shape) == 3:
        if starts is not None:
            raise ValueError("packed rows (starts) need [tokens, channels]")
        rows, tokens, channels = shape
    elif len(shape) == 2:
        tokens, channels = shape
        rows = 1
        if starts is not None:
            rows = starts.numel() - 1
            if rows < 0:
                raise ValueError("starts must hold rows + 1 elements")
    else:
        raise ValueError("x must be [rows, tokens, channels] or [tokens, channels]")
    if channels < 1:
        raise ValueError("x must have channels")
    return rows, tokens, channels, number, wide


def _states(t, name: str, channels: int, pool: int, here: int):
    """Address of fp32 states [pool, channels]; None for None."""
    if t is None:
        return None
    if t.get_device() == here and t.dtype is _F32 and t.shape == (pool, channels) and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != here:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if t.shape != (pool, channels) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{pool}, {channels}]")
    raise TypeError(f"{name} must be float32")


def gated_scan(x: torch.Tensor, gate: torch.Tensor, starts: torch.Tensor | None = None,
               initial: torch.Tensor | None = None, slots: torch.Tensor | None = None, kind: str = "decay",
               out: torch.Tensor | None = None, final: torch.Tensor | None = None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + b_t over every row's tokens,
    channel by channel, in fp32: ``kind`` "decay" (a = gate, b = x), "log" (a =
    exp(gate), b = x) or "sigmoid" (a = sigmoid(gate), b = (1 - a) x).

    ``x`` (float32, float16 or bfloat16) is [rows, tokens, channels], or
    [tokens, channels]: one row, or with ``starts`` (int32, rows + 1, as
    ``slot_map`` gives them) packed rows, of those tokens that there are; tokens in
    no row get 0.  ``gate`` has
    x's shape, and its type or float32.  Only the channels need to be
    contiguous.  ``initial`` (fp32 [states, channels]) holds the rows' h before
    their first token; ``slots`` (int32 per row) says where in it, and in
    ``final``, which takes h after their last token.  One token per row is the
    decode step.

    Carries no autograd graph; its gradients are :func:`gated_scan_backward`'s.
    Returns (out, final).  ``out`` may be ``x`` itself and ``final`` may be
    ``initial`` itself; without ``final``, rows with slots leave their states in
    ``initial``, and others in a new tensor."""
    suffix = _value_suffix(x)
    here = _device_of(x, "x")
    _no_graph("gated_scan", x, gate, initial)
    rows, tokens, channels, number, wide = _gated_rows(x, gate, starts, kind)
    empty = torch.empty if stream is None else _empty_on(stream)
    if final is None:
        if slots is None:
            final = empty(rows, channels, dtype=_F32, device=x.device)
        elif initial is None:
            raise ValueError("slots need initial or final to point into")
        else:
            final = initial
    pool = final.shape[0] if final.dim() else 0
    if slots is None and pool != rows:
        raise ValueError(f"final must hold {rows} states")
    shape, dtype = x.shape, x.dtype
    if out is None:
        out = empty(shape, dtype=dtype, device=x.device)
    x_at, x_row, x_token = _token_array(x, "x", shape, dtype, here)
    gate_at, gate_row, gate_token = _token_array(gate, "gate", shape, gate.dtype, here)
    out_at, out_row, out_token = _token_array(out, "out", shape, dtype, here)
    states = _states(final, "final", channels, pool, here)
    status = getattr(load(), "gated_scan_" + suffix)(
        x_at, x_row, x_token, gate_at, gate_row, gate_token, wide, rows, tokens, channels,
        None if starts is None else _vector(starts, "starts", _I32, rows + 1, here),
        states if initial is final else _states(initial, "initial", channels, pool, here),
        None if slots is None else _vector(slots, "slots", _I32, rows, here), pool, number, out_at, out_row, out_token,
        states, _stream_handle(stream))
    if status:
        _lib.check(status, "gated_scan_" + suffix)
    return out, final


def gated_scan_backward(grad: torch.Tensor, x: torch.Tensor | None, gate: torch.Tensor, y: torch.Tensor,
                        starts: torch.Tensor | None = None, initial: torch.Tensor | None = None,
                        grad_final: torch.Tensor | None = None, kind: str = "decay",
                        grad_x: torch.Tensor | None = None, grad_gate: torch.Tensor | None = None,
                        grad_initial: torch.Tensor | None = None, stream=None):
    """Gradients of :func:`gated_scan` (without slots): from those of its
    outputs, ``grad`` and ``grad_final`` (fp32 [rows, channels], optional), and
    from what it was given and gave (``y``, its ``out``), those of ``x`` and
    ``gate`` in their types and of ``initial``.  ``x`` is read for "sigmoid"
    only, and may be None otherwise.  Returns (grad_x, grad_gate,
    grad_initial), the last None where there is neither ``initial`` nor a
    tensor for it."""
    suffix = _value_suffix(y)
    here = _device_of(y, "y")
    _no_graph("gated_scan_backward", grad, x, gate, y, initial, grad_final)
    rows, tokens, channels, number, wide = _gated_rows(y, gate, starts, kind)
    shape, dtype, device = y.shape, y.dtype, y.device
    if kind == "sigmoid" and x is None:
        raise ValueError("sigmoid needs x")
    empty = torch.empty if stream is None else _empty_on(stream)
    if grad_x is None:
        grad_x = empty(shape, dtype=dtype, device=device)
    if grad_gate is None:
        grad_gate = empty(shape, dtype=gate.dtype, device=device)
    if grad_initial is None and initial is not None:
        grad_initial = empty(rows, channels, dtype=_F32, device=device)
    status = getattr(load(), "gated_scan_backward_" + suffix)(
        *_token_array(grad, "grad", shape, dtype, here),
        *((None, 0, 0) if x is None else _token_array(x, "x", shape, dtype, here)),
        *_token_array(gate, "gate", shape, gate.dtype, here), wide, *_token_array(y, "y", shape, dtype, here), rows,
        tokens, channels, _vector(starts, "starts", _I32, rows + 1, here),
        _states(initial, "initial", channels, rows, here), _states(grad_final, "grad_final", channels, rows, here),
        number, *_token_array(grad_x, "grad_x", shape, dtype, here),
        *_token_array(grad_gate, "grad_gate", shape, gate.dtype, here),
        _states(grad_initial, "grad_initial", channels, rows, here), _stream_handle(stream))
    if status:
        _lib.check(status, "gated_scan_backward_" + suffix)
    return grad_x, grad_gate, grad_initial


_IDS = {torch.int32: "expert_sort_i32", torch.int64: "expert_sort_i64"}


def expert_sort(experts: torch.Tensor, num_experts: int, align: int = 1, rows: int | None = None,
                starts: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                order: torch.Tensor | None = None, places: torch.Tensor | None = None, stream=None):
    """Sort the pairs (token, choice) of ``experts`` (int32 or int64 [tokens,
    choices], as a top-k gives them) stably by expert, every expert's rows
    rounded up to a multiple of ``align``.  Returns (starts, counts, order,
    places), all int32: each expert's first row and the number of rows
    [num_experts + 1], its number of pairs [num_experts], for every row the pair
    that lies there (-1: rounds up, -2: behind the last segment), and for
    every pair its row (-1 where its id is outside 0 .. num_experts - 1).
    ``rows`` is the number of rows that there are (by default what the pairs
    can need at most); pairs beyond have no place."""
    here = _device_of(experts, "experts")
    name = _IDS.get(experts.dtype)
    if name is None:
        raise TypeError("experts must be int32 or int64")
    if experts.dim() != 2 or not experts.is_contiguous():
        raise ValueError("experts must be a contiguous [tokens, choices]")
    tokens, choices = experts.shape
    num_experts, align = int(num_experts), int(align)
    if num_experts < 1 or align < 1 or choices < 1:
        raise ValueError("num_experts, align and choices must be positive")
    pairs = tokens * choices
    if rows is None:
        rows = order.numel() if order is not None else pairs + min(num_experts, pairs) * (align - 1)
    rows = int(rows)
    if rows < 0:
        raise ValueError("rows must not be negative")
    device = experts.device
    empty = torch.empty if stream is None else _empty_on(stream)
    if starts is None:
        starts = empty(num_experts + 1, dtype=_I32, device=device)
    if counts is None:
        counts = empty(num_experts, dtype=_I32, device=device)
    if order is None:
        order = empty(rows, dtype=_I32, device=device)
    if places is None:
        places = empty(tokens, choices, dtype=_I32, device=device)
    elif places.shape != experts.shape:
        raise ValueError("places must have the shape of experts")
    status = getattr(load(), name)(
        experts.data_ptr(), tokens, choices, num_experts, align, rows,
        _vector(starts, "starts", _I32, num_experts + 1, here), _vector(counts, "counts", _I32, num_experts, here),
        _vector(order, "order", _I32, rows, here), _vector(places, "places", _I32, pairs, here),
        _stream_handle(stream))
    if status:
        _lib.check(status, name)
    return starts, counts, order, places


def _check_rows(t: torch.Tensor, name: str, rows: int, width: int, dtype: torch.dtype, here: int) -> int:
    """A matrix of that size and device; returns its row stride."""
    strides = t.stride()
    if t.get_device() == here and t.dtype is dtype and t.shape == (rows, width) and strides[1] == 1 and strides[0] >= width:
        return strides[0]
    if t.get_device() != here:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    stride = _check_matrix(t, name)
    if t.shape[0] != rows or t.shape[1] != width:
        raise ValueError(f"{name} must be [{rows}, {width}]")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    return stride


def _check_places(places: torch.Tensor, here: int):
    if places.dim() != 2 or places.dtype is not _I32 or not places.is_contiguous():
        raise ValueError("places must be a contiguous int32 [tokens, choices]")
    if places.get_device() != here:
        raise ValueError("places must be on the current device")
    tokens, choices = places.shape
    if choices < 1:
        raise ValueError("places must hold a choice per token")
    return tokens, choices


def _per_pair(t, name: str, places: torch.Tensor, here: int):
    """Address of fp32 values in the places' order: of their shape (apart from
    dimensions of 1), or flat; None for None.  Another shape of as many elements,
    such as [choices, tokens], would be read in an order that is not its own."""
    if t is not None and t.shape != places.shape:
        sizes = [n for n in t.shape if n != 1]
        if len(sizes) > 1 and sizes != [n for n in places.shape if n != 1]:
            raise ValueError(f"{name} must have the shape of places")
    return _vector(t, name, _F32, places.numel(), here)


def expert_dispatch(x: torch.Tensor, places: torch.Tensor, order: torch.Tensor, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Copy every token's row of ``x`` (any type, [tokens, width]) to its
    ``places``; rows that round up a segment (``order`` -1) become 0, those
    behind the last segment are left as they were (in a new tensor: whatever is
    there).  Returns ``out`` [rows, width].  The gradient of x is
    ``expert_combine`` of out's, without weights."""
    here = _device_of(x, "x")
    _no_graph("expert_dispatch", x)
    tokens, choices = _check_places(places, here)
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError("x must be [tokens, width]")
    width, rows, size, dtype = x.shape[1], order.numel(), x.element_size(), x.dtype
    empty = torch.empty if stream is None else _empty_on(stream)
    if out is None:
        out = empty(rows, width, dtype=dtype, device=x.device)
    status = load().expert_dispatch(
        x.data_ptr(), _check_rows(x, "x", tokens, width, dtype, here) * size, width * size, tokens, choices,
        places.data_ptr(), rows, _vector(order, "order", _I32, rows, here), out.data_ptr(),
        _check_rows(out, "out", rows, width, dtype, here) * size, _stream_handle(stream))
    if status:
        _lib.check(status, "expert_dispatch")
    return out


def expert_combine(y: torch.Tensor, places: torch.Tensor, weights: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Bring the experts' rows back: out[t] = sum over its choices of
    ``weights`` (fp32 like ``places``; None: 1) times the rows of ``y`` [rows,
    width] (float32, float16 or bfloat16) at its ``places``, summed in fp32.  A
    token without any place gets 0."""
    suffix = _value_suffix(y)
    here = _device_of(y, "y")
    _no_graph("expert_combine", y, weights)
    tokens, choices = _check_places(places, here)
    if y.dim() != 2 or y.shape[1] < 1:
        raise ValueError("y must be [rows, width]")
    rows, width = y.shape
    dtype = y.dtype
    empty = torch.empty if stream is None else _empty_on(stream)
    if out is None:
        out = empty(tokens, width, dtype=dtype, device=y.device)
    status = getattr(load(), "expert_combine_" + suffix)(
        y.data_ptr(), _check_rows(y, "y", rows, width, dtype, here), rows, tokens, choices, width, places.data_ptr(),
        _per_pair(weights, "weights", places, here), out.data_ptr(),
        _check_rows(out, "out", tokens, width, dtype, here), _stream_handle(stream))
    if status:
        _lib.check(status, "expert_combine_" + suffix)
    return out


def expert_combine_backward(grad: torch.Tensor, y: torch.Tensor, places: torch.Tensor,
                            weights: torch.Tensor | None = None, order: torch.Tensor | None = None,
                            grad_y: torch.Tensor | None = None, grad_weights: torch.Tensor | None = None,
                            stream=None):
    """Gradients of :func:`expert_combine`: from ``grad`` [tokens, width] those
    of ``y`` and of the weights (fp32 like ``places``).  With ``order``, rows of
    grad_y that round up a segment become 0; rows without a pair are otherwise
    left as they were.  Returns (grad_y, grad_weights), the second None where
    there are neither ``weights`` nor a tensor for it."""
    suffix = _value_suffix(y)
    here = _device_of(y, "y")
    _no_graph("expert_combine_backward", grad, y, weights)
    tokens, choices = _check_places(places, here)
    if y.dim() != 2 or y.shape[1] < 1:
        raise ValueError("y must be [rows, width]")
    rows, width = y.shape
    dtype = y.dtype
    empty = torch.empty if stream is None else _empty_on(stream)
    if grad_y is None:
        grad_y = empty(rows, width, dtype=dtype, device=y.device)
    if grad_weights is None and weights is not None:
        grad_weights = empty(tokens, choices, dtype=_F32, device=y.device)
    status = getattr(load(), "expert_combine_backward_" + suffix)(
        grad.data_ptr(), _check_rows(grad, "grad", tokens, width, dtype, here), y.data_ptr(),
        _check_rows(y, "y", rows, width, dtype, here), rows, tokens, choices, width, places.data_ptr(),
        _per_pair(weights, "weights", places, here), _vector(order, "order", _I32, rows, here), grad_y.data_ptr(),
        _check_rows(grad_y, "grad_y", rows, width, dtype, here),
        _per_pair(grad_weights, "grad_weights", places, here), _stream_handle(stream))
    if status:
        _lib.check(status, "expert_combine_backward_" + suffix)
    return grad_y, grad_weights


_TENSOR_TYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_DTYPE_OF = operator.attrgetter("dtype")


def _norm(tensors, out, max_norm, norm, work, stream):
    tensors = list(tensors)
    outs = tensors if out is None else list(out)
    count = len(tensors)
    if len(outs) != count:
        raise ValueError("out must hold a tensor for each of tensors")
    here = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1
    of = torch.Tensor                              # a method for all tensors at once: there may be hundreds
    dtypes = list(map(_DTYPE_OF, tensors))
    kinds = list(map(_TENSOR_TYPE.get, dtypes))
    if None in kinds:
        raise TypeError(f"unsupported dtype {dtypes[kinds.index(None)]} (float32, float16, bfloat16)")
    sizes = list(map(of.numel, tensors))
    at = list(map(of.data_ptr, tensors))
    if count and (set(map(of.get_device, tensors)) != {here} or here < 0 or not all(map(of.is_contiguous, tensors))):
        raise ValueError("tensors must be contiguous, on the current CUDA device")
    to = at
    if out is not None:
        if (count and set(map(of.get_device, outs)) != {here} or not all(map(of.is_contiguous, outs))
                or list(map(of.numel, outs)) != sizes or list(map(_DTYPE_OF, outs)) != dtypes):
            raise ValueError("each of out must match its tensor in type, size and device, and be contiguous")
        to = list(map(of.data_ptr, outs))
    if max_norm is not None and len(set(to)) != count:
        held = [p for p, n in zip(to, sizes) if n]
        if len(set(held)) != len(held):
            raise ValueError("a tensor is to be clipped twice")
    table = array.array("Q", bytes(32 * max(count, 1)))   # of devscan_tensor, four words each
    for word, values in enumerate((at, to, sizes, kinds)):
        table[word:4 * count:4] = array.array("Q", values)
    empty = torch.empty if stream is None else _empty_on(stream)
    if norm is None:
        norm = empty((), dtype=_F32, device="cuda")
    need = _lib.norm_work_bytes(count)
    if work is None:
        work = empty(need, dtype=torch.uint8, device="cuda")
    here = _device_of(work, "work")
    if not work.is_contiguous():
        raise ValueError("work must be contiguous")
    size = work.numel() * work.element_size()
    if size < need:
        raise ValueError(f"work must hold {need} bytes")
    address, result = table.buffer_info()[0], _vector(norm, "norm", _F32, 1, here)
    if max_norm is None:
        _lib.check(load().grad_norm(address, count, result, work.data_ptr(), size, _stream_handle(stream)), "grad_norm")
    else:
        _lib.check(load().clip_grad_norm(address, count, max_norm, result, work.data_ptr(), size,
                                         _stream_handle(stream)), "clip_grad_norm")
    return norm, outs


def grad_norm(tensors, norm: torch.Tensor | None = None, work: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """2-norm over all elements of ``tensors`` (contiguous float32, float16 or
    bfloat16, mixed as they come): an fp32 scalar on the device, without an autograd
    graph.  Squares neither overflow nor vanish.  ``work`` may pass the scratch (any type,
    ``_lib.norm_work_bytes(len(tensors))`` bytes)."""
    return _norm(tensors, None, None, norm, work, stream)[0]


def clip_grad_norm(tensors, max_norm: float, out=None, norm: torch.Tensor | None = None,
                   work: torch.Tensor | None = None, stream=None):
    """Scale ``tensors`` by min(1, max_norm / (norm + 1e-6)), norm being that of
    :func:`grad_norm` over all of them; in place, or into the tensors of
    ``out``.  Tensors that are written must not overlap others in part (that is
    not checked).  A norm that is infinite or NaN clips nothing.  Returns (norm, the
    list of clipped tensors); nothing is read back to the host."""
    max_norm = float(max_norm)
    if not max_norm >= 0:
        raise ValueError("max_norm must not be negative")
    return _norm(tensors, out, max_norm, norm, work, stream)


def scan_host(x_host: torch.Tensor, inclusive: bool = False, op: str = "add", device="cuda",
              stream=None, out_host: torch.Tensor | None = None, work=None,
              synchronize: bool = True, as_uint32: bool = False) -> torch.Tensor:
    """Scan a host array end to end through the library's host entry
    (``scan_{inclusive,exclusive}_host_T``): host-to-device copy, device
    scan, device-to-host copy, all queued by the library on ``stream``.
    Pinned host tensors make the copies asynchronous.  ``work`` may pass
    preallocated (device input, device output) tensors.  With
    ``synchronize`` (the default) it returns once the result is in
    ``out_host``; without, it returns at once and the result is there when
    ``stream`` has reached this point, so calls on two streams overlap one
    call's download with the next one's upload."""
    if x_host.is_cuda:
        raise ValueError("x_host must be a host tensor")
    if not x_host.is_contiguous():
        raise ValueError("x_host must be contiguous")
    suffix = "u32" if as_uint32 else _SUFFIX.get(x_host.dtype)
    if suffix is None:
        raise TypeError(f"unsupported dtype {x_host.dtype} (int32, uint32, float32)")
    s = stream if stream is not None else torch.cuda.current_stream()
    empty = torch.empty if stream is None else _empty_on(stream)
    if work is None:
        d_in = empty(x_host.shape, dtype=x_host.dtype, device=device)
        d_out = _made_on(stream, torch.empty_like, d_in)
    else:
        d_in, d_out = work
        _check_cuda(d_in, "work[0]")
        _check_cuda(d_out, "work[1]")
        if d_in.numel() < x_host.numel() or d_out.numel() < x_host.numel():
            raise ValueError("work tensors are smaller than x_host")
    if out_host is None:
        out_host = torch.empty(x_host.shape, dtype=x_host.dtype, pin_memory=x_host.is_pinned())
    if out_host.is_cuda or out_host.numel() != x_host.numel() or out_host.dtype != x_host.dtype:
        raise ValueError("out_host must be a host tensor matching x_host")
    name = f"scan_{'inclusive' if inclusive else 'exclusive'}_host_{suffix}"
    _lib.check(getattr(load(), name)(x_host.data_ptr(), out_host.data_ptr(), x_host.numel(), OPS[op],
                                     d_in.data_ptr(), d_out.data_ptr(), _stream_handle(s)), name)
    if synchronize:
        s.synchronize()
    return out_host


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) its device-side status."""
    return load().devscan_device_status(_stream_handle(stream))


def set_carry_mode(mode: str) -> None:
    """Measurement hook (``devscan_measure_set_carry_mode``): 'default',
    'lookback' (one tile per block), 'rts' (reduce-then-scan), 'pipelined'
    (persistent warp-specialised single pass) or 'l2' (the cooperative forms:
    the L2-resident scan, the one-read bracket check, the two-launch
    compaction with flags and split).  Applies to the calling thread's later
    calls only."""
    code = {"default": 0, "lookback": 1, "rts": 2, "pipelined": 3, "l2": 4}[mode]
    _lib.check(load().devscan_measure_set_carry_mode(code), "devscan_measure_set_carry_mode")


def stream_release(stream=None) -> None:
    _lib.check(load().devscan_stream_release(_stream_handle(stream)), "devscan_stream_release")


def selftest_stalled_wait(spin_limit: int = 1000, stream=None) -> int:
    """Run the bounded-wait self-test and return the status that
    ``device_status`` then reports (DEVSCAN_ERR_TIMEOUT = 4 expected)."""
    _lib.check(load().devscan_selftest_stalled_wait(int(spin_limit), _stream_handle(stream)),
               "devscan_selftest_stalled_wait")
    return device_status(stream)
