"""Token draws whose cut lies next to zero: zeros of both signs at the end of a
range of ordered bits, with more denormal numbers below them than the list
holds.  The temperature is so high that all tokens weigh the same, and the noise
makes each one outrun those ahead of it, so that the token drawn is the last
that is kept."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def row_of(top, zeros, below, seed):
    """One token at the largest value, zeros of both signs and negative
    denormals of at most 22 bits, shuffled."""
    rng = np.random.default_rng(seed)
    bits = np.concatenate([[np.float32(top).view(np.uint32)], np.where(rng.random(zeros) < 0.5, 0x80000000, 0),
                           0x80000000 + rng.integers(1, 1 << 22, below)]).astype(np.uint32)
    x = rng.permutation(bits).view(np.float32)
    order = np.lexsort((np.arange(x.size), -x.astype(np.float64)))
    q = np.empty(x.size, np.float32)
    q[order] = np.exp2(-40.0 * np.arange(x.size) / x.size)
    return x, q, order


@pytest.mark.parametrize("rows", [1, 5, 330])
@pytest.mark.parametrize("t", [1e30, math.inf])
@pytest.mark.parametrize("zeros,below", [(20000, 20000), (3000, 37000), (1, 30000), (30000, 1100)])
@pytest.mark.parametrize("top", [np.nextafter(np.float32(2), np.float32(0)), 1.5, 0.0])
def test_cut_below_zero(ds, top, zeros, below, t, rows):
    x, q, order = row_of(top, zeros, below, zeros)
    vocab = x.size
    cut = zeros + below // 2                          # places 0 .. cut are kept
    p = (cut + 0.5) / vocab
    f = lambda v: torch.full((rows,), v, dtype=torch.float32, device="cuda")  # noqa: E731
    xs, qs = torch.from_numpy(x).cuda().expand(rows, vocab).contiguous(), torch.from_numpy(q).cuda().expand(rows, vocab).contiguous()
    tokens, logprobs = ds.sample_tokens(xs, qs, temperature=f(t), top_p=f(p))
    assert tokens.tolist() == [order[cut]] * rows
    # One of cut + 1 equal weights; a sum of as many fp32 terms, each off by 4u.
    assert bool(((logprobs.double() + math.log(cut + 1)).abs() <= 2.0 ** -16).all())
    # The first k of them, cut in the same place.
    k = vocab - 100
    tokens, _ = ds.sample_tokens(xs, qs, temperature=f(t), top_k=torch.full((rows,), k, dtype=torch.int32, device="cuda"),
                                 top_p=f((cut + 0.5) / k))
    assert tokens.tolist() == [order[cut]] * rows
