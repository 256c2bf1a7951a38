"""Cuts by mass far down a row's tail.  One token holds nearly all of the mass
and the rest lie many temperatures below it, so that top-p ends among weights
of 2^-27 to 2^-40.  The noise makes every token of the order outrun the ones
ahead of it: the one drawn is the last that is kept, and its place in the order
is compared with the definition's in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def row_of(vocab, depth, t, spread, seed, dtype):
    """Logits `depth` temperatures below the one at the top, give or take; the
    order; and noise by which score rises with the place in the order."""
    rng = np.random.default_rng(seed)
    x = -t * (depth + spread * rng.standard_normal(vocab))
    top = int(rng.integers(0, vocab))
    x[top] = 0.0
    x = torch.from_numpy(x.astype(np.float32)).to(dtype)
    v = x.float().numpy().astype(np.float64)
    order = np.lexsort((np.arange(vocab), -v))
    w = np.exp((v[order] - v[order[0]]) / t)
    q = np.empty(vocab, np.float32)
    q[order] = w * np.exp2(-60.0 * np.arange(vocab) / vocab)
    return x, order, w, q


def places(w, d, k, p):
    """The least and the largest place that the last kept token may have.  A
    weight is off by up to (3 |d| + 3) U of itself (the arithmetic of its
    exponent), and 1 not at all; the sums are of integers in units of 2^-45 or
    finer, one unit lost per bin of 1,024."""
    n = k if k > 0 else w.size
    w, d = w[:n], d[:n]
    ahead = np.concatenate([[0.0], np.cumsum(w)[:-1]])
    total = ahead[-1] + w[-1]
    room = 2 * (w * np.where(d == 0, 0.0, 3 * np.abs(d) + 3) * U).sum() + 1024 * 2.0 ** -45
    bar = p * total
    return int((ahead < bar - room).sum()) - 1, int((ahead < bar + room).sum()) - 1


CASES = [(20.0, 0.9999), (22.0, 0.99999), (22.5, 0.99999), (24.0, 0.999999), (18.0, 0.9995)]


@pytest.mark.parametrize("rows", [1, 6, 320])
@pytest.mark.parametrize("t", [1.0, 0.25])
@pytest.mark.parametrize("vocab,spread,dtype,k", [(131072, 0.3, torch.float32, 0), (131072, 1.0, torch.bfloat16, 0),
                                                  (1 << 18, 0.5, torch.float32, 0), (60001, 0.2, torch.float16, 0),
                                                  (131072, 0.3, torch.float32, 100000), (131072, 0.0, torch.float32, 0)])
def test_last_kept_token(ds, vocab, spread, dtype, k, t, rows):
    kinds = [row_of(vocab, depth, t, spread, i, dtype) for i, (depth, _) in enumerate(CASES)]
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    pick = [r % len(CASES) for r in range(rows)]
    xs, qs = torch.stack([c[0] for c in kinds]).cuda(), torch.from_numpy(np.stack([c[3] for c in kinds])).cuda()
    at = torch.tensor(pick, device="cuda")
    tokens, _ = ds.sample_tokens(xs[at], qs[at], temperature=f([t] * rows),
                                 top_k=torch.full((rows,), k, dtype=torch.int32, device="cuda"),
                                 top_p=f([CASES[i][1] for i in pick]))
    tokens = tokens.tolist()
    for i, (x, order, w, q) in enumerate(kinds):
        d = np.log(w)
        lo, hi = places(w, d, k, float(np.float32(CASES[i][1])))
        assert 0 < lo <= hi < vocab and hi - lo <= 2 + 0.002 * vocab, (i, lo, hi)
        place = {int(v): r for r, v in enumerate(order)}
        for r in range(i, rows, len(CASES)):
            assert lo <= place[tokens[r]] <= hi, (CASES[i], lo, place[tokens[r]], hi)
