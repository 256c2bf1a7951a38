"""Token draws that the other files look at in part only: rows that rise or fall
along their whole length, and every row of a large batch of wide cuts."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def rising_error(ds, rows, vocab, dtype, t, order, reach):
    """Races of all tokens whose logits rise (or fall) from -reach to 0: the
    tokens that are not the definition's within the room, and the largest error
    of a log-probability beyond its room."""
    rng = np.random.default_rng(vocab + rows)
    x = np.sort(-reach * rng.random((8, vocab)), axis=1)[:, ::order].copy()
    q = rng.exponential(1.0, (8, vocab)).astype(np.float32) + np.float32(1e-30)
    xt = torch.from_numpy(x.astype(np.float32)).to(dtype)
    at = torch.arange(rows, device="cuda") % 8
    tokens, logprobs = ds.sample_tokens(xt.cuda()[at], torch.from_numpy(q).cuda()[at],
                                        temperature=torch.full((rows,), t, dtype=torch.float32, device="cuda"))
    tokens, logprobs = tokens.cpu().numpy(), logprobs.cpu().numpy().astype(np.float64)
    v = xt.float().numpy().astype(np.float64)
    t = float(np.float32(t))
    wrong, worst = 0, 0.0
    # A thread holds its sum and its best score relative to the largest logit it
    # has seen, and rescales them when a larger one comes, once per 16-byte chunk
    # at the most: a chunk's distance d is off by 3 |d| U, the exponential and the
    # product by 5 U, and the distances add up to the token's own.
    each = 16 // xt.element_size()
    chunks = -(-vocab // each) + 1
    rescales = -(-chunks // 256)                             # a row in one block has the most to a thread
    for r in range(rows):
        d = (v[r % 8] - v[r % 8].max()) / t
        w = np.exp(d)
        near = (3 * np.abs(d) + 8 + 5 * rescales) * U
        score = w / q[r % 8]
        best = score[tokens[r]]
        wrong += int(best * (1 + near[tokens[r]]) < (score * (1 - near)).max())
        rest = w.sum() - 1
        room = ((near * w).sum() + 2.0 ** -16 * rest) / (1 + rest)
        value = d[tokens[r]] - math.log1p(rest)
        worst = max(worst, abs(logprobs[r] - value) - room - 4 * U * abs(value))
    return wrong, worst


@pytest.mark.parametrize("rows", [1, 40, 330])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("vocab,dtype", [(1 << 18, torch.float32), (131072, torch.float32), (50001, torch.float16),
                                         (131072, torch.bfloat16)])
@pytest.mark.parametrize("t,reach", [(1.0, 30.0), (0.7, 1.0), (1.0, 2000.0)])
def test_rows_in_order(ds, t, reach, vocab, dtype, order, rows):
    wrong, worst = rising_error(ds, rows, vocab, dtype, t, order, reach)
    assert wrong == 0 and worst <= 0.0


def test_every_row_of_a_batch_of_wide_cuts(ds):
    rows, vocab = 330, 36001
    rng = np.random.default_rng(41)
    x = rng.standard_normal((rows, vocab)).astype(np.float32) * 2
    x[::9] = np.round(x[::9])
    x[4::11][:, rng.random(vocab) < 0.7] = -math.inf
    q = rng.exponential(1.0, (rows, vocab)).astype(np.float32) + np.float32(1e-30)
    kinds = [(1.0, 20000, 1.0, 0.0), (1.0, 5000, 0.99, 0.0), (0.5, 0, 0.9999, 0.0), (30.0, 0, 0.97, 0.0),
             (1.0, 9999, 0.3, 0.01), (1.0, 36000, 0.999, 0.0), (1.0, 0, 0.9, 0.0), (0.8, 50, 0.9, 0.0)]
    asks = [kinds[(r + r // 8) % 8] for r in range(rows)]
    t, k, p, m = zip(*asks)
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    tokens, logprobs = ds.sample_tokens(torch.from_numpy(x).cuda(), torch.from_numpy(q).cuda(), temperature=f(t),
                                        top_k=torch.tensor(k, dtype=torch.int32, device="cuda"), top_p=f(p), min_p=f(m))
    tokens, logprobs = tokens.tolist(), logprobs.tolist()
    for r in range(rows):
        good, logprob = ref.draw(x[r], q[r], *(float(np.float32(v)) if i != 1 else v for i, v in enumerate(asks[r])))
        assert tokens[r] in good, (r, asks[r], tokens[r], sorted(good)[:4])
        value, room = logprob(tokens[r])
        assert abs(logprobs[r] - value) <= room, (r, asks[r], logprobs[r], value, room)
