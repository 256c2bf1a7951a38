"""The token draw's noise at and past the ends of what takes part: zero,
negative, NaN and infinite numbers lose, whatever their token weighs, and
numbers down to the smallest denormal count by their value, in every form of
the race."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

INF = math.inf
LOSING = (0.0, -0.0, -1.0, -1e-40, -INF, INF, math.nan)
TINY = tuple(np.float32(2.0 ** -149) * np.float32(k) for k in (1, 2, 3, 700, 5e5))   # denormal
ENDS = (2.0 ** -126, 2.0 ** -125, 1e-30, 2.0 ** 60, 2.0 ** 64)

# The race of all tokens, of a list, of a row that needs histograms (cut by
# count, by mass, and inside a tie) and of what min-p leaves.
FORMS = {"all": (1.0, 0, 1.0, 0.0), "list": (0.8, 40, 1.0, 0.0), "list and mass": (0.9, 50, 0.9, 0.0),
         "count": (1.0, 3000, 1.0, 0.0), "mass": (1.5, 0, 0.95, 0.0), "count and mass": (1.0, 5000, 0.97, 0.0),
         "min-p": (1.0, 0, 1.0, 0.01)}


@pytest.fixture(scope="module")
def ds():
    import stream_compaction_device_gb300 as m
    m.load()
    return m


def rows_of(rows, vocab, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, vocab)) * 1.5
    q = rng.exponential(1.0, (rows, vocab)) + 1e-30
    return x.astype(np.float32), q.astype(np.float32), rng


def settings(asks):
    t, k, p, m = zip(*asks)
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    return {"temperature": f(t), "top_k": torch.tensor(k, dtype=torch.int32, device="cuda"), "top_p": f(p),
            "min_p": f(m)}


def check(ds, x, q, asks, dtype=torch.float32, only=None):
    xt = torch.from_numpy(x).to(dtype)
    tokens, logprobs = ds.sample_tokens(xt.cuda(), torch.from_numpy(q).cuda(), **settings(asks))
    x, tokens, logprobs = xt.float().numpy(), tokens.tolist(), logprobs.tolist()
    for r in range(len(asks)) if only is None else only:
        t, k, p, m = asks[r]
        with np.errstate(invalid="ignore"):
            # Noise that loses: as if it came last of all.
            clean = np.where((q[r] > 0) & (q[r] < INF), q[r].astype(np.float64), INF)
        t, p, m = (float(np.float32(v)) for v in (t, p, m))
        good, logprob = ref.draw(x[r], clean, t, k, p, m)
        assert tokens[r] in good, (r, asks[r], tokens[r], sorted(good)[:4], q[r][tokens[r]], q[r][sorted(good)[:4]])
        value, room = logprob(tokens[r])
        assert abs(logprobs[r] - value) <= room, (r, asks[r])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vocab", [700, 5000, 36001])
@pytest.mark.parametrize("form", FORMS)
def test_losing_noise(ds, form, vocab, dtype):
    """A third of the tokens have noise that loses; the last rows' heaviest
    tokens, all of them."""
    x, q, rng = rows_of(8, vocab, vocab)
    bad = rng.random(q.shape) < 0.3
    q[bad] = rng.choice(np.array(LOSING, np.float32), int(bad.sum()))
    for r in (5, 6, 7):
        heavy = np.argsort(-x[r])[:6]
        q[r, heavy] = LOSING[r - 5]
    check(ds, x, q, [FORMS[form]] * 8, dtype)


@pytest.mark.parametrize("vocab", [700, 36001])
@pytest.mark.parametrize("form", FORMS)
def test_denormal_noise_counts_by_its_value(ds, form, vocab):
    """Some tokens of every kept set have noise below 2^-126: of these the one
    with the largest quotient is drawn, not the first."""
    x, q, rng = rows_of(8, vocab, vocab + 1)
    for r in range(8):
        heavy = np.argsort(-x[r])[:30]
        at = rng.choice(heavy, 8, replace=False)
        q[r, at] = rng.choice(np.array(TINY + LOSING[:2], np.float32), 8)
        q[r, heavy[heavy.size - r:]] = ENDS[r % len(ENDS)]
    check(ds, x, q, [FORMS[form]] * 8)


@pytest.mark.parametrize("form", FORMS)
def test_rows_left_to_the_second_launch(ds, form):
    rows, vocab = 330, 40000
    x, q, rng = rows_of(rows, vocab, 3)
    bad = rng.random((rows, 4000)) < 0.3
    q[:, ::10][bad] = rng.choice(np.array(LOSING + TINY, np.float32), int(bad.sum()))
    check(ds, x, q, [FORMS[form]] * rows, only=range(0, rows, 23))


@pytest.mark.parametrize("vocab", [64, 3000, 36001])
@pytest.mark.parametrize("form", FORMS)
def test_rows_whose_noise_all_loses(ds, form, vocab):
    x, _, rng = rows_of(len(LOSING) + 1, vocab, 5)
    q = np.repeat(np.array(LOSING, np.float32)[:, None], vocab, 1)
    q = np.concatenate([q, rng.choice(np.array(LOSING, np.float32), (1, vocab))])
    tokens, logprobs = ds.sample_tokens(torch.from_numpy(x).cuda(), torch.from_numpy(q).cuda(),
                                        **settings([FORMS[form]] * len(q)))
    assert tokens.tolist() == [-1] * len(q)
    assert logprobs.tolist() == [-INF] * len(q)


@pytest.mark.parametrize("vocab", [64, 36001])
def test_masked_tokens_are_not_drawn_for_want_of_noise(ds, vocab):
    """Masked tokens have good noise, the others none or, in odd rows, one."""
    x, q, _ = rows_of(6, vocab, 6)
    x[:, ::2] = -INF
    x[2:4, 4] = math.nan
    q[:, 1::2] = 0.0
    q[1::2, 33] = 5.0
    for ask in FORMS.values():
        if ask[1] == 40 or ask[1] == 50:
            x[1::2, 33] = 9.0               # inside every cut
        tokens, _ = ds.sample_tokens(torch.from_numpy(x).cuda(), torch.from_numpy(q).cuda(), **settings([ask] * 6))
        got = tokens.tolist()
        assert got[0::2] == [-1, -1, -1], ask
        assert all(t in (-1, 33) for t in got[1::2]), ask
