"""qmv_sample where the answer lies at an end of the running sum: rows whose
first or last tokens each weigh nothing, though many of them together would."""
import numpy as np
import pytest

import more_ref as M
from test_gpu_sample import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def whole_weights(x, t):
    """Weights of a row as whole multiples of 2^-39 of the largest."""
    return np.rint(np.exp((x.astype(np.float64) - x.max()) / t) * 2.0 ** 39)


@pytest.mark.parametrize("below", [28.0, 28.5, 29.0])
@pytest.mark.parametrize("t", [1.0, 0.7])
@pytest.mark.parametrize("vocab", [3000, 9000, 50001, 248320])
def test_tokens_that_weigh_nothing_are_not_drawn(vocab, t, below):
    """u at its ends, and rows that begin and end with thousands of tokens at
    2^-40.4 to 2^-41.8 of the largest, masked ones among them.  (Weights are
    right to 2^-22 of themselves: none lies that near to half a unit.)"""
    g = np.random.default_rng(vocab)
    rows = 6
    x = (2.0 * g.standard_normal((rows, vocab))).astype(np.float32)
    top = x.max(-1) + 3
    ends = vocab // 3 if vocab < 10000 else 4096
    for i in range(rows):
        x[i, vocab // 2] = top[i]
        x[i, :ends] = x[i, -ends:] = top[i] - np.float32(below * t)
        x[i, :ends - 1:2 + i] = x[i, -1::-97] = -np.inf
        x[i, vocab // 2 + 1:vocab - ends:701] = -np.inf
    u = np.array([0.0, 1.0, 0.0, 1.0, 1e-13, 0.99999994], dtype=np.float32)
    ids, lp = run(x, u, t=np.full(rows, t))
    for i in range(rows):
        w = whole_weights(x[i], float(np.float32(t)))
        there = np.nonzero(w)[0]
        if u[i] == 0.0:
            assert ids[i] == there[0]
        elif u[i] == 1.0:
            assert ids[i] == there[-1]
        assert w[ids[i]] > 0
        want = float(x[i, ids[i]] - np.float64(top[i])) / float(np.float32(t)) - np.log(w.sum() * 2.0 ** -39)
        assert M.sample_ok([(ids[i], want)], ids[i], lp[i])
    assert np.array_equal(run(x, u, t=np.full(rows, t), m=np.full(rows, 1e-20))[0][:4], ids[:4])


@pytest.mark.parametrize("vocab", [2, 20000])
def test_log_probabilities_are_not_off_to_one_side(vocab):
    """Log probabilities from -20 to -26, each rounded once to steps of 2^-19
    (most in one binade), so by half a step at most, and the mean of n by about
    0.29 / sqrt(n).  float32's ln 2 is 1.9e-9 above ln 2: where its low part is
    left out the mean is 0.03 steps off, where it is added with the wrong sign
    0.06 or 0.07."""
    g = np.random.default_rng(vocab)
    rows = 1 << 14 if vocab == 2 else 1 << 11
    t = np.float32(0.7)                       # (with 1 the logits lie on the steps themselves)
    d = g.uniform(14.0, 18.2, rows).astype(np.float32)
    x = np.full((rows, vocab), -np.inf, dtype=np.float32)
    x[:, 0], x[:, 1] = -d, 0.0
    # (u = 0: the first token that weighs anything)
    ids, lp = run(x, np.zeros(rows), t=np.full(rows, t))
    assert np.all(ids == 0)
    want = -d.astype(np.float64) / float(t)
    want -= np.log1p(np.exp(want))
    steps = (lp - want) * 2.0 ** 19
    # (the total's part above the largest, below 2^-28, and the roundings of the low parts are 0.01 steps)
    assert np.all(np.abs(steps) <= 0.51)
    assert abs(steps.mean()) <= 0.01 + 4 * 0.29 / np.sqrt(rows)


@pytest.mark.parametrize("vocab", [(1 << 24) - 1, 1 << 24])
def test_the_largest_vocabulary_all_alike(vocab):
    """Weights of the largest sum there is, 2^63 units; the first half of it with top_p."""
    x = np.full((3, vocab), -2.5, dtype=np.float32)
    u = np.array([0.0, 0.75, 1.0], dtype=np.float32)
    ids, lp = run(x, u)
    assert list(ids) == [0, int(0.75 * vocab), vocab - 1]
    assert all(M.sample_ok([(i, -np.log(vocab))], i, l) for i, l in zip(ids, lp))
    ids, lp = run(x, u, p=np.full(3, 0.5))
    half = (vocab + 1) // 2
    assert list(ids) == [0, int(0.75 * half), half - 1]
    assert all(M.sample_ok([(i, -np.log(half))], i, l) for i, l in zip(ids, lp))
