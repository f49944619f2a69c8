"""qmv_kv4_attend with queries that are no number: NaN for their rows and
heads, whatever the stored keys and the scale make of their products, and
nothing else changes.  Through every kernel: a few columns, a tile of them, a
wave's own, many, and sequences that are cut into pieces."""
import numpy as np
import pytest

import more_ref as M
import serve_ref as R
from test_gpu_attend4 import attend
from test_gpu_kv4 import seqs, to_gpu

pytestmark = pytest.mark.gpu
PAGE = 64
FORMS = {  # lens, new rows, heads to a key/value head, empty sequences, spare rows, hint of the longest
    "few": ([1, 5, 100], [1, 1, 1], 4, 0, 0, 100),
    "few, cut": ([3000, 1], [1, 1], 4, 0, 0, 3000),
    "tile": ([1, 70, 100], [1, 3, 9], 16, 0, 0, 100),
    "tile, cut": ([3000, 2], [2, 2], 16, 0, 0, 3000),
    "own": ([1, 70, 100], [1, 3, 70], 16, 1200, 0, 100),
    "many": ([130, 64, 200], [130, 1, 150], 2, 64, 10000, 1 << 20),
    "many, cut": ([300, 900], [130, 150], 2, 0, 0, 1 << 20),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


KINDS = [(w, s) for w in (np.inf, -np.inf, np.nan) for s in (0.125, -0.125, 0.0)]
# (all of them at one head dim; at the others products of either infinity, and a scale of 0)
CASES = [(64, w, s) for w, s in KINDS] + [(d, w, s) for d in (128, 256) for w, s in ((np.inf, -0.125), (-np.inf, 0.125), (-np.inf, 0.0))]


@pytest.mark.parametrize("dim,what,scale", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
def test_queries_that_are_no_number(form, dim, dtype, what, scale):
    lens, news, group, empty, spare, longest = FORMS[form]
    g = np.random.default_rng(dim)
    kv_heads, heads = 2, 2 * group
    counts = [-(-n // PAGE) for n in lens]
    c = M.Cache4(sum(counts), kv_heads, dim)
    # keys and values from 1/2 to 6: an infinite query's products are all infinite, of one sign
    for n in "kv":
        c.code[n] = g.integers(1, 8, size=c.code[n].shape).astype(np.uint8)
        c.byte[n][:] = 127
    table = np.full((len(lens) + empty, max(counts)), -1)
    ids = g.permutation(c.pages)
    for i, n in enumerate(counts):
        table[i, :n] = ids[sum(counts[:i]):sum(counts[:i]) + n]
    start = [0, *np.cumsum(news + [0] * empty).tolist()]
    rows = start[-1]
    q = R.bf16(g.standard_normal((rows + spare, heads, dim)).astype(np.float32))
    s = seqs(table, lens + [0] * empty, start, max(news + [spare]), longest)
    gpu = to_gpu(c)
    clean = attend(gpu, s, q, dtype, scale)[:rows]
    assert np.all(np.isfinite(clean))
    bad = np.zeros((rows, heads), dtype=bool)
    bad[0, 0] = bad[rows - 1, heads - 1] = bad[news[0], group] = True
    for at, ch in zip(np.argwhere(bad), (0, dim - 1, dim // 2 + 5)):
        q[at[0], at[1], ch] = what
    got = attend(gpu, s, q, dtype, scale)[:rows]
    assert np.array_equal(np.isnan(got).any(-1), bad) and np.array_equal(np.isnan(got).all(-1), bad)
    # both are within a half step of bfloat16, 2^-8, and attend_bound's 2^-10 of values up to 6
    assert np.all(np.abs(got[~bad] - clean[~bad]) <= 12 * (2.0 ** -8 + 2.0 ** -10))
