"""qmv_kv4_attend where whole pages hold zeros, tokens that are no number, or
values far above or below the other pages': outputs stay those of the formula,
within more_ref.attend_bound and what the header says of small values."""
import numpy as np
import pytest

import more_ref as M
import serve_ref as R
from block_quant_weight_amd import serve as S
from test_gpu_attend4 import FAR, attend, starts
from test_gpu_attend4 import check as check_random
from test_gpu_kv4 import put, seqs, to_gpu

pytestmark = pytest.mark.gpu
PAGE = 64
DIMS = [64, 128, 256]
# With many bfloat16 queries, values below this part of the largest of their
# sequence and head may count as 0; and in every call those below 2^-96.
LOST, LEAST = 2.0 ** -80, 2.0 ** -96
# Rows and sequences beside those of a test, without tokens: a call that looks
# large goes to the kernel for many also under a window, and is not cut.
SPARE_ROWS, SPARE_SEQS = 10000, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def inputs(seed, lens, kv_heads, dim):
    """Keys and values of all tokens of each sequence, values of a mean that is not 0."""
    g = np.random.default_rng(seed)
    k = [R.bf16(g.standard_normal((n, kv_heads, dim)).astype(np.float32)) for n in lens]
    v = [R.bf16((0.5 + g.standard_normal((n, kv_heads, dim))).astype(np.float32)) for n in lens]
    return g, k, v


def stored(c, table, lens, k, v):
    """What qmv_kv4_write makes of all tokens, into c."""
    seq = np.repeat(np.arange(len(lens)), lens)
    pos = np.concatenate([np.arange(n) for n in lens])
    page, t = table[seq, pos // PAGE], pos % PAGE
    none = ~(np.isfinite(k).all(-1) & np.isfinite(v).all(-1))
    for n, x, byte in (("k", k, 255), ("v", v, 2)):
        index, neg, e = M.quantize(np.where(none[..., None], 0, x))
        c.code[n][page, :, t] = np.where(none[..., None], 0, index + 8 * neg)
        c.byte[n][page, :, t] = np.where(none[..., None], byte, e + 127)


def check(g, k, v, news, heads, dtype, window=0, flat=1.0):
    """Writes the tokens with qmv_kv4_write, and attends with the last `news`
    of each sequence; sequences cut into pieces, and whole."""
    lens, (_, kv_heads, dim) = [len(x) for x in k], k[0].shape
    counts = [-(-n // PAGE) for n in lens]
    c = M.Cache4(sum(counts) + 2, kv_heads, dim)
    ids = g.permutation(c.pages)
    table = np.full((len(lens), max(counts)), -1)
    for i, n in enumerate(counts):
        table[i, :n] = ids[sum(counts[:i]):sum(counts[:i]) + n]
    gpu = to_gpu(c)
    all_k, all_v, at = np.concatenate(k), np.concatenate(v), starts(lens)
    S.qmv_kv4_write(gpu, seqs(table, lens, at), put(all_k, "bf16"), put(all_v, "bf16"))
    stored(c, table, lens, all_k, all_v)
    start = starts(news)
    rows = start[-1]
    q = R.bf16((flat * g.standard_normal((rows, heads, dim))).astype(np.float32))
    with np.errstate(all="ignore"):
        ref, b = M.attend(c, table, lens, start, q, np.float32(dim ** -0.5), window)
    # a row that sees a token that is no number is NaN, no other is
    nan = np.isnan(ref).any(-1)
    ref = np.where(nan[..., None], 0, ref)
    b = {n: np.where(nan[..., None], 1, x) for n, x in b.items()}
    tol = M.attend_bound(b, dim, max(lens), dtype, many=dtype == "bf16") + LEAST
    if dtype == "bf16":
        for i in range(len(lens)):
            big = [np.abs(x[np.isfinite(x)], dtype=np.float64).max() for x in (v[i][:, h] for h in range(kv_heads))]
            tol[start[i]:start[i + 1]] += LOST * np.repeat(big, heads // kv_heads)[None, :, None]
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    wide = np.concatenate([q, np.zeros((SPARE_ROWS, heads, dim), dtype=np.float32)])
    calls = [(q, seqs(table, lens, start, *FAR))]
    calls.append((wide, seqs(np.concatenate([table, np.full((SPARE_SEQS, table.shape[1]), -1)]), lens + [0] * SPARE_SEQS,
                             start + [rows] * SPARE_SEQS, SPARE_ROWS, 1 << 20)))
    for x, s in calls:
        got = attend(gpu, s, x, dtype, window=window)
        assert np.all(got[rows:] == 5.0), "rows of no sequence were written"
        got = got[:rows]
        assert np.array_equal(np.isnan(got).any(-1), nan) and np.array_equal(np.isnan(got).all(-1), nan)
        assert np.all(np.isfinite(got[~nan]))
        err = np.abs(np.where(nan[..., None], 0, got) - ref)
        assert np.all(err <= tol), f"worst {np.nanmax(err / tol):.3g} of the bound"
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [0.01, 1.0, 300.0])
@pytest.mark.parametrize("dim", DIMS)
def test_pages_of_zeros(dim, size, dtype):
    """Pages whose values are all 0 in one head: the first, some between
    others, the last; whole sequences and ones that are cut."""
    g, k, v = inputs(dim, [450, 900], 2, dim)
    for x in v:
        x *= np.float32(size)
        x[:] = R.bf16(x)
        x[128:192, 0] = 0
        x[256:384, 1] = 0
    v[0][-2:] = 0
    v[1][:64] = 0
    v[1][-100:, 0] = 0
    check(g, k, v, [40, 130], 4, dtype)
    check(g, k, v, [40, 130], 4, dtype, window=70)


@pytest.mark.parametrize("dim", DIMS)
def test_a_sequence_of_zeros(dim):
    g, k, v = inputs(dim + 1, [450, 300], 1, dim)
    v[0][:] = 0
    got = check(g, k, v, [130, 40], 2, "bf16")
    assert np.all(got[:130] == 0)


@pytest.mark.parametrize("flat", [0.0, 1.0])
@pytest.mark.parametrize("size", [1.0, 1000.0])
@pytest.mark.parametrize("dim", DIMS)
def test_last_page_of_one_token(dim, size, flat):
    """The only token of the last page that any row sees is 0, or no number:
    the rows before it, in the same tile, do not see that."""
    for last in (0.0, np.nan, np.inf):
        g, k, v = inputs(dim + 2, [193, 577], 1, dim)
        for x in v:
            x[:] = R.bf16(x * np.float32(size))
            x[-1] = last
        check(g, k, v, [30, 130], 2, "bf16", flat=flat)


@pytest.mark.parametrize("dim", DIMS)
def test_page_begun_by_tokens_that_are_no_number(dim):
    """A page of such tokens alone, under a window that later rows have moved past it."""
    g, k, v = inputs(dim + 3, [500], 1, dim)
    v[0][256:320, 0, 3] = np.nan
    check(g, k, v, [200], 2, "bf16", window=64)
    check(g, k, v, [200], 2, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exps", [(0, -100, 0, 0, -100, -100, 0), (60, -60, 60, -90, 0, 60, -60), (-90, -90, 40, -90, -30, -90, 40),
                                  (0, -60, -90, 0, -70, -66, 0), (-95, -50, 0, 50, 61, 0, -95)])
@pytest.mark.parametrize("dim", DIMS)
def test_pages_far_apart(dim, exps, dtype):
    """Values of the pages up to 2^156 apart; every row sees the largest
    before it, so what may count as 0 is no part of its output that counts,
    and under a window some see the small ones alone."""
    g, k, v = inputs(dim + 4, [440, 600], 1, dim)
    for x in v:
        for p in range(-(-len(x) // PAGE)):
            x[PAGE * p:PAGE * (p + 1)] *= np.float32(2.0 ** exps[p % len(exps)])
    check(g, k, v, [130, 60], 2, dtype)
    check(g, k, v, [130, 60], 2, dtype, window=40)


@pytest.mark.parametrize("window", [1, 2, 50, 64, 200])
@pytest.mark.parametrize("dim", DIMS)
def test_kernel_for_many_under_a_window(dim, window):
    """Edges of causality and window inside a page, groups that do not divide a
    tile, more rows than tokens, in a call that looks large enough for that
    kernel though a window leaves few pages."""
    empty = [0] * SPARE_SEQS
    for lens, news, heads, kv_heads in (([300, 40], [200, 40], 4, 2), ([400], [90], 5, 1), ([3, 70, 0], [80, 100, 9], 3, 1)):
        check_random(lens + empty, news + empty, heads, kv_heads, dim, "bf16", seed=dim + window, window=window,
                     spare=SPARE_ROWS, hints=(SPARE_ROWS, 1 << 20))
