"""qmv_sample against the draw in 64 bits.  A token may be another than the
reference's only where a border lies within more_ref.NEAR of the weights' own
error (derived there)."""
import numpy as np
import pytest

import more_ref as M
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def run(x, u, t=None, k=None, p=None, m=None):
    import torch
    dev = lambda a, dt=np.float32: None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()
    rows, vocab = x.shape
    ids = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), 9.0, device="cuda")
    ws = torch.full((max(S.qmv_sample_workspace(rows, vocab), 16),), 0xFF, dtype=torch.uint8, device="cuda")
    S.qmv_sample(dev(x), dev(u), ids, temperature=dev(t), top_k=dev(k, np.int32), top_p=dev(p), min_p=dev(m), lp=lp, workspace=ws)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), lp.cpu().numpy()


def check(x, u, t=None, k=None, p=None, m=None):
    rows = len(x)
    ids, lp = run(x, u, t, k, p, m)
    full = lambda a, v: np.full(rows, v) if a is None else np.asarray(a)
    t, k, p, m = full(t, np.float32(1)), full(k, 0), full(p, np.float32(1)), full(m, np.float32(0))
    for i in range(rows):
        ans = M.sample_answers(x[i], float(np.float32(u[i])), float(np.float32(t[i])), int(k[i]), float(np.float32(p[i])),
                               float(np.float32(m[i])))
        assert M.sample_ok(ans, ids[i], lp[i]), (i, ids[i], lp[i], ans, t[i], k[i], p[i], m[i], u[i])
    return ids


def logits(g, rows, vocab, likely=True):
    x = 2.2 * g.standard_normal((rows, vocab))
    if likely and vocab > 40:
        for r in range(rows):
            x[r, g.choice(vocab, 20, replace=False)] = 9 + 2.5 * g.standard_normal(20)
    return x.astype(np.float32)


def wishes(g, rows, vocab):
    return dict(u=g.random(rows).astype(np.float32), t=g.choice([0.0, 0.3, 0.7, 1.0, 2.0], rows),
                k=g.choice([0, 0, 1, 2, 7, 40, vocab, 3 * vocab], rows), p=g.choice([1.0, 1.0, 0.0, 0.3, 0.9, 0.999], rows),
                m=g.choice([0.0, 0.0, 0.01, 0.3, 1.0], rows))


@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 1000, 1025, 4096, 8191, 16385, 40001, 151936])
def test_all_filters(vocab):
    g = np.random.default_rng(vocab)
    rows = 24 if vocab > 10000 else 60
    check(logits(g, rows, vocab), **wishes(g, rows, vocab))


@pytest.mark.parametrize("vocab", [700, 50000])
@pytest.mark.parametrize("names", ["", "t", "k", "p", "m", "kp", "pm", "tkpm"])
def test_filters_left_out(vocab, names):
    g = np.random.default_rng(vocab + len(names))
    x, w = logits(g, 12, vocab), wishes(g, 12, vocab)
    check(x, w["u"], **{n: w[n] for n in names})


def test_flat_rows_and_many_kept():
    """No token stands out: the tokens that stay are a large part of the row."""
    g = np.random.default_rng(1)
    x = logits(g, 20, 60000, likely=False)
    w = wishes(g, 20, 60000)
    check(x, w["u"], t=[1.0, 5.0] * 10, k=[0, 0, 5000, 30000] * 5, p=[0.95, 0.5, 0.99, 1.0, 0.8] * 4, m=[0.0, 0.001] * 10)


def test_ties():
    """Equal logits stay by the lower index: rows of one value, of a few, and
    ties at every filter's border."""
    g = np.random.default_rng(2)
    for vocab in (64, 3000, 70000):
        x = np.round(g.standard_normal((30, vocab)) * 2).astype(np.float32)
        x[0] = 1.5
        x[1] = -0.0
        x[1, ::2] = 0.0
        w = wishes(g, 30, vocab)
        w["k"][:10], w["p"][:10], w["m"][:10], w["t"][:10] = 50, 1.0, 0, 1.0
        w["p"][10:20] = 0.5
        check(x, **w)


def test_clustered_rows():
    """All likely tokens beside each other, at the row's start, at its end and
    in the lanes of one thread."""
    g = np.random.default_rng(3)
    vocab = 100000
    x = logits(g, 8, vocab, likely=False)
    x[0, :700] += 14
    x[1, -700:] += 14
    x[2, 5000:9000] += 14
    x[3, ::1024] += 14
    x[4, 77::4096] += 14
    x[5, :vocab // 2] += 14
    x[6, :3] += 30
    x[7, ::64] += 14
    for k, p in ((0, 0.95), (600, 1.0), (50, 0.9), (5000, 0.99), (0, 1.0)):
        check(x, g.random(8).astype(np.float32), t=np.full(8, 0.9), k=np.full(8, k), p=np.full(8, p), m=np.zeros(8))


def test_rows_that_cannot_be_drawn_from():
    g = np.random.default_rng(4)
    for vocab in (100, 30000):
        x = logits(g, 12, vocab)
        x[0, 3], x[1, vocab - 1], x[2], x[3, ::2] = np.nan, np.inf, -np.inf, -np.inf
        x[4], x[4, vocab // 2] = -np.inf, -3.0
        x[5, :] = -3e38
        x[6, 1:] = 3e38
        x[6, 0] = -3e38
        t = np.array([1, 1, 1, 1, 1, 1, 1, -1, np.nan, np.inf, 1e-38, 1e38], dtype=np.float32)
        ids = check(x, g.random(12).astype(np.float32), t=t, k=[0, 0, 0, 5] * 3, p=[1, 0.9] * 6, m=np.zeros(12))
        assert list(ids[[0, 1, 2, 7, 8, 9]]) == [-1] * 6 and ids[4] == vocab // 2


def test_odd_wishes():
    """Numbers outside their range: u at and past its ends and NaN, p and m
    past theirs and NaN, negative k."""
    g = np.random.default_rng(5)
    x = logits(g, 10, 5000)
    u = np.array([0.0, 1.0, -3.0, 7.0, np.nan, 0.99999994, 0.5, 0.5, 0.5, 0.5], dtype=np.float32)
    k = np.array([0, 0, 0, 0, 0, 0, -4, -2147483648, 2147483647, 3])
    p = np.array([1, 1, 1, 1, 1, 1, np.nan, -1, 2, 1], dtype=np.float32)
    m = np.array([0, 0, 0, 0, 0, 0, np.nan, 0, -1, 5], dtype=np.float32)
    ids, lp = run(x, u, None, k, p, m)
    clean = lambda a, v: np.where(np.isnan(a), v, a)
    for i in range(10):
        ui = float(clean(u, 0)[i])
        ans = M.sample_answers(x[i], min(max(ui, 0.0), 1.0), 1.0, int(k[i]), float(np.clip(clean(p, 1), 0, None)[i]), float(np.clip(clean(m, 0), 0, 1)[i]))
        if ui >= 1.0:                              # the last token whose weight counts
            w = np.exp(x[i].astype(np.float64) - x[i].max())
            assert w[ids[i]] >= 2.0 ** -41 and np.all(w[ids[i] + 1:] < 2.0 ** -39)
        else:
            assert M.sample_ok(ans, ids[i], lp[i]), i


def test_the_draws_are_the_distribution():
    """u over an even grid: each token is drawn as often as its weight says,
    to one place of the grid at each border (and the borders' own error)."""
    n = 4096
    g = np.random.default_rng(6)
    x = np.repeat(g.standard_normal((1, 50)).astype(np.float32), n, 0)
    u = (np.arange(n) + 0.5) / n
    ids, _ = run(x, u, t=np.full(n, 0.8))
    w = np.exp(x[0].astype(np.float64) / np.float32(0.8))
    assert np.all(np.abs(np.bincount(ids, minlength=50) - n * w / w.sum()) <= 2)


def test_many_rows_alone_and_together():
    """A row's answer does not depend on the rows beside it, nor on lp being asked for."""
    import torch
    g = np.random.default_rng(7)
    x, w = logits(g, 300, 3001), wishes(g, 300, 3001)
    ids, lp = run(x, **w)
    for i in (0, 17, 299):
        one, l1 = run(x[i:i + 1], **{n: a[i:i + 1] for n, a in w.items()})
        assert one[0] == ids[i] and (l1[0] == lp[i] or np.isnan(lp[i]))
    out = torch.empty(300, dtype=torch.int32, device="cuda")
    S.qmv_sample(torch.from_numpy(x).cuda(), torch.from_numpy(w["u"]).cuda(), out,
                 temperature=torch.from_numpy(w["t"].astype(np.float32)).cuda(), top_k=torch.from_numpy(w["k"].astype(np.int32)).cuda(),
                 top_p=torch.from_numpy(w["p"].astype(np.float32)).cuda(), min_p=torch.from_numpy(w["m"].astype(np.float32)).cuda())
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), ids)


@pytest.mark.parametrize("rows,vocab", [(1, 248320), (5, 9000), (3, 70000)])
def test_capture(rows, vocab):
    """Replays follow the inputs; two graphs with a workspace each run at once."""
    import torch
    g = np.random.default_rng(8)
    st = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for i in range(2):
        d = dict(x=torch.from_numpy(logits(g, rows, vocab)).cuda(), u=torch.rand(rows, device="cuda"),
                 ids=torch.empty(rows, dtype=torch.int32, device="cuda"), lp=torch.empty(rows, device="cuda"),
                 p=torch.full((rows,), 0.9, device="cuda"), k=torch.full((rows,), 40, dtype=torch.int32, device="cuda"),
                 ws=S.workspace(S.qmv_sample_workspace(rows, vocab)))
        st[i].wait_stream(torch.cuda.current_stream())
        d["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(d["graph"], stream=st[i]):
            S.qmv_sample(d["x"], d["u"], d["ids"], top_k=d["k"], top_p=d["p"], lp=d["lp"], workspace=d["ws"], stream=st[i])
        sets.append(d)
    for turn in range(3):
        for d in sets:
            d["u"].uniform_()
            d["x"].add_(torch.randn_like(d["x"]))
        torch.cuda.synchronize()
        for i, d in enumerate(sets):
            with torch.cuda.stream(st[i]):
                d["graph"].replay()
        torch.cuda.synchronize()
        for d in sets:
            ids, lp = torch.empty_like(d["ids"]), torch.empty_like(d["lp"])
            S.qmv_sample(d["x"], d["u"], ids, top_k=d["k"], top_p=d["p"], lp=lp)
            torch.cuda.synchronize()
            assert torch.equal(ids, d["ids"]) and torch.equal(lp, d["lp"])


def test_refusals():
    import torch
    x, u = torch.zeros(2, 100, device="cuda"), torch.zeros(2, device="cuda")
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    S.qmv_sample(x, u, ids)
    for bad in (dict(u=u[:1]), dict(ids=ids[:1]), dict(logits=x[0]), dict(logits=x[:, ::2]), dict(lp=u[:1]), dict(top_k=ids[:1]),
                dict(logits=x.cpu())):
        with pytest.raises(ValueError):
            S.qmv_sample(**{**dict(logits=x, u=u, ids=ids), **bad})
    for bad in (dict(u=ids), dict(ids=u), dict(top_k=u), dict(logits=x.bfloat16())):
        with pytest.raises(TypeError):
            S.qmv_sample(**{**dict(logits=x, u=u, ids=ids), **bad})
    with pytest.raises(Q.QmvError):
        S.qmv_sample(x, u, ids, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
