"""qmv_logprobs against log probabilities, entropy and stable sorting in 64
bits; bounds are derived in serve_ref."""
import numpy as np
import pytest

import serve_ref as R
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def run(x, ids, top, offset=0):
    """From logits that start `offset` floats into a buffer and a workspace full of ones."""
    import torch
    rows, vocab = x.shape
    buf = torch.full((rows * vocab + offset + 8,), 1e30, device="cuda")
    xd = buf[offset:offset + rows * vocab].view(rows, vocab)
    xd.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    idd = torch.from_numpy(ids.astype(np.int32)).cuda()
    lp = torch.full(ids.shape, 3.0, device="cuda")
    h = torch.full((rows,), 3.0, device="cuda")
    ti = torch.full((rows, top), -7, dtype=torch.int32, device="cuda") if top else None
    tl = torch.full((rows, top), 3.0, device="cuda") if top else None
    n = S.qmv_logprobs_workspace(rows, vocab, top)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    S.qmv_logprobs(xd, idd, lp, h, ti, tl, workspace=ws)
    torch.cuda.synchronize()
    return {"lp": lp.cpu().numpy(), "entropy": h.cpu().numpy(),
            "top_ids": ti.cpu().numpy() if top else np.zeros((rows, 0), int),
            "top_lp": tl.cpu().numpy() if top else np.zeros((rows, 0))}


def check(x, ids, top, offset=0):
    got, ref = run(x, ids, top, offset), R.logprobs(x, ids, top)
    pieces = -(-x.shape[1] // 2048)
    ok = (ids >= 0) & (ids < x.shape[1])
    assert np.all(got["lp"][~ok] == 0)
    fin = np.isfinite(ref["lp"])
    assert np.array_equal(got["lp"][~fin], ref["lp"][~fin].astype(np.float32))
    lp = np.where(fin, ref["lp"], 0)
    assert np.all(np.abs(np.where(fin, got["lp"], 0) - lp) <= R.logprob_bound(ref, lp, pieces))
    assert np.all(np.abs(got["entropy"] - ref["entropy"]) <= R.entropy_bound(ref, pieces))
    assert np.array_equal(got["top_ids"], ref["top_ids"])
    fin = np.isfinite(ref["top_lp"])
    assert np.array_equal(got["top_lp"][~fin], ref["top_lp"][~fin].astype(np.float32))
    lp = np.where(fin, ref["top_lp"], 0)
    assert np.all(np.abs(np.where(fin, got["top_lp"], 0) - lp) <= R.logprob_bound(ref, lp, pieces))


def ids_of(g, rows, vocab, n):
    return g.integers(0, vocab, size=(rows, n))


# one element; around a thread's four, a group of lanes, a piece of 2048 and
# of 8192 (which many rows take); odd lengths whose rows start unaligned
@pytest.mark.parametrize("rows,vocab,n,top", [
    (1, 1, 1, 1), (2, 3, 2, 3), (1, 15, 1, 15), (3, 17, 5, 16), (2, 33, 1, 32), (1, 1000, 1, 20), (4, 2047, 1, 5),
    (3, 2048, 1, 32), (2, 2049, 1, 1), (5, 8193, 3, 20), (1, 50001, 1, 32), (700, 1023, 1, 7), (600, 8200, 2, 20),
    (2, 248320, 1, 20), (1, 300001, 1, 32), (9, 128, 1, 0)])
def test_shapes(rows, vocab, n, top):
    g = np.random.default_rng(rows * vocab + top)
    x = (3 * g.standard_normal((rows, vocab))).astype(np.float32)
    check(x, ids_of(g, rows, vocab, n), top)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_logits_at_any_float(offset):
    g = np.random.default_rng(offset)
    x = g.standard_normal((3, 4099)).astype(np.float32)
    check(x, ids_of(g, 3, 4099, 1), 20, offset)


@pytest.mark.parametrize("rows", [2, 600])
def test_ties_go_to_the_lowest_index(rows):
    g = np.random.default_rng(5)
    vocab = 9001
    x = g.integers(0, 4, size=(rows, vocab)).astype(np.float32)   # thousands of equal logits
    x[0] = 1.5                                                    # all equal
    x[1] = np.where(np.arange(vocab) % 2 == 0, 0.0, -0.0)         # -0 and 0 are equal
    check(x, ids_of(g, rows, vocab, 1), 32)


@pytest.mark.parametrize("rows", [1, 600])
def test_best_ones_side_by_side(rows):
    """All of the best in one lane's elements, one group, one piece, or spread."""
    g = np.random.default_rng(6)
    vocab = 20000
    for where in (np.arange(32) + 4096, np.arange(32) * 4 + 8192, np.arange(32) * 1024 % vocab,
                  vocab - 1 - np.arange(32), np.arange(32) * 600):
        x = g.standard_normal((rows, vocab)).astype(np.float32)
        x[:, where] += 20
        check(x, ids_of(g, rows, vocab, 1), 32)


def test_values_at_the_ends():
    g = np.random.default_rng(7)
    vocab = 5000
    x = g.standard_normal((6, vocab)).astype(np.float32)
    x[0, 100:] = -np.inf                       # a mask that leaves 100 tokens
    x[1, :] = -np.inf
    x[1, 4321] = -3.0                          # one token alone: entropy 0
    x[2] = -3.4028235e38                       # a type's lowest value as a mask
    x[2, 7] = 1.0
    x[3] *= 1000                               # nearly all mass on one
    x[4] *= np.float32(1e-20)
    x[5, 4000:] = -np.inf                      # whole pieces of -infinity
    ids = np.array([[50, 200], [4321, 0], [7, 8], [0, 1], [2, 3], [4999, 1]])
    check(x, ids, 32)


def test_ids_out_of_range_give_zero():
    g = np.random.default_rng(8)
    x = g.standard_normal((3, 777)).astype(np.float32)
    check(x, np.array([[-1, 777, 5], [2147483647, -2147483648, 776], [0, 1, 100000]]), 3)


@pytest.mark.parametrize("rows", [5, 300])
def test_rows_without_a_distribution(rows):
    """NaN, +infinity, or nothing but -infinity: NaN, for that row alone."""
    g = np.random.default_rng(9)
    vocab = 20000
    x = g.standard_normal((rows, vocab)).astype(np.float32)
    ids = ids_of(g, rows, vocab, 2)
    want = run(x, ids, 5)
    x[0, 9000] = np.nan
    x[1, 3] = np.inf
    x[2] = -np.inf
    x[3, :8192] = np.nan
    got = run(x, ids, 5)
    for k in ("lp", "entropy", "top_lp"):
        assert np.all(np.isnan(got[k][:4])), k
        assert np.array_equal(got[k][4:], want[k][4:])
    assert np.all((got["top_ids"] >= 0) & (got["top_ids"] < vocab))
    assert np.array_equal(got["top_ids"][4:], want["top_ids"][4:])


def test_outputs_one_by_one():
    import torch
    g = np.random.default_rng(10)
    x = g.standard_normal((4, 3001)).astype(np.float32)
    ids = ids_of(g, 4, 3001, 2)
    want = run(x, ids, 6)
    xd, idd = torch.from_numpy(x).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda()
    h = torch.empty(4, device="cuda")
    S.qmv_logprobs(xd, entropy=h)
    lp = torch.empty(4, 2, device="cuda")
    S.qmv_logprobs(xd, idd, lp)
    ti, tl = torch.empty(4, 6, dtype=torch.int32, device="cuda"), torch.empty(4, 6, device="cuda")
    S.qmv_logprobs(xd, top_ids=ti, top_lp=tl)
    assert np.array_equal(h.cpu().numpy(), want["entropy"]) and np.array_equal(lp.cpu().numpy(), want["lp"])
    assert np.array_equal(ti.cpu().numpy(), want["top_ids"]) and np.array_equal(tl.cpu().numpy(), want["top_lp"])


def test_capture_and_other_stream():
    import torch
    g = np.random.default_rng(11)
    x = g.standard_normal((3, 30000)).astype(np.float32)
    want = run(x, ids_of(g, 3, 30000, 1), 20)
    xd = torch.from_numpy(x).cuda()
    ti, tl = torch.empty(3, 20, dtype=torch.int32, device="cuda"), torch.empty(3, 20, device="cuda")
    ws = S.workspace(S.qmv_logprobs_workspace(3, 30000, 20))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        S.qmv_logprobs(xd, top_ids=ti, top_lp=tl, workspace=ws, stream=st)
    for _ in range(3):
        ti.fill_(-1)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ti.cpu().numpy(), want["top_ids"]) and np.array_equal(tl.cpu().numpy(), want["top_lp"])


def test_refuses_what_it_cannot_take():
    import torch
    x = torch.zeros(2, 100, device="cuda")
    h = torch.empty(2, device="cuda")
    with pytest.raises(Q.QmvError):
        S.qmv_logprobs(x)
    with pytest.raises(ValueError):
        S.qmv_logprobs(x.t(), entropy=h)
    with pytest.raises(ValueError):
        S.qmv_logprobs(x, entropy=h[:1])
    with pytest.raises(TypeError):
        S.qmv_logprobs(x.double(), entropy=h)
    with pytest.raises(TypeError):
        S.qmv_logprobs(x, torch.zeros(2, 1, dtype=torch.int64, device="cuda"), torch.empty(2, 1, device="cuda"))
    with pytest.raises(ValueError):
        S.qmv_logprobs(x, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.empty(2, 1, device="cuda"))
    with pytest.raises(Q.QmvError) as e:
        S.qmv_logprobs(x, top_ids=torch.zeros(2, 40, dtype=torch.int32, device="cuda"),
                       top_lp=torch.zeros(2, 40, device="cuda"))
    assert e.value.status == Q.QMV_E_SHAPE


@pytest.mark.parametrize("vocab", [1, 3, 5, 100, 2049, 2050])
def test_nan_at_the_end_of_a_row(vocab):
    """The top of a row of NaN, or with one last, is still of the row."""
    g = np.random.default_rng(14)
    x = g.standard_normal((3, vocab)).astype(np.float32)
    x[0] = np.nan
    x[1, -1] = np.nan
    top = min(vocab, 32)
    got = run(x, ids_of(g, 3, vocab, 1), top)
    assert np.all((got["top_ids"] >= 0) & (got["top_ids"] < vocab))
    assert all(len(set(r)) == top for r in got["top_ids"].tolist())
    assert np.all(np.isnan(got["top_lp"][:2])) and np.all(np.isfinite(got["top_lp"][2]))


def test_more_rows_than_workgroups():
    g = np.random.default_rng(15)
    x = g.standard_normal((300001, 40)).astype(np.float32)
    check(x, ids_of(g, 300001, 40, 1), 3)


@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("vocab", [1, 2, 31, 32, 33, 255, 1023, 1024, 1025, 2047, 2048, 2049, 4095, 4096, 4097,
                                   8191, 8192, 8193])
def test_rows_around_a_workgroups_size(rows, vocab):
    """Both sides of the sizes at which a row changes kernels, with values
    spread, equal, and in order (so that one wave has the best)."""
    g = np.random.default_rng(vocab)
    x = (3 * g.standard_normal((rows, vocab))).astype(np.float32)
    x[0] = 1.5
    x[1] = np.arange(vocab, dtype=np.float32) / 64
    x[2, vocab // 2:] = -np.inf if vocab > 1 else 0.0
    check(x, ids_of(g, rows, vocab, 300 if rows == 3 else 1), min(vocab // 2 if vocab in (2, 31) else vocab, 32))


def test_more_pieces_than_workgroups():
    """90000 rows of three pieces; sampled rows against the reference."""
    import torch
    rows, vocab, top = 90000, 8193, 4
    x = torch.randn(rows, vocab, device="cuda")
    ids = torch.randint(0, vocab, (rows, 1), device="cuda", dtype=torch.int32)
    lp, h = torch.empty(rows, 1, device="cuda"), torch.empty(rows, device="cuda")
    ti, tl = torch.empty(rows, top, dtype=torch.int32, device="cuda"), torch.empty(rows, top, device="cuda")
    S.qmv_logprobs(x, ids, lp, h, ti, tl)
    sel = [0, 1, 43690, 65535, 87381, 87382, rows - 2, rows - 1]
    ref = R.logprobs(x[sel].cpu().numpy(), ids[sel].cpu().numpy(), top)
    assert np.all(np.abs(lp[sel].cpu().numpy() - ref["lp"]) <= R.logprob_bound(ref, ref["lp"], 3))
    assert np.all(np.abs(h[sel].cpu().numpy() - ref["entropy"]) <= R.entropy_bound(ref, 3))
    assert np.array_equal(ti[sel].cpu().numpy(), ref["top_ids"])
    assert np.all(np.abs(tl[sel].cpu().numpy() - ref["top_lp"]) <= R.logprob_bound(ref, ref["top_lp"], 3))


@pytest.mark.parametrize("vocab", [5, 64, 1000, 1024, 2048, 3001, 4096, 8191, 8192, 8193, 20000])
@pytest.mark.parametrize("top", [1, 20, 32])
def test_rows_of_nan_and_infinity(vocab, top):
    """Rows that mix NaN with -infinity, in blocks and scattered: NaN, indexes
    of the row, each once; the ordinary row between them as it is alone."""
    g = np.random.default_rng(vocab + top)
    top = min(top, vocab)
    plain = g.standard_normal(vocab).astype(np.float32)
    rows = []
    for nans in sorted({1, vocab // 8, vocab // 2, vocab - vocab // 8, vocab - 1, vocab} - {0}):
        for infs in sorted({0, (vocab - nans) // 2, vocab - nans}):
            for order in range(4):
                x = np.concatenate([np.full(nans, np.nan), np.full(infs, -np.inf), plain[:vocab - nans - infs]])
                x = x[::-1] if order == 1 else (np.roll(x, infs) if order == 2 else (g.permutation(x) if order == 3 else x))
                rows.append(x.astype(np.float32))
    rows.append(plain)
    x = np.stack(rows)
    ids = ids_of(g, x.shape[0], vocab, 2)
    got = run(x, ids, top)
    for k in ("lp", "entropy", "top_lp"):
        assert np.all(np.isnan(got[k][:-1])), k
    assert np.all((got["top_ids"] >= 0) & (got["top_ids"] < vocab))
    assert all(len(set(r)) == top for r in got["top_ids"].tolist())
    check(plain[None], ids[-1:], top)
    assert np.array_equal(got["top_ids"][-1], R.logprobs(plain[None], ids[-1:], top)["top_ids"][0])
