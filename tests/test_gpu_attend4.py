"""qmv_kv4_attend against plain attention in 64 bits over the values that the
cache stands for; the bound is derived in more_ref.attend_bound."""
import numpy as np
import pytest

import more_ref as M
import serve_ref as R
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S
from test_gpu_kv4 import seqs, to_gpu

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def make(lens, kv_heads, dim, seed, extra=2, k_exp=(-3, 0), v_exp=(-9, 3)):
    """A cache of random codes and scales, garbage behind the sequences' ends, and its table."""
    g = np.random.default_rng(seed)
    counts = [-(-n // PAGE) for n in lens]
    pages = sum(counts) + extra
    c = M.Cache4(pages, kv_heads, dim)
    for n, (lo, hi) in (("k", k_exp), ("v", v_exp)):
        c.code[n] = g.integers(0, 16, size=c.code[n].shape).astype(np.uint8)
        c.byte[n] = (127 + g.integers(lo, hi, size=c.byte[n].shape)).astype(np.uint8)
    table = np.full((len(lens), max(max(counts), 1)), -1)
    ids = g.permutation(pages)
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = ids[at:at + n]
        at += n
        if n and lens[i] % PAGE:                  # what memory holds there does not matter
            for what in "kv":
                c.byte[what][table[i, n - 1], :, lens[i] % PAGE:] = g.integers(0, 256, size=c.byte[what][table[i, n - 1], :, lens[i] % PAGE:].shape)
    return g, c, table


def starts(news):
    s = [0]
    for m in news:
        s.append(s[-1] + m)
    return s


def attend(c, s, q, dtype, scale=None, window=0):
    """Outputs as float32, from a workspace full of NaN."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    qd = torch.from_numpy(q).cuda().to(dt)
    out = torch.full(q.shape, 5.0, dtype=dt, device="cuda")
    n = S.qmv_kv4_attend_workspace(c, s, qd, window)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    S.qmv_kv4_attend(c, s, qd, out, scale=scale, window=window, workspace=ws)
    torch.cuda.synchronize()
    return out.float().cpu().numpy()


def queries(g, rows, heads, dim, dtype="bf16"):
    q = R.bf16(g.standard_normal((rows, heads, dim)).astype(np.float32))
    return q if dtype == "bf16" else (q * np.float32(1.0003)).astype(np.float32)


def near(got, ref, b, dim, longest, dtype, many=False):
    tol = M.attend_bound(b, dim, longest, dtype, many)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of the bound"


def check(lens, news, heads, kv_heads, dim, dtype, seed, window=0, scale=None, spare=3, hints=(None, None)):
    g, c, table = make(lens, kv_heads, dim, seed)
    start = starts(news)
    q = queries(g, start[-1] + spare, heads, dim, dtype)
    sc = dim ** -0.5 if scale is None else scale
    got = attend(to_gpu(c), seqs(table, lens, start, *hints), q, dtype, scale, window)
    ref, b = M.attend(c, table, lens, start, q, np.float32(sc), window)
    m = start[-1]
    near(got[:m], ref[:m], {n: x[:m] for n, x in b.items()}, dim, max(lens), dtype)
    assert np.all(got[m:] == 5.0), "rows of no sequence were written"
    # a row that sees nothing is exactly 0
    assert np.all(got[:m][b["mass"][:m].max(-1) == 0] == 0)


SHAPES = [
    # lens, new rows, heads, kv_heads, dim: one token; lengths around pages;
    # groups of one, odd and more than a tile's columns
    ([1], [1], 1, 1, 64),
    ([1, 63, 64, 65, 129], [1, 1, 1, 1, 1], 8, 2, 64),
    ([200, 1, 70], [1, 1, 1], 5, 1, 128),
    ([100, 300], [1, 1], 32, 8, 128),
    ([90, 257], [1, 1], 24, 1, 128),
    ([130, 66], [1, 1], 6, 2, 256),
    # several rows: every row its own causal end; all of a sequence's tokens
    ([70, 64, 5], [7, 64, 5], 4, 4, 64),
    ([200], [33], 6, 2, 128),
    ([150, 80], [150, 2], 12, 4, 64),
    ([129], [129], 4, 1, 256),
    ([300, 40], [140, 40], 8, 2, 128),
    # sequences without rows or tokens between others
    ([0, 50, 64, 0], [0, 1, 0, 0], 4, 2, 64),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news,heads,kv_heads,dim", SHAPES)
def test_attend(lens, news, heads, kv_heads, dim, dtype):
    check(lens, news, heads, kv_heads, dim, dtype, seed=sum(lens) + dim)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 100, 5000])
def test_window(window, dtype):
    check([300, 70, 1], [1, 70, 1], 4, 2, 64, dtype, seed=window, window=window)
    check([260], [200], 8, 2, 128, dtype, seed=window + 1, window=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequences_in_pieces(dtype):
    """Lengths at which the pages of a sequence are shared by many workgroups,
    and long sequences beside short ones."""
    check([5000, 1200, 3], [1, 1, 1], 4, 2, 64, dtype, seed=1)
    check([4100], [3], 8, 1, 128, dtype, seed=2)
    check([3001], [2], 4, 2, 256, dtype, seed=3, window=2500)
    check([2500, 600], [40, 30], 4, 2, 128, dtype, seed=4)
    check([30] * 40 + [9000] + [100] * 29, [1] * 70, 2, 1, 64, dtype, seed=5)
    check([7000] + [0, 20] * 40, [2] + [0, 1] * 40, 4, 1, 64, dtype, seed=6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_columns(dtype):
    """Calls with columns enough that each wave, or a whole workgroup's tile, has its own."""
    check([300] * 6, [70] * 6, 32, 4, 64, dtype, seed=21)
    check([400, 130], [400, 130], 16, 4, 128, dtype, seed=22)
    check([260, 70], [260, 70], 8, 2, 256, dtype, seed=23, window=100)


FAR = (None, 1 << 20)      # a hint of long sequences: bfloat16 columns enough then go to the kernel for many


@pytest.mark.parametrize("window", [0, 1, 50, 64, 200])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_kernel_for_many(dim, window):
    """Tiles with and without rows to fill them, edges of causality and window
    inside a page, groups that do not divide a tile, empty sequences."""
    check([300, 40], [300, 40], 8, 2, dim, "bf16", seed=dim + window, window=window, hints=FAR)
    check([700], [90], 5, 1, dim, "bf16", seed=dim + window + 1, window=window, hints=FAR)
    check([0, 130, 64, 0, 1], [0, 130, 64, 3, 1], 24, 4, dim, "bf16", seed=dim + window + 2, window=window, hints=FAR)
    check([3, 70, 0], [80, 200, 90], 4, 2, dim, "bf16", seed=dim + window + 3, window=window, hints=FAR)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_kernel_for_many_in_pieces(dim):
    """One sequence's pages shared by workgroups, joined afterwards; page ids more than a wave looks up at once."""
    check([5000], [70], 4, 1, dim, "bf16", seed=dim, hints=FAR)
    check([4500, 100], [64, 64], 4, 1, dim, "bf16", seed=dim + 1, scale=-0.05, hints=FAR)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_kernel_for_many_rising_scores(dim):
    """Scores that rise along the sequence, so that references move all the
    time, and rows for which they fall; value scales that rise and fall by far
    between the pages."""
    g, c, table = make([900], 1, dim, 31, k_exp=(-2, -1))
    c.code["k"][:] = 4                             # 2
    for p in range(15):
        c.byte["k"][table[0, p]] = 127 - 8 + p
        c.byte["v"][table[0, p]] += (0, 30, 20, 60, 40, 10, 0, 3, 50, 0, 0, 25, 9, 1, 70)[p]
    q = queries(g, 200, 2, dim)
    q[::2] = np.abs(q[::2])
    q[1::2] = -np.abs(q[1::2])
    got = attend(to_gpu(c), seqs(table, [900], [0, 200], *((200, 1 << 20))), q, "bf16")
    ref, b = M.attend(c, table, [900], [0, 200], q, np.float32(dim ** -0.5), 0)
    near(got, ref, b, dim, 900, "bf16", many=True)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_kernel_for_many_and_what_is_not_there(dim):
    """Unknown pages between known ones, tokens and queries that are no number."""
    g, c, table = make([500, 300], 2, dim, 32)
    # page 0, which stands in for unknown ones, is in no table: its tokens move to one that is not
    spare = next(p for p in range(c.pages) if p not in table and p != 0)
    for n in "kv":
        c.code[n][spare], c.byte[n][spare] = c.code[n][0], c.byte[n][0]
    table[table == 0] = spare
    c.byte["v"][0, :, :, 0] = 255
    table = table.copy()
    table[0, 2], table[0, 5], table[1, 0] = -7, c.pages, -1
    c.byte["k"][table[0, 3], 1, 9], c.byte["v"][table[0, 3], 1, 9], c.code["v"][table[0, 3], 1, 9] = 255, 2, 0
    start = [0, 300, 500]
    q = queries(g, 500, 16, dim)
    q[123, 2, 3] = np.nan
    s = seqs(table, [500, 300], start, 300, 1 << 20)
    got = attend(to_gpu(c), s, q, "bf16")
    ref, b = M.attend(c, table, [500, 300], start, np.where(np.isnan(q), 0, q), np.float32(dim ** -0.5), 0)
    nan = np.zeros((500, 16), dtype=bool)
    nan[:300, 8:] = np.arange(200, 500)[:, None] >= 3 * 64 + 9
    nan[123, 2] = True
    assert np.array_equal(np.isnan(got).any(-1), nan) and np.array_equal(np.isnan(got).all(-1), nan)
    ref, got = np.where(nan[..., None], 0, ref), np.where(nan[..., None], 0, got)
    near(got, ref, {n: np.where(nan[..., None], 1, x) for n, x in b.items()}, dim, 500, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_rows_than_tokens(dtype):
    """Positions below 0 see nothing: zeros."""
    check([3, 0, 70], [5, 4, 80], 4, 2, 64, dtype, seed=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_hints_do_not_change_results(dtype):
    for hints in ((1, 1), (0, 0), (100000, 100000), (1, 100000), (100000, 1)):
        check([700, 90], [40, 90], 8, 2, 64, dtype, seed=6, hints=hints)
        check([1500, 90], [300, 90], 2, 2, 64, dtype, seed=7, hints=hints)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_negative_and_zero_scale(dtype):
    check([300, 40], [3, 1], 4, 2, 64, dtype, seed=8, scale=-0.2)
    check([300, 40], [200, 40], 16, 2, 64, dtype, seed=9, scale=-0.2)
    check([300, 40], [200, 40], 16, 2, 64, dtype, seed=9, scale=0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [[2, 3, 70], [130, 140, 70]])
def test_pages_that_are_not_there(dtype, news):
    """Unknown page ids and positions past the table are left out; a row whose
    pages are all unknown gets zeros."""
    g, c, table = make([300, 200, 70], 2, 64, 7)
    table = table[:, :4].copy()
    table[0, 1], table[0, 3] = -5, c.pages
    table[1, :] = -1
    table[2, 0] = 2147483647
    lens, start = [300, 200, 70], starts(news)
    q = queries(g, start[-1], 16, 64, dtype)
    got = attend(to_gpu(c), seqs(table, lens, start), q, dtype)
    ref, b = M.attend(c, table, lens, start, q, 0.125, 0)
    near(got, ref, b, 64, 300, dtype)
    assert np.all(got[start[1]:start[2]] == 0) and np.all(got[start[2]:start[3] - 6] == 0) and np.any(got[-6:] != 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [[1, 1, 1], [70, 80, 65], [180, 190, 200]])
def test_nan_touches_only_what_sees_it(dtype, news):
    """Tokens that are no number leave the rows that do not see them as they
    are; a row and head that sees one, or whose query is none, is NaN."""
    lens = [200, 200, 200]
    g, c, table = make(lens, 2, 64, 8, v_exp=(-5, -4))
    start = starts(news)
    rows = start[-1]
    q = queries(g, rows, 16, 64, dtype)
    window = 30
    clean = attend(to_gpu(c), seqs(table, lens, start), q, dtype, window=window)
    marks = [(0, 150, 0), (1, 190, 1), (1, 20, 0), (2, 3, 1)]
    for i, pos, h in marks:
        at = table[i, pos // 64]
        c.byte["k"][at, h, pos % 64], c.byte["v"][at, h, pos % 64] = 255, 2
        c.code["k"][at, h, pos % 64] = c.code["v"][at, h, pos % 64] = 0
    q[start[2] - 1, 0, 5] = np.nan              # the last row of sequence 1
    q[rows - 1, 15, 0] = np.inf
    got = attend(to_gpu(c), seqs(table, lens, start), q, dtype, window=window)
    nan = np.zeros((rows, 16), dtype=bool)
    for i, pos, h in marks:
        for t in range(news[i]):
            p = 200 - news[i] + t
            if p - window < pos <= p:
                nan[start[i] + t, 8 * h:8 * h + 8] = True
    nan[start[2] - 1, 0] = True
    nan[rows - 1, 15] = True
    assert np.array_equal(np.isnan(got).any(-1), nan) and np.array_equal(np.isnan(got).all(-1), nan)
    assert np.array_equal(got[~nan], clean[~nan])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [1, 200])
def test_sharp_and_flat_rows(dtype, news):
    """A zero query weighs all alike; a huge one picks one token; value scales
    far apart within a block of tokens and between pages; tokens far below the
    first one."""
    lens = [1000]
    g, c, table = make(lens, 1, 64, 9)
    c.byte["v"][table[0, 3]] = 127 - 60
    c.byte["v"][table[0, 4], 0, ::3] = 127 - 40
    c.byte["v"][table[0, 5], 0, 5, 1] = 127 + 30
    c.byte["v"][table[0, 6]] = 2
    c.byte["k"][table[0, 7]] = 60
    c.code["k"][table[0, 0], 0, 0] = 7
    q = queries(g, news, 16, 64, dtype)
    q[-1, 0] = 0
    q[-1, 1] *= 100
    q[-1, 2] = 0
    q[-1, 2, 0] = 1e-30
    q[-1, 3] = 0.5       # the first token, then nothing near it
    if dtype == "bf16":
        q = R.bf16(q)    # (what the call takes: a hundred times a bfloat16 value is none)
    start = [0, news]
    got = attend(to_gpu(c), seqs(table, lens, start), q, dtype)
    ref, b = M.attend(c, table, lens, start, q, 0.125, 0)
    near(got, ref, b, 64, 1000, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news", [([3000, 100], [1, 1]), ([400, 300], [200, 300])])
def test_out_may_be_q_and_capture(dtype, lens, news):
    import torch
    g, c, table = make(lens, 2, 128, 10)
    start = starts(news)
    q = queries(g, start[-1], 8, 128, dtype)
    cg, s = to_gpu(c), seqs(table, lens, start)
    want = attend(cg, s, q, dtype)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    first = torch.from_numpy(q).cuda().to(dt)
    qd = first.clone()
    ws = S.workspace(S.qmv_kv4_attend_workspace(cg, s, qd))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        S.qmv_kv4_attend(cg, s, qd, qd, workspace=ws, stream=st)
    for _ in range(3):
        qd.copy_(first)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(qd.float().cpu().numpy(), want)


def test_graph_as_lengths_grow():
    """One graph of a decode step, replayed as its sequences grow past what
    pieces the first length made, against eager calls."""
    import torch
    g, c, table = make([6000, 900], 2, 64, 14)
    lens = torch.tensor([1000, 64], dtype=torch.int32, device="cuda")
    i = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    s = S.KvSeqs(i(table), lens, i([0, 1, 2]), 1, 6000)
    cg = to_gpu(c)
    q = torch.from_numpy(queries(g, 2, 8, 64)).cuda()
    out, ref = torch.empty_like(q), torch.empty_like(q)
    ws = S.workspace(S.qmv_kv4_attend_workspace(cg, s, q))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        S.qmv_kv4_attend(cg, s, q, out, workspace=ws, stream=st)
    for n in ([1, 1], [1000, 64], [3000, 900], [6000, 1], [64, 65]):
        lens.copy_(i(n))
        graph.replay()
        S.qmv_kv4_attend(cg, s, q, ref)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        want, b = M.attend(c, table, n, [0, 1, 2], q.cpu().numpy(), 0.125, 0)
        near(out.cpu().numpy(), want, b, 64, max(n), "f32")


def test_two_calls_at_once():
    """Two streams, a workspace each, over one cache: as one after the other."""
    import torch
    g, c, table = make([6000, 900], 2, 128, 11)
    cg, s = to_gpu(c), seqs(table, [6000, 900], [0, 1, 2])
    qs = [queries(g, 2, 8, 128) for _ in range(2)]
    want = [attend(cg, s, q, "f32") for q in qs]
    qd = [torch.from_numpy(q).cuda() for q in qs]
    out = [torch.empty_like(x) for x in qd]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [S.workspace(S.qmv_kv4_attend_workspace(cg, s, qd[0])) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            S.qmv_kv4_attend(cg, s, qd[i], out[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(out[i].cpu().numpy(), want[i])


def test_cache_past_four_gib():
    """Pages whose codes lie beyond 32-bit offsets."""
    import torch
    heads, dim = 8, 256
    pages = (9 << 29) // (heads * PAGE * dim // 2)
    cg = S.Kv4Cache.empty(pages, heads, dim)
    g, c, table = make([250], heads, dim, 12)
    small = to_gpu(c)
    ids = [pages - 1, 3, pages - 2, pages // 2 + 7]
    for i, p in enumerate(ids):
        for name in ("k", "v", "k_scale", "v_scale"):
            getattr(cg, name)[p] = getattr(small, name)[int(table[0, i])]
    for dtype, new in (("f32", 1), ("bf16", 1), ("bf16", 100)):
        q = queries(g, new, 16, dim, dtype)
        got = attend(cg, seqs([ids], [250], [0, new]), q, dtype)
        want = attend(small, seqs(table, [250], [0, new]), q, dtype)
        assert np.array_equal(got, want)
    del cg
    torch.cuda.empty_cache()


def test_refuses_what_it_cannot_take():
    import torch
    g, c, table = make([5000], 2, 64, 13)
    cg, s = to_gpu(c), seqs(table, [5000], [0, 1])
    q = torch.zeros(1, 4, 64, device="cuda")
    with pytest.raises(Q.QmvError) as e:
        S.qmv_kv4_attend(cg, s, torch.zeros(1, 3, 64, device="cuda"), q[:, :3].contiguous())
    assert e.value.status == Q.QMV_E_SHAPE
    with pytest.raises(Q.QmvError) as e:
        S.qmv_kv4_attend(cg, s, q, q.clone(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == Q.QMV_E_ARG
    with pytest.raises(Q.QmvError):
        S.qmv_kv4_attend(cg, s, q, q.clone(), scale=float("nan"))
    with pytest.raises(TypeError):
        S.qmv_kv4_attend(cg, s, q, q.bfloat16())
    with pytest.raises(TypeError):
        S.qmv_kv4_attend(S.KvCache.empty(1, 2, 64), s, q, q)
    with pytest.raises(TypeError):
        S.qmv_kv_attend(cg, s, q, q)
    with pytest.raises(ValueError):
        S.qmv_kv4_attend(cg, s, torch.zeros(1, 4, 128, device="cuda"), q)
    with pytest.raises(ValueError):
        S.qmv_kv4_attend(cg, s, q, q.clone(), window=1 << 32)
