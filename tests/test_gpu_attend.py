"""qmv_kv_attend against plain attention in 64 bits over the values that the
cache stands for; the bound is derived in serve_ref.attend_bound."""
import numpy as np
import pytest

import serve_ref as R
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def make(lens, kv_heads, dim, seed, extra=2, spread=True):
    """A numpy cache of random codes and scales, and its table."""
    g = np.random.default_rng(seed)
    counts = [-(-n // PAGE) for n in lens]
    pages = sum(counts) + extra
    c = R.Cache(pages, kv_heads, dim)
    c.k = np.clip(np.rint(40 * g.standard_normal(c.k.shape)), -127, 127)
    c.v = np.clip(np.rint(40 * g.standard_normal(c.v.shape)), -127, 127)
    c.k_scale = 2.0 ** g.integers(-6, -4, size=c.k_scale.shape)
    c.v_scale = 2.0 ** (g.integers(-9, 3, size=c.v_scale.shape) if spread else np.full(c.v_scale.shape, -5))
    table = np.full((len(lens), max(max(counts), 1)), -1)
    ids = g.permutation(pages)
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = ids[at:at + n]
        at += n
    return g, c, table


def to_gpu(c):
    import torch
    return S.KvCache(torch.from_numpy(c.k.astype(np.int8)).cuda(),
                     torch.from_numpy(np.ascontiguousarray(c.v.transpose(0, 1, 3, 2)).astype(np.int8)).cuda(),
                     torch.from_numpy(c.k_scale.astype(np.float32)).cuda(),
                     torch.from_numpy(c.v_scale.astype(np.float32)).cuda())


def starts(news):
    s = [0]
    for m in news:
        s.append(s[-1] + m)
    return s


def seqs(table, lens, start, max_new=None, max_len=None):
    import torch
    def i32(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    news = [b - a for a, b in zip(start, start[1:])]
    return S.KvSeqs(i32(table), i32(lens), i32(start), max_new=max(news) if max_new is None else max_new,
                    max_len=max(lens) if max_len is None else max_len)


def attend(c, s, q, dtype, scale=None, window=0, rows=None):
    """Outputs as float32, from a workspace full of NaN."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    qd = torch.from_numpy(q).cuda().to(dt)
    out = torch.full(q.shape, 5.0, dtype=dt, device="cuda")
    n = S.qmv_kv_attend_workspace(c, s, qd, window)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    S.qmv_kv_attend(c, s, qd, out, scale=scale, window=window, workspace=ws)
    torch.cuda.synchronize()
    return out.float().cpu().numpy()


def queries(g, rows, heads, dim):
    return R.bf16(g.standard_normal((rows, heads, dim)).astype(np.float32))


def check(lens, news, heads, kv_heads, dim, dtype, seed, window=0, scale=None, spare=3, hints=None):
    g, c, table = make(lens, kv_heads, dim, seed)
    start = starts(news)
    q = queries(g, start[-1] + spare, heads, dim)
    if dtype == "f32":
        q = (q * np.float32(1.0003)).astype(np.float32)
    sc = dim ** -0.5 if scale is None else scale
    s = seqs(table, lens, start, *(hints or (None, None)))
    got = attend(to_gpu(c), s, q, dtype, scale, window)
    ref, b = R.attend(c, table, lens, start, q, np.float32(sc), window)
    tol = R.attend_bound(b, q, sc, max(lens), dtype)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    m = start[-1]
    err = np.abs(got[:m] - ref[:m])
    assert np.all(err <= tol[:m]), f"worst {np.nanmax(err / np.maximum(tol[:m], 1e-300)):.3g} of the bound"
    assert np.all(got[m:] == 5.0), "rows of no sequence were written"
    # a row that sees nothing is exactly 0
    assert np.all(got[:m][b["smax"][:m, :, 0] + b["vmax"][:m, :, 0] == 0] == 0)


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
    """Lengths at which the pages of a sequence are shared by many workgroups."""
    check([5000, 1200, 3], [1, 1, 1], 4, 2, 64, dtype, seed=1)
    check([4100], [3], 8, 1, 128, dtype, seed=2)
    check([3001], [2], 4, 2, 256, dtype, seed=3, window=2500)
    check([2500, 600], [40, 30], 4, 2, 128, dtype, seed=4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_rows_than_tokens(dtype):
    """Positions below 0 see nothing: zeros."""
    check([3, 0, 70], [5, 4, 80], 4, 2, 64, dtype, seed=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_hints_do_not_change_results(dtype):
    for hints in ((1, 1), (0, 0), (100000, 100000), (1, 100000)):
        check([700, 90], [40, 90], 8, 2, 64, dtype, seed=6, hints=hints)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_that_are_not_there(dtype):
    """Unknown page ids and positions past the table are left out; a row whose
    pages are all unknown gets zeros."""
    import torch
    g, c, table = make([300, 200, 70], 2, 64, 7)
    table = table[:, :4].copy()
    table[0, 1], table[0, 3] = -5, c.pages
    table[1, :] = -1
    table[2, 0] = 2147483647
    lens, start = [300, 200, 70], [0, 2, 5, 75]
    q = queries(g, 75, 4, 64)
    got = attend(to_gpu(c), seqs(table, lens, start), q, dtype)
    ref, b = R.attend(c, table, lens, start, q, 0.125, 0)
    tol = R.attend_bound(b, q, 0.125, 300, dtype)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol)
    assert np.all(got[2:5] == 0) and np.all(got[5:69] == 0) and np.any(got[69:] != 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [[1, 1, 1], [70, 80, 65]])
def test_nan_touches_only_what_sees_it(dtype, news):
    """NaN scales of pages that are masked (later pages, pages outside the
    window) leave a row as it is; where they are seen, and for a NaN or
    infinite query, the row and head is NaN."""
    lens = [200, 200, 200]
    g, c, table = make(lens, 2, 64, 8, spread=False)
    start = starts(news)
    rows = start[-1]
    q = queries(g, rows, 4, 64)
    window = 30
    clean = attend(to_gpu(c), seqs(table, lens, start), q, dtype, window=window)
    c.k_scale[table[0, 2], 0] = np.nan          # positions 128 .. 191, heads 0 and 1
    c.v_scale[table[1, 2], 1] = np.nan          # heads 2 and 3
    c.k_scale[table[1, 0], :] = np.nan          # outside every row's window
    c.v_scale[table[2, 0], :] = np.nan
    q[start[2] - 1, 0, 5] = np.nan              # the last row of sequence 1
    q[rows - 1, 3, 0] = np.inf
    got = attend(to_gpu(c), seqs(table, lens, start), q, dtype, window=window)
    nan = np.zeros((rows, 4), dtype=bool)
    for i, page, heads in ((0, 2, (0, 1)), (1, 2, (2, 3))):
        for t in range(news[i]):
            pos = 200 - news[i] + t
            if pos >= page * 64 and pos - window + 1 < page * 64 + 64:
                nan[start[i] + t, list(heads)] = True
    nan[start[2] - 1, 0] = True
    nan[rows - 1, 3] = True
    assert np.array_equal(np.isnan(got).any(-1), nan) and np.array_equal(np.isnan(got).all(-1), nan)
    assert np.array_equal(got[~nan], clean[~nan])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [1, 80])
def test_sharp_and_flat_rows(dtype, news):
    """A zero query weighs all alike; a huge one picks one token; V scales far
    apart; zero pages of K and V; many tokens far below the first one."""
    lens = [1000]
    g, c, table = make(lens, 1, 64, 9)
    c.v_scale[table[0, 3]] = 2.0 ** -60
    c.v_scale[table[0, 4]] = 0
    c.k_scale[table[0, 5]] = 0
    c.k[table[0, 0], 0, 0] = 127
    q = queries(g, news, 4, 64)
    q[-1, 0] = 0
    q[-1, 1] *= 100
    q[-1, 2] = 0
    q[-1, 2, 0] = 1e-30
    q[-1, 3] = 0.5       # the first token, then nothing near it
    start = [0, news]
    got = attend(to_gpu(c), seqs(table, lens, start), q, dtype)
    ref, b = R.attend(c, table, lens, start, q, 0.125, 0)
    tol = R.attend_bound(b, q, 0.125, 1000, dtype)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news", [([3000, 100], [1, 1]), ([400, 300], [200, 300])])
def test_out_may_be_q_and_capture(dtype, lens, news):
    import torch
    g, c, table = make(lens, 2, 128, 10)
    start = starts(news)
    q = queries(g, start[-1], 8, 128)
    cg, s = to_gpu(c), seqs(table, lens, start)
    want = attend(cg, s, q, dtype)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    first = torch.from_numpy(q).cuda().to(dt)
    qd = first.clone()
    ws = S.workspace(S.qmv_kv_attend_workspace(cg, s, qd))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        S.qmv_kv_attend(cg, s, qd, qd, workspace=ws, stream=st)
    for _ in range(3):
        qd.copy_(first)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(qd.float().cpu().numpy(), want)


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
    ws = [S.workspace(S.qmv_kv_attend_workspace(cg, s, qd[0])) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            S.qmv_kv_attend(cg, s, qd[i], out[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(out[i].cpu().numpy(), want[i])


def test_cache_past_four_gib():
    """Pages whose codes lie beyond 32-bit offsets."""
    import torch
    heads, dim = 8, 256
    pages = (5 << 30) // (heads * PAGE * dim)
    c = S.KvCache.empty(pages, heads, dim)
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = [pages - 1, 3, pages - 2, pages // 2 + 7]
    small = R.Cache(4, heads, dim)
    for i, p in enumerate(ids):
        for t in (c.k, c.v):
            t[p] = torch.randint(-127, 128, t[p].shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
        c.k_scale[p], c.v_scale[p] = 2.0 ** -7, 2.0 ** -6
        small.k[i], small.v[i] = c.k[p].cpu().numpy(), c.v[p].cpu().numpy().transpose(0, 2, 1)
    small.k_scale[:], small.v_scale[:] = 2.0 ** -7, 2.0 ** -6
    lens, rng = [250], np.random.default_rng(12)
    for dtype, new in (("f32", 1), ("bf16", 1), ("bf16", 100)):
        q = queries(rng, new, 16, dim)
        got = attend(c, seqs([ids], lens, [0, new]), q, dtype)
        ref, b = R.attend(small, [[0, 1, 2, 3]], lens, [0, new], q, dim ** -0.5, 0)
        tol = R.attend_bound(b, q, dim ** -0.5, 250, dtype)
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert np.all(np.abs(got - ref) <= tol)


def test_refuses_what_it_cannot_take():
    import torch
    g, c, table = make([5000], 2, 64, 13)
    cg, s = to_gpu(c), seqs(table, [5000], [0, 1])
    q = torch.zeros(1, 4, 64, device="cuda")
    with pytest.raises(Q.QmvError) as e:
        S.qmv_kv_attend(cg, s, torch.zeros(1, 3, 64, device="cuda"), q[:, :3].contiguous())
    assert e.value.status == Q.QMV_E_SHAPE
    with pytest.raises(Q.QmvError) as e:
        S.qmv_kv_attend(cg, s, q, q.clone(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == Q.QMV_E_ARG
    with pytest.raises(Q.QmvError):
        S.qmv_kv_attend(cg, s, q, q.clone(), scale=float("nan"))
    with pytest.raises(TypeError):
        S.qmv_kv_attend(cg, s, q, q.bfloat16())
    with pytest.raises(ValueError):
        S.qmv_kv_attend(cg, s, torch.zeros(1, 4, 128, device="cuda"), q)
    with pytest.raises(ValueError):
        S.qmv_kv_attend(cg, s, q[0], q)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 3, 4])
def test_single_tokens_of_up_to_four_heads(group, dim):
    """Decode: the columns of one product, over lengths of a page and beside it."""
    for dtype in ("f32", "bf16"):
        check([1, 64, 200, 0, 131], [1, 1, 1, 0, 1], 2 * group, 2, dim, dtype, seed=group + dim)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_short_sequences(dtype):
    """More sequences than compute units, some without tokens or rows."""
    g = np.random.default_rng(11)
    lens = [int(n) for n in g.integers(0, 140, size=400)]
    check(lens, [int(n > 0 and n % 7 != 3) for n in lens], 3, 1, 64, dtype, seed=12)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hints", [(1, 1), (200, 100000), (0, 0), (33, 64)])
def test_any_hints(hints, dtype):
    """Hints far from the truth choose another launch, of other tiles and pieces."""
    check([300, 9, 1500], [9, 9, 1], 4, 1, 64, dtype, seed=13, hints=hints)
    check([150, 140], [150, 130], 2, 1, 256, dtype, seed=14, hints=hints)


@pytest.mark.parametrize("window", [0, 40, 130])
@pytest.mark.parametrize("lens,news,heads,kv_heads", [
    ([300, 190], [150, 128], 2, 2), ([130, 70, 600], [129, 70, 45], 12, 4), ([257], [257], 5, 5)])
def test_wide_heads_of_many_rows(lens, news, heads, kv_heads, window):
    check(lens, news, heads, kv_heads, 256, "bf16", seed=sum(lens) + window, window=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [1, 140])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_maxima_that_grow_and_values_far_apart(dim, news, dtype):
    """Keys that double from page to page, so that each page's largest score
    is far above the last one's; values' scales between 2^-40 and 2^40."""
    g, c, table = make([700], 1, dim, seed=dim + news)
    for n, page in enumerate(table[0]):
        c.k_scale[page] = 2.0 ** (n - 11)
        c.v_scale[page] = 2.0 ** int(g.integers(-40, 41))
    q = queries(g, news, 2, dim)
    ref, b = R.attend(c, table, [700], [0, news], q, np.float32(dim ** -0.5), 0)
    got = attend(to_gpu(c), seqs(table, [700], [0, news]), q, dtype)
    tol = R.attend_bound(b, q, dim ** -0.5, 700, dtype)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_any_scale(scale, dtype):
    check([200, 90], [3, 1], 4, 2, 64, dtype, seed=15, scale=scale)
    check([260], [140], 2, 2, 128, dtype, seed=16, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [1, 150])
def test_length_past_the_table(news, dtype):
    """A sequence that claims 2^31 - 1 tokens of a table of four pages: its
    rows see what is there."""
    g, c, table = make([256], 2, 64, seed=17)
    q = queries(g, news, 2, 64)
    got = attend(to_gpu(c), seqs(table, [2 ** 31 - 1], [0, news], max_len=256), q, dtype)
    ref, b = R.attend(c, np.repeat(table, news, 0), [256] * news, list(range(news + 1)), q, np.float32(0.125), 0)
    tol = R.attend_bound(b, q, 0.125, 256, dtype)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol)


def test_device_and_streams(monkeypatch):
    """A cache of another device is refused; a call on a stream without a
    workspace allocates one in that stream's order."""
    import torch
    g, c, table = make([3000], 1, 64, seed=18)
    cg, s = to_gpu(c), seqs(table, [3000], [0, 1])
    qd = torch.from_numpy(queries(g, 1, 4, 64)).cuda()
    want, got = torch.empty_like(qd), torch.empty_like(qd)
    assert S.qmv_kv_attend_workspace(cg, s, qd) > 0
    S.qmv_kv_attend(cg, s, qd, want)
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        got.zero_()
        torch.cuda.synchronize()
        S.qmv_kv_attend(cg, s, qd, got, stream=stream)
        st.synchronize()
        assert torch.equal(got, want)
    monkeypatch.setattr(cg, "device", 1)
    with pytest.raises(ValueError, match="device"):
        S.qmv_kv_attend(cg, s, qd, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_wave_for_each_tile(dim, dtype):
    """Many short pieces: 40 sequences, some without rows, ends inside a tile
    of 16 columns and inside a workgroup's four."""
    g = np.random.default_rng(19)
    lens = [int(n) for n in g.integers(1, 120, size=40)]
    news = [min(n, int(m)) for n, m in zip(lens, g.integers(0, 40, size=40))]
    check(lens, news, 5 if dim == 64 else 3, 1, dim, dtype, seed=20)
    check([130, 20], [130, 20], 4, 4, dim, dtype, seed=21, window=40, hints=(130, 64))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_pages_than_a_wave_looks_up_at_once(dtype):
    """More than 64 pages in one wave."""
    check([4500], [70], 64, 1, 64, dtype, seed=22, hints=(70, 64))


@pytest.mark.parametrize("dim,scale", [(64, 0.125), (64, 0.5), (128, 0.25), (256, 0.0625)])
def test_digits_of_a_probability_agree(dim, scale):
    """Some 800000 probabilities that matter, whose digits are made in
    different lanes: one whose lanes differ by a last bit next to a border of
    a digit is off by a hundredth of itself."""
    check([64] * 400, [1] * 400, 32, 8, dim, "f32", seed=23, scale=scale)


def test_refuses_negative_sizes():
    import torch
    g, c, table = make([100], 1, 64, seed=25)
    for new, longest in ((-1, 100), (1, -100)):
        with pytest.raises(ValueError):
            seqs(table, [100], [0, 1], new, longest)
    q = torch.zeros(1, 2, 64, device="cuda")
    s = seqs(table, [100], [0, 1])
    with pytest.raises(ValueError):
        S.qmv_kv_attend(to_gpu(c), s, q, q, window=-1)
    with pytest.raises(ValueError):
        S.qmv_kv_attend_workspace(to_gpu(c), s, q, window=-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_shared_by_sequences(dtype):
    """Two sequences with the same first pages, and a page twice in a table."""
    g, c, table = make([300, 250], 2, 128, seed=26)
    table[1, :3] = table[0, :3]
    table[0, 3] = table[0, 1]
    start, lens = [0, 1, 41], [300, 250]
    q = queries(g, 41, 6, 128)
    got = attend(to_gpu(c), seqs(table, lens, start), q, dtype)
    sc = np.float32(128 ** -0.5)
    ref, b = R.attend(c, table, lens, start, q, sc, 0)
    tol = R.attend_bound(b, q, sc, 300, dtype)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol)


def held(c, table, lens, start, q, dtype, window=0, b=None):
    """A call against its reference; b: what replaces the bound's sizes."""
    dim = q.shape[2]
    got = attend(to_gpu(c), seqs(table, lens, start), q, dtype, window=window)
    ref, sizes = R.attend(c, table, lens, start, q, np.float32(dim ** -0.5), window)
    sizes.update(b or {})
    tol = R.attend_bound(sizes, q, dim ** -0.5, max(lens), dtype)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(got[:start[-1]] - ref[:start[-1]])
    assert np.all(err <= tol[:start[-1]]), f"worst {np.nanmax(err / np.maximum(tol[:start[-1]], 1e-300)):.3g} of the bound"


# exponents of the values' scales, page by page: a large page that later rows of
# the tile do not see, at the borders of what f16 holds of the smaller ones (24
# below it) and far past them; a small page that earlier rows see alone; up to
# 2^96 apart
FAR = [[0, -20, -24, -5], [0, -25, -25, -26], [0, -30, 0, -30], [-40, 0, -41, 5], [6, -18, 5, 11],
       [10, -70, -72, 24], [-60, 30, -60, 36], [-90, -90, 5, -90], [36, 36, -20, -60]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exps", FAR, ids=lambda e: "_".join(map(str, e)))
def test_scales_of_pages_that_a_row_does_not_see(exps, dim, dtype):
    """Rows under a window, each held against the values that it sees itself."""
    narrow_windows(exps, dim, dtype, (1, 20, 64))


def narrow_windows(exps, dim, dtype, windows):
    g, c, table = make([64 * len(exps)], 1, dim, seed=27)
    for page, e in zip(table[0], exps):
        c.v_scale[page] = 2.0 ** e
    q = queries(g, 200, 2, dim)
    for window in windows:
        held(c, table, [64 * len(exps)], [0, 200], q, dtype, window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exps", FAR, ids=lambda e: "_".join(map(str, e)))
def test_scales_of_pages_without_weight(exps, dim, dtype):
    """No window, but keys so that every row's weight lies on its own page: the
    earlier pages' is below e^-200 of it, where neither float32 nor float16 has
    anything left, so each row is held against its own page's values."""
    g, c, table = make([64 * len(exps)], 1, dim, seed=28)
    for n, page in enumerate(table[0]):
        c.v_scale[page] = 2.0 ** exps[n]
        c.k_scale[page] = 2.0 ** -6
        c.k[page] = np.rint(c.k[page] / 40)
        c.k[page, 0, :, 0] = 20 * n
    q = queries(g, 200, 2, dim)
    q[:, :, 0] = 64 * 12 * dim ** 0.5              # a score of 240 a page
    q = R.bf16(q.astype(np.float32))
    own = np.zeros((200, 2, 1))
    for t in range(200):
        pos = 64 * len(exps) - 200 + t
        own[t] = np.abs(c.v[table[0, pos // 64], 0]).max() * 2.0 ** exps[pos // 64]
    held(c, table, [64 * len(exps)], [0, 200], q, dtype, b={"vmax": own})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exps", [[0, -105, -112, 0], [50, -100, -120, -126], [-60, 50, -75, -126], [50, 0, -126, -60]],
                         ids=lambda e: "_".join(map(str, e)))
def test_scales_further_apart_than_float32(exps, dim, dtype):
    """Rows that see all of the pages: what is far below the rest does not show,
    and nothing leaves float32 on the way."""
    g, c, table = make([64 * len(exps)], 1, dim, seed=29)
    for page, e in zip(table[0], exps):
        c.v_scale[page] = 2.0 ** e
    held(c, table, [64 * len(exps)], [0, 64], queries(g, 64, 2, dim), dtype)
