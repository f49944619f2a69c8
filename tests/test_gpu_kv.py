"""qmv_kv_write and qmv_kv_read against the cache in plain numpy: codes,
scales and values bit for bit, over many calls that fill, rescale, roll back
and begin pages anew; what a call must not touch stays as it was."""
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


class Pair:
    """A cache on the GPU and the same one in numpy."""

    def __init__(self, pages, heads, dim):
        import torch
        self.ref = R.Cache(pages, heads, dim)
        self.gpu = S.KvCache(torch.zeros(pages, heads, PAGE, dim, dtype=torch.int8, device="cuda"),
                             torch.zeros(pages, heads, dim, PAGE, dtype=torch.int8, device="cuda"),
                             torch.zeros(pages, heads, device="cuda"), torch.zeros(pages, heads, device="cuda"))

    def seqs(self, table, lens, news, max_new=None):
        import torch
        start = [0]
        for m in news:
            start.append(start[-1] + m)
        self.start = start
        t = torch.tensor(np.asarray(table), dtype=torch.int32, device="cuda")
        return S.KvSeqs(t, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                        torch.tensor(start, dtype=torch.int32, device="cuda"),
                        max_new=max(news) if max_new is None else max_new, max_len=max(lens))

    def write(self, table, lens, news, k, v, dtype="f32", max_new=None):
        import torch
        s = self.seqs(table, lens, news, max_new)
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        S.qmv_kv_write(self.gpu, s, torch.from_numpy(k).cuda().to(dt), torch.from_numpy(v).cuda().to(dt))
        torch.cuda.synchronize()
        self.ref.write(table, lens, self.start, k, v)

    def check(self, what=""):
        k = self.gpu.k.cpu().numpy()
        v = self.gpu.v.cpu().numpy().transpose(0, 1, 3, 2)
        ks, vs = self.gpu.k_scale.cpu().numpy(), self.gpu.v_scale.cpu().numpy()
        assert np.array_equal(ks, self.ref.k_scale.astype(np.float32), equal_nan=True), what
        assert np.array_equal(vs, self.ref.v_scale.astype(np.float32), equal_nan=True), what
        assert np.array_equal(k, self.ref.k), what
        assert np.array_equal(v, self.ref.v), what

    def check_read(self, table, lens, news, dtype="f32", rows=None):
        import torch
        s = self.seqs(table, lens, news)
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        n = self.start[-1] if rows is None else rows
        k = torch.full((n, self.ref.heads, self.ref.dim), 7.0, dtype=dt, device="cuda")
        v = torch.full_like(k, 9.0)
        S.qmv_kv_read(self.gpu, s, k, v)
        torch.cuda.synchronize()
        m = self.start[-1]
        for got, what, fill in ((k, "k", 7.0), (v, "v", 9.0)):
            got = got.float().cpu().numpy()
            assert np.array_equal(got[:m], self.ref.read(table, lens, self.start, what, m).astype(np.float32),
                                  equal_nan=True), what
            assert np.all(got[m:] == fill), "rows of no sequence were written"


def normal(g, n, heads, dim, size=1.0):
    return R.bf16((size * g.standard_normal((n, heads, dim))).astype(np.float32))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_of_odd_lengths(dim, dtype):
    g = np.random.default_rng(dim)
    lens = [1, 63, 64, 65, 200, 0]
    table = np.full((6, 5), -1)
    ids = g.permutation(20)
    at = 0
    for i, n in enumerate(lens):
        c = -(-n // PAGE)
        table[i, :c] = ids[at:at + c]
        at += c
    p = Pair(20, 3, dim)
    n = sum(lens)
    k, v = normal(g, n, 3, dim), normal(g, n, 3, dim, 0.1)
    if dtype == "f32":
        k = (k * np.float32(1.0001)).astype(np.float32)
    p.write(table, lens, lens, k, v, dtype)
    p.check()
    p.check_read(table, lens, lens, dtype)
    p.check_read(table, lens, [1, 1, 64, 2, 130, 0], dtype, rows=203)


def test_tokens_one_by_one_rescale():
    """A page filled token by token with values that grow: codes are rescaled
    each time, and every value stays within one final scale."""
    g = np.random.default_rng(2)
    p = Pair(4, 2, 64)
    table = np.array([[2, 0], [3, 1]])
    size = np.exp(np.linspace(-3, 3, 100))
    k = np.stack([normal(g, 2, 2, 64, s) for s in size])      # [step, seq, heads, dim]
    v = np.stack([normal(g, 2, 2, 64, s) for s in size[::-1]])
    for t in range(100):
        p.write(table, [t + 1, t + 1], [1, 1], k[t], v[t])
        if t % 9 == 0 or t > 60:
            p.check(t)
    p.check_read(table, [100, 100], [100, 70])
    for what, x in (("k", k), ("v", v)):
        got, _ = p.ref.rows(table[0], 100, what)
        scale = (p.ref.k_scale if what == "k" else p.ref.v_scale)[table[0][np.arange(100) // PAGE]]
        assert np.all(np.abs(got - x[:, 0]) <= scale[:, :, None])


@pytest.mark.parametrize("dim", [64, 256])
def test_roll_back_and_pieces(dim):
    """Pieces that start and end inside pages, then a shorter length written
    over, then a page begun anew by another sequence."""
    g = np.random.default_rng(4)
    p = Pair(6, 2, dim)
    table = np.array([[5, 1, 3, 0]])
    for length, new, size in ((30, 30, 1.0), (50, 20, 5.0), (64, 14, 0.1), (150, 86, 1.0), (151, 1, 9.0),
                              (140, 6, 2.0), (128, 1, 40.0), (130, 2, 0.01), (256, 126, 0.5)):
        k, v = normal(g, new, 2, dim, size), normal(g, new, 2, dim, 1 / size)
        p.write(table, [length], [new], k, v)
        p.check((length, new))
        p.check_read(table, [length], [length])
    other = np.array([[1, 2]])
    p.write(other, [70], [70], normal(g, 70, 2, dim, 0.001), normal(g, 70, 2, dim, 0.001))
    p.check("begun anew")


def test_hints_do_not_change_results():
    g = np.random.default_rng(6)
    p = Pair(12, 1, 64)
    table = g.permutation(12).reshape(2, 6)
    k, v = normal(g, 500, 1, 64), normal(g, 500, 1, 64)
    p.write(table, [300, 200], [300, 200], k, v, max_new=1)
    p.check()
    s = p.seqs(table, [300, 200], [300, 200], max_new=0)
    import torch
    out = torch.empty(500, 1, 64, device="cuda")
    S.qmv_kv_read(p.gpu, s, out)
    assert np.array_equal(out.cpu().numpy(), p.ref.read(table, [300, 200], [0, 300, 500], "k", 500).astype(np.float32))


def test_places_that_are_not_there():
    """Pages outside the cache, positions below 0 and past the table: nothing
    is written, zeros are read."""
    g = np.random.default_rng(8)
    p = Pair(5, 2, 64)
    table = np.array([[0, -1, 2], [5, 1, 2147483647], [3, 4, -2147483648]])
    lens, news = [150, 100, 260], [150, 100, 100]             # the third one's last tokens are past the table
    n = sum(news)
    p.write(table, lens, news, normal(g, n, 2, 64), normal(g, n, 2, 64))
    p.check()
    p.check_read(table, lens, news)
    p.check_read(table, [3, 0, 10], [10, 5, 70])              # more rows than tokens
    before = [t.clone() for t in (p.gpu.k, p.gpu.v, p.gpu.k_scale, p.gpu.v_scale)]
    p.write(table, [0, 0, 0], [4, 0, 3], normal(g, 7, 2, 64), normal(g, 7, 2, 64))
    for a, b in zip(before, (p.gpu.k, p.gpu.v, p.gpu.k_scale, p.gpu.v_scale)):
        assert bool((a == b).all())


def test_starts_out_of_range_are_held():
    """start beyond the rows, or decreasing: rows are held to the array."""
    import torch
    g = np.random.default_rng(9)
    p = Pair(4, 1, 64)
    table = torch.tensor([[0], [1], [2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 5, 5], dtype=torch.int32, device="cuda")
    start = torch.tensor([-3, 4, 2, 1000], dtype=torch.int32, device="cuda")   # rows 0-3, none, 2-9
    k, v = normal(g, 10, 1, 64), normal(g, 10, 1, 64)
    s = S.KvSeqs(table, lens, start, max_new=5, max_len=5)
    S.qmv_kv_write(p.gpu, s, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    torch.cuda.synchronize()
    t = np.array([[0], [1], [2]])
    p.ref.write(t[:1], [5], [0, 4], k, v)
    p.ref.write(t[2:], [5], [2, 10], k, v)
    p.check()


def test_extreme_values():
    """Zero pages, the ends of the range, infinities and NaN."""
    g = np.random.default_rng(10)
    p = Pair(8, 2, 64)
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 7]])
    k = normal(g, 40, 2, 64)
    v = normal(g, 40, 2, 64)
    k[0:10] = 0
    v[0:10, 0] = 0
    k[10:20] *= np.float32(2.0 ** 125)
    v[10:20] *= np.float32(2.0 ** -130)
    k[20, 0, 0] = np.float32(3.4028235e38)
    v[20:30, 1] = np.float32(1e-45)
    k[35, 1, 3] = np.inf
    v[36, 0, 9] = np.nan
    p.write(table, [10, 10, 10, 10], [10, 10, 10, 10], k, v)
    p.check()
    p.check_read(table, [10, 10, 10, 10], [10, 10, 10, 10])
    p.check_read(table, [10, 10, 10, 10], [10, 10, 10, 10], "bf16")
    # later tokens: a zero page gets a scale, a NaN one stays, until begun anew
    k2, v2 = normal(g, 40, 2, 64), normal(g, 40, 2, 64)
    p.write(table, [20, 20, 20, 20], [10, 10, 10, 10], k2, v2)
    p.check()
    assert np.isnan(p.ref.k_scale[6, 1]) and np.isnan(p.ref.v_scale[6, 0])
    p.write(table[3:], [8], [8], k2[:8], v2[:8])
    p.check()
    assert np.all(np.isfinite(p.ref.k_scale))


def test_halves_and_scale_borders():
    """x / d on halves rounds to even; amax at 127 d and just above."""
    p = Pair(5, 1, 64)
    k = np.zeros((5, 1, 64), dtype=np.float32)
    k[0, 0] = np.arange(64) / 2
    k[0, 0, 63] = 127.0                                      # d = 1
    k[1, 0, 0] = np.nextafter(np.float32(127.0), np.float32(200.0))
    k[1, 0, 1:4] = (1.0, 3.0, 5.0)                           # d = 2: halves
    k[2, 0, 0] = 127.0 * 2.0 ** -126
    k[3, 0, 0] = np.nextafter(np.float32(127.0 * 2.0 ** 120), np.float32(1e38))       # just below
    k[4, 0, 0] = np.nextafter(np.float32(127.0 * 2.0 ** 120), np.float32(np.inf))     # just above
    p.write(np.array([[0], [1], [2], [3], [4]]), [1] * 5, [1] * 5, k, -k)
    p.check()
    assert [float(s) for s in p.ref.k_scale[:, 0]] == [1.0, 2.0, 2.0 ** -126, 2.0 ** 120, 2.0 ** 121]


def test_one_of_two_and_capture():
    import torch
    g = np.random.default_rng(12)
    p = Pair(4, 2, 128)
    table = np.array([[3, 1]])
    k, v = normal(g, 100, 2, 128), normal(g, 100, 2, 128)
    s = p.seqs(table, [100], [100])
    kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    out = torch.empty(100, 2, 128, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        S.qmv_kv_write(p.gpu, s, kd, vd, stream=st)
        S.qmv_kv_read(p.gpu, s, None, out, stream=st)
    p.ref.write(table, [100], p.start, k, v)
    want = p.ref.read(table, [100], p.start, "v", 100).astype(np.float32)
    for _ in range(3):
        p.gpu.v.zero_()
        out.fill_(np.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), want)
        p.check()


def test_refuses_what_it_cannot_take():
    import torch
    p = Pair(4, 2, 64)
    s = p.seqs(np.array([[0]]), [3], [3])
    k = torch.zeros(3, 2, 64, device="cuda")
    for bad in (k[:, :1], k[..., :32].contiguous(), k.half(), k.transpose(0, 1)):
        with pytest.raises((ValueError, TypeError)):
            S.qmv_kv_write(p.gpu, s, bad, k)
    with pytest.raises(TypeError):
        S.qmv_kv_write(p.gpu, s, k, k.bfloat16())
    with pytest.raises(ValueError):
        S.qmv_kv_write(p.gpu, s, k, k[:2])
    with pytest.raises(Q.QmvError):
        S.qmv_kv_read(p.gpu, s)
    c = p.gpu
    with pytest.raises(ValueError):
        S.KvCache(c.k[:, :, :32].contiguous(), c.v, c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        S.KvCache(c.k, c.k, c.k_scale[:3], c.v_scale)
    with pytest.raises(ValueError):
        S.KvSeqs(s.table[0], s.len, s.start, 3, 3)
    with pytest.raises(ValueError):
        S.KvSeqs(s.table, s.len, s.start[:1], 3, 3)
    with pytest.raises(TypeError):
        S.KvSeqs(s.table.long(), s.len, s.start, 3, 3)
