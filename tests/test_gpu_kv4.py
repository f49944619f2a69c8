"""qmv_kv4_write and qmv_kv4_read against plain quantization: the same bytes,
and the same values read back."""
import numpy as np
import pytest

import more_ref as M
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


def to_gpu(c):
    import torch
    k, v, ks, vs = (torch.from_numpy(a).cuda() for a in c.arrays())
    codes, scales = (c.pages, c.heads, 64, c.dim // 2), (c.pages, c.heads, 64, c.dim // 32)
    return S.Kv4Cache(k.view(codes), v.view(codes), ks.view(scales), vs.view(scales))


def same_bytes(gpu, c):
    for t, a in zip((gpu.k, gpu.v, gpu.k_scale, gpu.v_scale), c.arrays()):
        assert np.array_equal(t.cpu().numpy().reshape(a.shape), a)


def seqs(table, lens, start, max_new=None, max_len=None):
    import torch
    i = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    news = [b - a for a, b in zip(start, start[1:])]
    return S.KvSeqs(i(table), i(lens), i(start), max(news) if max_new is None else max_new, max(lens) if max_len is None else max_len)


def tokens(g, rows, heads, dim, dtype):
    x = g.standard_normal((rows, heads, dim)) * 2.0 ** g.integers(-8, 9, size=(rows, heads, 1))
    x = x.astype(np.float32)
    return R.bf16(x) if dtype == "bf16" else x


def put(x, dtype):
    import torch
    return torch.from_numpy(x).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16)


def read_back(gpu, s, rows, heads, dim, dtype):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    k, v = (torch.full((rows, heads, dim), 5.0, dtype=dt, device="cuda") for _ in range(2))
    S.qmv_kv4_read(gpu, s, k, v)
    torch.cuda.synchronize()
    return k.float().cpu().numpy(), v.float().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 3])
def test_write_and_read(dim, heads, dtype):
    """Prompts, then tokens over page ends; every byte, and what is read."""
    g = np.random.default_rng(dim + heads)
    c = M.Cache4(9, heads, dim)
    gpu = to_gpu(c)
    table = np.array([[8, 2, 5], [0, 3, 1], [6, 4, 7]])
    lens, start = [100, 63, 1], [0, 100, 163, 164]
    for turn in range(3):
        rows = start[-1] + 2                      # two rows of no sequence
        k, v = tokens(g, rows, heads, dim, dtype), tokens(g, rows, heads, dim, dtype)
        s = seqs(table, lens, start)
        S.qmv_kv4_write(gpu, s, put(k, dtype), put(v, dtype))
        c.write(table, lens, start, k, v)
        same_bytes(gpu, c)
        got = read_back(gpu, s, rows, heads, dim, dtype)
        for x, what in zip(got, "kv"):
            ref = c.read(table, lens, start, what, rows)
            assert np.array_equal(x[:start[-1]], ref[:start[-1]].astype(np.float32))
            assert np.all(x[start[-1]:] == 5.0)
        new = [1, 2, 70][turn]
        lens = [n + new for n in lens] if turn < 2 else lens
        start = [0, new, 2 * new, 3 * new]


def test_every_rounding():
    """Values at, below and above the middle between neighbours, at the ends
    of the scales, zeros of both signs, subnormals."""
    edge = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.5, 7])
    around = np.concatenate([np.nextafter(edge.astype(np.float32), np.float32(-9)), edge.astype(np.float32),
                             np.nextafter(edge.astype(np.float32), np.float32(9))]).astype(np.float32)
    around = around[np.abs(around) <= 7]
    rows = []
    for exp in (-149, -140, -126, -125, -124, -40, 0, 1, 60, 124, 125):
        for at in range(0, len(around), 30):
            part = np.zeros(32, np.float64)
            part[:len(around[at:at + 30])] = around[at:at + 30]
            part[30], part[31] = 7.0, -0.0
            with np.errstate(over="ignore"):
                x = (part * 2.0 ** exp).astype(np.float32)
            rows.append(np.where(np.isfinite(x), x, np.float32(3e38)))
            rows.append(-rows[-1])
    rows.append(np.zeros(32, np.float32))
    while len(rows) % 2:
        rows.append(np.zeros(32, np.float32))
    x = np.stack(rows).reshape(-1, 1, 64)
    n = len(x)
    assert n <= 64
    c = M.Cache4(1, 1, 64)
    gpu = to_gpu(c)
    s = seqs([[0]], [n], [0, n])
    S.qmv_kv4_write(gpu, s, put(x, "f32"), put(-x, "f32"))
    c.write([[0]], [n], [0, n], x, -x)
    same_bytes(gpu, c)
    k, v = read_back(gpu, s, n, 1, 64, "f32")
    assert np.array_equal(k, c.read([[0]], [n], [0, n], "k", n).astype(np.float32))
    assert np.array_equal(v, -k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_numbers(dtype):
    """A NaN or infinity makes its token's keys and values of that head NaN,
    and no others; writing the token again heals it."""
    g = np.random.default_rng(5)
    k, v = tokens(g, 70, 2, 128, dtype), tokens(g, 70, 2, 128, dtype)
    fine = k.copy(), v.copy()
    k[3, 0, 17], v[5, 1, 127], k[69, 1, 0], v[64, 0, 64] = np.nan, np.inf, -np.inf, np.nan
    c = M.Cache4(2, 2, 128)
    gpu = to_gpu(c)
    s = seqs([[1, 0]], [70], [0, 70])
    S.qmv_kv4_write(gpu, s, put(k, dtype), put(v, dtype))
    c.write([[1, 0]], [70], [0, 70], k, v)
    same_bytes(gpu, c)
    bad = {(3, 0), (5, 1), (69, 1), (64, 0)}
    for x in read_back(gpu, s, 70, 2, 128, dtype):
        nan = np.isnan(x)
        assert np.array_equal(nan.any(-1), nan.all(-1))
        assert {(int(a), int(b)) for a, b in zip(*np.nonzero(nan.any(-1)))} == bad
    S.qmv_kv4_write(gpu, s, put(fine[0], dtype), put(fine[1], dtype))
    assert all(np.isfinite(x).all() for x in read_back(gpu, s, 70, 2, 128, dtype))


@pytest.mark.parametrize("dim", [64, 256])
def test_places_that_are_not_there(dim):
    """Unknown pages, positions past the table or below 0: nothing written,
    zeros read; nothing else of the cache changes."""
    g = np.random.default_rng(6)
    c = M.Cache4(4, 2, dim)
    for n in "kv":
        c.code[n][:] = g.integers(0, 16, size=c.code[n].shape)
        c.byte[n][:] = g.integers(100, 140, size=c.byte[n].shape)
    gpu = to_gpu(c)
    table = np.array([[1, -3], [4, 0], [2147483647, 2]])
    lens, start = [128, 150, 3], [0, 100, 150, 158]
    k, v = tokens(g, 158, 2, dim, "f32"), tokens(g, 158, 2, dim, "f32")
    s = seqs(table, lens, start)
    S.qmv_kv4_write(gpu, s, put(k, "f32"), put(v, "f32"))
    c.write(table, lens, start, k, v)
    same_bytes(gpu, c)
    for x, what in zip(read_back(gpu, s, 158, 2, dim, "f32"), "kv"):
        assert np.array_equal(x, c.read(table, lens, start, what, 158).astype(np.float32))


def test_hints_one_array_and_bad_starts():
    """Hints only shape the launch; starts are held to the rows; keys or values alone can be read."""
    import torch
    g = np.random.default_rng(7)
    k, v = tokens(g, 90, 2, 64, "f32"), tokens(g, 90, 2, 64, "f32")
    table, lens = np.array([[0, 1], [2, 3]]), [80, 64]
    want = M.Cache4(4, 2, 64)
    want.write(table, lens, [0, 70, 90], k, v)
    for hints in ((1, 1), (0, 0), (100000, 1 << 30)):
        gpu = to_gpu(M.Cache4(4, 2, 64))
        s = seqs(table, lens, [-5, 70, 1000], *hints)
        S.qmv_kv4_write(gpu, s, put(k, "f32"), put(v, "f32"))
        same_bytes(gpu, want)
        only = torch.full((90, 2, 64), 5.0, device="cuda")
        S.qmv_kv4_read(gpu, s, v=only)
        torch.cuda.synchronize()
        assert np.array_equal(only.cpu().numpy(), want.read(table, lens, [0, 70, 90], "v", 90).astype(np.float32))


def test_capture():
    import torch
    g = np.random.default_rng(8)
    gpu, c = to_gpu(M.Cache4(3, 2, 128)), M.Cache4(3, 2, 128)
    lens = torch.tensor([62], dtype=torch.int32, device="cuda")
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    s = S.KvSeqs(table, lens, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1, 192)
    k, v, ko, vo = (torch.zeros(1, 2, 128, device="cuda") for _ in range(4))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        S.qmv_kv4_write(gpu, s, k, v, stream=st)
        S.qmv_kv4_read(gpu, s, ko, vo, stream=st)
    for n in range(63, 68):
        a, b = tokens(g, 1, 2, 128, "f32"), tokens(g, 1, 2, 128, "f32")
        k.copy_(torch.from_numpy(a))
        v.copy_(torch.from_numpy(b))
        lens.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        c.write([[2, 0, 1]], [n], [0, 1], a, b)
        for x, what in ((ko, "k"), (vo, "v")):
            assert np.array_equal(x.cpu().numpy(), c.read([[2, 0, 1]], [n], [0, 1], what, 1).astype(np.float32))
    same_bytes(gpu, c)


def test_cache_past_four_gib():
    """Codes beyond 32-bit offsets."""
    import torch
    heads, dim = 8, 256
    pages = (9 << 29) // (heads * 64 * dim // 2)
    gpu = S.Kv4Cache.empty(pages, heads, dim)
    g = np.random.default_rng(9)
    table, lens, start = np.array([[pages - 1, 0, pages // 2 + 3]]), [150], [0, 150]
    k, v = tokens(g, 150, heads, dim, "bf16"), tokens(g, 150, heads, dim, "bf16")
    s = seqs(table, lens, start)
    S.qmv_kv4_write(gpu, s, put(k, "bf16"), put(v, "bf16"))
    small = M.Cache4(3, heads, dim)
    small.write(np.array([[0, 1, 2]]), lens, start, k, v)
    for x, what in zip(read_back(gpu, s, 150, heads, dim, "bf16"), "kv"):
        assert np.array_equal(x, small.read(np.array([[0, 1, 2]]), lens, start, what, 150).astype(np.float32))
    del gpu
    torch.cuda.empty_cache()


def test_refusals():
    import torch
    gpu = S.Kv4Cache.empty(2, 2, 64)
    eight = S.KvCache.empty(2, 2, 64)
    s = seqs([[0]], [3], [0, 3])
    x = torch.zeros(3, 2, 64, device="cuda")
    for call in (lambda: S.qmv_kv4_write(eight, s, x, x), lambda: S.qmv_kv_write(gpu, s, x, x), lambda: S.qmv_kv4_read(eight, s, x),
                 lambda: S.qmv_kv_read(gpu, s, x), lambda: S.qmv_kv4_write(gpu, s, x.half(), x.half()), lambda: S.qmv_kv4_write(gpu, s, x, x.bfloat16())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: S.qmv_kv4_write(gpu, s, x[:, :1].contiguous(), x), lambda: S.qmv_kv4_write(gpu, s, x, x[:2]),
                 lambda: S.qmv_kv4_write(gpu, s, x.cpu(), x), lambda: S.Kv4Cache(gpu.k[:, :1], gpu.v, gpu.k_scale, gpu.v_scale),
                 lambda: S.Kv4Cache(gpu.k, gpu.v, gpu.k_scale[..., :1].contiguous(), gpu.v_scale), lambda: S.Kv4Cache.empty(1, 1, 48)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(Q.QmvError):
        S.qmv_kv4_read(gpu, s)
    with pytest.raises(Q.QmvError):
        S.qmv_kv4_write(S.Kv4Cache.empty(2, 2, 96), s, torch.zeros(3, 2, 96, device="cuda"), torch.zeros(3, 2, 96, device="cuda"))
    with pytest.raises(AttributeError):
        gpu.k = gpu.k.clone()
