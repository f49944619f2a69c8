"""Sizes past what a launch's grid holds at once, where workgroups go round, and
calls beside each other: each against the same rows in calls of their own, which
other tests hold against their references."""
import numpy as np
import pytest

import more_ref as M
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def ints(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def generator(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_rotate_more_rows_than_workgroups():
    import torch
    rows, heads, dim = (1 << 22) + 5, 2, 16
    g = generator(1)
    q = torch.randn(rows, heads, dim, generator=g, device="cuda")
    pos = torch.randint(0, 1 << 20, (rows,), generator=g, device="cuda", dtype=torch.int32)
    freq = torch.tensor([1.0, 0.3, 0.1, 0.03, 0.01, 3e-3, 1e-3, 3e-4], device="cuda")
    out = torch.empty_like(q)
    S.qmv_qk_rotate(q, None, pos, freq, out, None)
    at = [0, 1 << 21, (1 << 22) - 1, 1 << 22, rows - 4, rows - 1]
    some = torch.empty(len(at), heads, dim, device="cuda")
    S.qmv_qk_rotate(q[at].contiguous(), None, pos[at].contiguous(), freq, some, None)
    torch.cuda.synchronize()
    assert torch.equal(out[at], some)


def test_rotate_more_heads_than_workgroups():
    """One row of 2^20 heads: 65535 workgroups of 16 have some twice."""
    import torch
    heads, dim = 1 << 20, 128
    q = torch.randn(1, heads, dim, generator=generator(2), device="cuda")
    w, pos, freq = torch.ones(dim, device="cuda"), ints([77]), torch.rand(dim // 2, generator=generator(3), device="cuda")
    out = torch.empty_like(q)
    S.qmv_qk_rotate(q, None, pos, freq, out, None, q_w=w)
    at = [0, 65535 * 8, 65535 * 8 + 7, heads - 1]
    some = torch.empty(1, len(at), dim, device="cuda")
    S.qmv_qk_rotate(q[:, at].contiguous(), None, pos, freq, some, None, q_w=w)
    torch.cuda.synchronize()
    assert torch.equal(out[:, at], some)


def test_cache_more_tokens_than_workgroups():
    """A prompt whose tokens and heads are more than 65535 groups, written and
    read at once and in parts."""
    import torch
    n, heads, dim = 150001, 8, 128
    pages = -(-n // 64)
    g = generator(4)
    k, v = (torch.randn(n, heads, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(1, -1)
    one, two = S.Kv4Cache.empty(pages, heads, dim), S.Kv4Cache.empty(pages, heads, dim)
    for c in (one, two):
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            t.zero_()
    whole = S.KvSeqs(table, ints([n]), ints([0, n]), max_new=n, max_len=n)
    S.qmv_kv4_write(one, whole, k, v)
    for a in range(0, n, 40000):
        b = min(a + 40000, n)
        S.qmv_kv4_write(two, S.KvSeqs(table, ints([b]), ints([0, b - a]), max_new=b - a, max_len=b), k[a:b], v[a:b])
    for a, b in zip((one.k, one.v, one.k_scale, one.v_scale), (two.k, two.v, two.k_scale, two.v_scale)):
        assert torch.equal(a, b)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    S.qmv_kv4_read(one, whole, ko, vo)
    for a in (0, 65535 * 2 // 2, n - 3):
        kp, vp = torch.empty_like(k[:3]), torch.empty_like(v[:3])
        S.qmv_kv4_read(one, S.KvSeqs(table, ints([a + 3]), ints([0, 3]), max_new=3, max_len=a + 3), kp, vp)
        torch.cuda.synchronize()
        assert torch.equal(ko[a:a + 3], kp) and torch.equal(vo[a:a + 3], vp)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_more_tiles_than_workgroups(dtype):
    """A whole prompt under a narrow window, its tiles more than 65535; rows of
    it alone, as single tokens of sequences that end there."""
    import torch
    n, heads, dim, window = (1 << 20) + 77, 5 if dtype == "f32" else 9, 64, 50
    pages = -(-n // 64)
    g = generator(5)
    c = S.Kv4Cache.empty(pages, 1, dim)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.int32))
    for t in (c.k_scale, c.v_scale):             # scales 2^-3 to 1
        t.copy_(torch.randint(124, 128, t.shape, generator=g, device="cuda", dtype=torch.int32))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    q = torch.randn(n, heads, dim, generator=g, device="cuda").to(dt)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(1, -1)
    s = S.KvSeqs(table, ints([n]), ints([0, n]), max_new=n, max_len=n)
    out = torch.full_like(q, 5.0)
    S.qmv_kv4_attend(c, s, q, out, window=window, workspace=S.workspace(max(S.qmv_kv4_attend_workspace(c, s, q, window), 16)))
    at = [0, 49, 64, 1000, 65535 * 16 // heads, 65535 * 16 // heads + 1, n - 2, n - 1]
    m = len(at)
    s = S.KvSeqs(table.expand(m, -1).contiguous(), ints([a + 1 for a in at]), ints(range(m + 1)), max_new=1, max_len=n)
    qs = q[at].contiguous()
    some = torch.empty_like(qs)
    S.qmv_kv4_attend(c, s, qs, some, window=window, workspace=S.workspace(max(S.qmv_kv4_attend_workspace(c, s, qs, window), 16)))
    torch.cuda.synchronize()
    # each side is within attend_bound of the truth: sizes by the largest key and value, 6
    x = qs.float().abs().sum(-1).max().item() * 6 * dim ** -0.5
    b = {"mass": np.float64(6), "smax": np.float64(x), "qk": np.float64(x), "vmax": np.float64(6)}
    tol = 2 * M.attend_bound(b, dim, window, dtype, many=True)
    got, want = out[at].float(), some.float()
    if dtype == "bf16":
        tol = tol + 2 * 2.0 ** -8 * (want.abs() + tol)
    assert torch.all((got - want).abs() <= tol)


def test_sample_more_rows_than_workgroups():
    import torch
    rows, vocab = 66001, 8200
    g = generator(6)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 3
    u = torch.rand(rows, generator=g, device="cuda")
    p, k = torch.full((rows,), 0.9, device="cuda"), torch.full((rows,), 50, device="cuda", dtype=torch.int32)

    def draw(x, u, p, k):
        ids, lp = torch.empty(len(x), dtype=torch.int32, device="cuda"), torch.empty(len(x), device="cuda")
        S.qmv_sample(x, u, ids, top_k=k, top_p=p, lp=lp, workspace=S.workspace(S.qmv_sample_workspace(*x.shape)))
        torch.cuda.synchronize()
        return ids, lp
    ids, lp = draw(x, u, p, k)
    at = list(range(0, rows, 4999)) + [65534, 65535, 65536, rows - 1]
    some = draw(x[at].contiguous(), u[at].contiguous(), p[at].contiguous(), k[at].contiguous())
    assert torch.equal(ids[at], some[0]) and torch.equal(lp[at], some[1])


def test_sample_long_rows():
    """Vocabularies at and past the longest of which a list is kept."""
    from test_gpu_sample import check, logits
    g = np.random.default_rng(7)
    for vocab in (1 << 19, (1 << 19) + 1, 700001):
        n = 4
        check(logits(g, n, vocab), g.random(n).astype(np.float32), t=np.array([0.0, 0.7, 1.0, 1.0], dtype=np.float32),
              k=np.array([0, 40, 0, 0]), p=np.array([1.0, 0.9, 0.3, 1.0], dtype=np.float32), m=np.array([0.0, 0.0, 0.01, 0.0], dtype=np.float32))


def test_two_draws_and_two_rotations_at_once():
    """On two streams, a workspace each, over and over: the same bits as alone."""
    import torch
    g = generator(8)
    x = [torch.randn(r, v, generator=g, device="cuda") * 3 for r, v in ((5, 60000), (70, 20001))]
    u = [torch.rand(len(a), generator=g, device="cuda") for a in x]
    p = [torch.full((len(a),), 0.8, device="cuda") for a in x]
    q = [torch.randn(n, 6, 96, generator=g, device="cuda") for n in (3, 900)]
    pos = [torch.arange(len(a), device="cuda", dtype=torch.int32) for a in q]
    freq = torch.rand(24, generator=g, device="cuda")
    ws = [S.workspace(S.qmv_sample_workspace(*a.shape)) for a in x]

    def run(i, ids, lp, out, stream):
        S.qmv_sample(x[i], u[i], ids, top_p=p[i], lp=lp, workspace=ws[i], stream=stream)
        S.qmv_qk_rotate(q[i], None, pos[i], freq, out, None, neighbours=i == 1, stream=stream)

    def outs(i):
        return torch.full((len(x[i]),), -5, dtype=torch.int32, device="cuda"), torch.empty(len(x[i]), device="cuda"), torch.empty_like(q[i])
    want = [outs(i) for i in range(2)]
    for i in range(2):
        run(i, *want[i], None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[outs(i) for _ in range(20)] for i in range(2)]
    torch.cuda.synchronize()
    for turn in range(20):
        for i in range(2):
            run(i, *got[i][turn], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(o, want[i]))
