"""qmv_qk_rotate against the formula in 64 bits.

Bound, in units of 2^-24 of |a| + |b| of a pair: the norm's r rounds its
argument (half a unit), its root and its quotient, x r and (x r) w once each:
4.5; the angle's fraction of a turn rounds to 2^-26 of a turn, 2 pi of them:
1.6; cosine and sine are right to 4 units; mscale, two products and a sum round
once each: 2.5.  13 in all; a channel that stays has the norm's 4.5.  bfloat16
outputs add half a step, 2^-8 of the result."""
import numpy as np
import pytest

import more_ref as M
import serve_ref as R
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def tensor(x, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16)


def ok(got, x, w, pos, freq, neighbours, mscale, out):
    ref, size = M.rotate(x, w, EPS, pos, freq, neighbours, mscale)
    tol = 13 * 2.0 ** -24 * size + 1e-44
    if out == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    got = got.float().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


def inputs(rows, heads, kv_heads, dim, dtype, seed, most=100000):
    g = np.random.default_rng(seed)
    q = g.standard_normal((rows, heads, dim)).astype(np.float32) * 2
    k = g.standard_normal((rows, kv_heads, dim)).astype(np.float32) * 2
    if dtype == "bf16":
        q, k = R.bf16(q), R.bf16(k)
    qw, kw = ((1 + .1 * g.standard_normal(dim)).astype(np.float32) for _ in range(2))
    return q, k, qw, kw, g.integers(0, most, size=rows).astype(np.int32)


def frequencies(rot, base=1e6):
    return (base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)


SHAPES = [  # rows, heads, kv_heads, dim, rot
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 5, 1, 80, 80), (7, 6, 2, 96, 32), (33, 16, 4, 256, 64),
    (2, 3, 3, 8, 0), (2, 2, 1, 512, 512), (5, 1, 1, 16, 16), (130, 20, 4, 128, 112), (1, 200, 50, 64, 32),
]


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,heads,kv_heads,dim,rot", SHAPES)
def test_rotate(rows, heads, kv_heads, dim, rot, dtype, out, neighbours):
    import torch
    q, k, qw, kw, pos = inputs(rows, heads, kv_heads, dim, dtype, rows + dim)
    freq, m = frequencies(rot), 1.1
    dt = torch.float32 if out == "f32" else torch.bfloat16
    qo, ko = (torch.full(x.shape, 7.0, dtype=dt, device="cuda") for x in (q, k))
    f, p = torch.from_numpy(freq).cuda(), torch.from_numpy(pos).cuda()
    for weights in ((qw, kw), (None, None), (None, kw)):
        dw = [None if w is None else torch.from_numpy(w).cuda() for w in weights]
        S.qmv_qk_rotate(tensor(q, dtype), tensor(k, dtype), p, f, qo, ko, q_w=dw[0], k_w=dw[1], eps=EPS,
                        neighbours=neighbours, mscale=m)
        torch.cuda.synchronize()
        ok(qo, q, weights[0], pos, freq, neighbours, m, out)
        ok(ko, k, weights[1], pos, freq, neighbours, m, out)


def test_positions_far_and_negative():
    import torch
    q, k, qw, kw, _ = inputs(6, 2, 1, 64, "f32", 1)
    pos = np.array([0, 1, -1, 1 << 20, (1 << 24) + 1, -(1 << 20)], dtype=np.int32)
    freq = frequencies(64, 1e4)
    qo, ko = torch.empty(6, 2, 64, device="cuda"), torch.empty(6, 1, 64, device="cuda")
    S.qmv_qk_rotate(tensor(q, "f32"), tensor(k, "f32"), torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), qo, ko)
    torch.cuda.synchronize()
    ok(qo, q, None, pos, freq, False, 1.0, "f32")
    assert np.array_equal(qo[0].cpu().numpy(), q[0])          # position 0 turns nothing


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_one_array_in_place(dtype):
    """Queries and keys as slices of all projections, turned where they lie;
    what is beside them stays, and either may be given alone."""
    import torch
    rows, h, kvh, dim = 9, 6, 2, 128
    q, k, qw, kw, pos = inputs(rows, h, kvh, dim, dtype, 2)
    g = np.random.default_rng(3)
    v = R.bf16(g.standard_normal((rows, kvh * dim)).astype(np.float32))
    freq = frequencies(128)
    all3 = tensor(np.concatenate([q.reshape(rows, -1), k.reshape(rows, -1), v], 1), dtype)
    p, f = torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda()
    w = [torch.from_numpy(x).cuda() for x in (qw, kw)]
    qs, ks = all3[:, :h * dim].unflatten(1, (h, dim)), all3[:, h * dim:(h + kvh) * dim].unflatten(1, (kvh, dim))
    alone = torch.empty(rows, kvh, dim, device="cuda")
    S.qmv_qk_rotate(None, ks, p, f, None, alone, k_w=w[1], eps=EPS)
    S.qmv_qk_rotate(qs, ks, p, f, qs, ks, q_w=w[0], k_w=w[1], eps=EPS)
    torch.cuda.synchronize()
    ok(qs, q, qw, pos, freq, False, 1.0, dtype)
    ok(ks, k, kw, pos, freq, False, 1.0, dtype)
    ok(alone, k, kw, pos, freq, False, 1.0, "f32")
    assert np.array_equal(all3[:, (h + kvh) * dim:].float().cpu().numpy(), v)


def test_zeros_infinities_and_large_values_stay_in_their_head():
    import torch
    q, k, qw, kw, pos = inputs(2, 5, 1, 64, "f32", 4)
    q[0, 0], q[0, 1, 3], q[0, 2, 5], q[0, 3] = 0, np.nan, np.inf, q[0, 3] * 1e30
    freq = frequencies(64)
    qo, ko = torch.empty(2, 5, 64, device="cuda"), torch.empty(2, 1, 64, device="cuda")
    S.qmv_qk_rotate(tensor(q, "f32"), tensor(k, "f32"), torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), qo, ko,
                    q_w=torch.from_numpy(qw).cuda(), k_w=torch.from_numpy(kw).cuda(), eps=EPS)
    torch.cuda.synchronize()
    got = qo.cpu().numpy()
    assert np.all(got[0, 0] == 0) and np.all(np.isnan(got[0, 1]))
    assert np.isnan(got[0, 2, [5, 37]]).all() and np.isfinite(np.delete(got[0, 2], [5, 37])).all()
    for r, h in ((0, 3), (0, 4), (1, 0), (1, 1), (1, 2), (1, 3), (1, 4)):
        ref, size = M.rotate(q[r:r + 1, h:h + 1], qw, EPS, pos[r:r + 1], freq, False, 1.0)
        assert np.all(np.abs(got[r, h] - ref[0, 0]) <= 13 * 2.0 ** -24 * size[0, 0]), (r, h)


def test_capture_and_streams():
    """A graph of the call gives, at every replay, what the eager call gives."""
    import torch
    q, k, qw, kw, pos = inputs(4, 8, 2, 128, "f32", 5)
    f, p = torch.from_numpy(frequencies(128)).cuda(), torch.from_numpy(pos).cuda()
    x, y = tensor(q, "f32"), tensor(k, "f32")
    out = [torch.empty_like(t) for t in (x, y, x, y)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        S.qmv_qk_rotate(x, y, p, f, out[0], out[1], stream=st)
    for turn in range(3):
        p.add_(17)
        x.mul_(1.25)
        graph.replay()
        S.qmv_qk_rotate(x, y, p, f, out[2], out[3])
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])


def test_refusals():
    import torch
    q, k = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda")
    p, f = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(32, device="cuda")
    call = lambda **a: S.qmv_qk_rotate(**{**dict(q=q, k=k, pos=p, freq=f, q_out=q.clone(), k_out=k.clone()), **a})
    call()
    for bad in (dict(pos=p[:1]), dict(q_out=None), dict(k_out=None), dict(q_w=f), dict(k=torch.zeros(3, 2, 64, device="cuda")),
                dict(q=q.cpu()), dict(q=torch.zeros(2, 64, 4, device="cuda").transpose(1, 2)), dict(freq=f.view(2, 16))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(k=k.bfloat16()), dict(k_out=k.bfloat16()), dict(pos=p.long()), dict(q=q.half(), q_out=q.half())):
        with pytest.raises(TypeError):
            call(**bad)
    odd = torch.zeros(2, 4 * 64 + 4, device="cuda")[:, :256].unflatten(1, (4, 64))
    for bad in (dict(freq=torch.zeros(4, device="cuda")), dict(freq=torch.zeros(40, device="cuda")), dict(eps=-1.0),
                dict(mscale=float("nan")), dict(q=odd)):
        with pytest.raises(Q.QmvError):
            call(**bad)
