"""CPU checks of qmv_qk_rotate, qmv_kv4_* and qmv_sample: every refusal that is
made on the host before anything is launched, and the references the GPU tests
use against brute force."""
import ctypes

import numpy as np
import pytest

import more_ref as M
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S
from test_serve_cpu import BAD_KV, cache, seqs

P = 1 << 20           # an aligned address that is never used
OK, ARG, SHAPE = Q.QMV_OK, Q.QMV_E_ARG, Q.QMV_E_SHAPE


@pytest.mark.parametrize("c,s,want", BAD_KV)
def test_kv4_refusals(c, s, want):
    L = S.lib()
    n = ctypes.c_uint64(7)
    assert L.qmv_kv4_write(cache(**c), seqs(**s), 0, P, P, None) == want
    assert L.qmv_kv4_read(cache(**c), seqs(**s), 0, P, P, None) == want
    assert L.qmv_kv4_attend_workspace(cache(**c), seqs(**s), 0, 4, 0, ctypes.byref(n)) == want
    assert n.value == 0
    assert L.qmv_kv4_attend(cache(**c), seqs(**s), 0, 4, 1.0, 0, P, P, P, 1 << 62, None) == want


def test_kv4_calls_refuse():
    L = S.lib()
    assert L.qmv_kv4_write(None, seqs(), 0, P, P, None) == ARG
    assert L.qmv_kv4_write(cache(), None, 0, P, P, None) == ARG
    assert L.qmv_kv4_write(cache(), seqs(), 2, P, P, None) == ARG
    for k, v in ((None, P), (P, None), (P + 8, P), (P, P + 2)):
        assert L.qmv_kv4_write(cache(), seqs(), 0, k, v, None) == ARG
    for k, v in ((None, None), (P + 8, None), (None, P + 4)):
        assert L.qmv_kv4_read(cache(), seqs(), 0, k, v, None) == ARG

    def attend(heads=4, scale=1.0, q=P, out=P, ws=P, nb=1 << 62, **s):
        return L.qmv_kv4_attend(cache(), seqs(**s), 0, heads, scale, 0, q, out, ws, nb, None)
    for a in (dict(q=None), dict(out=None), dict(q=P + 8), dict(out=P + 4), dict(ws=P + 8), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert attend(**a) == ARG, a
    for a in (dict(heads=0), dict(heads=3), dict(heads=1 << 25), dict(rows=1 << 28, heads=8)):
        assert attend(**a) == SHAPE, a
    n = ctypes.c_uint64(0)
    assert L.qmv_kv4_attend_workspace(cache(), seqs(max_len=100000), 0, 4, 0, ctypes.byref(n)) == OK and n.value > 0
    assert attend(ws=None, max_len=100000) == ARG and attend(nb=n.value - 1, max_len=100000) == ARG
    assert L.qmv_kv4_attend_workspace(cache(), seqs(), 0, 4, 0, None) == ARG


def heads(**kw):
    a = dict(x=P, y=2 * P, w=P, x_stride=256, y_stride=256, heads=4)
    a.update(kw)
    return S._pack_heads(*[v or 0 for v in a.values()])


def test_rotate_refuses():
    L = S.lib()

    def call(q=heads(), k=None, rows=2, dim=64, dtype=0, out=0, eps=1e-6, pos=P, freq=P, rot=64, m=1.0):
        return L.qmv_qk_rotate(q, k, rows, dim, dtype, out, eps, pos, freq, rot, 0, m, None)
    nan, inf = float("nan"), float("inf")
    for a in (dict(q=None), dict(rows=0), dict(dtype=2), dict(out=2), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(pos=None),
              dict(pos=P + 2), dict(freq=None), dict(freq=P + 1), dict(m=nan), dict(m=inf), dict(q=heads(x=None)), dict(q=heads(y=None)),
              dict(q=heads(heads=0)), dict(q=heads(x=P + 8)), dict(q=heads(y=P + 8)), dict(q=heads(w=P + 4)),
              dict(q=heads(y=P, y_stride=512)), dict(q=heads(y=P), out=1), dict(k=heads(x=None)), dict(k=heads(y=P + 4))):
        assert call(**a) == ARG, a
    for a in (dict(dim=0), dict(dim=60), dict(dim=520), dict(rot=8), dict(rot=80), dict(rows=1 << 31), dict(q=heads(heads=5)),
              dict(q=heads(x_stride=260)), dict(q=heads(y_stride=248)), dict(q=heads(x_stride=1 << 41)), dict(k=heads(heads=1 << 21)),
              dict(q=heads(heads=(1 << 20) + 1, x_stride=1 << 30, y_stride=1 << 30))):
        assert call(**a) == SHAPE, a
    assert len(heads()) == 48


def test_sample_refuses():
    L = S.lib()
    n = ctypes.c_uint64(7)
    assert L.qmv_sample_workspace(3, 5000, None) == ARG
    for r, v, want in ((0, 5, ARG), (5, 0, ARG), (1, (1 << 24) + 1, SHAPE), ((1 << 22) + 1, 5, SHAPE)):
        assert L.qmv_sample_workspace(r, v, ctypes.byref(n)) == want and n.value == 0
    assert L.qmv_sample_workspace(3, 5000, ctypes.byref(n)) == OK

    def call(x=P, rows=3, vocab=5000, u=P, t=P, k=P, p=P, m=P, ids=P, lp=P, ws=P, nb=1 << 62):
        return L.qmv_sample(x, rows, vocab, u, t, k, p, m, ids, lp, ws, nb, None)
    for a in (dict(x=None), dict(u=None), dict(ids=None), dict(rows=0), dict(vocab=0), dict(ws=None), dict(ws=P + 8), dict(nb=n.value - 1)):
        assert call(**a) == ARG, a
    for name in ("x", "u", "t", "k", "p", "m", "ids", "lp"):
        assert call(**{name: P + 2}) == ARG, name
    assert call(vocab=1 << 25) == SHAPE
    for sizes in (((1 << 32) + 1, 100), (1, (1 << 32) + 100), (-1, 100)):
        with pytest.raises(ValueError):
            S.qmv_sample_workspace(*sizes)


def test_the_reference_quantizes_to_the_nearest():
    """Against all sixteen values of a block, and the scale against all exponents."""
    g = np.random.default_rng(0)
    x = (g.standard_normal((40, 32)) * 2.0 ** g.integers(-20, 20, size=(40, 1))).astype(np.float32)
    index, neg, e = M.quantize(x)
    for row, i, n, ex in zip(x.astype(np.float64), index, neg, e[:, 0]):
        amax = np.abs(row).max()
        assert amax <= 7 * 2.0 ** ex and amax > 7 * 2.0 ** (ex - 1)
        every = np.concatenate([M.LEVELS, -M.LEVELS]) * 2.0 ** ex
        got = np.where(n, -1, 1) * M.LEVELS[i] * 2.0 ** ex
        assert np.all(np.abs(got - row) <= np.abs(every[None] - row[:, None]).min(1))


def test_the_reference_packs_every_place_once():
    for dim in (64, 128, 256):
        c = M.Cache4(1, 1, dim)
        for n in "kv":
            c.code[n][:] = 15
            c.byte[n][:] = 200
        for a in c.arrays():
            assert np.all((a == 255) | (a == 200))


def test_the_reference_draws_the_whole_distribution():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0], dtype=np.float64)).astype(np.float32)
    draws = [M.sample(x, u, 1.0, 0, 1.0, 0.0)[0] for u in (0.0, 0.12, 0.13, 0.62, 0.63, 0.87, 0.88, 0.999)]
    assert draws == [0, 0, 1, 1, 2, 2, 3, 3]
    assert M.sample(x, 0.99, 1.0, 1, 1.0, 0.0)[0] == 1
    assert M.sample(x, 0.99, 1.0, 3, 1.0, 0.0)[0] == 2 and M.sample(x, 0.0, 1.0, 3, 1.0, 0.0)[0] == 0
    assert M.sample(x, 0.99, 1.0, 0, 0.51, 0.0)[0] == 2 and M.sample(x, 0.99, 1.0, 0, 0.49, 0.0)[0] == 1
    assert M.sample(x, 0.99, 1.0, 0, 1.0, 0.4)[0] == 2 and M.sample(x, 0.99, 1.0, 0, 1.0, 0.6)[0] == 1
