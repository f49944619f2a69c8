"""CPU checks of the calls of include/qmv_serve.h: exports, and every refusal
that is made on the host before anything is launched."""
import ctypes
import os
import re

import pytest

from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20           # an aligned address that is never used
OK, ARG, SHAPE = Q.QMV_OK, Q.QMV_E_ARG, Q.QMV_E_SHAPE


def test_library_exports_every_declared_function():
    txt = open(os.path.join(ROOT, "include", "qmv_serve.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    declared = set(re.findall(r"\b(qmv_[a-z0-9_]+)\s*\(", txt))
    assert declared == set(S.EXPORTS)
    for name in declared:
        assert hasattr(S.lib(), name), name


def cache(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, pages=8, kv_heads=2, head_dim=64)
    a.update(kw)
    return ctypes.byref(S._Cache(*[a[f] for f, _ in S._Cache._fields_]))


def seqs(**kw):
    a = dict(table=P, len=P, start=P, seqs=2, table_stride=4, rows=3, max_new=2, max_len=200)
    a.update(kw)
    return ctypes.byref(S._Seqs(*[a[f] for f, _ in S._Seqs._fields_]))


BAD_KV = [
    (dict(k=None), {}, ARG), (dict(v=None), {}, ARG), (dict(k_scale=None), {}, ARG),
    (dict(v_scale=None), {}, ARG), (dict(k=P + 8), {}, ARG), (dict(v=P + 4), {}, ARG),
    (dict(k_scale=P + 4), {}, ARG), (dict(v_scale=P + 8), {}, ARG), (dict(pages=0), {}, ARG),
    (dict(kv_heads=0), {}, ARG), (dict(head_dim=0), {}, SHAPE), (dict(head_dim=32), {}, SHAPE),
    (dict(head_dim=96), {}, SHAPE), (dict(head_dim=512), {}, SHAPE), (dict(kv_heads=65536), {}, SHAPE),
    (dict(pages=1 << 31), {}, SHAPE),
    ({}, dict(table=None), ARG), ({}, dict(len=None), ARG), ({}, dict(start=None), ARG),
    ({}, dict(table=P + 2), ARG), ({}, dict(len=P + 1), ARG), ({}, dict(start=P + 3), ARG),
    ({}, dict(seqs=0), ARG), ({}, dict(table_stride=0), ARG), ({}, dict(rows=0), ARG),
    ({}, dict(rows=1 << 31), SHAPE), ({}, dict(seqs=1 << 30), SHAPE),
]


@pytest.mark.parametrize("c,s,want", BAD_KV)
def test_kv_refusals(c, s, want):
    L = S.lib()
    n = ctypes.c_uint64(7)
    assert L.qmv_kv_write(cache(**c), seqs(**s), 0, P, P, None) == want
    assert L.qmv_kv_read(cache(**c), seqs(**s), 0, P, P, None) == want
    assert L.qmv_kv_attend_workspace(cache(**c), seqs(**s), 0, 4, 0, ctypes.byref(n)) == want
    assert n.value == 0
    assert L.qmv_kv_attend(cache(**c), seqs(**s), 0, 4, 1.0, 0, P, P, P, 1 << 40, None) == want


def test_kv_call_refusals():
    L = S.lib()
    c, s = cache(), seqs()
    n = ctypes.c_uint64(0)
    assert L.qmv_kv_write(None, s, 0, P, P, None) == ARG
    assert L.qmv_kv_write(c, None, 0, P, P, None) == ARG
    assert L.qmv_kv_write(c, s, 2, P, P, None) == ARG
    assert L.qmv_kv_write(c, s, 0, None, P, None) == ARG
    assert L.qmv_kv_write(c, s, 0, P, None, None) == ARG
    assert L.qmv_kv_write(c, s, 1, P + 2, P, None) == ARG
    assert L.qmv_kv_write(c, s, 0, P, P + 4, None) == ARG
    assert L.qmv_kv_read(c, s, 0, None, None, None) == ARG
    assert L.qmv_kv_read(c, s, 0, P + 8, P, None) == ARG
    assert L.qmv_kv_read(c, s, 3, P, P, None) == ARG
    assert L.qmv_kv_attend_workspace(c, s, 0, 4, 0, None) == ARG
    for heads in (0, 1, 3, 5, 1 << 25):
        assert L.qmv_kv_attend_workspace(c, s, 0, heads, 0, ctypes.byref(n)) == SHAPE
        assert L.qmv_kv_attend(c, s, 0, heads, 1.0, 0, P, P, P, 1 << 40, None) == SHAPE
    assert L.qmv_kv_attend(c, s, 2, 4, 1.0, 0, P, P, P, 1 << 40, None) == ARG
    for q, out, ws, scale in ((None, P, P, 1.0), (P, None, P, 1.0), (P + 2, P, P, 1.0), (P, P + 8, P, 1.0),
                              (P, P, P + 4, 1.0), (P, P, P, float("nan")), (P, P, P, float("inf"))):
        assert L.qmv_kv_attend(c, s, 0, 4, scale, 0, q, out, ws, 1 << 40, None) == ARG
    # a workspace that is needed and too small, or missing
    long = seqs(max_len=100000, table_stride=2000)
    assert L.qmv_kv_attend_workspace(c, long, 0, 4, 0, ctypes.byref(n)) == OK and n.value > 0
    assert L.qmv_kv_attend(c, long, 0, 4, 1.0, 0, P, P, P, n.value - 1, None) == ARG
    assert L.qmv_kv_attend(c, long, 0, 4, 1.0, 0, P, P, None, n.value, None) == ARG


def test_norm_refusals():
    def call(x=P, res=P, w=P, eps=1e-5, rows=2, cols=64, sum=P, y=P, yb=None, q=None, d=None):
        return S.lib().qmv_rms_norm(x, res, w, eps, rows, cols, sum, y, yb, q, d, None)
    assert call(x=None) == ARG and call(w=None) == ARG and call(rows=0) == ARG
    assert call(sum=None, y=None) == ARG
    assert call(q=P) == ARG and call(d=P) == ARG
    assert call(eps=-1e-9) == ARG and call(eps=float("nan")) == ARG and call(eps=float("inf")) == ARG
    for name in ("x", "res", "w", "sum", "y", "yb"):
        assert call(**{name: P + 4}) == ARG, name
    assert call(q=P + 8, d=P) == ARG and call(q=P, d=P + 8) == ARG
    for cols in (0, 1, 31, 48, (1 << 24) + 32):
        assert call(cols=cols) == SHAPE, cols


def test_logprobs_refusals():
    L = S.lib()
    n = ctypes.c_uint64(0)

    def call(x=P, rows=2, vocab=1000, ids=P, n_ids=1, top=3, lp=P, h=P, ti=P, tl=P, ws=P, nb=1 << 40):
        return L.qmv_logprobs(x, rows, vocab, ids, n_ids, top, lp, h, ti, tl, ws, nb, None)
    assert L.qmv_logprobs_workspace(2, 1000, 3, None) == ARG
    for rows, vocab, top, want in ((0, 10, 0, ARG), (1, 0, 0, ARG), (1, (1 << 24) + 1, 0, SHAPE),
                                   (1, 10, 11, SHAPE), (1, 1000, 33, SHAPE), ((1 << 22) + 1, 10, 0, SHAPE)):
        assert L.qmv_logprobs_workspace(rows, vocab, top, ctypes.byref(n)) == want
        assert call(rows=rows, vocab=vocab, top=top) == want
    assert L.qmv_logprobs_workspace(2, 1000, 3, ctypes.byref(n)) == OK and n.value > 0
    assert call(x=None) == ARG
    assert call(lp=None, h=None, ti=None, tl=None, top=0) == ARG
    assert call(ids=None) == ARG and call(n_ids=0) == ARG
    assert call(ti=None) == ARG and call(tl=None) == ARG and call(top=0) == ARG
    assert call(ti=None, tl=None, top=3) == ARG
    assert call(ws=None) == ARG and call(ws=P + 8) == ARG and call(nb=n.value - 1) == ARG
    for name in ("x", "ids", "lp", "h", "ti", "tl"):
        assert call(**{name: P + 2}) == ARG, name


def test_structs_match_the_header():
    assert ctypes.sizeof(S._Cache) == 48 and ctypes.sizeof(S._Seqs) == 48
    assert S.QMV_KV_PAGE == 64 and (S.QMV_F32, S.QMV_BF16) == (0, 1)


def test_launch_limits():
    """Sizes that a launch, or 32-bit places, cannot hold."""
    L = S.lib()
    for c, s in ((dict(kv_heads=4), dict(seqs=(1 << 20) + 1, table_stride=1)),
                 (dict(pages=1 << 30), {}), ({}, dict(seqs=1 << 20, table_stride=1 << 11)),
                 ({}, dict(rows=0x7FFF0001))):
        assert L.qmv_kv_write(cache(**c), seqs(**s), 0, P, P, None) == SHAPE
        assert L.qmv_kv_read(cache(**c), seqs(**s), 0, P, P, None) == SHAPE
        assert L.qmv_kv_attend(cache(**c), seqs(**s), 0, 4, 1.0, 0, P, P, P, 1 << 62, None) == SHAPE
    assert L.qmv_kv_attend(cache(), seqs(rows=1 << 28), 0, 8, 1.0, 0, P, P, P, 1 << 62, None) == SHAPE


@pytest.mark.parametrize("window", [-1, 1 << 32, (1 << 32) + 5, 1 << 64])
def test_windows_that_32_bits_do_not_hold(window):
    """(2^32 + 5 would be a window of 5.)"""
    import torch
    q = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError, match="window"):
        S.qmv_kv_attend(None, None, q, q, window=window)
    with pytest.raises(ValueError, match="window"):
        S.qmv_kv_attend_workspace(None, None, q, window=window)


def test_sizes_that_32_bits_do_not_hold():
    assert S.qmv_logprobs_workspace(1, 10000, 3) > 0
    for sizes in (((1 << 32) + 1, 10000, 3), (1, (1 << 32) + 10000, 3), (1, 10000, (1 << 32) + 3), (-1, 10000, 0)):
        with pytest.raises(ValueError):
            S.qmv_logprobs_workspace(*sizes)


def test_hints_past_32_bits_count_as_the_largest(monkeypatch):
    """A hint is only a hint: 2^32 is not 0."""
    import torch
    monkeypatch.setattr(S, "_dev", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(S, "_first", lambda t, *a: t.data_ptr())
    t = torch.zeros(1, 4, dtype=torch.int32)
    c = S.KvSeqs(t, t, t, 1 << 32, 1 << 40).c
    assert c.max_new == c.max_len == 0xFFFFFFFF


def test_tensors_of_a_handle_are_changed_in_place_only(monkeypatch):
    """A handle holds addresses: another tensor in an attribute's place would
    leave the calls reading the first one's memory, which nothing keeps."""
    import torch
    monkeypatch.setattr(S, "_dev", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(S, "_first", lambda t, *a: t.data_ptr())
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)
    s = S.KvSeqs(i(2, 3), i(2), i(3), 1, 1)
    c = S.KvCache(torch.zeros(4, 1, 64, 64, dtype=torch.int8), torch.zeros(4, 1, 64, 64, dtype=torch.int8),
                  torch.zeros(4, 1), torch.zeros(4, 1))
    for handle, names in ((s, ("table", "len", "start")), (c, ("k", "v", "k_scale", "v_scale"))):
        for name in names:
            t = getattr(handle, name)
            with pytest.raises(AttributeError, match="in place"):
                setattr(handle, name, t.clone())
            assert getattr(handle, name) is t and t.data_ptr() == getattr(handle.c, name)
    s.len += 1
    s.table[:] = 2
    assert s.len.tolist() == [1, 1] and s.len.data_ptr() == s.c.len and int(s.table.sum()) == 12
