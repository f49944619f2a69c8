"""qmv_rms_norm against the plain norm in 64 bits.

Tolerance of y: r, h r and (h r) w round once each, 3 * 2^-24 (1 + 2^-20) of
the value; bfloat16 adds half a step, 2^-8.  Codes and scales are compared
with the activation quantizer's rule on the call's own float32 y, bit for
bit."""
import numpy as np
import pytest

import oracle as O
import serve_ref as R
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def data(rows, cols, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)).astype(np.float32)
    res = (3 * g.standard_normal((rows, cols))).astype(np.float32)
    w = (1 + 0.1 * g.standard_normal(cols)).astype(np.float32)
    return x, res, w


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(x, res, w, eps=EPS, outs=("sum", "y", "yb", "q")):
    import torch
    rows, cols = x.shape
    o = {"sum": torch.full((rows, cols), np.nan, device="cuda"), "y": torch.full((rows, cols), np.nan, device="cuda"),
         "yb": torch.full((rows, cols), np.nan, device="cuda", dtype=torch.bfloat16),
         "q": torch.full((rows, cols), -128, device="cuda", dtype=torch.int8),
         "d": torch.full((rows, cols // 32), -1.0, device="cuda")}
    rd = None if res is None else dev(res)
    kw = dict(res=rd, sum=o["sum"] if "sum" in outs else None)
    if "q" in outs:
        kw.update(q=o["q"], d=o["d"])
    xd, wd = dev(x), dev(w)
    if "y" in outs:
        S.qmv_rms_norm(xd, wd, eps, y=o["y"], **kw)
    if "yb" in outs:
        S.qmv_rms_norm(xd, wd, eps, y=o["yb"], **kw)
    torch.cuda.synchronize()
    return {k: (v.float() if k == "yb" else v).cpu().numpy() for k, v in o.items()}


def check(x, res, w, o, eps=EPS):
    h, y = R.norm(x, res, w, eps)
    assert np.array_equal(o["sum"].view(np.uint32), h.view(np.uint32))
    tol = 3.01 * 2.0 ** -24 * np.abs(y)
    assert np.all(np.abs(o["y"] - y) <= tol)
    assert np.all(np.abs(o["yb"] - y) <= tol + 2.0 ** -8 * np.abs(y))
    assert np.array_equal(o["yb"], R.bf16(o["y"]))
    for i in range(x.shape[0]):
        q, d = O.quantize_q8(o["y"][i])
        assert np.array_equal(o["q"][i], q) and np.array_equal(o["d"][i].view(np.uint32), d.view(np.uint32)), i


# one block, odd counts of blocks, every launch shape and both sides of its
# borders, and rows longer than a workgroup holds
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (5, 1024), (2, 1056), (1, 4096), (7, 4096), (3, 4128),
                                       (2, 8192), (2, 8224), (2, 16384), (2, 16416), (1, 65568), (300, 2048)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(rows, cols, residual):
    x, res, w = data(rows, cols, rows * 7 + cols)
    res = res if residual else None
    check(x, res, w, run(x, res, w))


@pytest.mark.parametrize("cols", [96, 4096, 20000 // 32 * 32])
def test_in_place(cols):
    """sum may be res, or x."""
    import torch
    x, res, w = data(3, cols, cols)
    h, y = R.norm(x, res, w, EPS)
    for which in ("res", "x"):
        xd, rd, out = dev(x), dev(res), torch.empty(3, cols, device="cuda")
        S.qmv_rms_norm(xd, dev(w), EPS, res=rd, sum=rd if which == "res" else xd, y=out)
        got, other = (rd, xd) if which == "res" else (xd, rd)
        assert np.array_equal(got.cpu().numpy(), h)
        assert np.array_equal(other.cpu().numpy(), x if which == "res" else res)
        assert np.all(np.abs(out.cpu().numpy() - y) <= 3.01 * 2.0 ** -24 * np.abs(y))


def test_single_outputs_write_nothing_else():
    x, res, w = data(4, 160, 5)
    whole = run(x, res, w)
    for outs in (("y",), ("yb",), ("sum", "y"), ("q", "y")):
        o = run(x, res, w, outs=outs)
        for k in ("sum", "y", "yb", "q", "d"):
            if k in outs or (k == "d" and "q" in outs):
                assert np.array_equal(o[k], whole[k]), (outs, k)
            else:
                assert np.all(np.isnan(o[k]) | (o[k] == -128) | (o[k] == -1)), (outs, k)


def test_values_at_the_ends():
    """Zero rows, tiny and huge values, rows that hold an infinity or NaN."""
    x, res, w = data(8, 128, 9)
    x[0] = 0
    x[1] *= np.float32(1e-25)
    x[2] *= np.float32(1e30)
    x[3] = 0
    x[3, 77] = np.float32(1e-30)
    x[4, 5] = np.inf
    x[5, 100] = np.nan
    x[6] *= np.float32(1e-42)
    o = run(x, None, w)
    with np.errstate(all="ignore"):
        h, y = R.norm(x, None, w, EPS)
    for i in (0, 1, 2, 3, 6, 7):
        # products below the normal range round to whole steps of 2^-149
        assert np.all(np.abs(o["y"][i] - y[i]) <= 3.01 * 2.0 ** -24 * np.abs(y[i]) + 3 * 2.0 ** -149), i
        q, d = O.quantize_q8(o["y"][i])
        assert np.array_equal(o["q"][i], q) and np.array_equal(o["d"][i], d)
    # an infinite row: r = 0, so inf * 0 is NaN there and the rest is 0
    assert np.isnan(o["y"][4, 5]) and np.isnan(o["d"][4, 0]) and np.all(o["q"][4, :32] == 0)
    assert np.all(np.delete(o["y"][4], 5) == 0) and np.all(o["d"][4, 1:] == 0)
    assert np.all(np.isnan(o["y"][5])) and np.all(np.isnan(o["d"][5])) and np.all(o["q"][5] == 0)


def test_eps_zero_and_zero_row():
    x, _, w = data(2, 64, 3)
    o = run(x, None, w, eps=0.0)
    check(x, None, w, o, eps=0.0)


def test_capture_and_other_stream():
    import torch
    x, res, w = data(6, 4096, 11)
    want = run(x, res, w)
    xd, rd, wd = dev(x), dev(res), dev(w)
    q = torch.empty(6, 4096, dtype=torch.int8, device="cuda")
    d = torch.empty(6, 128, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        S.qmv_rms_norm(xd, wd, EPS, res=rd, q=q, d=d, stream=s)
    for _ in range(3):
        q.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(q.cpu().numpy(), want["q"]) and np.array_equal(d.cpu().numpy(), want["d"])


def test_refuses_what_it_cannot_take():
    import torch
    x = torch.zeros(2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(Q.QmvError) as e:
        S.qmv_rms_norm(x, w, EPS)
    assert e.value.status == Q.QMV_E_ARG
    with pytest.raises(ValueError):
        S.qmv_rms_norm(x.t(), w, EPS, y=x)
    with pytest.raises(ValueError):
        S.qmv_rms_norm(x, w[:32], EPS, y=x)
    with pytest.raises(TypeError):
        S.qmv_rms_norm(x.half(), w, EPS, y=x)
    with pytest.raises(TypeError):
        S.qmv_rms_norm(x, w, EPS, y=x.half())
    with pytest.raises(ValueError):
        S.qmv_rms_norm(x.cpu(), w, EPS, y=x)


def test_arrays_past_the_caches():
    """Arrays of 64 MB and more, and one float4 a thread of rows that do not fill it."""
    for rows, cols in ((4100, 4096), (2100, 8224)):
        x, res, w = data(rows, cols, cols)
        o = run(x, res, w)
        sel = np.r_[0:9, rows // 2 - 3:rows // 2, rows - 9:rows]
        check(x[sel], res[sel], w, {k: v[sel] for k, v in o.items()})


def test_more_rows_than_workgroups():
    rows = (1 << 20) + 300
    x, res, w = data(rows, 32, 5)
    o = run(x, res, w)
    sel = np.r_[0:300, (1 << 20) - 2:rows]
    check(x[sel], res[sel], w, {k: v[sel] for k, v in o.items()})
