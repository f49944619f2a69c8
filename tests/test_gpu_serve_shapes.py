"""The binding of qmv_serve.h takes arrays of the documented shape alone: one
of another shape that holds enough elements would be filled in another order,
or in part."""
import pytest

from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def others(t):
    """Contiguous tensors that hold as many elements as t, or more, in other shapes."""
    import torch
    more = torch.zeros(t.shape[0] + 1, *t.shape[1:], dtype=t.dtype, device=t.device)
    flat = t.reshape(-1)
    return [more, t.unsqueeze(0)] + ([flat, t.transpose(0, 1).contiguous()] if t.dim() > 1 else [])


def each_refused(call, args, names):
    """call(**args) runs; with any of the named arrays in another shape it is refused and writes nothing."""
    import torch
    call(**args)
    torch.cuda.synchronize()
    for name in names:
        for bad in others(args[name]):
            if bad.shape == args[name].shape:
                continue
            before = {n: t.clone() for n, t in args.items() if n != name}
            was = bad.clone()
            with pytest.raises(ValueError, match="must be|holds"):
                call(**{**args, name: bad})
            torch.cuda.synchronize()
            assert torch.equal(bad, was), name
            assert all(torch.equal(before[n], args[n]) for n in before), name


def zeros(*shape, dtype=None):
    import torch
    return torch.zeros(*shape, dtype=dtype or torch.float32, device="cuda")


def test_norm():
    import torch
    args = dict(x=zeros(3, 64) + 1, w=zeros(64) + 1, res=zeros(3, 64), sum=zeros(3, 64), y=zeros(3, 64),
                q=zeros(3, 64, dtype=torch.int8), d=zeros(3, 2))
    each_refused(lambda **a: S.qmv_rms_norm(eps=1e-5, **a), args, ("w", "res", "sum", "y", "q", "d"))
    args["y"] = zeros(3, 64, dtype=torch.bfloat16)
    each_refused(lambda **a: S.qmv_rms_norm(eps=1e-5, **a), args, ("y",))


@pytest.mark.parametrize("bits", [32, 16])
def test_cache_and_attention(bits):
    import torch
    dt = torch.float32 if bits == 32 else torch.bfloat16
    c = S.KvCache.empty(2, 2, 64)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    s = S.KvSeqs(i32(0, 1).view(1, 2), i32(5), i32(0, 5), 5, 5)
    kv = dict(k=zeros(5, 2, 64, dtype=dt), v=zeros(5, 2, 64, dtype=dt))
    each_refused(lambda **a: S.qmv_kv_write(c, s, **a), kv, ("v",))
    each_refused(lambda **a: S.qmv_kv_read(c, s, **a), kv, ("v",))
    args = dict(q=zeros(5, 4, 64, dtype=dt), out=zeros(5, 4, 64, dtype=dt))
    each_refused(lambda **a: S.qmv_kv_attend(c, s, **a), args, ("out",))


def test_longer_lengths_and_starts():
    """Of longer lengths and starts the first elements are taken."""
    import torch
    c = S.KvCache.empty(2, 1, 64)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    x = torch.randn(5, 1, 64, device="cuda")
    out = [zeros(5, 1, 64) for _ in range(2)]
    for o, s in zip(out, (S.KvSeqs(i32(0, 1).view(1, 2), i32(5), i32(0, 5), 5, 5),
                          S.KvSeqs(i32(0, 1).view(1, 2), i32(5, 9), i32(0, 5, 9, 9), 5, 5))):
        S.qmv_kv_write(c, s, x, x)
        S.qmv_kv_read(c, s, o)
    assert torch.equal(out[0], out[1]) and bool((out[0] != 0).any())


def test_log_probabilities():
    import torch
    args = dict(logits=torch.randn(3, 50, device="cuda"), ids=zeros(3, 2, dtype=torch.int32), lp=zeros(3, 2),
                entropy=zeros(3), top_ids=zeros(3, 4, dtype=torch.int32), top_lp=zeros(3, 4))
    each_refused(S.qmv_logprobs, args, ("lp", "entropy", "top_lp"))
    for bad in (dict(lp=args["lp"]), dict(top_lp=args["top_lp"])):
        with pytest.raises(Q.QmvError) as e:
            S.qmv_logprobs(args["logits"], **bad)
        assert e.value.status == Q.QMV_E_ARG
