"""qmv_kv4_attend's kernel for many queries as a program has it: captured and
replayed, in place, two graphs at once with a workspace each; and every kernel's
answer the same bits in every call."""
import numpy as np
import pytest

from block_quant_weight_amd import serve as S
from test_gpu_attend4 import FAR, attend, make, queries, starts
from test_gpu_attend4_queries import FORMS
from test_gpu_kv4 import seqs, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_two_graphs_of_the_kernel_for_many(dim, cut):
    """Whole sequences, and ones that are cut and joined through the workspace."""
    import torch
    sides = []
    for i in range(2):
        lens, news = ([900, 70], [140, 70]) if cut else ([300, 70], [200, 70])
        g, c, table = make(lens, 2, dim, 40 + i)
        start = starts(news)
        gpu, q = to_gpu(c), queries(g, start[-1] + (0 if cut else 10000), 4, dim)
        empty = 0 if cut else 64
        s = seqs(np.concatenate([table, np.full((empty, table.shape[1]), -1)]), lens + [0] * empty, start + [start[-1]] * empty,
                 *(FAR if cut else (10000, 1 << 20)))
        want = attend(gpu, s, q, "bf16")
        want[start[-1]:] = q[start[-1]:]          # (in place: rows of no sequence stay)
        d = dict(keep=(gpu, s), first=torch.from_numpy(q).cuda().bfloat16(), want=want, stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph())
        d["q"] = d["first"].clone()
        nbytes = S.qmv_kv4_attend_workspace(gpu, s, d["q"])
        assert (nbytes > 0) == cut
        d["ws"] = S.workspace(nbytes)
        torch.cuda.synchronize()
        with torch.cuda.graph(d["graph"], stream=d["stream"]):
            S.qmv_kv4_attend(gpu, s, d["q"], d["q"], workspace=d["ws"], stream=d["stream"])
        sides.append(d)
    for _ in range(4):
        for d in sides:
            d["q"].copy_(d["first"])
            d["ws"].fill_(0xFF)
        torch.cuda.synchronize()
        for d in sides:
            with torch.cuda.stream(d["stream"]):
                d["graph"].replay()
        torch.cuda.synchronize()
        for d in sides:
            assert np.array_equal(d["q"].float().cpu().numpy(), d["want"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("form", FORMS)
def test_the_same_bits_in_every_call(form, dim, dtype):
    import torch
    lens, news, group, empty, spare, longest = FORMS[form]
    g, c, table = make(lens, 2, dim, dim + 7)
    start = starts(news + [0] * empty)
    q = torch.from_numpy(queries(g, start[-1] + spare, 2 * group, dim, dtype)).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16)
    gpu = to_gpu(c)
    s = seqs(np.concatenate([table, np.full((empty, table.shape[1]), -1)]), lens + [0] * empty, start, max(news + [spare]), longest)
    ws = S.workspace(S.qmv_kv4_attend_workspace(gpu, s, q))
    first = None
    for turn in range(20):
        out = torch.zeros_like(q)
        ws.fill_(turn)
        S.qmv_kv4_attend(gpu, s, q, out, workspace=ws)
        torch.cuda.synchronize()
        first = out if first is None else first
        assert torch.equal(out.view(torch.uint8), first.view(torch.uint8))
