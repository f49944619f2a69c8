"""The attention kernel for many bfloat16 queries at sizes where a call would
not choose it: hints of long sequences and, for the launch that does not split
them, many rows of no sequence behind the last one."""
import numpy as np
import pytest

import test_gpu_attend as A
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.fixture(params=["split", "whole"])
def many(request, monkeypatch):
    """split: the pages of a sequence over workgroups that are joined; whole: not."""
    import torch
    real_seqs = A.seqs

    def seqs(table, lens, start, max_new=None, max_len=None):
        return real_seqs(table, lens, start, max_new=1 << 20, max_len=1 << 24)

    def attend(c, s, q, dtype, scale=None, window=0, rows=None):
        assert dtype == "bf16"
        n, heads, dim = q.shape
        group = heads // c.kv_heads
        # 8192 / dim columns or, whole, at least 256 workgroups' of 256
        cols = (1 << 18 if window else 1 << 16) if request.param == "whole" else 16384 // dim
        all_rows = max(n, -(-cols // group))
        # (what chooses the kernel: columns, and products of 16 with a page)
        pages = -(-(min(window + 16, 1 << 24) if window else 1 << 24) // 64) + 1
        cols = all_rows * group
        assert cols * dim >= 16384 and s.seqs * c.kv_heads * -(-cols // 16) * pages * dim >= 2.4e6
        qd = torch.full((all_rows, heads, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
        qd[:n] = torch.from_numpy(q)
        out = torch.full_like(qd, 5.0)
        size = S.qmv_kv_attend_workspace(c, s, qd, window)
        assert (size == 0) == (request.param == "whole")
        ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        S.qmv_kv_attend(c, s, qd, out, scale=scale, window=window, workspace=ws)
        assert bool((out[n:] == 5.0).all()), "rows of no sequence were written"
        return out[:n].float().cpu().numpy()

    monkeypatch.setattr(A, "seqs", seqs)
    monkeypatch.setattr(A, "attend", attend)


@pytest.mark.parametrize("lens,news,heads,kv_heads,dim", A.SHAPES)
def test_attend(many, lens, news, heads, kv_heads, dim):
    A.test_attend(lens, news, heads, kv_heads, dim, "bf16")


@pytest.mark.parametrize("many", ["whole"], indirect=True)
@pytest.mark.parametrize("window", [1, 63, 64, 65, 100, 5000])
def test_window(many, window):
    A.test_window(window, "bf16")


@pytest.mark.parametrize("many,window", [("split", 0), ("whole", 0), ("whole", 40), ("whole", 130)],
                         indirect=["many"])
def test_wide_heads(many, window):
    A.test_wide_heads_of_many_rows([300, 190], [150, 128], 2, 2, window)
    A.test_wide_heads_of_many_rows([130, 70, 600], [129, 70, 45], 12, 4, window)


@pytest.mark.parametrize("news", [1, 140])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_maxima_that_grow_and_values_far_apart(many, dim, news):
    A.test_maxima_that_grow_and_values_far_apart(dim, news, "bf16")


@pytest.mark.parametrize("news", [1, 80])
def test_sharp_and_flat_rows(many, news):
    A.test_sharp_and_flat_rows("bf16", news)


@pytest.mark.parametrize("many", ["whole"], indirect=True)
@pytest.mark.parametrize("news", [[1, 1, 1], [70, 80, 65]])
def test_nan_touches_only_what_sees_it(many, news):
    A.test_nan_touches_only_what_sees_it("bf16", news)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_any_scale(many, scale):
    A.test_any_scale(scale, "bf16")


@pytest.mark.parametrize("news", [1, 150])
def test_length_past_the_table(many, news):
    A.test_length_past_the_table(news, "bf16")


def test_rows_without_tokens_and_pages(many):
    A.test_more_rows_than_tokens("bf16")
    A.test_pages_that_are_not_there("bf16")


@pytest.mark.parametrize("many", ["split"], indirect=True)
def test_out_may_be_q_and_capture(many):
    A.test_out_may_be_q_and_capture("bf16", [400, 300], [200, 300])


@pytest.mark.parametrize("many", ["whole"], indirect=True)
def test_many_short_sequences(many):
    A.test_many_short_sequences("bf16")


@pytest.mark.parametrize("many", ["whole"], indirect=True)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exps", A.FAR, ids=lambda e: "_".join(map(str, e)))
def test_scales_of_pages_that_a_row_does_not_see(many, exps, dim):
    # (at head dims of 64 narrower ones are too little work to choose this kernel)
    A.narrow_windows(exps, dim, "bf16", (50, 64) if dim == 64 else (1, 20, 64))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exps", A.FAR, ids=lambda e: "_".join(map(str, e)))
def test_scales_of_pages_without_weight(many, exps, dim):
    A.test_scales_of_pages_without_weight(exps, dim, "bf16")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exps", [[0, -105, -112, 0], [50, -100, -120, -126], [-60, 50, -75, -126], [50, 0, -126, -60]],
                         ids=lambda e: "_".join(map(str, e)))
def test_scales_further_apart_than_float32(many, exps, dim):
    A.test_scales_further_apart_than_float32(exps, dim, "bf16")
