"""The calls of qmv_serve.h in the order of a model's step, with the products
between them: norm, q/k/v products, cache write, attention, output product,
norm with the residual, LM head, log probabilities.  Every stage is held
against its 64-bit reference from the stage's own inputs, so each has its own
derived bound; then the step as a graph is held against the eager one."""
import numpy as np
import pytest

import cases as K
import oracle as O
import serve_ref as R
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S

pytestmark = pytest.mark.gpu
HIDDEN, HEADS, KV, DIM, VOCAB, TOP = 256, 4, 2, 64, 500, 5
EPS = 1e-5
MATRICES = [("q", 2, HEADS * DIM, HIDDEN), ("k", 1, KV * DIM, HIDDEN), ("v", 1, KV * DIM, HIDDEN),
            ("o", 2, HIDDEN, HEADS * DIM), ("head", 1, VOCAB, HIDDEN)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


class Model:
    def __init__(self):
        self.img, self.h = {}, {}
        for i, (name, wt, rows, cols) in enumerate(MATRICES):
            self.img[name] = K.make_image(70, i, wt, 1, rows, cols)
            self.h[name] = K.upload(self.img[name], wt, 1, rows, cols)
        g = np.random.default_rng(70)
        self.norm1 = (1 + 0.1 * g.standard_normal(HIDDEN)).astype(np.float32)
        self.norm2 = (1 + 0.1 * g.standard_normal(HIDDEN)).astype(np.float32)
        self.w1, self.w2 = K.dev(self.norm1), K.dev(self.norm2)

    def close(self):
        for h in self.h.values():
            Q.qmv_destroy(h)


@pytest.fixture()
def model():
    m = Model()
    yield m
    m.close()


class Step:
    """Buffers of a step of `rows` rows, and the step."""

    def __init__(self, m, cache, table, lens, start, coded):
        import torch
        rows = start[-1]
        f = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")
        i = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
        news = [b - a for a, b in zip(start, start[1:])]
        self.m, self.cache, self.coded = m, cache, coded
        self.table, self.len = i(table), i(lens)
        self.seqs = S.KvSeqs(self.table, self.len, i(start), max_new=max(news), max_len=64 * self.table.shape[1])
        self.x, self.ids = f(rows, HIDDEN), f(rows, 1, dtype=torch.int32)
        self.y, self.xq, self.xd = f(rows, HIDDEN), f(rows, HIDDEN, dtype=torch.int8), f(rows, HIDDEN // 32)
        self.q, self.k, self.v = f(rows, HEADS, DIM), f(rows, KV, DIM), f(rows, KV, DIM)
        self.att, self.o, self.sum = f(rows, HEADS, DIM), f(rows, HIDDEN), f(rows, HIDDEN)
        self.y2, self.logits = f(rows, HIDDEN), f(rows, VOCAB)
        self.lp, self.h = f(rows, 1), f(rows)
        self.ti, self.tl = f(rows, TOP, dtype=torch.int32), f(rows, TOP)
        self.ws = S.workspace(S.qmv_kv_attend_workspace(cache, self.seqs, self.q))
        self.ws2 = S.workspace(S.qmv_logprobs_workspace(rows, VOCAB, TOP))

    def run(self, stream=None):
        m, s = self.m, stream
        if self.coded:                           # quantized activations, as prompts take them
            S.qmv_rms_norm(self.x, m.w1, EPS, q=self.xq, d=self.xd, stream=s)
            for name, out in (("q", self.q), ("k", self.k), ("v", self.v)):
                Q.qmv_gemm_q8(m.h[name], self.xq, self.xd, out.view(out.shape[0], -1), stream=s)
        else:
            S.qmv_rms_norm(self.x, m.w1, EPS, y=self.y, stream=s)
            for name, out in (("q", self.q), ("k", self.k), ("v", self.v)):
                Q.qmv_gemv(m.h[name], self.y, out.view(out.shape[0], -1), stream=s)
        S.qmv_kv_write(self.cache, self.seqs, self.k, self.v, stream=s)
        S.qmv_kv_attend(self.cache, self.seqs, self.q, self.att, workspace=self.ws, stream=s)
        Q.qmv_gemv(m.h["o"], self.att.view(-1, HIDDEN), self.o, stream=s)
        S.qmv_rms_norm(self.o, m.w2, EPS, res=self.x, sum=self.sum, y=self.y2, stream=s)
        Q.qmv_gemv(m.h["head"], self.y2, self.logits, stream=s)
        S.qmv_logprobs(self.logits, self.ids, self.lp, self.h, self.ti, self.tl, workspace=self.ws2, stream=s)

    OUT = ("y", "xq", "xd", "q", "k", "v", "att", "o", "sum", "y2", "logits", "lp", "h", "ti", "tl")

    def outputs(self):
        import torch
        torch.cuda.synchronize()
        return {n: getattr(self, n).cpu().numpy() for n in self.OUT}


def product_ok(m, name, x, y):
    _, wt, rows, cols = next(t for t in MATRICES if t[0] == name)
    ref, norm = O.product(m.img[name], wt, 1, rows, cols, x, threads=K.THREADS)
    assert O.within_tolerance(y, ref, norm)[0], name


def stages_ok(m, st, x, ids, ref_cache, table, lens, start):
    """Every stage of a step that ran, from the stage's own inputs."""
    o = st.outputs()
    rows = x.shape[0]
    _, y = R.norm(x, None, m.norm1, EPS)
    if st.coded:
        # codes round to half a step of d; y / d and d round by 2^-22 and
        # less, at most 127 of them 2^-15 of a step
        dec = o["xq"].reshape(rows, -1, 32) * o["xd"][:, :, None].astype(np.float64)
        assert np.all(np.abs(dec.reshape(y.shape) - y) <= 0.51 * np.repeat(o["xd"], 32, 1) + 1e-6 * np.abs(y))
        for name in ("q", "k", "v"):
            _, wt, n, cols = next(t for t in MATRICES if t[0] == name)
            ref, bound = O.gemm_q8act(m.img[name], wt, 1, n, cols, o["xq"], o["xd"], threads=K.THREADS)
            assert O.q8act_within_tolerance(o[name].reshape(rows, n), ref, bound, cols)[0], name
    else:
        assert np.all(np.abs(o["y"] - y) <= 3.01 * 2.0 ** -24 * np.abs(y))
        for name in ("q", "k", "v"):
            product_ok(m, name, o["y"], o[name].reshape(rows, -1))
    ref_cache.write(table, lens, start, o["k"], o["v"])
    used = sorted({int(p) for t, n in zip(table, lens) for p in t[:-(-n // 64)]})
    c = st.cache
    for name in ("k_scale", "v_scale"):
        assert np.array_equal(getattr(c, name).cpu().numpy()[used], getattr(ref_cache, name)[used].astype(np.float32))
    ref, b = R.attend(ref_cache, table, lens, start, o["q"], np.float32(DIM ** -0.5), 0)
    assert np.all(np.abs(o["att"] - ref) <= R.attend_bound(b, o["q"], DIM ** -0.5, max(lens), "f32"))
    product_ok(m, "o", o["att"].reshape(rows, -1), o["o"])
    h, y = R.norm(o["o"], x, m.norm2, EPS)
    assert np.array_equal(o["sum"], h) and np.all(np.abs(o["y2"] - y) <= 3.01 * 2.0 ** -24 * np.abs(y))
    product_ok(m, "head", o["y2"], o["logits"])
    ref = R.logprobs(o["logits"], ids, TOP)
    assert np.all(np.abs(o["lp"] - ref["lp"]) <= R.logprob_bound(ref, ref["lp"], 1))
    assert np.all(np.abs(o["h"] - ref["entropy"]) <= R.entropy_bound(ref, 1))
    assert np.array_equal(o["ti"], ref["top_ids"])
    assert np.all(np.abs(o["tl"] - ref["top_lp"]) <= R.logprob_bound(ref, ref["top_lp"], 1))
    return o


def test_prompt_then_tokens(model):
    """A prompt of three sequences, then tokens one by one over a page's end,
    eager and as a graph that is replayed as the lengths grow."""
    import torch
    g = np.random.default_rng(71)
    prompt = [70, 9, 126]
    table = np.array([[4, 1, 7], [0, 9, 5], [3, 8, 2]])
    cache, ref = S.KvCache.empty(10, KV, DIM), R.Cache(10, KV, DIM)
    start = [0, 70, 79, 205]
    x, ids = g.standard_normal((205, HIDDEN)).astype(np.float32), g.integers(0, VOCAB, size=(205, 1))
    st = Step(model, cache, table, prompt, start, coded=True)
    st.x.copy_(torch.from_numpy(x))
    st.ids.copy_(torch.from_numpy(ids.astype(np.int32)))
    st.run()
    stages_ok(model, st, x, ids, ref, table, prompt, start)

    # tokens: the eager step and, from the same state of the cache, the graph
    def clone():
        return S.KvCache(*(t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    other = clone()
    one = [0, 1, 2, 3]
    eager = Step(model, cache, table, prompt, one, coded=False)
    graphed = Step(model, other, table, prompt, one, coded=False)
    graphed.x.zero_()
    graphed.ids.zero_()
    # (the first call of a shape may set up what a capture could not; the
    # token it writes is written again by the first replay, at a place that a
    # scale of zeros does not change)
    graphed.len.copy_(torch.tensor([n + 1 for n in prompt], dtype=torch.int32))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphed.run(stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        graphed.run(stream)
    lens = list(prompt)
    for turn in range(4):
        lens = [n + 1 for n in lens]
        x, ids = g.standard_normal((3, HIDDEN)).astype(np.float32), g.integers(0, VOCAB, size=(3, 1))
        for s in (eager, graphed):
            s.x.copy_(torch.from_numpy(x))
            s.ids.copy_(torch.from_numpy(ids.astype(np.int32)))
            s.len.copy_(torch.tensor(lens, dtype=torch.int32))
        eager.run()
        want = stages_ok(model, eager, x, ids, ref, table, lens, one)
        graph.replay()
        got = graphed.outputs()
        for name in want:
            if name not in ("xq", "xd"):         # (not this step's)
                assert np.array_equal(got[name], want[name]), (turn, name)
