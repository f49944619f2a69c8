"""A model's step from a token to the next one with the heads' rotation, the
4-bit cache and the draw, and the framework's products and norms between them.
Every stage is held against its 64-bit reference from the stage's own inputs,
so each has its own derived bound; then the step as a graph, each token drawn
being the next one's input, is held against the eager one."""
import numpy as np
import pytest

import cases as K
import more_ref as M
import oracle as O
import serve_ref as R
from block_quant_weight_amd import qmv as Q
from block_quant_weight_amd import serve as S
from test_gpu_kv4 import to_gpu

pytestmark = pytest.mark.gpu
HIDDEN, HEADS, KV, DIM, ROT, VOCAB = 256, 4, 2, 64, 32, 500
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
            self.img[name] = K.make_image(72, i, wt, 1, rows, cols)
            self.h[name] = K.upload(self.img[name], wt, 1, rows, cols)
        g = np.random.default_rng(72)
        near = lambda n: (1 + 0.1 * g.standard_normal(n)).astype(np.float32)
        self.norm, self.out_norm, self.q_norm, self.k_norm = near(HIDDEN), near(HIDDEN), near(DIM), near(DIM)
        self.freq = (1e4 ** (-2.0 * np.arange(ROT // 2) / ROT)).astype(np.float32)
        self.embed = g.standard_normal((VOCAB, HIDDEN)).astype(np.float32)
        self.dev = {n: K.dev(getattr(self, n)) for n in ("norm", "out_norm", "q_norm", "k_norm", "freq", "embed")}

    def close(self):
        for h in self.h.values():
            Q.qmv_destroy(h)




class Step:
    """Buffers of a step of `rows` rows, and the step."""

    OUT = ("x", "y", "q", "k", "v", "qr", "kr", "att", "o", "sum", "y2", "logits", "ids", "lp")

    def __init__(self, m, cache, table, lens, start, wish):
        import torch
        rows, dev = start[-1], "cuda"
        f = lambda *s: torch.empty(*s, device=dev)
        i = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)
        news = [b - a for a, b in zip(start, start[1:])]
        self.m, self.cache = m, cache
        self.len, self.pos = i(lens), i(np.zeros(rows))
        self.seqs = S.KvSeqs(i(table), self.len, i(start), max_new=max(news), max_len=64 * table.shape[1])
        self.ids, self.lp, self.u = i(np.zeros(rows)), f(rows), f(rows)
        self.wish = {n: torch.from_numpy(np.ascontiguousarray(a)).cuda() for n, a in wish.items()}
        self.x, self.y = f(rows, HIDDEN), f(rows, HIDDEN)
        self.q, self.k, self.v = f(rows, HEADS, DIM), f(rows, KV, DIM), f(rows, KV, DIM)
        self.qr, self.kr = f(rows, HEADS, DIM), f(rows, KV, DIM)
        self.att, self.o, self.sum = f(rows, HEADS, DIM), f(rows, HIDDEN), f(rows, HIDDEN)
        self.y2, self.logits = f(rows, HIDDEN), f(rows, VOCAB)
        self.ws = S.workspace(max(S.qmv_kv4_attend_workspace(cache, self.seqs, self.q), 16))
        self.ws2 = S.workspace(max(S.qmv_sample_workspace(rows, VOCAB), 16))

    def run(self, stream=None):
        import torch
        m, s = self.m, stream
        torch.index_select(m.dev["embed"], 0, self.ids, out=self.x)
        S.qmv_rms_norm(self.x, m.dev["norm"], EPS, y=self.y, stream=s)
        for name, out in (("q", self.q), ("k", self.k), ("v", self.v)):
            Q.qmv_gemv(m.h[name], self.y, out.view(out.shape[0], -1), stream=s)
        S.qmv_qk_rotate(self.q, self.k, self.pos, m.dev["freq"], self.qr, self.kr, q_w=m.dev["q_norm"], k_w=m.dev["k_norm"],
                        eps=EPS, stream=s)
        S.qmv_kv4_write(self.cache, self.seqs, self.kr, self.v, stream=s)
        S.qmv_kv4_attend(self.cache, self.seqs, self.qr, self.att, workspace=self.ws, stream=s)
        Q.qmv_gemv(m.h["o"], self.att.view(-1, HEADS * DIM), self.o, stream=s)
        S.qmv_rms_norm(self.o, m.dev["out_norm"], EPS, res=self.x, sum=self.sum, y=self.y2, stream=s)
        Q.qmv_gemv(m.h["head"], self.y2, self.logits, stream=s)
        S.qmv_sample(self.logits, self.u, self.ids, lp=self.lp, workspace=self.ws2, stream=s, **self.wish)

    def give(self, lens, pos, u, ids=None):
        import torch
        self.len.copy_(torch.tensor(lens, dtype=torch.int32))
        self.pos.copy_(torch.from_numpy(pos.astype(np.int32)))
        self.u.copy_(torch.from_numpy(u))
        if ids is not None:
            self.ids.copy_(torch.from_numpy(ids.astype(np.int32)))

    def outputs(self):
        import torch
        torch.cuda.synchronize()
        return {n: getattr(self, n).cpu().numpy() for n in self.OUT}


def product_ok(m, name, x, y):
    _, wt, rows, cols = next(t for t in MATRICES if t[0] == name)
    ref, norm = O.product(m.img[name], wt, 1, rows, cols, x, threads=K.THREADS)
    assert O.within_tolerance(y, ref, norm)[0], name


def stages_ok(m, st, ids, pos, u, wish, ref_cache, table, lens, start):
    """Every stage of a step that ran, from the stage's own inputs."""
    o = st.outputs()
    rows = len(ids)
    assert np.array_equal(o["x"], m.embed[ids])
    _, y = R.norm(o["x"], None, m.norm, EPS)
    assert np.all(np.abs(o["y"] - y) <= 3.01 * 2.0 ** -24 * np.abs(y))
    for name in ("q", "k", "v"):
        product_ok(m, name, o["y"], o[name].reshape(rows, -1))
    for name, w in (("q", m.q_norm), ("k", m.k_norm)):
        # (the bound of the rotation's own tests)
        ref, size = M.rotate(o[name], w, EPS, pos, m.freq, False, 1.0)
        assert np.all(np.abs(o[name + "r"] - ref) <= 13 * 2.0 ** -24 * size + 1e-44), name
    ref_cache.write(table, lens, start, o["kr"], o["v"])
    c = st.cache
    for got, want in zip((c.k, c.v, c.k_scale, c.v_scale), ref_cache.arrays()):
        assert np.array_equal(got.cpu().numpy().reshape(want.shape), want)
    ref, b = M.attend(ref_cache, table, lens, start, o["qr"], np.float32(DIM ** -0.5), 0)
    assert np.all(np.abs(o["att"] - ref) <= M.attend_bound(b, DIM, max(lens), "f32"))
    product_ok(m, "o", o["att"].reshape(rows, -1), o["o"])
    h, y = R.norm(o["o"], o["x"], m.out_norm, EPS)
    assert np.array_equal(o["sum"], h) and np.all(np.abs(o["y2"] - y) <= 3.01 * 2.0 ** -24 * np.abs(y))
    product_ok(m, "head", o["y2"], o["logits"])
    f = lambda a, i: float(np.float32(a[i]))
    for i in range(rows):
        answers = M.sample_answers(o["logits"][i], f(u, i), f(wish["temperature"], i), int(wish["top_k"][i]), f(wish["top_p"], i),
                                   f(wish["min_p"], i))
        assert M.sample_ok(answers, o["ids"][i], o["lp"][i]), i
    return o


def wishes(g, rows):
    return dict(temperature=g.choice([0.0, 0.7, 5.0], rows).astype(np.float32), top_k=g.choice([0, 40], rows).astype(np.int32),
                top_p=g.choice([1.0, 0.9], rows).astype(np.float32), min_p=g.choice([0.0, 0.02], rows).astype(np.float32))


def test_prompt_then_tokens():
    """A prompt of three sequences, then tokens one by one over a page's end,
    each drawn from the step before, eager and as a graph replayed as the
    lengths grow."""
    import torch
    m = Model()
    try:
        g = np.random.default_rng(73)
        prompt = [70, 9, 126]
        table = np.array([[4, 1, 7], [0, 9, 5], [3, 8, 2]])
        ref = M.Cache4(10, KV, DIM)
        cache = to_gpu(ref)
        start = [0, 70, 79, 205]
        ids, u, wish = g.integers(0, VOCAB, size=205), g.random(205).astype(np.float32), wishes(g, 205)
        pos = np.concatenate([np.arange(n) for n in prompt])
        st = Step(m, cache, table, prompt, start, wish)
        st.give(prompt, pos, u, ids)
        st.run()
        o = stages_ok(m, st, ids, pos, u, wish, ref, table, prompt, start)
        ids = o["ids"][[n - 1 for n in start[1:]]]          # each sequence's next token

        # tokens: the eager step and, from the same state of the cache, the graph
        other = S.Kv4Cache(*(t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
        one, wish = [0, 1, 2, 3], wishes(g, 3)
        eager, graphed = Step(m, cache, table, prompt, one, wish), Step(m, other, table, prompt, one, wish)
        lens = list(prompt)
        # (the first call of a shape may set up what a capture could not; the
        # token that it writes is written again by the first replay)
        graphed.give([n + 1 for n in lens], np.array(lens), np.zeros(3, dtype=np.float32), ids)
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            graphed.run(stream)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            graphed.run(stream)
        eager.give(lens, np.array(lens), np.zeros(3, dtype=np.float32), ids)
        graphed.give(lens, np.array(lens), np.zeros(3, dtype=np.float32), ids)
        for turn in range(4):
            pos, lens, u = np.array(lens), [n + 1 for n in lens], g.random(3).astype(np.float32)
            for s in (eager, graphed):
                s.give(lens, pos, u)
            eager.run()
            want = stages_ok(m, eager, ids, pos, u, wish, ref, table, lens, one)
            graph.replay()
            got = graphed.outputs()
            for name in want:
                assert np.array_equal(got[name], want[name]), (turn, name)
            ids = want["ids"]
    finally:
        m.close()
