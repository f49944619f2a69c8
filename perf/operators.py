"""The operators between a quantized model's products, as they are measured:
the norm in front of a product, the 8-bit key/value cache (written and read
back), attention over that cache, and the log probabilities of the LM head's
logits.

`run` with own = False computes each operator in plain torch; with own = True
it makes the calls of block_quant_weight_amd.serve.  A case is a dict of plain
values; prepare(case, seed) makes its inputs on the GPU, exact(case, seed)
the same results in 64 bits."""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
PAGE = 64          # tokens of a cache page, which share one scale per head
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # -- norm: (rows, cols) of the residual stream in front of a product
        # one decode token in front of qmv_gemv (dim 4096 of the decode layer): latency
        {"name": "norm_1x4096_f32", "op": "norm", "rows": 1, "cols": 4096, "out": "f32", "residual": True},
        # a prefill batch of 512 tokens in front of qmv_gemm_q8: Q8_0 activations
        {"name": "norm_512x4096_q8", "op": "norm", "rows": 512, "cols": 4096, "out": "q8", "residual": True},
        # a long prompt in front of qmv_gemm: bfloat16 activations
        {"name": "norm_8191x4096_bf16", "op": "norm", "rows": 8191, "cols": 4096, "out": "bf16", "residual": True},
        # -- cache: 8 KV heads of 128
        # one new token for each of 64 sequences, float32 from the vector product; the last 100 tokens read back
        {"name": "cache_append_64x1_f32", "op": "cache", "seqs": 64, "len": 2000, "new": 1, "back": 100,
         "kv_heads": 8, "dim": 128, "dtype": "f32"},
        # prompts of up to 4096 tokens written page by page and read back whole
        {"name": "cache_prompt_4x4096_bf16", "op": "cache", "seqs": 4, "len": 4096, "new": 4096, "back": 4096,
         "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # -- attention
        # the smallest call: one sequence of 100 tokens, one new token
        {"name": "attend_1x100_f32", "op": "attend", "seqs": 1, "len": 100, "new": 1, "heads": 8, "kv_heads": 2,
         "dim": 64, "dtype": "f32", "window": 0},
        # an ordinary decode step: 32 sequences of 1000 to 4000 tokens, 32 heads on 8 KV heads of 128
        {"name": "attend_32x4000_f32", "op": "attend", "seqs": 32, "len": 4000, "new": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "dtype": "f32", "window": 0},
        # decode on a few very long contexts
        {"name": "attend_2x131072_bf16", "op": "attend", "seqs": 2, "len": 131072, "new": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "window": 0},
        # a whole prompt of 8192 tokens
        {"name": "attend_prompt_1x8192_bf16", "op": "attend", "seqs": 1, "len": 8192, "new": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "window": 0},
        # pieces of up to 500 tokens of three prompts under a sliding window, heads of 256
        {"name": "attend_piece_3x500_window", "op": "attend", "seqs": 3, "len": 6000, "new": 500, "heads": 16,
         "kv_heads": 4, "dim": 256, "dtype": "bf16", "window": 1024},
        # -- log probabilities: the 248320-row LM head's logits
        # one sampled token with its 20 best alternatives
        {"name": "logprobs_1x248320", "op": "logprobs", "rows": 1, "vocab": 248320, "ids": 1, "top": 20},
        # a decode batch of 64
        {"name": "logprobs_64x248320", "op": "logprobs", "rows": 64, "vocab": 248320, "ids": 1, "top": 20},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "cache", "attend", "attend", "logprobs"))
    if op == "norm":
        cols = 32 * _log(rng, 1, 512)
        return {"op": op, "rows": min(_log(rng, 1, 8191), (7000 * 4096) // cols), "cols": cols,
                "out": rng.choice(("f32", "bf16", "q8")), "residual": rng.random() < 0.75}
    if op == "logprobs":
        vocab = _log(rng, 500, 262144)
        return {"op": op, "rows": min(_log(rng, 1, 2048), (63 * 248320) // vocab), "vocab": vocab,
                "ids": rng.choice((1, 1, 2, 5)), "top": rng.choice((0, 1, 5, 20, 32))}
    kv_heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 128, 256))
    dtype = rng.choice(("f32", "bf16"))
    per = kv_heads * dim                      # values a token keeps
    if op == "cache":
        size = 5 if dtype == "f32" else 3
        length = min(_log(rng, 1, 16000), 120_000_000 // (4 * per * size))
        seqs = max(1, min(_log(rng, 1, 128), 120_000_000 // (4 * per * size * length)))
        new = rng.choice((1, _log(rng, 1, length), length))
        return {"op": op, "seqs": seqs, "len": length, "new": new, "back": rng.choice((new, length)),
                "kv_heads": kv_heads, "dim": dim, "dtype": dtype}
    group = rng.choice((1, 2, 4, 5, 8))
    kind = rng.choice(("decode", "decode", "few", "prompt"))
    if kind == "prompt":
        length = _log(rng, 16, 8192)
        new = rng.choice((length, _log(rng, 16, min(length, 2048))))
        heads = kv_heads * group
        new = min(new, 130_000_000_000 // (length * heads * dim))
        seqs = max(1, min(_log(rng, 1, 16), 130_000_000_000 // (length * new * heads * dim), (1 << 30) // (length * new * heads)))
    else:
        length = _log(rng, 1, 131072)
        new = 1 if kind == "decode" else min(length, rng.randint(2, 9))
        seqs = max(1, min(_log(rng, 1, 64), (2 * 131072 * 1024) // (length * per)))
    return {"op": op, "seqs": seqs, "len": length, "new": new, "heads": kv_heads * group, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "window": rng.choice((0, 0, 0, _log(rng, 16, 4096)))}


def _lengths(case):
    """(tokens in the cache with the new ones, new tokens) of every sequence:
    the first sequence has the most, the others between a quarter and all."""
    r = random.Random(case["seqs"] * 1000003 + case["len"] * 101 + case["new"])
    lens, news = [], []
    for i in range(case["seqs"]):
        n = case["len"] if i == 0 else r.randint(max(1, case["len"] // 4), case["len"])
        m = case["new"] if i == 0 else r.randint((case["new"] + 1) // 2, case["new"])
        lens.append(n)
        news.append(min(n, m))
    return lens, news


def _pairs(n, m, window):
    """Query-key pairs of a sequence of n tokens whose last m are queries, and the keys that any of them sees."""
    if window == 0:
        return m * (n - m) + m * (m + 1) // 2, n
    k = max(0, min(m, window - (n - m)))      # queries that see everything before them
    return k * (n - m) + k * (k + 1) // 2 + (m - k) * window, min(n, window + m - 1)


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["cols"]
        out = {"f32": 4 * n, "bf16": 2 * n, "q8": n + n // 8}[case["out"]]
        return {"bytes": 4 * n * (3 if case["residual"] else 1) + out + 4 * case["cols"], "flops": 5 * n}
    if op == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": 4 * n + case["rows"] * (8 * case["ids"] + 8 * case["top"] + 4), "flops": 5 * n}
    lens, news = _lengths(case)
    size = 4 if case["dtype"] == "f32" else 2
    per = case["kv_heads"] * case["dim"]
    if op == "cache":
        new, back = sum(news), sum(min(case["back"], n) for n in lens)
        return {"bytes": 2 * per * (new * (size + 1) + back * (size + 1)), "flops": 2 * per * (4 * new + back)}
    pairs, keys = (sum(v) for v in zip(*(_pairs(n, m, case["window"]) for n, m in zip(lens, news))))
    q = sum(news) * case["heads"] * case["dim"]
    return {"bytes": 2 * per * keys + 2 * size * q, "flops": 4 * case["heads"] * case["dim"] * pairs}


# ---- inputs ----------------------------------------------------------------

def _power(amax):
    """The scale of a page: the least power of two d with amax <= 127 d (0 for a page of zeros)."""
    m, e = torch.frexp(amax)
    e = torch.clamp(torch.where(m <= 127.0 / 128.0, e - 7, e - 6), min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _codes(x, d):
    """Whole multiples of d nearest to x, in 8 bits."""
    return torch.round(x / torch.where(d > 0, d, torch.ones_like(d))).to(torch.int8)


def _cache_state(case, g):
    """A cache whose pages are handed out in no order, filled up to each
    sequence's last `new` tokens, and what says which page holds what."""
    lens, news = _lengths(case)
    counts = [-(-n // PAGE) for n in lens]
    pages, most = sum(counts) + 3, max(counts)
    kvh, dim = case["kv_heads"], case["dim"]
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32).cpu()
    table = torch.full((case["seqs"], most), -1, dtype=torch.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    start = [0]
    for m in news:
        start.append(start[-1] + m)
    # keys have channels that stand out, values do not
    width = 1.0 + 4.0 * (torch.rand(dim, generator=g, device=DEVICE) < 0.05)
    k = torch.empty(pages, kvh, PAGE, dim, dtype=torch.int8, device=DEVICE)
    v = torch.empty(pages, kvh, dim, PAGE, dtype=torch.int8, device=DEVICE)
    ks = torch.empty(pages, kvh, device=DEVICE)
    vs = torch.empty(pages, kvh, device=DEVICE)
    step = max(1, (1 << 26) // (kvh * PAGE * dim))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        x = torch.randn(b - a, kvh, PAGE, dim, generator=g, device=DEVICE) * width
        ks[a:b] = _power(x.abs().amax((2, 3)))
        k[a:b] = _codes(x, ks[a:b, :, None, None])
        x = torch.randn(b - a, kvh, dim, PAGE, generator=g, device=DEVICE)
        vs[a:b] = _power(x.abs().amax((2, 3)))
        v[a:b] = _codes(x, vs[a:b, :, None, None])
    s = {"k": k, "v": v, "k_scale": ks, "v_scale": vs, "table": table.to(DEVICE), "width": width,
         "len": torch.tensor(lens, dtype=torch.int32, device=DEVICE),
         "start": torch.tensor(start, dtype=torch.int32, device=DEVICE),
         "max_len": max(lens), "max_new": max(news), "rows": start[-1]}
    s.update(_places(lens, news, table, "row_"))
    return s


def _places(lens, news, table, what):
    """Sequence, position and page of the last `news` tokens of every sequence, one after the other."""
    seq = torch.tensor([i for i, m in enumerate(news) for _ in range(m)], dtype=torch.int64)
    pos = torch.tensor([p for n, m in zip(lens, news) for p in range(n - m, n)], dtype=torch.int64)
    page = table[seq, pos // PAGE].to(torch.int64)
    return {what + "seq": seq.to(DEVICE), what + "pos": pos.to(DEVICE), what + "page": page.to(DEVICE)}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    op = case["op"]
    if op == "norm":
        n, c = case["rows"], case["cols"]
        s = {"case": case, "x": normal(n, c), "w": 1.0 + 0.1 * normal(c),
             "res": 3.0 * normal(n, c) if case["residual"] else None}
        s["sum"] = torch.empty(n, c, device=DEVICE) if case["residual"] else None
        if case["out"] == "q8":
            s["q"] = torch.empty(n, c, dtype=torch.int8, device=DEVICE)
            s["d"] = torch.empty(n, c // 32, device=DEVICE)
        else:
            s["y"] = torch.empty(n, c, dtype=DTYPES[case["out"]], device=DEVICE)
        return s
    if op == "logprobs":
        n, v, top = case["rows"], case["vocab"], case["top"]
        s = {"case": case, "x": 2.5 * normal(n, v),
             "ids": torch.randint(0, v, (n, case["ids"]), generator=g, device=DEVICE).to(torch.int32),
             "lp": torch.empty(n, case["ids"], device=DEVICE), "entropy": torch.empty(n, device=DEVICE),
             "top_ids": torch.empty(n, top, dtype=torch.int32, device=DEVICE) if top else None,
             "top_lp": torch.empty(n, top, device=DEVICE) if top else None}
        s["x"][:, :max(1, v // 1000)] *= 2.0      # a few likely tokens, and ties among the others
        s["x"] = torch.round(s["x"] * 4096.0) / 4096.0
        if own:
            from block_quant_weight_amd import serve
            s["workspace"] = serve.workspace(serve.qmv_logprobs_workspace(n, v, top), DEVICE)
        return s
    s = _cache_state(case, g)
    s["case"] = case
    dtype = DTYPES[case["dtype"]]
    kvh, dim = case["kv_heads"], case["dim"]
    if op == "cache":
        # some of the new tokens are larger than what their page holds so far
        big = 1.0 + 2.0 * (torch.rand(s["rows"], 1, 1, generator=g, device=DEVICE) < 0.1)
        s["new_k"] = (normal(s["rows"], kvh, dim) * s["width"] * big).to(dtype)
        s["new_v"] = (normal(s["rows"], kvh, dim) * big).to(dtype)
        lens, news = _lengths(case)
        backs = [min(case["back"], n) for n in lens]
        first = [0]
        for m in backs:
            first.append(first[-1] + m)
        s.update(_places(lens, backs, s["table"].cpu(), "back_"))
        s["touched"] = torch.unique(s["row_page"])
        s["back_start"] = torch.tensor(first, dtype=torch.int32, device=DEVICE)
        s["out_k"] = torch.empty(first[-1], kvh, dim, dtype=dtype, device=DEVICE)
        s["out_v"] = torch.empty(first[-1], kvh, dim, dtype=dtype, device=DEVICE)
    else:
        s["q"] = (2.0 * normal(s["rows"], case["heads"], dim)).to(dtype)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(dim)
    if own:      # the handles that a program keeps: of the cache, and of a step's sequences for all its layers
        from block_quant_weight_amd import serve
        s["cache"] = serve.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["seqs"] = serve.KvSeqs(s["table"], s["len"], s["start"], max_new=s["max_new"], max_len=s["max_len"])
        if op == "cache":
            s["back_seqs"] = serve.KvSeqs(s["table"], s["len"], s["back_start"],
                                          max_new=min(case["back"], s["max_len"]), max_len=s["max_len"])
        else:
            s["workspace"] = serve.workspace(serve.qmv_kv_attend_workspace(
                s["cache"], s["seqs"], s["q"], window=case["window"]), DEVICE)
    return s


# ---- one pass --------------------------------------------------------------

def run(s):
    if own:
        return {"norm": _own_norm, "cache": _own_cache, "attend": _own_attend, "logprobs": _own_logprobs}[s["case"]["op"]](s)
    return {"norm": _norm, "cache": _cache, "attend": _attend, "logprobs": _logprobs}[s["case"]["op"]](s)


def _values(q, d):
    """What Q8_0 activations stand for."""
    return (q.view(q.shape[0], -1, 32) * d.unsqueeze(-1)).view(q.shape)


def _own_norm(s):
    from block_quant_weight_amd import serve
    if s["case"]["out"] == "q8":
        serve.qmv_rms_norm(s["x"], s["w"], EPS, res=s["res"], sum=s["sum"], q=s["q"], d=s["d"])
        return {"sum": s["sum"], "y": _values(s["q"], s["d"])}
    serve.qmv_rms_norm(s["x"], s["w"], EPS, res=s["res"], sum=s["sum"], y=s["y"])
    return {"sum": s["sum"], "y": s["y"]}


def _norm(s):
    x, res = s["x"], s["res"]
    h = x if res is None else x + res
    mean = h.double().square().mean(-1, keepdim=True)       # 64 bits: the codes lie next to borders
    y = h * (1.0 / torch.sqrt(mean + EPS)).float() * s["w"]
    total = None if res is None else h
    if s["case"]["out"] != "q8":
        return {"sum": total, "y": y.to(DTYPES[s["case"]["out"]])}
    b = y.view(y.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, 127.0)                      # a tensor: a number would be divided by with its reciprocal
    d = torch.where(amax < 1e-30, 0.0, amax / top)
    q = torch.trunc(b * torch.where(amax < 1e-30, 0.0, top / amax) + torch.copysign(torch.full_like(b, 0.5), b))
    q = torch.where(amax < 1e-30, 0.0, q.clamp(-127, 127))
    return {"sum": total, "y": (q * d).view(y.shape)}


def _own_cache(s):
    from block_quant_weight_amd import serve
    serve.qmv_kv_write(s["cache"], s["seqs"], s["new_k"], s["new_v"])
    serve.qmv_kv_read(s["cache"], s["back_seqs"], s["out_k"], s["out_v"])
    return {"k": s["out_k"], "v": s["out_v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _write(s, codes, scale, x, swap):
    """New tokens x [rows, heads, dim] into their pages of codes [pages,
    heads, 64, dim] (swap: [pages, heads, dim, 64]), in place."""
    page, off, touched = s["row_page"], s["row_pos"] % PAGE, s["touched"]
    x = x.float()
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    fresh = torch.zeros(scale.shape[0], dtype=torch.int32, device=scale.device)
    fresh = fresh.index_add_(0, page, (off == 0).to(torch.int32))[touched].unsqueeze(-1) > 0
    old = torch.where(fresh, 0.0, scale[touched])
    d = torch.maximum(old, _power(amax[touched]))
    ratio = torch.where(d > 0, old / torch.where(d > 0, d, 1.0), 0.0)
    codes[touched] = torch.round(codes[touched].float() * ratio[:, :, None, None]).to(torch.int8)
    scale[touched] = d
    q = _codes(x, scale[page].unsqueeze(-1))
    if swap:
        codes.transpose(2, 3)[page, :, off] = q
    else:
        codes[page, :, off] = q


def _cache(s):
    _write(s, s["k"], s["k_scale"], s["new_k"], False)
    _write(s, s["v"], s["v_scale"], s["new_v"], True)
    page, off = s["back_page"], s["back_pos"] % PAGE
    dtype = s["new_k"].dtype
    return {"k": (s["k"][page, :, off] * s["k_scale"][page].unsqueeze(-1)).to(dtype),
            "v": (s["v"].transpose(2, 3)[page, :, off] * s["v_scale"][page].unsqueeze(-1)).to(dtype),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _own_attend(s):
    from block_quant_weight_amd import serve
    serve.qmv_kv_attend(s["cache"], s["seqs"], s["q"], s["out"], scale=s["scale"], window=s["case"]["window"],
                        workspace=s["workspace"])
    return s["out"]


def _attend(s):
    case = s["case"]
    kvh, dim, group = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    n, new = case["seqs"], s["max_new"]
    pages = s["table"].long().clamp(min=0)                  # [n, pages]
    k = (s["k"][pages] * s["k_scale"][pages][..., None, None]).transpose(2, 3).reshape(n, -1, kvh, dim)
    v = (s["v"][pages] * s["v_scale"][pages][..., None, None]).permute(0, 1, 4, 2, 3).reshape(n, -1, kvh, dim)
    keys = k.shape[1]
    length, start = s["len"].long(), s["start"].long()
    count = start[1:] - start[:-1]
    t = torch.arange(new, device=k.device)
    row = (start[:-1, None] + t).clamp(max=s["rows"] - 1)   # [n, new]: rows of q, those past a sequence's end unused
    pos = (length - count).unsqueeze(1) + t
    q = s["q"].float()[row].view(n, new, kvh, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kvh, group * new, dim)
    p = torch.matmul(q, k.permute(0, 2, 3, 1)).view(n, kvh, group, new, keys) * s["scale"]
    j = torch.arange(keys, device=k.device)
    seen = (j <= pos.unsqueeze(-1)) & (j < length[:, None, None])
    if case["window"]:
        seen &= j > pos.unsqueeze(-1) - case["window"]
    p.masked_fill_(~seen[:, None, None], float("-inf"))
    p -= p.amax(-1, keepdim=True)
    p.exp_()
    p /= p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, kvh, group * new, keys), v.transpose(1, 2)).view(n, kvh, group, new, dim)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, new, case["heads"], dim)
    at = s["row_pos"] - (length - count)[s["row_seq"]]
    return o[s["row_seq"], at].to(s["q"].dtype)


def _own_logprobs(s):
    from block_quant_weight_amd import serve
    serve.qmv_logprobs(s["x"], s["ids"], s["lp"], s["entropy"], s["top_ids"], s["top_lp"], workspace=s["workspace"])
    return {"lp": s["lp"], "entropy": s["entropy"], "top_ids": s["top_ids"], "top_lp": s["top_lp"]}


def _logprobs(s):
    x, top = s["x"], s["case"]["top"]
    z = x - x.amax(-1, keepdim=True)
    e = z.exp()
    total = e.sum(-1, keepdim=True)
    lp = z - total.log()
    got = {"lp": lp.gather(1, s["ids"].long()), "entropy": -(e * lp).sum(-1) / total[:, 0], "top_ids": None, "top_lp": None}
    if top:
        # the larger value first, then the lower index: whole numbers in the order of the values, above the index
        b = (x + 0.0).view(torch.int32).long()
        b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
        key = b * (1 << 31) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
        at = key.topk(top, -1).indices
        got["top_ids"], got["top_lp"] = at.to(torch.int32), lp.gather(1, at)
    return got


# ---- the same in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "cache": _exact_cache, "attend": _exact_attend, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_norm(s):
    x, w = s["x"].cpu().numpy(), s["w"].cpu().numpy()
    # the sum is stored in 32 bits, and what follows is computed from what is stored
    h = x if s["res"] is None else (x.astype(np.float64) + s["res"].cpu().numpy()).astype(np.float32)
    total = None if s["res"] is None else x.astype(np.float64) + s["res"].cpu().numpy()
    hd = h.astype(np.float64)
    r = 1.0 / np.sqrt(np.mean(hd * hd, axis=1, keepdims=True) + EPS)
    if s["case"]["out"] != "q8":
        return {"sum": total, "y": hd * r * w.astype(np.float64)}
    # the operator's codes come from its 32-bit values: y rounded after each of its two products
    y = (h * r.astype(np.float32)) * w
    b = y.reshape(y.shape[0], -1, 32)
    amax = np.abs(b).max(-1, keepdims=True)
    q = np.clip(np.trunc(b * (np.float32(127.0) / amax) + np.copysign(np.float32(0.5), b)), -127, 127)
    return {"sum": total, "y": (q.astype(np.float64) * (amax / np.float32(127.0))).reshape(y.shape)}


def _exact_cache(s):
    """Page by page, in the order of the positions."""
    got = {}
    start, lens = s["start"].tolist(), s["len"].tolist()
    first = s["back_start"].tolist()
    table = s["table"].tolist()
    for name, codes, scale, new in (("k", s["k"], s["k_scale"], s["new_k"]),
                                    ("v", s["v"].transpose(2, 3), s["v_scale"], s["new_v"])):
        new = new.double()
        scale = scale.double().clone()
        out = torch.zeros(first[-1], new.shape[1], new.shape[2], dtype=torch.float64, device=new.device)
        for i, n in enumerate(lens):
            m = start[i + 1] - start[i]
            back = first[i + 1] - first[i]
            for page in range(min(n - m, n - back) // PAGE, (n - 1) // PAGE + 1):
                at = table[i][page]
                a, b = page * PAGE, min(n, page * PAGE + PAGE)
                lo = max(a, n - m)                                     # the first new token of the page
                value = codes[at, :, :b - a].double().transpose(0, 1)  # [tokens, heads, dim]
                if lo < b:
                    x = new[start[i] + lo - (n - m):start[i] + b - (n - m)]
                    need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((0, 2)) / 127.0)))
                    d = need if lo == a else torch.maximum(need, scale[at])
                    kept = torch.round(value[:lo - a] * (scale[at] / d)[:, None])
                    value = torch.cat([kept, torch.round(x / d[:, None])])
                    scale[at] = d
                value = value * scale[at][:, None]
                keep = max(a, n - back)
                if keep < b:
                    out[first[i] + keep - (n - back):first[i] + b - (n - back)] = value[keep - a:]
        got[name], got[name + "_scale"] = out, scale
    return got


def _exact_attend(s):
    case = s["case"]
    group = case["heads"] // case["kv_heads"]
    start, lens = s["start"].tolist(), s["len"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(lens):
        a, b = start[i], start[i + 1]
        pages = s["table"][i, :-(-n // PAGE)].long()
        for h in range(case["kv_heads"]):
            k = (s["k"][pages, h].double() * s["k_scale"][pages, h].double()[:, None, None]).reshape(-1, case["dim"])[:n]
            v = (s["v"][pages, h].double() * s["v_scale"][pages, h].double()[:, None, None]).transpose(1, 2)
            v = v.reshape(-1, case["dim"])[:n].contiguous()
            kt = k.t().contiguous()
            for c in range(a, b, 1024):
                e = min(b, c + 1024)
                pos = torch.arange(n - (b - c), n - (b - e), device=out.device)[:, None]
                j = torch.arange(n, device=out.device)[None]
                unseen = j > pos
                if case["window"]:
                    unseen = unseen | (j <= pos - case["window"])
                for f in range(h * group, (h + 1) * group):
                    t = torch.mm(s["q"][c:e, f].double().contiguous(), kt) / math.sqrt(case["dim"])
                    out[c:e, f] = torch.mm(torch.softmax(t.masked_fill(unseen, -math.inf), -1), v)
    return out


def _exact_logprobs(s):
    x = s["x"].double().cpu().numpy()
    ids, top = s["ids"].cpu().numpy(), s["case"]["top"]
    m = x.max(1, keepdims=True)
    lse = m + np.log(np.exp(x - m).sum(1, keepdims=True))
    lp = x - lse
    got = {"lp": np.take_along_axis(lp, ids.astype(np.int64), 1), "entropy": -(np.exp(lp) * lp).sum(1),
           "top_ids": None, "top_lp": None}
    if top:
        best = np.argsort(-x, axis=1, kind="stable")[:, :top]
        got["top_ids"], got["top_lp"] = best.astype(np.int32), np.take_along_axis(lp, best, 1)
    return got
