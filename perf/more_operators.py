"""More operators of a decoding step around a quantized model's products, as
they are measured: the norm of every query and key head with the position's
rotation, a key/value cache in 4 bits (written and read back), attention over
that cache, and the next token drawn from the LM head's logits.

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
PAGE = 64          # tokens of a cache page
BLOCK = 32         # channels of one token and head that share a scale
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # -- rotation: queries and keys as slices of one array of all three projections
        # one decode token, 32 heads on 8 KV heads of 128 (a layer of dim 4096): latency
        {"name": "rotate_1x32_f32", "op": "rotate", "rows": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "norm": True, "dtype": "f32", "out": "f32"},
        # pieces of prompts, heads of 256 of which a quarter is rotated, in the neighbouring order
        {"name": "rotate_1500x16_part_bf16", "op": "rotate", "rows": 1500, "heads": 16, "kv_heads": 4, "dim": 256,
         "rot": 64, "pairs": "neighbours", "norm": True, "dtype": "bf16", "out": "bf16"},
        # a long prompt: float32 products become bfloat16 queries and keys
        {"name": "rotate_8191x32_bf16", "op": "rotate", "rows": 8191, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "pairs": "halves", "norm": True, "dtype": "f32", "out": "bf16"},
        # -- cache: 8 KV heads of 128
        # one new token for each of 64 sequences, float32 from the vector product; the last 100 tokens read back
        {"name": "cache4_append_64x1_f32", "op": "cache", "seqs": 64, "len": 2000, "new": 1, "back": 100,
         "kv_heads": 8, "dim": 128, "dtype": "f32"},
        # prompts of up to 4096 tokens written and read back whole
        {"name": "cache4_prompt_4x4096_bf16", "op": "cache", "seqs": 4, "len": 4096, "new": 4096, "back": 4096,
         "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # -- attention
        # the smallest call: one sequence of 100 tokens, one new token
        {"name": "attend4_1x100_f32", "op": "attend", "seqs": 1, "len": 100, "new": 1, "heads": 8, "kv_heads": 2,
         "dim": 64, "dtype": "f32", "window": 0},
        # an ordinary decode step: 32 sequences of 1000 to 4000 tokens, 32 heads on 8 KV heads of 128
        {"name": "attend4_32x4000_f32", "op": "attend", "seqs": 32, "len": 4000, "new": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "f32", "window": 0},
        # decode on a few very long contexts
        {"name": "attend4_2x131072_bf16", "op": "attend", "seqs": 2, "len": 131072, "new": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "window": 0},
        # a whole prompt of 8192 tokens
        {"name": "attend4_prompt_1x8192_bf16", "op": "attend", "seqs": 1, "len": 8192, "new": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "window": 0},
        # pieces of up to 500 tokens of three prompts under a sliding window, heads of 256
        {"name": "attend4_piece_3x500_window", "op": "attend", "seqs": 3, "len": 6000, "new": 500, "heads": 16,
         "kv_heads": 4, "dim": 256, "dtype": "bf16", "window": 1024},
        # -- the next token, from the 248320-row LM head's logits
        # one sequence, the usual filters
        {"name": "sample_1x248320", "op": "sample", "rows": 1, "vocab": 248320, "how": "usual"},
        # a decode batch of 64 whose requests ask for different filters
        {"name": "sample_64x248320", "op": "sample", "rows": 64, "vocab": 248320, "how": "mixed"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotate", "cache", "attend", "attend", "sample"))
    if op == "sample":
        vocab = _log(rng, 500, 262144)
        return {"op": op, "rows": min(_log(rng, 1, 2048), (63 * 248320) // vocab), "vocab": vocab,
                "how": rng.choice(("greedy", "plain", "usual", "top_k", "top_p", "min_p", "mixed"))}
    kv_heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 128, 256))
    group = rng.choice((1, 2, 4, 5, 8))
    dtype = rng.choice(("f32", "bf16"))
    per = kv_heads * dim                      # values a token keeps
    if op == "rotate":
        rows = min(_log(rng, 1, 8191), (8000 * 40 * 128) // (per * (group + 1)))
        return {"op": op, "rows": rows, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice((dim, dim, dim // 2, dim // 4)), "pairs": rng.choice(("halves", "halves", "neighbours")),
                "norm": rng.random() < 0.7, "dtype": dtype, "out": rng.choice(("f32", "bf16"))}
    if op == "cache":
        size = 4.6 if dtype == "f32" else 2.6
        length = min(_log(rng, 1, 16000), int(100_000_000 / (4 * per * size)))
        seqs = max(1, min(_log(rng, 1, 128), int(100_000_000 / (4 * per * size * length))))
        new = rng.choice((1, _log(rng, 1, length), length))
        return {"op": op, "seqs": seqs, "len": length, "new": new, "back": rng.choice((new, length)),
                "kv_heads": kv_heads, "dim": dim, "dtype": dtype}
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
    if op == "rotate":
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        size = {"f32": 4, "bf16": 2}
        weights = 8 * case["dim"] if case["norm"] else 0
        return {"bytes": n * (size[case["dtype"]] + size[case["out"]]) + weights + 4 * case["rows"] + 2 * case["rot"],
                "flops": n * (4 if case["norm"] else 0) + 3 * n * case["rot"] // case["dim"]}
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": 4 * n + 28 * case["rows"], "flops": 5 * n}
    lens, news = _lengths(case)
    size = 4 if case["dtype"] == "f32" else 2
    per = case["kv_heads"] * case["dim"]
    stored = per // 2 + per // BLOCK          # bytes of a token's keys, and of its values
    if op == "cache":
        new, back = sum(news), sum(min(case["back"], n) for n in lens)
        return {"bytes": 2 * (new + back) * (size * per + stored), "flops": 2 * per * (4 * new + back)}
    pairs, keys = (sum(v) for v in zip(*(_pairs(n, m, case["window"]) for n, m in zip(lens, news))))
    q = sum(news) * case["heads"] * case["dim"]
    return {"bytes": 2 * stored * keys + 2 * size * q, "flops": 4 * case["heads"] * case["dim"] * pairs}


# ---- the 4-bit format --------------------------------------------------------
# A block of 32 channels of one token and head has a scale 2^(byte - 127) and
# 32 codes: a sign above an index into 0, .5, 1, 1.5, 2, 3, 4, 6.

def _scale(byte):
    """2^(byte - 127) of bytes from 2 to 252."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _codes(x):
    """(codes, scale bytes) of x [..., dim], float32: the least scale d with the block's largest magnitude <= 7 d, and
    the nearest codes, halves to the even one."""
    b = x.view(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 3, e - 2).clamp(-125, 125)
    byte = torch.where(amax > 0, e + 127, 2).to(torch.uint8)
    y = b / _scale(byte).unsqueeze(-1)
    a = y.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(y).to(torch.uint8) * 8
    return code.view(x.shape), byte


def _table():
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=DEVICE)


def _packed(code):
    """Two codes to a byte, the first in its low half."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(packed, byte):
    """packed [..., dim / 2], byte [..., dim / 32] as what they stand for."""
    c = torch.stack([packed & 15, packed >> 4], -1).view(*packed.shape[:-1], -1, BLOCK)
    return (_table()[c.int()] * _scale(byte).unsqueeze(-1)).view(*packed.shape[:-1], -1)


# The arrays of a page and head: where token t = 16 a + 4 b + i keeps its
# bytes.  Keys lie token by token; their scales [16 tokens t % 16][blocks][4 a].
# Values lie in groups of four tokens: [16 groups 4 a + b][16 channel
# sixteenths][4 i][dim / 32 bytes], their scales [4 b][blocks][4 a][4 i].

def _k_scales(s):
    p, h = s["k_scale"].shape[:2]
    return s["k_scale"].view(p, h, 16, -1, 4)


def _v_codes(s):
    p, h = s["v"].shape[:2]
    return s["v"].view(p, h, 16, 16, 4, -1)


def _v_scales(s):
    p, h = s["v_scale"].shape[:2]
    return s["v_scale"].view(p, h, 4, -1, 4, 4)


def _tokens(s, what, page, t):
    """Packed codes [n, heads, dim / 2] and scale bytes [n, heads, dim / 32] of tokens t of pages `page`."""
    if what == "k":
        return s["k"][page, :, t], _k_scales(s)[page, :, t % 16, :, t // 16]
    return _v_codes(s)[page, :, t // 4, :, t % 4].flatten(2), _v_scales(s)[page, :, t % 16 // 4, :, t // 16, t % 4]


def _put(s, what, page, t, packed, byte):
    if what == "k":
        s["k"][page, :, t] = packed
        _k_scales(s)[page, :, t % 16, :, t // 16] = byte
    else:
        _v_codes(s)[page, :, t // 4, :, t % 4] = packed.unflatten(2, (16, -1))
        _v_scales(s)[page, :, t % 16 // 4, :, t // 16, t % 4] = byte


def _whole(s, what, pages):
    """Values of whole pages [..., heads, 64, dim] for page ids [...]."""
    if what == "k":
        codes = s["k"][pages]
        byte = _k_scales(s)[pages].movedim(-1, -3).flatten(-3, -2)
    else:
        codes = _v_codes(s)[pages].transpose(-3, -2).flatten(-2).flatten(-3, -2)
        byte = _v_scales(s)[pages].movedim(-3, -1).movedim(-4, -3).flatten(-4, -2)
    return _values(codes, byte)


# ---- inputs ----------------------------------------------------------------

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
    s = {"k": torch.empty(pages, kvh, PAGE, dim // 2, dtype=torch.uint8, device=DEVICE),
         "v": torch.empty(pages, kvh, PAGE, dim // 2, dtype=torch.uint8, device=DEVICE),
         "k_scale": torch.empty(pages, kvh, PAGE, dim // BLOCK, dtype=torch.uint8, device=DEVICE),
         "v_scale": torch.empty(pages, kvh, PAGE, dim // BLOCK, dtype=torch.uint8, device=DEVICE)}
    step = max(1, (1 << 25) // (kvh * PAGE * dim))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        code, byte = _codes(torch.randn(b - a, kvh, PAGE, dim, generator=g, device=DEVICE) * width)
        s["k"][a:b] = _packed(code)
        _k_scales(s)[a:b] = byte.unflatten(2, (4, 16)).movedim(2, -1)
        code, byte = _codes(torch.randn(b - a, kvh, PAGE, dim, generator=g, device=DEVICE))
        _v_codes(s)[a:b] = _packed(code).unflatten(3, (16, -1)).unflatten(2, (16, 4)).transpose(3, 4)
        _v_scales(s)[a:b] = byte.unflatten(2, (4, 4, 4)).permute(0, 1, 3, 5, 2, 4)
    s.update({"table": table.to(DEVICE), "width": width,
              "len": torch.tensor(lens, dtype=torch.int32, device=DEVICE),
              "start": torch.tensor(start, dtype=torch.int32, device=DEVICE),
              "max_len": max(lens), "max_new": max(news), "rows": start[-1]})
    s.update(_places(lens, news, table, "row_"))
    return s


def _places(lens, news, table, what):
    """Sequence, position and page of the last `news` tokens of every sequence, one after the other."""
    seq = torch.tensor([i for i, m in enumerate(news) for _ in range(m)], dtype=torch.int64)
    pos = torch.tensor([p for n, m in zip(lens, news) for p in range(n - m, n)], dtype=torch.int64)
    page = table[seq, pos // PAGE].to(torch.int64)
    return {what + "seq": seq.to(DEVICE), what + "pos": pos.to(DEVICE), what + "page": page.to(DEVICE)}


def _sample_params(case, g):
    """Temperature, top_k, top_p, min_p and random number of every row."""
    n, how = case["rows"], case["how"]

    def pick(*values):
        return torch.tensor(values, device=DEVICE)[torch.randint(0, len(values), (n,), generator=g, device=DEVICE)]

    def same(value):
        return torch.full((n,), value, device=DEVICE)

    t, k, p, m = same(1.0), same(0), same(1.0), same(0.0)
    if how == "greedy":
        t = same(0.0)
    elif how == "usual":
        t, k, p, m = same(0.8), same(40), same(0.95), same(0.05)
    elif how == "top_k":
        t, k = pick(0.7, 1.0, 1.3), pick(1, 2, 20, 50, 200, 1000)
    elif how == "top_p":
        t, p = pick(0.6, 0.8, 1.0), pick(0.5, 0.8, 0.9, 0.95, 0.99)
    elif how == "min_p":
        t, m = pick(0.7, 1.0, 1.5), pick(0.02, 0.05, 0.1)
    elif how == "mixed":
        t, k = pick(0.0, 0.6, 0.7, 0.8, 1.0, 1.0), pick(0, 0, 20, 40, 50, 100)
        p, m = pick(1.0, 0.8, 0.9, 0.95, 0.95), pick(0.0, 0.0, 0.05, 0.1)
    return {"temperature": t, "top_k": k.to(torch.int32), "top_p": p, "min_p": m,
            "u": torch.rand(n, generator=g, device=DEVICE)}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    op = case["op"]
    if op == "rotate":
        n, h, kvh, dim = case["rows"], case["heads"], case["kv_heads"], case["dim"]
        both = (2.0 * normal(n, (h + 2 * kvh) * dim)).to(DTYPES[case["dtype"]])   # queries, keys, values
        first = int(torch.randint(0, 100000, (1,), generator=g, device=DEVICE))
        rot = case["rot"]
        return {"case": case, "q": both[:, :h * dim].unflatten(1, (h, dim)),
                "k": both[:, h * dim:(h + kvh) * dim].unflatten(1, (kvh, dim)),
                "q_w": 1.0 + 0.1 * normal(dim) if case["norm"] else None,
                "k_w": 1.0 + 0.1 * normal(dim) if case["norm"] else None,
                "pos": torch.arange(first, first + n, dtype=torch.int32, device=DEVICE),
                "freq": 1e6 ** (-2.0 * torch.arange(rot // 2, device=DEVICE) / rot),
                "q_out": torch.empty(n, h, dim, dtype=DTYPES[case["out"]], device=DEVICE),
                "k_out": torch.empty(n, kvh, dim, dtype=DTYPES[case["out"]], device=DEVICE)}
    if op == "sample":
        n, v = case["rows"], case["vocab"]
        x = 2.2 * normal(n, v)
        # some dozens of likely tokens a row, of more weight in some rows than in others, and a few ties
        m = min(60, v // 8)
        likely = torch.randint(0, v // m, (n, m), generator=g, device=DEVICE) + v // m * torch.arange(m, device=DEVICE)
        level = 12.0 + 5.0 * torch.rand(n, 1, generator=g, device=DEVICE)
        x.scatter_(1, likely, level + 2.5 * normal(n, m))
        s = {"case": case, "x": torch.round(x * 4096.0) / 4096.0, "ids": torch.empty(n, dtype=torch.int32, device=DEVICE),
             "lp": torch.empty(n, device=DEVICE), **_sample_params(case, g)}
        if own:
            from block_quant_weight_amd import serve
            s["workspace"] = serve.workspace(serve.qmv_sample_workspace(n, v), DEVICE)
        return s
    s = _cache_state(case, g)
    s["case"] = case
    dtype = DTYPES[case["dtype"]]
    kvh, dim = case["kv_heads"], case["dim"]
    if op == "cache":
        s["new_k"] = (normal(s["rows"], kvh, dim) * s["width"]).to(dtype)
        s["new_v"] = normal(s["rows"], kvh, dim).to(dtype)
        lens, news = _lengths(case)
        backs = [min(case["back"], n) for n in lens]
        first = [0]
        for m in backs:
            first.append(first[-1] + m)
        s.update(_places(lens, backs, s["table"].cpu(), "back_"))
        s["back_start"] = torch.tensor(first, dtype=torch.int32, device=DEVICE)
        s["out_k"] = torch.empty(first[-1], kvh, dim, dtype=dtype, device=DEVICE)
        s["out_v"] = torch.empty(first[-1], kvh, dim, dtype=dtype, device=DEVICE)
    else:
        s["q"] = (2.0 * normal(s["rows"], case["heads"], dim)).to(dtype)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(dim)
    if own:      # the handles that a program keeps: of the cache, and of a step's sequences for all its layers
        from block_quant_weight_amd import serve
        s["cache"] = serve.Kv4Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["seqs"] = serve.KvSeqs(s["table"], s["len"], s["start"], max_new=s["max_new"], max_len=s["max_len"])
        if op == "cache":
            s["back_seqs"] = serve.KvSeqs(s["table"], s["len"], s["back_start"],
                                          max_new=min(case["back"], s["max_len"]), max_len=s["max_len"])
        else:
            s["workspace"] = serve.workspace(serve.qmv_kv4_attend_workspace(
                s["cache"], s["seqs"], s["q"], window=case["window"]), DEVICE)
    return s


# ---- one pass --------------------------------------------------------------

def run(s):
    if own:
        return {"rotate": _own_rotate, "cache": _own_cache, "attend": _own_attend, "sample": _own_sample}[s["case"]["op"]](s)
    return {"rotate": _rotate, "cache": _cache, "attend": _attend, "sample": _sample}[s["case"]["op"]](s)


def _own_rotate(s):
    from block_quant_weight_amd import serve
    serve.qmv_qk_rotate(s["q"], s["k"], s["pos"], s["freq"], s["q_out"], s["k_out"], q_w=s["q_w"], k_w=s["k_w"],
                        eps=EPS, neighbours=s["case"]["pairs"] == "neighbours")
    return {"q": s["q_out"], "k": s["k_out"]}


def _rotated(s, x, w):
    case = s["case"]
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    rot = case["rot"]
    angle = s["pos"].double()[:, None, None] * s["freq"].double()      # 64 bits: far positions
    c, n = angle.cos().float(), angle.sin().float()
    if case["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1).to(DTYPES[case["out"]])


def _rotate(s):
    return {"q": _rotated(s, s["q"], s["q_w"]), "k": _rotated(s, s["k"], s["k_w"])}


def _own_cache(s):
    from block_quant_weight_amd import serve
    serve.qmv_kv4_write(s["cache"], s["seqs"], s["new_k"], s["new_v"])
    serve.qmv_kv4_read(s["cache"], s["back_seqs"], s["out_k"], s["out_v"])
    return {"k": s["out_k"], "v": s["out_v"]}


def _cache(s):
    page, t = s["row_page"], s["row_pos"] % PAGE
    code, byte = _codes(s["new_k"].float())
    _put(s, "k", page, t, _packed(code), byte)
    code, byte = _codes(s["new_v"].float())
    _put(s, "v", page, t, _packed(code), byte)
    page, t = s["back_page"], s["back_pos"] % PAGE
    dtype = s["new_k"].dtype
    return {"k": _values(*_tokens(s, "k", page, t)).to(dtype), "v": _values(*_tokens(s, "v", page, t)).to(dtype)}


def _own_attend(s):
    from block_quant_weight_amd import serve
    serve.qmv_kv4_attend(s["cache"], s["seqs"], s["q"], s["out"], scale=s["scale"], window=s["case"]["window"],
                         workspace=s["workspace"])
    return s["out"]


def _attend(s):
    case = s["case"]
    kvh, dim, group = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    n, new = case["seqs"], s["max_new"]
    pages = s["table"].long().clamp(min=0)                  # [n, pages]
    k = _whole(s, "k", pages).transpose(2, 3).reshape(n, -1, kvh, dim)
    v = _whole(s, "v", pages).transpose(2, 3).reshape(n, -1, kvh, dim)
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


def _own_sample(s):
    from block_quant_weight_amd import serve
    serve.qmv_sample(s["x"], s["u"], s["ids"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                     min_p=s["min_p"], lp=s["lp"], workspace=s["workspace"])
    return {"ids": s["ids"], "lp": s["lp"]}


def _sample(s):
    x, v = s["x"].double(), s["case"]["vocab"]              # 64 bits: sums next to borders
    best, order = x.sort(dim=-1, descending=True, stable=True)  # the larger first, then the lower index
    t = s["temperature"].double().unsqueeze(1)
    greedy = t == 0
    rank = torch.arange(v, device=x.device)
    w = torch.exp((best - best[:, :1]) / torch.where(greedy, 1.0, t))
    k = torch.where(greedy[:, 0], 1, torch.where(s["top_k"] > 0, s["top_k"], v)).unsqueeze(1)
    w = torch.where(rank < k, w, 0.0)
    before = w.cumsum(-1) - w
    p = s["top_p"].double().unsqueeze(1)
    w = torch.where((rank == 0) | (p >= 1) | (before < p * w.sum(-1, keepdim=True)), w, 0.0)
    w = torch.where(w >= s["min_p"].double().unsqueeze(1), w, 0.0)
    kept = torch.zeros_like(x).scatter_(1, order, w)        # by index again
    total = kept.sum(-1, keepdim=True)
    ids = (kept.cumsum(-1) > s["u"].double().unsqueeze(1) * total).int().argmax(-1, keepdim=True)
    lp = (kept.gather(1, ids) / total).log()
    return {"ids": ids[:, 0].to(torch.int32), "lp": lp[:, 0].float()}


# ---- the same in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "cache": _exact_cache, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s)


def _exact_rotate(s):
    """Each pair as a complex number, times e^(i angle)."""
    case, got = s["case"], {}
    rot = case["rot"]
    turn = np.exp(1j * np.outer(s["pos"].cpu().numpy().astype(np.float64), s["freq"].cpu().numpy().astype(np.float64)))
    for name, x, w in (("q", s["q"], s["q_w"]), ("k", s["k"], s["k_w"])):
        x = x.double().cpu().numpy()
        if case["norm"]:
            x = x / np.sqrt(np.einsum("rhd,rhd->rh", x, x)[..., None] / case["dim"] + EPS) * w.double().cpu().numpy()
        y = x.copy()
        first = slice(0, rot // 2) if case["pairs"] == "halves" else slice(0, rot, 2)
        second = slice(rot // 2, rot) if case["pairs"] == "halves" else slice(1, rot, 2)
        z = (x[..., first] + 1j * x[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        got[name] = y
    return got


def _stored(x):
    """What is stored of x [..., dim], in 64 bits."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    d = torch.exp2(torch.ceil(torch.log2(amax / 7.0)).clamp(-125, 125))
    a = (b / d).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.where(amax > 0, torch.copysign(a, b) * d, torch.zeros_like(b)).flatten(-2)


def _token_values(s, what, page, t):
    """Values of token t of page `page` [heads, dim], code by code as the format says."""
    dim = s["case"]["dim"]
    if what == "k":
        codes = s["k"][page, :, t]
        byte = s["k_scale"][page].reshape(-1, 16, dim // BLOCK, 4)[:, t % 16, :, t // 16]
    else:
        codes = s["v"][page].reshape(-1, 16, 16, 4, dim // 32)[:, t // 4, :, t % 4].reshape(-1, dim // 2)
        byte = s["v_scale"][page].reshape(-1, 4, dim // BLOCK, 4, 4)[:, t // 4 % 4, :, t // 16, t % 4]
    c = torch.stack([codes % 16, codes // 16], -1).reshape(-1, dim // BLOCK, BLOCK).double()
    a = c % 8
    # an exponent of two bits above one bit of fraction, the least exponent without the leading one
    e = torch.floor(a / 2)
    a = torch.where(e > 0, (1 + (a % 2) / 2) * torch.exp2(e - 1), (a % 2) / 2)
    d = torch.exp2(byte.double() - 127).unsqueeze(-1)
    return (torch.where(c >= 8, -a, a) * d).reshape(-1, dim)


def _exact_cache(s):
    """The new tokens from what was written, the others token by token from the arrays."""
    lens, start, first = s["len"].tolist(), s["start"].tolist(), s["back_start"].tolist()
    table, got = s["table"].tolist(), {}
    old = sum(max(0, (first[i + 1] - first[i]) - (start[i + 1] - start[i])) for i in range(len(lens)))
    if old > 40000:
        return None
    for name, new in (("k", s["new_k"]), ("v", s["new_v"])):
        stored, rows = _stored(new), []
        for i, n in enumerate(lens):
            m, back = start[i + 1] - start[i], first[i + 1] - first[i]
            rows += [_token_values(s, name, table[i][p // PAGE], p % PAGE).unsqueeze(0) for p in range(n - back, n - m)]
            rows.append(stored[start[i + 1] - min(m, back):start[i + 1]])
        got[name] = torch.cat(rows)
    return got


def _exact_attend(s):
    case = s["case"]
    group, dim = case["heads"] // case["kv_heads"], case["dim"]
    start, lens = s["start"].tolist(), s["len"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    level = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=s["q"].device) / 2
    level = torch.cat([level, -level])

    def values(codes, byte):
        c = torch.stack([codes % 16, codes // 16], -1).reshape(-1, dim // BLOCK, BLOCK).long()
        return (level[c] * torch.exp2(byte.double() - 127).unsqueeze(-1)).reshape(-1, dim)

    for i, n in enumerate(lens):
        a, b = start[i], start[i + 1]
        pages = s["table"][i, :-(-n // PAGE)].long()
        for h in range(case["kv_heads"]):
            byte = s["k_scale"][pages, h].reshape(-1, 16, dim // BLOCK, 4).permute(0, 3, 1, 2).reshape(-1, dim // BLOCK)
            k = values(s["k"][pages, h].reshape(-1, dim // 2), byte)[:n]
            byte = s["v_scale"][pages, h].reshape(-1, 4, dim // BLOCK, 4, 4).permute(0, 3, 1, 4, 2).reshape(-1, dim // BLOCK)
            codes = s["v"][pages, h].reshape(-1, 16, 16, 4, dim // 32).transpose(2, 3).reshape(-1, dim // 2)
            v = values(codes, byte)[:n].contiguous()
            kt = k.t().contiguous()
            for c in range(a, b, 1024):
                e = min(b, c + 1024)
                pos = torch.arange(n - (b - c), n - (b - e), device=out.device)[:, None]
                j = torch.arange(n, device=out.device)[None]
                unseen = j > pos
                if case["window"]:
                    unseen = unseen | (j <= pos - case["window"])
                for f in range(h * group, (h + 1) * group):
                    t = torch.mm(s["q"][c:e, f].double().contiguous(), kt) / math.sqrt(dim)
                    out[c:e, f] = torch.mm(torch.softmax(t.masked_fill(unseen, -math.inf), -1), v)
    return out


def _exact_sample(s):
    """Row by row: how many of the best tokens stay, then the draw over these in the order of their indexes."""
    x = s["x"].cpu().numpy().astype(np.float64)
    t, k, p, m, u = (s[n].cpu().numpy().astype(np.float64) for n in ("temperature", "top_k", "top_p", "min_p", "u"))
    ids, lp = np.empty(len(x), np.int32), np.empty(len(x))
    for i, row in enumerate(x):
        order = np.argsort(-row, kind="stable")
        if t[i] == 0:
            ids[i], lp[i] = order[0], 0.0
            continue
        n = int(k[i]) if 0 < k[i] < len(row) else len(row)
        q = np.exp((row[order[:n]] - row[order[0]]) / t[i])
        if p[i] < 1:
            n = min(n, max(1, 1 + int(np.searchsorted(np.cumsum(q), p[i] * math.fsum(q), side="left"))))
        n = min(n, int(np.count_nonzero(q >= m[i])))
        chosen = np.sort(order[:n])
        q = np.exp((row[chosen] - row[order[0]]) / t[i])
        total = math.fsum(q)
        at = int(np.argmax(np.cumsum(q) > u[i] * total))
        ids[i], lp[i] = chosen[at], (row[chosen[at]] - row[order[0]]) / t[i] - math.log(total)
    return {"ids": ids, "lp": lp}
