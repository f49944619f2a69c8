"""The 4-bit cache, the heads' rotation and the draw of a token in plain numpy
and 64 bits (tests of qmv_qk_rotate, qmv_kv4_* and qmv_sample)."""
import itertools
import math

import numpy as np

PAGE, BLOCK = 64, 32
LEVELS = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


# ---- rotation ---------------------------------------------------------------

def rotate(x, w, eps, pos, freq, neighbours, mscale):
    """(y, size): y in 64 bits; size: |a| + |b| of the pair a value comes from
    (|y| of a channel that stays), times mscale where turned."""
    y = x.astype(np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps))) * w.astype(np.float64)
    half = len(freq)
    rot = 2 * half
    angle = pos.astype(np.float64)[:, None, None] * freq.astype(np.float64)
    c, s = float(np.float32(mscale)) * np.cos(angle), float(np.float32(mscale)) * np.sin(angle)
    first = slice(0, rot, 2) if neighbours else slice(0, half)
    second = slice(1, rot, 2) if neighbours else slice(half, rot)
    out, size = y.copy(), np.abs(y)
    a, b = y[..., first], y[..., second]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = (np.abs(a) + np.abs(b)) * abs(mscale)
    return out, size


# ---- cache ------------------------------------------------------------------

def quantize(x):
    """(level indexes with sign as +-, exponents) of x [..., dim]: nearest of
    the levels, ties to the even index, by distances."""
    b = x.astype(np.float64).reshape(*x.shape[:-1], -1, BLOCK)
    e = np.full(b.shape[:-1], -125)
    amax = np.abs(b).max(-1)
    while np.any((amax > 7 * 2.0 ** e) & (e < 125)):
        e = np.where((amax > 7 * 2.0 ** e) & (e < 125), e + 1, e)
    a = np.abs(b) / (2.0 ** e)[..., None]
    dist = np.abs(a[..., None] - LEVELS)
    best = dist.min(-1, keepdims=True)
    near = dist == best                           # one level, or two neighbours
    low = near.argmax(-1)
    index = np.where((near.sum(-1) == 2) & (low % 2 == 1), low + 1, low)
    return index.reshape(x.shape), np.signbit(x), e


def values(index, neg, e):
    v = LEVELS[index].reshape(*index.shape[:-1], -1, BLOCK) * (2.0 ** e)[..., None].astype(np.float64)
    return np.where(neg, -1.0, 1.0) * v.reshape(index.shape)


class Cache4:
    """codes [pages, heads, 64, dim] and exponent bytes [pages, heads, 64, dim / 32] of keys and values."""

    def __init__(self, pages, heads, dim):
        self.pages, self.heads, self.dim = pages, heads, dim
        self.code = {n: np.zeros((pages, heads, PAGE, dim), dtype=np.uint8) for n in "kv"}
        self.byte = {n: np.full((pages, heads, PAGE, dim // BLOCK), 2, dtype=np.uint8) for n in "kv"}

    def place(self, table, pos):
        if pos < 0 or pos // PAGE >= len(table):
            return None
        p = int(table[pos // PAGE])
        return (p, pos % PAGE) if 0 <= p < self.pages else None

    def write(self, table, lens, start, k, v):
        for i in range(len(lens)):
            new = start[i + 1] - start[i]
            for t in range(new):
                at = self.place(table[i], int(lens[i]) - new + t)
                if at is None:
                    continue
                row = start[i] + t
                for h in range(self.heads):
                    fine = np.isfinite(k[row, h]).all() and np.isfinite(v[row, h]).all()
                    for n, x in (("k", k), ("v", v)):
                        if fine:
                            index, neg, e = quantize(x[row, h])
                            self.code[n][at[0], h, at[1]] = index + 8 * neg
                            self.byte[n][at[0], h, at[1]] = e + 127
                        else:
                            self.code[n][at[0], h, at[1]] = 0
                            self.byte[n][at[0], h, at[1]] = 255 if n == "k" else 2

    def rows(self, table, length, what):
        out = np.zeros((max(length, 0), self.heads, self.dim))
        there = np.zeros(max(length, 0), dtype=bool)
        for pos in range(length):
            at = self.place(table, pos)
            if at is not None:
                c = self.code[what][at[0], :, at[1]]
                out[pos] = values(c % 8, c >= 8, self.byte[what][at[0], :, at[1]].astype(np.int64) - 127)
                out[pos][(self.byte["k"][at[0], :, at[1]] == 255).any(-1)] = np.nan
                there[pos] = True
        return out, there

    def read(self, table, lens, start, what, rows):
        out = np.zeros((rows, self.heads, self.dim))
        for i in range(len(lens)):
            new = start[i + 1] - start[i]
            full, _ = self.rows(table[i], int(lens[i]), what)
            for t in range(new):
                pos = int(lens[i]) - new + t
                if pos >= 0:
                    out[start[i] + t] = full[pos]
        return out

    def arrays(self):
        """k, v, k_scale, v_scale as the header lays them out."""
        p, h, d = self.pages, self.heads, self.dim
        e = d // 16
        got = {}
        for n in "kv":
            got[n] = np.zeros((p, h, PAGE * d // 2), dtype=np.uint8)
            got[n + "s"] = np.zeros((p, h, PAGE * d // BLOCK), dtype=np.uint8)
        for t in range(PAGE):
            for c in range(0, d, 2):
                for n in "kv":
                    at = t * d // 2 + c // 2 if n == "k" else ((t // 4 * 16 + c // e) * 4 + t % 4) * (e // 2) + c % e // 2
                    got[n][..., at] = self.code[n][:, :, t, c] | self.code[n][:, :, t, c + 1] << 4
            for b in range(d // BLOCK):
                got["ks"][..., ((t % 16) * (d // BLOCK) + b) * 4 + t // 16] = self.byte["k"][:, :, t, b]
                got["vs"][..., ((t // 4 % 4 * (d // BLOCK) + b) * 4 + t // 16) * 4 + t % 4] = self.byte["v"][:, :, t, b]
        return got["k"], got["v"], got["ks"], got["vs"]


def attend(cache, table, lens, start, q, scale, window):
    """(out, sizes): outputs in 64 bits; mass: sum p |v|; smax: the largest |s|;
    qk: the largest |scale| sum |q| |k|; vmax: the largest |v|, of every row and head."""
    rows, heads, dim = q.shape
    g = heads // cache.heads
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    smax, qk, vmax = np.zeros((rows, heads, 1)), np.zeros((rows, heads, 1)), np.zeros((rows, heads, 1))
    for i in range(len(lens)):
        n, new = int(lens[i]), start[i + 1] - start[i]
        if new == 0:
            continue
        k, there = cache.rows(table[i], n, "k")
        v, _ = cache.rows(table[i], n, "v")
        for t in range(new):
            pos, row = n - new + t, start[i] + t
            lo = max(0, pos - window + 1) if window else 0
            sel = [j for j in range(lo, pos + 1) if there[j]] if pos >= 0 else []
            if not sel:
                continue
            for h in range(heads):
                kk, vv, qq = k[sel, h // g], v[sel, h // g], q[row, h].astype(np.float64)
                with np.errstate(all="ignore"):
                    s = scale * (kk @ qq)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[row, h], mass[row, h] = p @ vv, p @ np.abs(vv)
                    smax[row, h] = np.abs(s).max()
                    qk[row, h] = abs(scale) * (np.abs(kk) @ np.abs(qq)).max()
                    vmax[row, h] = np.abs(vv).max()
    return out, {"mass": mass, "smax": smax, "qk": qk, "vmax": vmax}


def attend_bound(b, dim, longest, dtype, many=False):
    """How far an output may be off.

    A score is a sum of at most 3 dim products (three parts of a float32 query
    value), each addition rounding to 2^-24 of at most sum |q| |k|; its
    multiple and exponent round at most eight times relative to the largest
    score, the exponential to 2^-21.  That error d changes every p by at most a
    factor e^d, the quotient by e^2d.  Sums: of at most 3 parts of each token
    (and pieces: fifty more), each addition rounding to 2^-24 of the sum of
    magnitudes.  With bfloat16 the probabilities may be rounded to 11 bits,
    2^-11 of each product and of each term of the sum: 2^-10; the output rounds
    by half a step, 2^-8 (added by the caller).  In the kernel for many they are
    float16 numbers of which the largest is at least 4, so that the least are off
    by up to 2^-25, 2^-27 of the sum: that times |v|max, for each token."""
    d = 3 * dim * 2.0 ** -24 * b["qk"] + 8 * 2.0 ** -24 * b["smax"] + 2.0 ** -21
    rel = np.expm1(2 * d) + (3 * longest + 50) * 2.0 ** -23
    return b["mass"] * (rel + (2.0 ** -10 if dtype == "bf16" else 0.0)) + (longest * 2.0 ** -27 * b["vmax"] if many else 0.0)


# ---- the draw ---------------------------------------------------------------

def sample(x, u, t, k, p, m):
    """(id, lp) of one row in 64 bits; None for a row that cannot be drawn from."""
    x = x.astype(np.float64) + 0.0
    if not np.all(x < np.inf) or np.isnan(x).any() or x.max() == -np.inf or not (0 <= t < np.inf):
        return None
    order = np.argsort(-x, kind="stable")
    if t == 0:
        return int(order[0]), 0.0
    w = np.exp((x - x.max()) / t)
    n = int(k) if 0 < k < len(x) else len(x)
    if p < 1:
        ws = w[order[:n]]
        before = np.cumsum(ws) - ws
        n = max(1, int(np.count_nonzero(before < p * math.fsum(ws))))
    if m > 0:
        n = max(1, int(np.count_nonzero(w[order[:n]] >= min(m, 1.0))))
    kept = np.sort(order[:n])
    total = math.fsum(w[kept])
    past = np.nonzero(np.cumsum(w[kept]) > min(max(u, 0.0), 1 - 1e-12) * total)[0]
    at = kept[past[0] if len(past) else len(kept) - 1]
    with np.errstate(divide="ignore"):
        return int(at), float(np.log(w[at] / total))


# A weight is right to 2^-22 of itself (the exponent's two parts and the
# exponential) and half a unit of 2^-39 of the largest; a sum to the same, so
# whatever lies further than NEAR of itself from a border is on its side of it.
NEAR = 2.0 ** -20


def sample_answers(x, u, t, k, p, m):
    """What may be answered for a row: the answers with every border moved by
    no more than NEAR."""
    if sample(x, u, t, k, p, m) is None:
        return None
    got = set()
    for du, dp, dm in itertools.product((-1, 0, 1), repeat=3):
        got.add(sample(x, u + du * NEAR, t, k, p if p >= 1 else p * (1 + dp * NEAR), m * (1 + dm * NEAR)))
    return got


def sample_ok(answers, at, lp):
    if answers is None:
        return at == -1 and np.isnan(lp)
    # lp = ln w - ln total: 2^-21 both together, and its own rounding
    return any(at == i and abs(lp - v) <= 2.0 ** -20 + 2.0 ** -23 * abs(v) for i, v in answers)
