"""The calls of qmv_serve.h in plain numpy and 64 bits, and seeded inputs."""
import numpy as np

PAGE = 64


def bf16(x):
    """x rounded to bfloat16 (halves to even), as float32."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


# ---- norm -------------------------------------------------------------------

def norm(x, res, w, eps):
    """(h, y): h as the operator stores it (float32), y in 64 bits from it."""
    h = x if res is None else x + res           # float32, one rounding
    hd = h.astype(np.float64)
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((hd * hd).mean(1, keepdims=True) + float(np.float32(eps)))
        return h, hd * r * w.astype(np.float64)


# ---- cache ------------------------------------------------------------------

def scale_for(amax):
    """Least power of two d from 2^-126 with amax <= 127 d, at most 2^121."""
    if amax == 0:
        return 0.0
    if not np.isfinite(amax):
        return np.nan
    d = 2.0 ** -126
    while amax > 127 * d and d < 2.0 ** 121:
        d *= 2
    return d


class Cache:
    """k, v: codes [pages, heads, 64, dim]; k_scale, v_scale [pages, heads]."""

    def __init__(self, pages, heads, dim):
        self.pages, self.heads, self.dim = pages, heads, dim
        self.k = np.zeros((pages, heads, PAGE, dim))
        self.v = np.zeros((pages, heads, PAGE, dim))
        self.k_scale = np.zeros((pages, heads))
        self.v_scale = np.zeros((pages, heads))

    def place(self, table, pos):
        """Page id and place of a position, or None."""
        if pos < 0 or pos // PAGE >= len(table):
            return None
        p = int(table[pos // PAGE])
        return (p, pos % PAGE) if 0 <= p < self.pages else None

    def write(self, table, lens, start, k, v):
        for i in range(len(lens)):
            new = start[i + 1] - start[i]
            by_page = {}
            for t in range(new):
                pos = int(lens[i]) - new + t
                at = self.place(table[i], pos)
                if at is not None:
                    by_page.setdefault(at[0], []).append((at[1], start[i] + t))
            for page, tokens in by_page.items():
                for codes, scales, x in ((self.k, self.k_scale, k), (self.v, self.v_scale, v)):
                    for h in range(self.heads):
                        vals = np.stack([x[row, h] for _, row in tokens]).astype(np.float64)
                        need = scale_for(np.abs(vals).max()) if np.isfinite(vals).all() else np.nan
                        first = tokens[0][0]
                        old = 0.0 if first == 0 else scales[page, h]
                        d = need if np.isnan(need) or first == 0 else (old if np.isnan(old) else max(old, need))
                        if d > 0:
                            if first > 0 and old < d:
                                codes[page, h, :first] = np.rint(codes[page, h, :first] * (old / d))
                            q = np.clip(np.rint(vals / d), -127, 127)
                        else:
                            q = np.zeros_like(vals)
                        scales[page, h] = d
                        for (off, _), c in zip(tokens, q):
                            codes[page, h, off] = c

    def rows(self, table, length, what):
        """Values of positions 0 .. length - 1 as [length, heads, dim], and which of them have a place."""
        codes, scales = (self.k, self.k_scale) if what == "k" else (self.v, self.v_scale)
        out = np.zeros((max(length, 0), self.heads, self.dim))
        there = np.zeros(max(length, 0), dtype=bool)
        for pos in range(length):
            at = self.place(table, pos)
            if at is not None:
                out[pos] = codes[at[0], :, at[1]] * scales[at[0]][:, None]
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


def attend(cache, table, lens, start, q, scale, window):
    """(out, bound_a, bound_b): outputs [rows, heads, dim] in 64 bits (rows of
    no sequence are 0); per output sum p |v|, and the largest |v| that the
    row sees; plus per (row, head) the largest score's and key's sizes for
    the tolerance: dict."""
    rows, heads, dim = q.shape
    g = heads // cache.heads
    out = np.zeros(q.shape)
    mass, vmax = np.zeros(q.shape), np.zeros((rows, heads, 1))
    smax, ksum = np.zeros((rows, heads, 1)), np.zeros((rows, heads, 1))
    for i in range(len(lens)):
        n, new = int(lens[i]), start[i + 1] - start[i]
        k, there = cache.rows(table[i], n, "k")
        v, _ = cache.rows(table[i], n, "v")
        for t in range(new):
            pos = n - new + t
            row = start[i] + t
            lo = max(0, pos - window + 1) if window else 0
            sel = [j for j in range(lo, pos + 1) if there[j]] if pos >= 0 else []
            if not sel:
                continue
            for h in range(heads):
                kk, vv = k[sel, h // g], v[sel, h // g]
                with np.errstate(all="ignore"):
                    s = scale * (kk @ q[row, h].astype(np.float64))
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[row, h] = p @ vv
                    mass[row, h] = p @ np.abs(vv)
                    vmax[row, h] = np.abs(vv).max()
                    smax[row, h] = np.abs(s).max()
                    ksum[row, h] = np.abs(kk).sum(1).max()
    return out, {"mass": mass, "vmax": vmax, "smax": smax, "ksum": ksum}


def attend_bound(b, q, scale, longest, dtype):
    """How far an output may be off.

    A score: the query's digits are off by half of |q|max / (127 2^16), below
    2^-22 |q|max a value (bfloat16 queries of many columns are exact); the
    score's products and its exponent round at most eight times relative to
    the largest score.  That error d
    changes every p by at most a factor e^d, the quotient by e^2d.  Sums of
    pages: two roundings a page and about twenty others, each 2^-24 of the
    sum.  Probabilities in digits: half of 1 / (127 2^16) < 2^-23.9 each, 64
    of them relative to the page's largest p (which the sum holds at least
    once a page): 2^-17.9 |v|max, and the exponential's own error, 2^-21.
    bfloat16 outputs: half a step, 2^-8; their probabilities and values may
    be rounded to 11 bits on the way (2^-11 of each product, of the sum of
    magnitudes), and so may the sum's terms not be: 2^-10."""
    qmax = np.abs(q).max(-1, keepdims=True)
    d = abs(scale) * 2.0 ** -22 * qmax * b["ksum"] + 8 * 2.0 ** -24 * b["smax"] + 2.0 ** -21
    pages = longest // PAGE + 2
    rel = np.expm1(2 * d) + (2 * pages + 20) * 2.0 ** -24
    if dtype == "bf16":
        rel = rel + 2.0 ** -10
    return b["mass"] * rel + 2.0 ** -17.9 * b["vmax"]


# ---- log probabilities --------------------------------------------------------

def logprobs(x, ids, top):
    x = x.astype(np.float64) + 0.0
    with np.errstate(all="ignore"):
        m = x.max(1, keepdims=True)
        d = x - m
        e = np.exp(d)
        s0 = e.sum(1, keepdims=True)
        p = e / s0
        pd = np.where(e > 0, p * d, 0.0)
        lp = d - np.log(s0)
        h = np.log(s0[:, 0]) - pd.sum(1)
        # sizes for the tolerance: E|d|, E d^2
        ed, ed2 = -pd.sum(1), np.where(e > 0, p * d * d, 0.0).sum(1)
    best = np.argsort(-x, axis=1, kind="stable")[:, :top]
    ok = (ids >= 0) & (ids < x.shape[1])
    at = np.where(ok, ids, 0)
    return {"lp": np.where(ok, np.take_along_axis(lp, at, 1), 0.0), "entropy": h, "top_ids": best,
            "top_lp": np.take_along_axis(lp, best, 1), "ln": np.log(s0[:, 0]), "ed": ed, "ed2": ed2}


def logprob_bound(r, lp, pieces):
    """lp = (x - m) - ln S0: x - m and the difference round once each; a term
    e^d of S0 is off by at most 2^-22 + 2 |d| 2^-24 of itself (the argument
    d log2 e rounds, as does the exponential), on the average over the terms
    2^-22 + 2^-23 E|d|; the sums of 32 terms a thread, 9 levels of lanes and
    waves and the pieces round 2^-24 each."""
    s = 2.0 ** -22 + 2.0 ** -23 * r["ed"] + (64 + pieces) * 2.0 ** -24 + 2.0 ** -22 * np.abs(r["ln"])
    ln = r["ln"][:, None]
    return s[:, None] + 2.0 ** -24 * (np.abs(lp + ln) + np.abs(lp))


def entropy_bound(r, pieces):
    """ln S0 - S1 / S0: the terms e^d d of S1 are off by twice what those of
    S0 are, weighted by |d|."""
    s = 2.0 ** -22 + (64 + pieces) * 2.0 ** -24
    return (s + 2.0 ** -23 * r["ed"] + 2.0 ** -22 * np.abs(r["ln"])
            + r["ed"] * (2 * s + 2.0 ** -23 * r["ed"]) + 2.0 ** -22 * r["ed2"] + 2.0 ** -23 * r["ed"])
