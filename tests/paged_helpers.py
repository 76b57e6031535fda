"""Seeded paged caches and references of their operators: 64 bits where the definition is real
arithmetic, f32 step by step where the definition names f32 roundings."""
import math

import numpy as np

BLOCK = 16
TOP = {"i8": 127.0, "e4m3": 448.0}
U = 2.0**-24


def e4m3_table():
    """The value of each 8-bit code (sign, 4 exponent bits with bias 7, 3 of fraction; 0x7F and 0xFF NaN)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, (c & 7) / 8.0
    v = np.where(e == 0, f * 2.0**-6, (1 + f) * 2.0 ** (e.astype(float) - 7))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


E4M3 = e4m3_table()


def decode(codes, fmt):
    """uint8 codes -> their values in 64 bits."""
    return codes.view(np.int8).astype(np.float64) if fmt == "i8" else E4M3[codes]


def encode(x, fmt):
    """f32 value / scale -> uint8 codes: nearest, ties away from zero (i8) or to the even code (e4m3)."""
    x = np.asarray(x, np.float64)
    if fmt == "i8":
        return (np.sign(x) * np.minimum(np.floor(np.abs(x) + 0.5), 127)).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    up = E4M3[:127]
    hi = np.clip(np.searchsorted(up, a), 1, 126)
    lo = hi - 1
    d0, d1 = a - up[lo], up[hi] - a
    pick = np.where(d0 < d1, lo, np.where(d1 < d0, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def frequencies(theta, rot, scaling="none", factor=1.0, trained=0, low=1.0, high=32.0):
    """Radians per position of each pair and the magnitude, from the formulas in the header."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "turns":
        w = np.clip((trained * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return f * (w + (1 - w) / factor), 1.0
    if scaling == "pairs":
        d = lambda r: rot * math.log(trained / (2 * math.pi * r)) / (2 * math.log(theta))  # noqa: E731
        first, last = max(math.floor(d(high)), 0), min(math.ceil(d(low)), rot - 1)
        w = np.array([min(max(1 - (k - first) / max(last - first, 0.001), 0), 1) for k in range(rot // 2)])
        return f * (w + (1 - w) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def cos_sin(turns, pos, magnitude):
    """f32 (cos, sin) [len(pos)][pairs] of exact angles: position times turns modulo 2^64 in integers,
    quadrant and remainder in integers, the rest in 64 bits, rounded once."""
    c = np.empty((len(pos), len(turns)))
    s = np.empty_like(c)
    for a, p in enumerate(pos):
        for b, t in enumerate(turns):
            at = (int(p) * (int(t) & (2**64 - 1))) % 2**64
            quad = ((at + 2**61) >> 62) % 4
            x = (at - (((at + 2**61) >> 62) << 62)) * (math.pi / 2**63)
            co, si = math.cos(x), math.sin(x)
            c[a, b], s[a, b] = [(co, si), (-si, co), (-co, -si), (si, -co)][quad]
    return (c * magnitude).astype(np.float32), (s * magnitude).astype(np.float32)


def rotate(x, cs, rot, pairing):
    """x [rows][heads][hd] f32, rotated by (cos, sin) [rows][rot / 2] f32 in 64 bits, rounded once."""
    y = np.array(x, np.float32)
    c, s = (a.astype(np.float64)[:, None] for a in cs)
    half = pairing == "half"
    at0, at1 = (np.arange(rot // 2), np.arange(rot // 2) + rot // 2) if half else (np.arange(0, rot, 2), np.arange(1, rot, 2))
    x0, x1 = x[..., at0].astype(np.float64), x[..., at1].astype(np.float64)
    y[..., at0] = (x0 * c - x1 * s).astype(np.float32)
    y[..., at1] = (x0 * s + x1 * c).astype(np.float32)
    return y


class Cache:
    """A paged cache on the host: uint8 codes [pages][heads][tokens][hd], f32 scales, the table."""

    def __init__(self, rng, seqs, heads, hd, tokens, need, fmt, width=None, spare=3):
        self.fmt, self.heads, self.hd, self.tokens = fmt, heads, hd, tokens
        need = [-(-n // tokens) for n in need]
        pages = sum(need) + spare
        self.width = width or max(max(need), 1)
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((seqs, self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at : at + n]
            at += n
        shape = (pages, heads, tokens, hd)
        self.k, self.v = (self.random(rng, shape) for _ in range(2))
        self.ks, self.vs = (rng.uniform(0.01, 0.03, (pages, heads, tokens // BLOCK)).astype(np.float32) for _ in range(2))

    def random(self, rng, shape):
        if self.fmt == "i8":
            return rng.integers(-127, 128, shape).astype(np.int8).view(np.uint8)
        c = rng.integers(0, 256, shape).astype(np.uint8)
        return np.where((c & 127) == 127, 0, c).astype(np.uint8)

    def values(self, seq, head, n):
        """(codes, scales) of keys and of values at positions 0..n-1, 64 bits."""
        pages = self.table[seq, : -(-n // self.tokens)]
        out = []
        for codes, scale in ((self.k, self.ks), (self.v, self.vs)):
            c = decode(codes[pages, head].reshape(-1, self.hd)[:n], self.fmt)
            out += [c, np.repeat(scale[pages, head].reshape(-1), BLOCK)[:n].astype(np.float64)]
        return out

    def put(self, seq, pos, k, v):
        """Append k, v [rows][heads][hd] (f32, rotated already) at pos, block by block."""
        n = min(len(k), self.width * self.tokens - pos)
        f32 = np.float32
        for lo in range(pos // BLOCK * BLOCK, pos + n, BLOCK):
            a, z = max(lo, pos), min(lo + BLOCK, pos + n)
            page = self.table[seq, lo // self.tokens]
            if not 0 <= page < len(self.k):
                continue
            j, r = lo % self.tokens // BLOCK, lo % self.tokens
            for x, codes, scale in ((k, self.k, self.ks), (v, self.v, self.vs)):
                for h in range(self.heads):
                    new = x[a - pos : z - pos, h]
                    old = scale[page, h, j] if a > lo else f32(0)
                    with np.errstate(all="ignore"):
                        mine = f32(np.abs(new).max()) / f32(TOP[self.fmt])
                        now = f32(np.nan) if np.isnan(old) or not np.isfinite(new).all() else max(old, mine)
                        held = codes[page, h, r : r + a - lo]
                        if now > old and a > lo:
                            again = (decode(held, self.fmt).astype(f32) * old) / now
                            codes[page, h, r : r + a - lo] = encode(again, self.fmt)
                        into = encode(new / now, self.fmt) if now > 0 else np.zeros(new.shape, np.uint8)
                    codes[page, h, r + a - lo : r + z - lo] = into
                    scale[page, h, j] = now


def attn_ref(q, ck, sk, cv, sv, p, scale, window):
    """One row and head in 64 bits over positions 0..p: (out [hd], the bound of each output's error).
    With weights w_j that sum to 1, an output sum_j w_j v_j moves by at most sum_j w_j e_j (|v_j| + |o|)
    when every weight is off by a factor 1 + e_j.  A score is hd products of exact codes and of q, which
    is off by 2^-22 of each value (two parts, and the product with the scale before) and 2^-40 of the
    row's largest, and hd + 8 f32 additions and products: (hd + 16) 2^-24 of sum |q k|; exp2 and the
    weight's parts and scales add 16 * 2^-24.  The sums over n positions (at most n / 16 + 64 additions one
    after the other) and the products' own 8 half steps add (n / 16 + 72) 2^-24 of sum w |v| and of |o|;
    weights end 2^-38 below the largest w * scale of the row (a unit that its scales may stay 2^-2 below)."""
    lo = max(0, p - window + 1) if window else 0
    ck, sk, cv, sv = ck[lo : p + 1], sk[lo : p + 1], cv[lo : p + 1], sv[lo : p + 1]
    q, hd = q.astype(np.float64), ck.shape[1]
    s = (ck @ q) * sk * scale
    size = (np.abs(ck) @ np.abs(q)) * sk * abs(scale)
    w = np.exp(s - s.max())
    w /= w.sum()
    v = cv * sv[:, None]
    o = w @ v
    end_q = 2.0**-39 * np.abs(q).max() * np.abs(ck).sum(1) * sk * abs(scale)
    rel = (hd + 16) * U * size + end_q + 16 * U
    tol = (w * rel) @ (np.abs(v) + np.abs(o)) + (len(w) / 16 + 72) * U * (w @ np.abs(v) + np.abs(o))
    return o, tol + 2.0**-37 * (w * sv).max() * np.abs(cv).sum(0)


def attn_all(cache, q, row_start, pos, group, scale, window):
    """(out, bound) of every packed row; NaN where no sequence has the row."""
    out = np.full(q.shape, np.nan)
    tol = np.zeros(q.shape)
    for b in range(len(pos)):
        t = row_start[b + 1] - row_start[b]
        for h in range(q.shape[1]):
            if t:
                ck, sk, cv, sv = cache.values(b, h // group, pos[b] + t)
            for i in range(t):
                r = row_start[b] + i
                out[r, h], tol[r, h] = attn_ref(q[r, h], ck, sk, cv, sv, pos[b] + i, scale, window)
    return out, tol
