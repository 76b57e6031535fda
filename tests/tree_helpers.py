"""Seeded trees of drafted tokens and 64-bit references of the tree-verification operators."""
import numpy as np

HD = 64


def random_tree(rng, n):
    """parent [n] with parent[c] < c, and the ancestor relation [n][n] (a node is its own)."""
    parent = np.full(n, -1, np.int32)
    anc = np.eye(n, dtype=bool)
    for c in range(1, n):
        parent[c] = rng.integers(0, c)
        anc[c] |= anc[parent[c]]
    return parent, anc


def mask_bits(anc):
    """[..., n, n] booleans -> [..., n] int64 bit patterns."""
    n = anc.shape[-1]
    w = (np.uint64(1) << np.arange(n, dtype=np.uint64))
    return np.where(anc, w, np.uint64(0)).sum(-1, dtype=np.uint64).view(np.int64)


def attn_ref(q, k, v, kd, vd, pos, anc, cnt, hq, hk):
    """One sequence in 64 bits: out [cnt][hq][64] and, for the tolerance, the largest
    sum |q k| / 8 of a score and |v| (over what the rows see)."""
    q, k, v, kd, vd = (np.asarray(a, np.float64) for a in (q, k, v, kd, vd))
    out = np.zeros((cnt, hq, HD))
    smax = vmax = 0.0
    for h in range(hq):
        g = h // (hq // hk)
        for i in range(cnt):
            keep = [j for j in range(cnt) if anc[i, j]]
            kk = np.concatenate([k[g, :pos], kd[g, keep]])
            vv = np.concatenate([v[g, :pos], vd[g, keep]])
            if not len(kk):
                continue
            s = kk @ q[i, h] / 8.0
            w = np.exp(s - s.max())
            out[i, h] = (w @ vv) / w.sum()
            smax = max(smax, float((np.abs(kk) @ np.abs(q[i, h])).max() / 8.0))
            vmax = max(vmax, float(np.abs(vv).max()))
    return out, smax, vmax


def attn_tol(n, smax, vmax):
    """Bound of an output's error.  A score is a 64-term sum of products, each operand off by
    at most 2^-22 of the largest (the two-part split) or 2^-24: (64 + 8) 2^-24 + 2 * 2^-22 of
    sum |q k| / 8, and its weight is off by that much relatively, twice (numerator and
    denominator).  The weights (exp2: 2^-22; two-part split: 2^-22) and the sums over n
    positions (at most n / 16 + 64 f32 additions one after the other) add the rest."""
    ds = smax * (80 * 2.0**-24)
    return vmax * (2 * ds + 2 * (n / 16 + 64) * 2.0**-24 + 4 * 2.0**-22)


def attn_bound(q, k, v, kd, vd, pos, anc, cnt, hq, hk, f16):
    """One sequence in 64 bits: out [cnt][hq][64] and the bound of each output's own error.
    With weights w_j that sum to 1, an output sum_j w_j v_j moves by at most
    sum_j w_j e_j (|v_j| + |o|) when every weight is off by a factor 1 + e_j: a score is off by
    80 * 2^-24 of its own sum |q k| / 8 (64 f32 additions and two operands to 2^-21 each, as in
    attn_tol) and exp2 and the weight's parts by 8 * 2^-24.  The sums over n positions (n / 16 + 64
    additions one after the other, as in attn_tol) and the parts of v (8 half steps) add
    (n / 16 + 72) * 2^-24 of sum w |v| and of |o|.  Nothing here grows with another dimension of
    the value, or with a row that has no weight.  A binary16 cache: weights and queries in two
    binary16 parts, which end 2^-40 below the largest of the row."""
    q, k, v, kd, vd = (np.asarray(a, np.float64) for a in (q, k, v, kd, vd))
    u = 2.0**-24
    out, tol = np.zeros((cnt, hq, HD)), np.zeros((cnt, hq, HD))
    for h in range(hq):
        g = h // (hq // hk)
        for i in range(cnt):
            keep = [j for j in range(cnt) if anc[i, j]]
            kk = np.concatenate([k[g, :pos], kd[g, keep]])
            vv = np.concatenate([v[g, :pos], vd[g, keep]])
            s = kk @ q[i, h] / 8.0
            w = np.exp(s - s.max())
            rel = 80 * u * (np.abs(kk) @ np.abs(q[i, h])) / 8.0 + 8 * u
            w /= w.sum()
            o = w @ vv
            end = 0.0
            if f16:
                rel = rel + 2 * 2.0**-40 * np.abs(q[i, h]).max() * np.abs(kk).sum(1) / 8.0
                end = 2 * 2.0**-40 * w.max() * (np.abs(vv).sum(0) + len(vv) * np.abs(o))
            out[i, h] = o
            tol[i, h] = (w * rel) @ (np.abs(vv) + np.abs(o)) + (len(vv) / 16 + 72) * u * (w @ np.abs(vv) + np.abs(o)) + end
    return out, tol


def attn_plain(q, k, v, kd, vd, pos, anc, cnt, hq, hk, dtype=np.float32, part=lambda name, a: a):
    """One sequence in `dtype`, a head's rows at once: out [cnt][hq][64].  part(name, a) stands for
    what becomes of an operand ("q", "k", "p", "v") on its way into a product."""
    q, k, v, kd, vd = (np.asarray(a, dtype) for a in (q, k, v, kd, vd))
    out = np.zeros((cnt, hq, HD), dtype)
    sees = np.concatenate([np.ones((cnt, pos), bool), anc[:cnt, :cnt]], 1)
    for h in range(hq):
        g = h // (hq // hk)
        kk, vv = np.concatenate([k[g, :pos], kd[g, :cnt]]), np.concatenate([v[g, :pos], vd[g, :cnt]])
        s = part("q", q[:cnt, h] * dtype(0.125)) @ part("k", kk).T
        s = np.where(sees, s, dtype(-np.inf))
        p = np.exp(s - s.max(1, keepdims=True))
        out[:, h] = (part("p", p) @ part("v", vv)) / p.sum(1, keepdims=True)
    return out


def rms(a):
    return float(np.sqrt(np.mean(np.square(np.asarray(a, np.float64)))))


def logprobs_ref(x, tokens, top_k):
    """(logprob, entropy, top_idx, top_logprob) of one row in 64 bits."""
    x = np.asarray(x, np.float64)
    n = len(x)
    m = np.fmax.reduce(x)
    with np.errstate(all="ignore"):
        bad = np.isnan(x).any() or not np.isfinite(m)
        first = int(np.nanargmax(x)) if not np.isnan(x).all() else 0
        d = x - m
        e = np.exp(d)
        e[first] = 0.0
        r = e.sum()
        lse = np.nan if bad else np.log1p(r)
        h = np.where(e > 0, -e * d, 0.0).sum() / (1 + r) + lse
        lp = d - lse
    order = sorted(range(n), key=lambda i: (np.isnan(x[i]), -x[i] if not np.isnan(x[i]) else 0.0, i))[:top_k]
    return (np.array([lp[t] if 0 <= t < n else -np.inf for t in tokens]), h, np.array(order, np.int32),
            lp[order] if top_k else np.zeros(0))


def commit_ref(tokens, parent, chosen, cnt, pos, max_ctx):
    """(path, next token) of one sequence."""
    if pos < 0 or pos > max_ctx or min(cnt, max_ctx - pos) < 1:
        return [], -1
    path = [0]
    while len(path) < max_ctx - pos:
        cur = path[-1]
        on = [c for c in range(cur + 1, cnt) if parent[c] == cur and tokens[c] == chosen[cur]]
        if not on:
            break
        path.append(on[0])
    return path, int(chosen[path[-1]])
