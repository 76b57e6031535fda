"""Measured cases of the operators of a paged key/value cache in 8 bits.

The cache of a served model is cut into pages that sequences take as they grow; keys and values
are held as 8-bit codes with one f32 scale for each 16 positions of a key head.  `rope_tokens`
rotates the heads of packed tokens at any positions, part of the head and scaled for long contexts;
`paged_append` rotates queries and keys on the way and quantises keys and values into the pages;
`paged_attn` attends over the pages, one new token a sequence or many; `paged_read` gives sequences
back as the contiguous caches that the other operators take.

`run` computes each operator in elementary torch operations where `own` is false, and through
quantized_decode_gemv_gb300 where it is true.  Head layouts and contexts are those of the models
here (9 heads over 3, 32 over 32, head dimension 64, context 4096), with grouped layouts, head
dimension 128 and longer contexts beside them.

A cache's values: codes times the scale of their block.  A block's scale is the largest magnitude of
what was put into it over 127 (codes -127..127, nearest, ties away from zero) or over 448 (e4m3
codes, nearest, ties to even), divisions and scales in f32; where a later token of the block is
larger, the scale grows and the codes before it are rounded again.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16  # positions that share a scale
TOP = {"i8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence of the 135M shape early in its context, one new token: latency
        dict(name="attn_135m_1seq", op="attn", heads=9, kv_heads=3, hd=64, seqs=1, rows=1, longest=200, ragged=False,
             page=16, fmt="i8", window=0),
        # the 1.7B shape with 16 sequences of different lengths up to its context: served load
        dict(name="attn_1p7b_b16", op="attn", heads=32, kv_heads=32, hd=64, seqs=16, rows=1, longest=4096, ragged=True,
             page=64, fmt="i8", window=0),
        # 100 sequences with grouped heads, head dimension 128: a full server
        dict(name="attn_gqa4_b100", op="attn", heads=32, kv_heads=8, hd=128, seqs=100, rows=1, longest=8100,
             ragged=True, page=32, fmt="i8", window=0),
        # one long document: the walk has to be split
        dict(name="attn_long_131k", op="attn", heads=32, kv_heads=8, hd=128, seqs=1, rows=1, longest=131000,
             ragged=False, page=64, fmt="e4m3", window=0),
        # a prompt's second thousand tokens in one piece
        dict(name="attn_chunk_1024", op="attn", heads=32, kv_heads=8, hd=128, seqs=1, rows=1024, longest=2040,
             ragged=False, page=64, fmt="i8", window=0),
        # a mixed step: pieces of prompts and single tokens, eight query heads to a key head, sliding window
        dict(name="attn_mixed_window", op="attn", heads=8, kv_heads=1, hd=64, seqs=7, rows=45, longest=3001,
             ragged=True, page=16, fmt="e4m3", window=1000),
        # one new token of each of 16 sequences of the 135M shape, then the caches as drafting takes them
        dict(name="append_135m_b16", op="append", heads=9, kv_heads=3, hd=64, seqs=16, rows=1, longest=250,
             ragged=True, page=16, fmt="i8", rot=64, pairing="half", scaling="none", out="f32"),
        # prompts of different lengths in one packed batch, half of each head rotated, a stretched context
        dict(name="append_prompts", op="append", heads=32, kv_heads=8, hd=128, seqs=6, rows=1500, longest=2300,
             ragged=True, page=64, fmt="i8", rot=64, pairing="adjacent", scaling="pairs", out="f16"),
        # one short sequence handed over to tree verification
        dict(name="read_135m_1seq", op="read", heads=9, kv_heads=3, hd=64, seqs=1, rows=1, longest=200, ragged=False,
             page=16, fmt="i8", out="f32"),
        # 16 sequences moved out of the pages
        dict(name="read_b16", op="read", heads=32, kv_heads=8, hd=128, seqs=16, rows=1, longest=4096, ragged=True,
             page=32, fmt="e4m3", out="f16"),
        # the queries and keys of a decode step of 16 sequences far into a stretched context
        dict(name="rope_16tok_far", op="rope", heads=9, kv_heads=3, hd=64, tokens=16, rot=32, pairing="adjacent",
             scaling="turns", far=1000000),
        # the queries and keys of a prompt
        dict(name="rope_8000tok", op="rope", heads=32, kv_heads=8, hd=128, tokens=8000, rot=128, pairing="half",
             scaling="linear", far=120000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "read", "rope"])
    most = {}
    for c in listed():
        w = work(c)
        for k in ("bytes", "flops"):
            most[k] = max(most.get(k, 0), w[k] if c["op"] == op else 0)
    while True:
        heads, kv_heads = rng.choice([(9, 3), (32, 32), (32, 8), (8, 1), (6, 2), (5, 5), (16, 1), (40, 8)])
        case = dict(op=op, heads=heads, kv_heads=kv_heads, hd=rng.choice([64, 128]))
        if op == "rope":
            case.update(tokens=_log(rng, 1, 8000), rot=rng.choice([16, 32, 48, 64, case["hd"]]),
                        pairing=rng.choice(["half", "adjacent"]),
                        scaling=rng.choice(["none", "linear", "ntk", "turns", "pairs"]), far=_log(rng, 300, 1000000))
        else:
            seqs = _log(rng, 1, 100)
            longest = _log(rng, 17, 131000) if op == "attn" else _log(rng, 17, 5000)
            rows = 1 if op == "read" or rng.random() < 0.5 else min(_log(rng, 2, 1500), longest)
            case.update(seqs=seqs, rows=rows, longest=longest, ragged=rng.random() < 0.7,
                        page=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["i8", "e4m3"]))
            if op == "attn":
                case.update(window=rng.choice([0, 0, _log(rng, 1, longest)]))
            else:
                case.update(out=rng.choice(["f32", "f16"]))
            if op == "append":
                case.update(rot=rng.choice([16, 32, 64, case["hd"]]), pairing=rng.choice(["half", "adjacent"]),
                            scaling=rng.choice(["none", "linear", "ntk", "turns", "pairs"]))
            # what the plain forms hold: whole sequences in f32, and a score for each of them
            held = 8 * seqs * longest * kv_heads * case["hd"]
            scores = 4 * seqs * rows * heads * longest if op == "attn" else 0
            if held > 8 << 30 or scores > 1 << 30 or seqs * rows > 16000:
                continue
        w = work(case)
        if all(w[k] <= most[k] for k in most):
            return case


def _new(case):
    """New tokens of each sequence; a case has the same ones with every seed, as its outputs' shapes go by them."""
    b, t = case["seqs"], case["rows"]
    new = np.full(b, t)
    if case["ragged"]:
        new = np.random.default_rng([b, t, case["longest"]]).integers(1, t + 1, b)
        new[0] = t
        if b > 2:
            new[1], new[2] = 1, t
    return new


def _lengths(case, rng):
    """Positions that each sequence holds before the call, and its new tokens."""
    new, top = _new(case), case["longest"]
    total = np.full(case["seqs"], top)
    if case["ragged"]:
        total = rng.integers(new, top + 1)
        total[0] = top
        if case["seqs"] > 2:
            total[2] = new[2]  # a prompt from its start
    return (total - new).astype(np.int32), new.astype(np.int32)


def _frequencies(case):
    """Angle per position of each rotated pair (radians, 64 bits), and what cos and sin are multiplied by."""
    rot, theta, factor, trained, low, high = case["rot"], 1e4, 8.0, 4096, 1.0, 32.0
    i = np.arange(rot // 2, dtype=np.float64)
    kind = case["scaling"]
    if kind == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "turns":  # what turns often within the trained context stays, what hardly turns is stretched
        w = np.clip((trained * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return f * (w + (1 - w) / factor), 1.0
    if kind == "pairs":  # the same by the pairs' index, with larger products for the longer context
        at = lambda turns: rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(theta))  # noqa: E731
        first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        w = 1 - np.clip((i - first) / max(last - first, 0.001), 0, 1)
        return f * (w + (1 - w) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ------------------------------------------------------------------------------ inputs
def _codes(case, shape, g):
    """Codes as a cache of activations holds them, near normal and within their range."""
    x = torch.randn(shape, generator=g, device="cuda")
    if case["fmt"] == "i8":
        return x.mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    return x.mul_(130.0).clamp_(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    rng = np.random.default_rng([seed, 12])
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    h, hk, hd = case["heads"], case["kv_heads"], case["hd"]
    s = dict(case={k: v for k, v in case.items() if k != "name"})
    if case["op"] == "rope":
        n = case["tokens"]
        s["x"] = torch.randn(n, h + hk, hd, generator=g, device="cuda")  # queries and keys of the fused projection
        first = rng.integers(0, case["far"] + 1, 16)
        at = first[np.arange(n) * 16 // n] + np.arange(n)  # 16 runs of neighbouring positions
        s["pos"] = dev(np.minimum(at, case["far"]).astype(np.int32))
        s["out"] = torch.empty_like(s["x"])
    else:
        b, page = case["seqs"], case["page"]
        pos, new = _lengths(case, rng)
        need = -(-(pos + new) // page)  # pages of each sequence
        width, pages = -(-case["longest"] // page), int(need.sum()) + 3
        table = np.full((b, width), -1, np.int32)
        order = rng.permutation(pages)
        at = np.concatenate([[0], np.cumsum(need)])
        for i in range(b):
            table[i, : need[i]] = order[at[i] : at[i + 1]]
        s["table"], s["pos"], s["len"] = dev(table), dev(pos), dev(pos + new)
        s["row_start"] = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        s["n"], s["most"] = int(new.sum()), int(new.max())
        blocks = (pages, hk, page // BLOCK)
        for k in ("k", "v"):
            s[k + "_pages"] = _codes(case, (pages, hk, page, hd), g)
            s[k + "_scale"] = (0.7 + 0.6 * torch.rand(blocks, generator=g, device="cuda")) / (36.0 if case["fmt"] == "i8" else 130.0)
        n = s["n"]
        if case["op"] == "attn":
            s["q"] = torch.randn(n, h, hd, generator=g, device="cuda") * 1.5
            s["out"] = torch.zeros(n, h, hd, device="cuda")
        else:
            kind = torch.float32 if case["out"] == "f32" else torch.float16
            s["k_out"] = torch.zeros(b, hk, case["longest"], hd, dtype=kind, device="cuda")
            s["v_out"] = torch.zeros(b, hk, case["longest"], hd, dtype=kind, device="cuda")
        if case["op"] == "append":
            s["qkv"] = torch.randn(n, h + 2 * hk, hd, generator=g, device="cuda")
            s["qkv"][:, h : h + hk, ::17] *= 4.0  # some dimensions of keys are larger than the others
            s["q_out"] = torch.zeros(n, h, hd, device="cuda")
    if "rot" in case:
        f, s["magnitude"] = _frequencies(case)
        s["freq"] = dev(f)
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        return _OWN[c["op"]](s, c)
    return _PLAIN[c["op"]](s, c)


def _rotated(x, pos, s, c):
    """x [tokens][heads][hd], its first `rot` dimensions turned; angles and products in 64 bits, cos and sin
    rounded to f32 as the tables of the other operators hold them."""
    a = pos.double()[:, None] * s["freq"]
    cos, sin = ((f(a) * s["magnitude"]).float().double()[:, None] for f in (torch.cos, torch.sin))
    r = c["rot"]
    y = x[..., :r].double()
    if c["pairing"] == "half":
        y0, y1 = y[..., : r // 2], y[..., r // 2 :]
        y = torch.cat([y0 * cos - y1 * sin, y0 * sin + y1 * cos], dim=-1)
    else:
        y0, y1 = y[..., 0::2], y[..., 1::2]
        y = torch.stack([y0 * cos - y1 * sin, y0 * sin + y1 * cos], dim=-1).flatten(-2)
    return torch.cat([y.float(), x[..., r:]], dim=-1)


def _plain_rope(s, c):
    return _rotated(s["x"], s["pos"], s, c)


def _rows(s):
    """The sequence of each packed row, and its position."""
    at = torch.arange(s["n"], device="cuda")
    seq = torch.searchsorted(s["row_start"].long(), at, right=True) - 1
    return seq, s["pos"].long()[seq] + at - s["row_start"].long()[seq]


def _round(x, fmt):
    """Codes of x / scale, as f32 values."""
    if fmt == "i8":
        return torch.trunc(x.double() + torch.where(x < 0, -0.5, 0.5)).clamp(-127, 127).float()
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).float()


def _plain_put(x, pages, scale, s, c):
    """(codes as f32, scales) of a cache after the rows x [n][kv heads][hd] went into it."""
    seq, p = _rows(s)
    page = s["table"].long()[seq, p // c["page"]]
    block = page * (c["page"] // BLOCK) + p % c["page"] // BLOCK  # of all pages
    slot = p % BLOCK
    nb, hk, hd = scale.shape[0] * scale.shape[2], c["kv_heads"], c["hd"]
    most = torch.zeros(nb, hk, device="cuda").scatter_reduce(0, block[:, None].expand(-1, hk), x.abs().amax(-1), "amax")
    first = torch.full((nb,), BLOCK, device="cuda").scatter_reduce(0, block, slot, "amin")
    old = scale.transpose(1, 2).reshape(nb, hk)
    held = torch.where((first > 0)[:, None], old, 0.0)
    new = torch.where((first < BLOCK)[:, None], torch.maximum(held, (most.double() / TOP[c["fmt"]]).float()), old)
    codes = pages.float().view(-1, hk, c["page"] // BLOCK, BLOCK, hd).transpose(1, 2).reshape(nb, hk, BLOCK, hd)
    grown = (new > old)[..., None, None] & (torch.arange(BLOCK, device="cuda") < first[:, None])[:, None, :, None]
    again = _round(codes * old[..., None, None] / new[..., None, None], c["fmt"])
    codes = torch.where(grown & (first < BLOCK)[:, None, None, None], again, codes)
    codes[block, :, slot] = _round(x / new[block][..., None], c["fmt"])
    return codes, new


def _plain_values(codes, scale, s, c, kind, out):
    """Contiguous caches [sequence][kv head][position][hd] of codes [block][kv head][16][hd]; `out` behind the ends."""
    per, hk = c["page"] // BLOCK, c["kv_heads"]
    x = (codes * scale[..., None, None]).to(kind).view(-1, per, hk, BLOCK, c["hd"])[s["table"].long().clamp(min=0)]
    x = x.permute(0, 3, 1, 2, 4, 5).reshape(c["seqs"], hk, -1, c["hd"])[:, :, : c["longest"]]
    live = torch.arange(c["longest"], device="cuda") < s["len"][:, None]
    return torch.where(live[:, None, :, None], x, out)


def _blocks(pages, scale, c):
    per, hk = c["page"] // BLOCK, c["kv_heads"]
    codes = pages.float().view(-1, hk, per, BLOCK, c["hd"]).transpose(1, 2).reshape(-1, hk, BLOCK, c["hd"])
    return codes, scale.transpose(1, 2).reshape(-1, hk)


def _plain_append(s, c):
    h, hk = c["heads"], c["kv_heads"]
    _, p = _rows(s)
    qk = _rotated(s["qkv"][:, : h + hk], p, s, c)
    k, ks = _plain_put(qk[:, h:], s["k_pages"], s["k_scale"], s, c)
    v, vs = _plain_put(s["qkv"][:, h + hk :], s["v_pages"], s["v_scale"], s, c)
    kind = s["k_out"].dtype
    return qk[:, :h], _plain_values(k, ks, s, c, kind, s["k_out"]), _plain_values(v, vs, s, c, kind, s["v_out"])


def _plain_read(s, c):
    kind = s["k_out"].dtype
    return tuple(_plain_values(*_blocks(s[x + "_pages"], s[x + "_scale"], c), s, c, kind, s[x + "_out"]) for x in "kv")


def _plain_attn(s, c):
    b, t, h, hk, hd, n = c["seqs"], s["most"], c["heads"], c["kv_heads"], c["hd"], c["longest"]
    seq, p = _rows(s)
    i = p - s["pos"].long()[seq]
    zero = torch.zeros((), device="cuda")
    k, v = (_plain_values(*_blocks(s[x + "_pages"], s[x + "_scale"], c), s, c, torch.float32, zero) for x in "kv")
    q = torch.zeros(b, t, h, hd, device="cuda")
    q[seq, i] = s["q"]
    q = q.view(b, t, hk, h // hk, hd).permute(0, 2, 1, 3, 4).reshape(b, hk, t * (h // hk), hd)
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(1 / math.sqrt(hd)).view(b, hk, t, h // hk, n)
    at = torch.arange(n, device="cuda")
    last = s["pos"][:, None] + torch.arange(t, device="cuda")
    sees = at <= last[..., None]
    if c["window"]:
        sees &= at > last[..., None] - c["window"]
    scores.masked_fill_(~sees[:, None, :, None], -math.inf)
    w = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(b, hk, t * (h // hk), n), v).view(b, hk, t, h // hk, hd) / total
    return o.permute(0, 2, 1, 3, 4).reshape(b, t, h, hd)[seq, i]


_PLAIN = dict(attn=_plain_attn, append=_plain_append, read=_plain_read, rope=_plain_rope)


def _plan(s, c):
    """The rotation that a program lays out once: turns per position, and the magnitude."""
    import quantized_decode_gemv_gb300 as qd

    if "plan" not in s:
        turns, magnitude = qd.rope_plan(1e4, c["rot"], c["scaling"], factor=8.0, trained_ctx=4096, low=1.0, high=32.0)
        s["plan"] = turns.cuda(), magnitude
    return s["plan"]


def _cache(s, c):
    """The handle of a paged cache that a program keeps."""
    import quantized_decode_gemv_gb300 as qd

    if "cache" not in s:
        s["cache"] = qd.PagedKV(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], fmt=c["fmt"])
    return s["cache"]


def _own_rope(s, c):
    import quantized_decode_gemv_gb300 as qd

    turns, magnitude = _plan(s, c)
    width = (c["heads"] + c["kv_heads"]) * c["hd"]
    qd.rope_tokens(s["x"], width, s["out"], width, c["tokens"], c["heads"] + c["kv_heads"], c["hd"], c["rot"], s["pos"],
                   c["pairing"], turns, magnitude)
    return s["out"]


def _own_append(s, c):
    import quantized_decode_gemv_gb300 as qd

    turns, magnitude = _plan(s, c)
    h, hk, qkv = c["heads"], c["kv_heads"], s["qkv"]
    kv = _cache(s, c)
    qd.paged_append(kv, qkv, qkv[:, h:], qkv[:, h + hk :], (h + 2 * hk) * c["hd"], s["q_out"], h, s["n"], s["row_start"],
                    s["pos"], c["seqs"], c["rot"], c["pairing"], turns, magnitude)
    qd.paged_read(kv, s["len"], c["seqs"], c["longest"], s["k_out"], s["v_out"], out_f16=c["out"] == "f16")
    return s["q_out"], s["k_out"], s["v_out"]


def _own_read(s, c):
    import quantized_decode_gemv_gb300 as qd

    qd.paged_read(_cache(s, c), s["len"], c["seqs"], c["longest"], s["k_out"], s["v_out"], out_f16=c["out"] == "f16")
    return s["k_out"], s["v_out"]


def _own_attn(s, c):
    import quantized_decode_gemv_gb300 as qd

    kv = _cache(s, c)
    if "ws" not in s:
        size = qd.paged_attn_workspace(kv, c["heads"], s["n"], c["seqs"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    qd.paged_attn(kv, s["q"], c["heads"] * c["hd"], s["out"], c["heads"], s["n"], s["row_start"], s["pos"], c["seqs"],
                  1 / math.sqrt(c["hd"]), c["window"], s["ws"])
    return s["out"]


_OWN = dict(attn=_own_attn, append=_own_append, read=_own_read, rope=_own_rope)


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    h, hk, hd = case["heads"], case["kv_heads"], case["hd"]
    if case["op"] == "rope":
        n = case["tokens"] * (h + hk)
        return {"bytes": 8 * n * hd + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    # lengths of the ragged cases are drawn evenly from a sequence's new tokens to the longest
    b, top = case["seqs"], case["longest"]
    rows = float(_new(case).mean())
    mean = (top + rows) / 2 if case["ragged"] and b > 1 else top
    held = b * hk * (hd + 4 / BLOCK)  # bytes of a position of keys, or of values
    if case["op"] == "attn":
        window = case["window"] or top
        keys = min(mean, window + rows)
        seen = min(mean - rows / 2, window)
        return {"bytes": int(2 * held * keys + 8 * b * rows * h * hd), "flops": int(4 * b * rows * seen * h * hd)}
    e = 4 if case["out"] == "f32" else 2
    back = 2 * mean * (held + b * hk * hd * e)
    if case["op"] == "read":
        return {"bytes": int(back), "flops": int(2 * b * mean * hk * hd)}
    return {"bytes": int(back + rows * (b * hd * 4 * (2 * h + 2 * hk) + 2 * held)),
            "flops": int(2 * b * mean * hk * hd + b * rows * hd * (3 * (h + hk) + 6 * hk))}


# ------------------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed), case)


def _turned(x, pos, s, c):
    """Pairs as complex numbers, turned by unit ones (held in f32, as the definition says)."""
    a = pos.double()[:, None] * s["freq"]
    z = torch.complex((s["magnitude"] * torch.cos(a)).float().double(), (s["magnitude"] * torch.sin(a)).float().double())
    r, x = c["rot"], x.double()
    if c["pairing"] == "half":
        y = torch.complex(x[..., : r // 2].contiguous(), x[..., r // 2 : r].contiguous()) * z[:, None]
        y = torch.cat([y.real, y.imag], -1)
    else:
        y = torch.view_as_real(torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2)) * z[:, None]).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _exact_rope(s, c):
    return _turned(s["x"], s["pos"], s, c)


def _sequence(s, c, i, n):
    """Positions 0..n of sequence i: codes [kv head][n][hd], scales [kv head][n] of keys and values, 64 bits."""
    pages = s["table"][i, : -(-n // c["page"])].long()
    got = []
    for x in "kv":
        codes = s[x + "_pages"][pages].double().transpose(0, 1).reshape(c["kv_heads"], -1, c["hd"])[:, :n]
        scale = s[x + "_scale"][pages].double().transpose(0, 1).reshape(c["kv_heads"], -1)
        got += [codes, scale.repeat_interleave(BLOCK, 1)[:, :n]]
    return got


def _exact_read(s, c):
    out = [s["k_out"].double(), s["v_out"].double()]
    for i, n in enumerate(s["len"].tolist()):
        k, ks, v, vs = _sequence(s, c, i, n)
        out[0][i, :, :n], out[1][i, :, :n] = k * ks[..., None], v * vs[..., None]
    return tuple(out)


def _nearest(x, fmt):
    """The code of each value, by counting steps in 64 bits."""
    if fmt == "i8":
        return torch.sign(x) * torch.floor(x.abs() + 0.5).clamp(max=127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0**-6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s, c):
    """Block by block, the new rows in the order of their positions."""
    h, hk = c["heads"], c["kv_heads"]
    q = s["q_out"].double()
    out = [s["k_out"].double(), s["v_out"].double()]
    start = s["row_start"].tolist()
    for i, (p0, n) in enumerate(zip(s["pos"].tolist(), s["len"].tolist())):
        x = s["qkv"][start[i] : start[i + 1]]
        qk = _turned(x[:, : h + hk], torch.arange(p0, n, device="cuda"), s, c)
        q[start[i] : start[i + 1]] = qk[:, :h]
        parts = _sequence(s, c, i, n)
        for which, rows in ((0, qk[:, h:].float()), (1, x[:, h + hk :])):
            codes, scale = parts[2 * which], parts[2 * which + 1]
            for lo in range(p0 // BLOCK * BLOCK, n, BLOCK):
                a, z = max(lo, p0), min(lo + BLOCK, n)
                new = rows[a - p0 : z - p0].transpose(0, 1)  # [kv head][rows][hd]
                was = scale[:, lo].float() if a > lo else torch.zeros(hk, device="cuda")
                now = torch.maximum(was, (new.abs().amax((1, 2)).double() / TOP[c["fmt"]]).float())
                if a > lo:
                    old = (codes[:, lo:a].float() * was[:, None, None]) / now[:, None, None]
                    grows = (now > was)[:, None, None]
                    codes[:, lo:a] = torch.where(grows, _nearest(old.double(), c["fmt"]), codes[:, lo:a])
                codes[:, a:z] = _nearest((new / now[:, None, None]).double(), c["fmt"])
                scale[:, lo:z] = now.double()[:, None]
            out[which][i, :, :n] = codes * scale[..., None]
    return (q, *out)


def _exact_attn(s, c):
    """Each sequence by itself, its keys and values in 64 bits."""
    out = s["out"].double()
    start, group = s["row_start"].tolist(), c["heads"] // c["kv_heads"]
    for i, (p0, n) in enumerate(zip(s["pos"].tolist(), s["len"].tolist())):
        k, ks, v, vs = _sequence(s, c, i, n)
        last = torch.arange(p0, n, device="cuda")[:, None]
        at = torch.arange(n, device="cuda")
        hidden = at > last
        if c["window"]:
            hidden |= at <= last - c["window"]
        for h in range(c["heads"]):
            a = s["q"][start[i] : start[i + 1], h].double() @ k[h // group].t() * ks[h // group] / math.sqrt(c["hd"])
            w = torch.softmax(a.masked_fill(hidden, -math.inf), dim=1)
            out[start[i] : start[i + 1], h] = (w * vs[h // group]) @ v[h // group]
    return out


_EXACT = dict(attn=_exact_attn, append=_exact_append, read=_exact_read, rope=_exact_rope)
