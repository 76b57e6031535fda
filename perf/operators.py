"""Measured cases of the operators that verify a tree of drafted tokens in one pass.

A draft proposes, for each sequence, a tree of up to 64 tokens: node 0 is the last token that
was sampled, every other node continues its parent.  One pass of the model then runs all the
nodes: `tree_append` rotates the nodes' queries and keys and lays keys and values out in draft
buffers, `tree_attn` lets every node attend to the cached context and to its own ancestors,
`token_logprobs` scores the drafted tokens in the nodes' logits and names the alternatives, and
`tree_commit` walks the accepted path and copies its rows into the cache.

`run` computes each operator in elementary torch operations where `own` is false, and through
quantized_decode_gemv_gb300 where it is true.  Head layouts, cache types, context and vocabulary
are those of the models here (9 heads over 3, 32 over 32, head dimension 64, vocabulary 49152,
context 4096), with grouped layouts up to 8 heads to a key head and longer contexts beside them.
"""
import math

import numpy as np
import torch

own = False

HEAD_DIM = 64
LOG2_64 = 0.125  # 1 / sqrt(64)


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence of the 135M shape with a small tree early in its context: latency
        dict(name="attn_135m_t8_ctx100", op="attn", heads=9, kv_heads=3, batch=1, nodes=8, ctx=256, longest=100,
             ragged=False, kv_f16=False),
        # the 1.7B shape, one sequence near the end of its 4096 positions, f32 cache
        dict(name="attn_1p7b_t16_ctx4080", op="attn", heads=32, kv_heads=32, batch=1, nodes=16, ctx=4096,
             longest=4080, ragged=False, kv_f16=False),
        # the 1.7B shape with 16 sequences of different lengths and a binary16 cache: served load
        dict(name="attn_1p7b_b16_f16", op="attn", heads=32, kv_heads=32, batch=16, nodes=16, ctx=4096, longest=4095,
             ragged=True, kv_f16=True),
        # grouped heads, the widest tree over a long document
        dict(name="attn_gqa4_t64_ctx32k", op="attn", heads=32, kv_heads=8, batch=1, nodes=64, ctx=32768,
             longest=32700, ragged=False, kv_f16=True),
        # one key head for eight query heads, an odd tree, ragged lengths with an empty context among them
        dict(name="attn_g8_t27_ragged", op="attn", heads=8, kv_heads=1, batch=5, nodes=27, ctx=3001, longest=3001,
             ragged=True, kv_f16=False),
        # sampling: one row of logits, its token and the top 8
        dict(name="logprobs_1row", op="logprobs", rows=1, vocab=49152, tokens=1, top=8, masked=0.0),
        # the children of 37 tree nodes over an odd vocabulary, half of it ruled out by a grammar
        dict(name="logprobs_37rows_odd_masked", op="logprobs", rows=37, vocab=50257, tokens=4, top=20, masked=0.5),
        # scoring of a 2048-token prompt
        dict(name="logprobs_2048rows", op="logprobs", rows=2048, vocab=49152, tokens=1, top=5, masked=0.0),
        # one small tree of the 135M shape: latency
        dict(name="append_135m_t8", op="append", heads=9, kv_heads=3, batch=1, nodes=8, ctx=2048, kv_f16=False,
             pairing="half", ragged=False),
        # 16 sequences of the 1.7B shape with the widest tree
        dict(name="append_1p7b_b16_t64", op="append", heads=32, kv_heads=32, batch=16, nodes=64, ctx=4096, kv_f16=True,
             pairing="adjacent", ragged=True),
        # the 135M shape's 30 layers, one sequence
        dict(name="commit_135m_t16", op="commit", layers=30, kv_heads=3, batch=1, nodes=16, ctx=256, kv_f16=False,
             match=0.8),
        # the 1.7B shape's 24 layers, eight sequences, a short cache so that whole caches can be compared
        dict(name="commit_1p7b_b8_t32", op="commit", layers=24, kv_heads=32, batch=8, nodes=32, ctx=96, kv_f16=True,
             match=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "logprobs", "logprobs", "append", "commit"])
    most = {}
    for c in listed():
        w = work(c)
        for k in ("bytes", "flops"):
            most[k] = max(most.get(k, 0), w[k] if c["op"] == op else 0)
    while True:
        heads, kv_heads = rng.choice([(9, 3), (32, 32), (32, 8), (8, 1), (6, 2), (5, 5)])
        nodes = _log(rng, 1, 64)
        batch = rng.randint(1, 16)
        if op == "attn":
            ctx = _log(rng, 17, 32768)
            case = dict(op=op, heads=heads, kv_heads=kv_heads, batch=batch, nodes=nodes, ctx=ctx,
                        longest=rng.randint(ctx // 2, ctx), ragged=rng.random() < 0.6, kv_f16=rng.random() < 0.5)
        elif op == "logprobs":
            case = dict(op=op, rows=_log(rng, 1, 2048), vocab=_log(rng, 300, 152000), tokens=rng.randint(1, 8),
                        top=rng.randint(0, 32), masked=rng.choice([0.0, 0.0, 0.5, 0.99]))
        elif op == "append":
            case = dict(op=op, heads=heads, kv_heads=kv_heads, batch=batch, nodes=nodes, ctx=_log(rng, 128, 4096),
                        kv_f16=rng.random() < 0.5, pairing=rng.choice(["half", "adjacent"]),
                        ragged=rng.random() < 0.6)
        else:
            case = dict(op=op, layers=rng.randint(1, 30), kv_heads=kv_heads, batch=batch, nodes=nodes,
                        ctx=rng.randint(nodes + 1, 256), kv_f16=rng.random() < 0.5, match=rng.uniform(0.3, 1.0))
        w = work(case)
        cache = 2 * case.get("layers", 0) * batch * kv_heads * case.get("ctx", 0) * HEAD_DIM * 4
        if all(w[k] <= most[k] for k in most) and cache <= 512 << 20:
            return case


def _shape(case):
    return {k: v for k, v in case.items() if k != "name"}


def _lengths(case, rng):
    """Positions that each sequence holds, and its number of nodes."""
    b, n = case["batch"], case["nodes"]
    if case["op"] == "attn":
        top = case["longest"]
    else:
        top = case["ctx"] - n
    if not case.get("ragged", case["op"] == "commit"):
        return np.full(b, top, np.int32), np.full(b, n, np.int32)
    pos = rng.integers(0, top + 1, b).astype(np.int32)
    cnt = rng.integers(max(1, n // 2), n + 1, b).astype(np.int32)
    pos[0], cnt[0] = top, n
    if b > 2:
        pos[1] = 0
    return pos, cnt


def _trees(n, batch, rng):
    """parent [batch][n] (parent[c] < c), depth, and every node's set of ancestors and itself as bits."""
    parent = np.zeros((batch, n), np.int32)
    depth = np.zeros((batch, n), np.int32)
    mask = np.zeros((batch, n), np.uint64)
    for b in range(batch):
        parent[b, 0] = -1
        mask[b, 0] = 1
        for c in range(1, n):
            # drafts are deeper than they are wide: a recent node is the likelier parent
            p = max(0, c - 1 - int(rng.geometric(0.45) - 1))
            parent[b, c] = p
            depth[b, c] = depth[b, p] + 1
            mask[b, c] = mask[b, p] | np.uint64(1 << c)
    return parent, depth, mask


def _rope_table(theta, ctx):
    a = np.arange(ctx)[:, None] * theta ** (-2.0 * np.arange(HEAD_DIM // 2) / HEAD_DIM)[None, :]
    return np.stack([np.cos(a), np.sin(a)], axis=-1).astype(np.float32)


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    rng = np.random.default_rng([seed, 11])
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    normal = lambda *s, scale=1.0: torch.randn(*s, generator=g, device="cuda") * scale  # noqa: E731
    s = dict(case=_shape(case))
    if case["op"] == "logprobs":
        rows, v = case["rows"], case["vocab"]
        # logits of a trained head: a wide bulk and a few tokens far above it
        x = normal(rows, v, scale=2.0)
        hot = torch.randint(0, v, (rows, 12), generator=g, device="cuda")
        x.scatter_add_(1, hot, 6.0 + normal(rows, 12, scale=3.0))
        if case["masked"]:
            ruled_out = torch.rand(rows, v, generator=g, device="cuda") < case["masked"]
            x.masked_fill_(ruled_out, -math.inf)
            x[:, v // 2] = 1.0  # a grammar leaves one token at least
        s["logits"] = x
        t = torch.randint(0, v, (rows, case["tokens"]), generator=g, device="cuda", dtype=torch.int32)
        t[:, 0] = hot[:, 0]
        s["tokens"] = t
        f32 = dict(dtype=torch.float32, device="cuda")
        s["logprob"] = torch.empty(rows, case["tokens"], **f32)
        s["entropy"] = torch.empty(rows, **f32)
        s["top_idx"] = torch.empty(rows, case["top"], dtype=torch.int32, device="cuda")
        s["top_logprob"] = torch.empty(rows, case["top"], **f32)
        return s

    n, b, hk = case["nodes"], case["batch"], case["kv_heads"]
    pos, cnt = _lengths(case, rng)
    parent, depth, mask = _trees(n, b, rng)
    s["pos"], s["count"] = dev(pos), dev(cnt)
    s["parent"], s["depth"], s["mask"] = dev(parent), dev(depth), dev(mask.view(np.int64))
    kv = torch.float16 if case["kv_f16"] else torch.float32
    if case["op"] == "attn":
        h = case["heads"]
        s["q"] = normal(b, n, h, HEAD_DIM, scale=1.5)
        s["k"] = normal(b, hk, case["ctx"], HEAD_DIM).to(kv)
        s["v"] = normal(b, hk, case["ctx"], HEAD_DIM).to(kv)
        s["k_draft"] = normal(b, hk, n, HEAD_DIM).to(kv)
        s["v_draft"] = normal(b, hk, n, HEAD_DIM).to(kv)
        s["out"] = torch.zeros(b, n, h, HEAD_DIM, device="cuda")
    elif case["op"] == "append":
        h = case["heads"]
        s["qkv"] = normal(b, n, h + 2 * hk, HEAD_DIM)  # the rows of the fused projection
        s["table"] = dev(_rope_table(1e4, case["ctx"]))
        s["q_out"] = torch.zeros(b, n, h, HEAD_DIM, device="cuda")
        s["k_draft"] = torch.zeros(b, hk, n, HEAD_DIM, dtype=kv, device="cuda")
        s["v_draft"] = torch.zeros(b, hk, n, HEAD_DIM, dtype=kv, device="cuda")
    else:
        la = case["layers"]
        tokens = rng.integers(0, 49152, (b, n)).astype(np.int32)
        chosen = rng.integers(0, 49152, (b, n)).astype(np.int32)
        for i in range(b):
            for c in range(n - 1, 0, -1):  # the model agrees with one of a node's children, more often than not
                if rng.random() < case["match"]:
                    chosen[i, parent[i, c]] = tokens[i, c]
        s["tokens"], s["chosen"] = dev(tokens), dev(chosen)
        s["k"] = normal(la, b, hk, case["ctx"], HEAD_DIM).to(kv)
        s["v"] = normal(la, b, hk, case["ctx"], HEAD_DIM).to(kv)
        s["k_draft"] = normal(la, b, hk, n, HEAD_DIM).to(kv)
        s["v_draft"] = normal(la, b, hk, n, HEAD_DIM).to(kv)
        s["path"] = torch.zeros(b, n, dtype=torch.int32, device="cuda")
        s["accepted"], s["next"], s["pos_out"] = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(3))
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        return _OWN[c["op"]](s, c)
    return _PLAIN[c["op"]](s, c)


def _bits(mask, n):
    """[batch][n][n]: whether node i sees node j."""
    return ((mask[..., None] >> torch.arange(n, device=mask.device)) & 1).bool()


def _plain_attn(s, c):
    b, n, h, hk, ctx = c["batch"], c["nodes"], c["heads"], c["kv_heads"], c["longest"]
    group = h // hk
    k = torch.cat([s["k"][:, :, :ctx], s["k_draft"]], dim=2).float()
    v = torch.cat([s["v"][:, :, :ctx], s["v_draft"]], dim=2).float()
    q = s["q"].reshape(b, n, hk, group, HEAD_DIM).permute(0, 2, 1, 3, 4).reshape(b, hk, n * group, HEAD_DIM)
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(LOG2_64).view(b, hk, n, group, ctx + n)
    cached = torch.arange(ctx, device="cuda") < s["pos"][:, None]
    sees = torch.cat([cached[:, None].expand(b, n, ctx), _bits(s["mask"], n)], dim=2)
    real = torch.arange(n, device="cuda") < s["count"][:, None]
    scores.masked_fill_(~sees[:, None, :, None], -math.inf)
    p = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, n * group, ctx + n), v).view(b, hk, n, group, HEAD_DIM) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(b, n, h, HEAD_DIM)
    return torch.where(real[:, :, None, None], o, s["out"])


def _plain_logprobs(s, c):
    x = s["logits"]
    m = x.amax(1, keepdim=True)
    d = x - m
    e = d.exp()
    total = e.sum(1, keepdim=True)
    lse = total.log()
    entropy = lse[:, 0] - torch.where(e > 0, e * d, 0.0).sum(1) / total[:, 0]
    logprob = d.gather(1, s["tokens"].long()) - lse
    # the largest values, the lowest index first among equal ones
    bits = x.view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = (order << 32) + (0xFFFFFFFF - torch.arange(c["vocab"], device="cuda"))
    idx = 0xFFFFFFFF - (key.topk(c["top"], dim=1).values & 0xFFFFFFFF)
    return logprob, entropy, idx.int(), d.gather(1, idx) - lse


def _plain_append(s, c):
    b, n, h, hk = c["batch"], c["nodes"], c["heads"], c["kv_heads"]
    cs = s["table"][(s["pos"][:, None] + s["depth"]).long()][:, :, None]  # [b][n][1][32][2]
    cos, sin = cs[..., 0], cs[..., 1]
    x = s["qkv"][:, :, : h + hk]
    if c["pairing"] == "half":
        x0, x1 = x[..., : HEAD_DIM // 2], x[..., HEAD_DIM // 2 :]
        y = torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], dim=-1)
    else:
        x0, x1 = x[..., 0::2], x[..., 1::2]
        y = torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], dim=-1).flatten(-2)
    real = (torch.arange(n, device="cuda") < s["count"][:, None])[:, :, None, None]
    q = torch.where(real, y[:, :, :h], s["q_out"])
    real = real.transpose(1, 2)
    k = torch.where(real, y[:, :, h:].transpose(1, 2).to(s["k_draft"].dtype), s["k_draft"])
    v = torch.where(real, s["qkv"][:, :, h + hk :].transpose(1, 2).to(s["v_draft"].dtype), s["v_draft"])
    return q, k, v


def _plain_commit(s, c):
    b, n = c["batch"], c["nodes"]
    at = torch.arange(n, device="cuda")
    parent, tokens = s["parent"].clamp(min=0).long(), s["tokens"]
    agrees = tokens == s["chosen"].gather(1, parent)
    twin = (parent[:, :, None] == parent[:, None]) & (tokens[:, :, None] == tokens[:, None])
    twin &= (at[None, :] < at[:, None]) & (at[None, :] > 0)  # an earlier child of the same node with the same token
    good = agrees & ~twin.any(2)
    good[:, 0] = True
    accepted = ~(_bits(s["mask"], n) & ~good[:, None]).any(2) & (at < s["count"][:, None])
    length = accepted.sum(1, dtype=torch.int32)
    order = torch.where(accepted, at, n).sort(1).values
    on = at < length[:, None]
    path = torch.where(on, order, -1).int()
    last = order.gather(1, (length - 1)[:, None].long())
    row = order.clamp(max=n - 1)
    dest = s["pos"][:, None].long() + at
    src = torch.arange(b, device="cuda")[:, None]
    for cache, draft in ((s["k"], s["k_draft"]), (s["v"], s["v_draft"])):
        keep = on[:, :, None, None, None]
        cache[:, src, :, dest] = torch.where(keep, draft[:, src, :, row], cache[:, src, :, dest])
    return path, length, s["chosen"].gather(1, last)[:, 0], s["pos"] + length, s["k"], s["v"]


_PLAIN = dict(attn=_plain_attn, logprobs=_plain_logprobs, append=_plain_append, commit=_plain_commit)


def _own_attn(s, c):
    import quantized_decode_gemv_gb300 as qd

    b, n, h, hk = c["batch"], c["nodes"], c["heads"], c["kv_heads"]
    if "ws" not in s:
        size = qd.tree_attn_workspace(h, hk, HEAD_DIM, n, c["ctx"], b)
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    qd.tree_attn(s["q"], n * h * HEAD_DIM, s["k"], s["v"], s["k_draft"], s["v_draft"], s["out"], h, hk, HEAD_DIM,
                 s["pos"], s["mask"], s["count"], n, c["ctx"], b, s["ws"], kv_f16=c["kv_f16"])
    return s["out"]


def _own_logprobs(s, c):
    import quantized_decode_gemv_gb300 as qd

    qd.token_logprobs(s["logits"], c["vocab"], c["vocab"], c["rows"], s["tokens"], c["tokens"], s["logprob"],
                      s["entropy"], c["top"], s["top_idx"], s["top_logprob"])
    return s["logprob"], s["entropy"], s["top_idx"], s["top_logprob"]


def _own_append(s, c):
    import quantized_decode_gemv_gb300 as qd

    b, n, h, hk = c["batch"], c["nodes"], c["heads"], c["kv_heads"]
    width = (h + 2 * hk) * HEAD_DIM
    qkv = s["qkv"]
    qd.tree_append(qkv, qkv[:, :, h:], qkv[:, :, h + hk :], n * width, width, s["q_out"], s["k_draft"], s["v_draft"],
                   h, hk, HEAD_DIM, s["pos"], s["depth"], s["count"], n, c["pairing"], s["table"], c["ctx"], b,
                   kv_f16=c["kv_f16"])
    return s["q_out"], s["k_draft"], s["v_draft"]


def _own_commit(s, c):
    import quantized_decode_gemv_gb300 as qd

    b, n, hk = c["batch"], c["nodes"], c["kv_heads"]
    qd.tree_commit(s["tokens"], s["parent"], s["chosen"], 1, s["count"], n, s["k_draft"], s["v_draft"], s["k"], s["v"],
                   c["layers"], b * hk * c["ctx"] * HEAD_DIM, hk, HEAD_DIM, s["pos"], c["ctx"], b, s["path"],
                   s["accepted"], s["next"], s["pos_out"], kv_f16=c["kv_f16"])
    return s["path"], s["accepted"], s["next"], s["pos_out"], s["k"], s["v"]


_OWN = dict(attn=_own_attn, logprobs=_own_logprobs, append=_own_append, commit=_own_commit)


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "logprobs":
        rows, v = case["rows"], case["vocab"]
        # a comparison, a subtraction, an exp, two sums and a product for each logit
        return {"bytes": 4 * rows * (v + 2 * case["tokens"] + 1 + 2 * case["top"]), "flops": 6 * rows * v}
    n, b, hk = case["nodes"], case["batch"], case["kv_heads"]
    e = 2 if case["kv_f16"] else 4
    # lengths of the ragged cases are drawn evenly from 0 to the longest and from half the nodes to all
    mean_pos = 0.5 if case.get("ragged") else 1.0
    mean_n = 0.75 if case.get("ragged") else 1.0
    if op == "attn":
        h, ctx = case["heads"], case["longest"] * mean_pos
        return {"bytes": int(b * (2 * hk * (ctx + n) * HEAD_DIM * e + 2 * 4 * n * mean_n * h * HEAD_DIM + 8 * n)),
                "flops": int(4 * b * h * n * mean_n * (ctx + n / 2) * HEAD_DIM)}
    if op == "append":
        h = case["heads"]
        return {"bytes": int(b * n * mean_n * HEAD_DIM * ((h + 2 * hk) * 4 + 4 * h + 2 * hk * e + 4)),
                "flops": int(b * n * mean_n * 3 * HEAD_DIM * (h + hk))}
    # the accepted path is a few nodes long; its rows are read once and written once
    path = min(n, 1 + 2 * math.log2(n + 1) * case["match"])
    return {"bytes": int(case["layers"] * b * hk * path * HEAD_DIM * e * 4 + 16 * b * n), "flops": int(b * n)}


# ------------------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed), case)


def _exact_attn(s, c):
    """Each sequence by itself: softmax over the cached positions and the node's ancestors."""
    group = c["heads"] // c["kv_heads"]
    out = s["out"].double()
    masks = s["mask"].cpu().numpy().view(np.uint64)
    for b, (pos, cnt) in enumerate(zip(s["pos"].tolist(), s["count"].tolist())):
        sees = torch.tensor([[bool(int(masks[b, i]) >> j & 1) for j in range(cnt)] for i in range(cnt)], device="cuda")
        for kvh in range(c["kv_heads"]):
            k = torch.cat([s["k"][b, kvh, :pos], s["k_draft"][b, kvh, :cnt]]).double()
            v = torch.cat([s["v"][b, kvh, :pos], s["v_draft"][b, kvh, :cnt]]).double()
            for h in range(kvh * group, (kvh + 1) * group):
                a = s["q"][b, :cnt, h].double() @ k.t() / math.sqrt(HEAD_DIM)
                a[:, pos:][~sees] = -math.inf
                w = torch.softmax(a, dim=1)
                out[b, :cnt, h] = w @ v
    return out


def _exact_logprobs(s, c):
    parts = [[], [], [], []]
    for r0 in range(0, c["rows"], 256):
        lp = torch.log_softmax(s["logits"][r0 : r0 + 256].double(), dim=1)
        idx = s["logits"][r0 : r0 + 256].sort(dim=1, descending=True, stable=True).indices[:, : c["top"]]
        parts[0].append(lp.gather(1, s["tokens"][r0 : r0 + 256].long()))
        parts[1].append(-torch.xlogy(lp.exp(), lp.exp()).sum(1))
        parts[2].append(idx.int())
        parts[3].append(lp.gather(1, idx))
    return tuple(torch.cat(p) for p in parts)


def _exact_append(s, c):
    """Pairs as complex numbers, turned by the table's angles."""
    h, hk, n = c["heads"], c["kv_heads"], c["nodes"]
    q, k, v = s["q_out"].double(), s["k_draft"].double(), s["v_draft"].double()
    x = s["qkv"].double()
    if c["pairing"] == "half":
        z = torch.complex(x[..., :32], x[..., 32:])
    else:
        z = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous())
    table = torch.view_as_complex(s["table"].double())
    for b, (pos, cnt) in enumerate(zip(s["pos"].tolist(), s["count"].tolist())):
        for i in range(cnt):
            t = z[b, i] * table[pos + int(s["depth"][b, i])]
            t = torch.cat([t.real, t.imag], -1) if c["pairing"] == "half" else torch.view_as_real(t).flatten(-2)
            q[b, i], k[b, :, i], v[b, :, i] = t[:h], t[h : h + hk], x[b, i, h + hk :]
    return q, k, v


def _exact_commit(s, c):
    """The walk from the root, child by child."""
    b, n = c["batch"], c["nodes"]
    tokens, parent, chosen = (s[k].tolist() for k in ("tokens", "parent", "chosen"))
    path = np.full((b, n), -1, np.int32)
    length, nxt = np.zeros(b, np.int32), np.zeros(b, np.int32)
    k, v = s["k"].double(), s["v"].double()
    for i, (pos, cnt) in enumerate(zip(s["pos"].tolist(), s["count"].tolist())):
        walk = [0]
        while True:
            at = walk[-1]
            on = [x for x in range(1, cnt) if parent[i][x] == at and tokens[i][x] == chosen[i][at]]
            if not on:
                break
            walk.append(on[0])
        path[i, : len(walk)] = walk
        length[i], nxt[i] = len(walk), chosen[i][walk[-1]]
        for j, node in enumerate(walk):
            k[:, i, :, pos + j] = s["k_draft"][:, i, :, node].double()
            v[:, i, :, pos + j] = s["v_draft"][:, i, :, node].double()
    t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return t(path), t(length), t(nxt), s["pos"] + t(length), k, v


_EXACT = dict(attn=_exact_attn, logprobs=_exact_logprobs, append=_exact_append, commit=_exact_commit)
