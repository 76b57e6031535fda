"""The paged 8-bit cache on the GPU against 64-bit references: rotation, append, attention, read
back, and a step's calls in a row."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import dev
from paged_helpers import BLOCK, Cache, attn_all, attn_ref, cos_sin, decode, rotate

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ helpers
def _plan(qd, rot, scaling="none", **more):
    turns, mag = qd.rope_plan(1e4, rot, scaling, **more)
    return turns.numpy().view(np.uint64), turns.cuda(), mag


def _handle(qd, c):
    """The cache on the device: (handle, its tensors by name)."""
    t = dict(k=dev(c.k.view(np.int8)), v=dev(c.v.view(np.int8)), ks=dev(c.ks), vs=dev(c.vs), table=dev(c.table))
    return qd.PagedKV(t["k"], t["v"], t["ks"], t["vs"], t["table"], fmt=c.fmt), t


def _starts(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def _near_f32(got, want, share):
    """Equal bits but for a share of values that are the neighbouring f32."""
    got, want = np.asarray(got, np.float32), np.asarray(want, np.float32)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    off = (got != want) & ~np.isnan(want)
    assert off.sum() <= 1 + share * off.size, f"{off.sum()} of {off.size} differ"
    up, down = np.nextafter(want, np.float32(np.inf)), np.nextafter(want, np.float32(-np.inf))
    assert np.all((got[off] == up[off]) | (got[off] == down[off]))


def _near_rotated(got, x, pos, turns, mag, rot, pairing):
    """Rotated rows within 4 * 2^-24 of |x0| + |x1| (times the magnitude): one product rounded, the fused step
    rounded, the reference rounded (each 2^-24 of at most that) and cos or sin the neighbouring f32 value (2^-24 of
    it, as values up to 1 have steps of 2^-24)."""
    want = rotate(x, cos_sin(turns, pos, mag), rot, pairing).astype(np.float64)
    off = np.abs(np.asarray(got, np.float64) - want)
    if pairing == "half":
        pair = np.abs(x[..., : rot // 2]) + np.abs(x[..., rot // 2 : rot])
        most = np.concatenate([pair, pair], -1)
    else:
        most = np.repeat(np.abs(x[..., 0:rot:2]) + np.abs(x[..., 1:rot:2]), 2, -1)
    assert np.array_equal(np.asarray(got)[..., rot:], x[..., rot:])
    assert np.all(off[..., :rot] <= 4 * 2.0**-24 * most * max(mag, 1.0))


# ------------------------------------------------------------------ angles and rotation
@pytest.mark.parametrize("scaling,more", [
    ("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
    ("turns", dict(factor=8.0, trained_ctx=4096, low=1.0, high=4.0)),
    ("pairs", dict(factor=16.0, trained_ctx=4096, low=1.0, high=32.0))])
def test_angles_are_the_rounded_exact_ones(qd, scaling, more):
    """Heads of ones and zeros give (cos, sin) themselves, at any position an int32 holds.  The series is
    within 2^-43 (its terms are to 2^-45 and a handful of operations follow), so one value in 2^18 may round
    to its neighbour."""
    rot = 128
    turns, d_turns, mag = _plan(qd, rot, scaling, **more)
    rng = np.random.default_rng(5)
    pos = np.concatenate([np.arange(40), [4095, 99999, 2**24 + 1, 2**31 - 1], rng.integers(0, 2**31, 120),
                          rng.integers(0, 2**17, 120)]).astype(np.int32)
    x = np.zeros((len(pos), 1, rot), np.float32)
    x[..., 0::2] = 1
    out = torch.zeros(len(pos), 1, rot, device="cuda")
    qd.rope_tokens(dev(x), rot, out, rot, len(pos), 1, rot, rot, dev(pos), "adjacent", d_turns, mag)
    c, s = cos_sin(turns, pos, mag)
    got = out.cpu().numpy()[:, 0]
    _near_f32(got[:, 0::2], c, 2.0**-17)
    _near_f32(got[:, 1::2], s, 2.0**-17)


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("n,heads,hd,rot", [(1, 1, 8, 8), (1, 12, 64, 64), (3, 5, 64, 16), (37, 3, 96, 48), (300, 2, 128, 120),
                                            (2, 1, 1024, 1024), (5, 40, 128, 128), (700, 12, 64, 32)])
def test_rope_tokens(qd, pairing, n, heads, hd, rot):
    rng = np.random.default_rng([n, heads, hd, rot])
    turns, d_turns, mag = _plan(qd, rot, "pairs", factor=8.0, trained_ctx=4096)
    x = rng.normal(size=(n, heads, hd)).astype(np.float32)
    pos = rng.integers(0, 40000, n).astype(np.int32)
    if n > 2:
        pos[1] = -1  # a padded row
    gap = 4 * (n % 3)
    wide = torch.full((n, heads * hd + gap), 7.0, device="cuda")
    wide[:, : heads * hd] = dev(x).view(n, -1)
    out = torch.full((n, heads, hd), 5.0, device="cuda")
    d_pos = dev(pos)
    qd.rope_tokens(wide, heads * hd + gap, out, heads * hd, n, heads, hd, rot, d_pos, pairing, d_turns, mag)
    got, live = out.cpu().numpy(), pos >= 0
    assert np.all(got[~live] == 5.0)
    _near_rotated(got[live], x[live], pos[live], turns, mag, rot, pairing)
    # in place: the same bits, the padded row and the gap as they were
    qd.rope_tokens(wide, heads * hd + gap, wide, heads * hd + gap, n, heads, hd, rot, d_pos, pairing, d_turns, mag)
    live = dev(live)
    assert torch.equal(wide[:, : heads * hd].reshape(n, heads, hd)[live], out[live])
    assert torch.equal(wide[~live][:, : heads * hd].reshape(-1, heads, hd), dev(x)[~live])
    assert torch.all(wide[:, heads * hd :] == 7.0)


def test_rope_tokens_infinities_stay_in_their_pair(qd):
    turns, d_turns, mag = _plan(qd, 64)
    x = np.random.default_rng(6).normal(size=(1, 2, 64)).astype(np.float32)
    y = x.copy()
    y[0, 0, 3], y[0, 1, 40] = np.inf, np.nan
    pos = np.array([1], np.int32)
    out = torch.zeros(1, 2, 64, device="cuda")
    qd.rope_tokens(dev(y), 128, out, 128, 1, 2, 64, 64, dev(pos), "half", d_turns, mag)
    got = out.cpu().numpy()
    assert np.isinf(got[0, 0, [3, 35]]).all() and np.isnan(got[0, 1, [8, 40]]).all()
    x[0, 0, [3, 35]] = x[0, 1, [8, 40]] = got[0, 0, [3, 35]] = got[0, 1, [8, 40]] = 0
    _near_rotated(got, x, pos, turns, mag, 64, "half")


# ------------------------------------------------------------------ append
def _append_case(qd, seed, heads, hk, hd, tokens, fmt, pos, rows, rot, pairing, width=None, change=None):
    """One append on the device and by the reference; returns (host cache after, device tensors, the arguments); the queries are checked here."""
    rng = np.random.default_rng([seed, hk, hd, tokens])
    pos = np.array(pos, np.int32)
    need = [max(int(p) + int(t), 0) if p >= 0 else 0 for p, t in zip(pos, rows)]
    if width:
        need = [min(n, width * tokens) for n in need]
    c = Cache(rng, len(pos), hk, hd, tokens, need, fmt, width)
    start = _starts(rows)
    n = int(start[-1])
    spare = 2  # rows behind the last sequence
    x = rng.normal(size=(n + spare, heads + 2 * hk, hd)).astype(np.float32)
    x[:, heads : heads + hk, ::13] *= 5
    if change:
        change(c, x)
    turns, d_turns, mag = _plan(qd, rot, "linear", factor=3.0)
    kv, t = _handle(qd, c)
    q_out = torch.full((n + spare, heads, hd), 9.0, device="cuda")
    d = dev(x)
    stride = (heads + 2 * hk) * hd
    args = (kv, d, d[:, heads:], d[:, heads + hk :], stride, q_out, heads, n + spare, dev(start), dev(pos), len(pos), rot,
            pairing, d_turns, mag)
    qd.paged_append(*args)
    q = []  # rows, queries and positions that are rotated
    cap = c.width * tokens
    for b, p in enumerate(pos):
        if p < 0 or p > cap or not rows[b]:
            continue
        r = slice(start[b], start[b + 1])
        at = np.arange(p, p + rows[b])
        y = rotate(x[r, : heads + hk], cos_sin(turns, at, mag), rot, pairing)
        q.append((r, x[r, :heads], at))
        if p < cap:
            c.put(b, int(p), y[:, heads:], x[r, heads + hk :])
    got, left = q_out.cpu().numpy(), np.ones(n + spare, bool)
    for r, rows_q, at in q:
        _near_rotated(got[r], rows_q, at, turns, mag, rot, pairing)
        left[r] = False
    assert np.all(got[left] == 9.0)
    return c, t, args


def _same_cache(t, c):
    """Codes and scales bit for bit, over the whole pool."""
    for name, want in (("k", c.k), ("v", c.v)):
        got = t[name].cpu().numpy().view(np.uint8)
        assert np.array_equal(decode(got, c.fmt), decode(want, c.fmt), equal_nan=True), name
    for name, want in (("ks", c.ks), ("vs", c.vs)):
        assert np.array_equal(t[name].cpu().numpy(), want, equal_nan=True), name


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("heads,hk,hd,tokens,pos,rows,rot,pairing", [
    (1, 1, 64, 16, [0], [1], 64, "half"),
    (9, 3, 64, 16, [5, 16, 0, 31, 47], [1, 1, 1, 1, 1], 32, "adjacent"),
    (4, 4, 128, 64, [0, 63, 17], [100, 1, 33], 128, "half"),
    (8, 1, 128, 48, [13, 0, 95, 0], [3, 0, 50, 16], 64, "adjacent"),  # an empty sequence, pages of no power of two
    (6, 2, 64, 1024, [1023, 0], [2, 15], 8, "half"),
    (32, 32, 64, 32, [100, 7, 0], [17, 31, 1], 64, "adjacent"),
    (16, 1, 64, 16, [0], [500], 64, "half"),
    (5, 5, 64, 16, list(range(70)), [1] * 70, 16, "half"),  # more sequences than lanes
])
def test_append(qd, fmt, heads, hk, hd, tokens, pos, rows, rot, pairing):
    c, t, args = _append_case(qd, 1, heads, hk, hd, tokens, fmt, pos, rows, rot, pairing)
    _same_cache(t, c)
    qd.paged_append(*args)  # the same call again stores the same values
    _same_cache(t, c)


def test_append_256_sequences(qd):
    pos = [(37 * b) % 50 for b in range(256)]
    c, t, _ = _append_case(qd, 2, 2, 2, 64, 16, "i8", pos, [(b * 7) % 4 for b in range(256)], 64, "half")
    _same_cache(t, c)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_append_positions_and_pages_out_of_range(qd, fmt):
    """A negative position, one behind the table, one that runs out of it in the middle, and entries that are
    no pages: nothing else changes."""
    def change(c, x):
        c.table[3, 1], c.table[4, 0] = len(c.k), -5

    c, t, _ = _append_case(qd, 3, 4, 2, 64, 16, fmt, [-1, 1000, 40, 10, 3, 48], [3, 3, 20, 30, 4, 2], 64, "half",
                                     width=3, change=change)
    _same_cache(t, c)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_append_values_at_the_edges(qd, fmt):
    """Zeros, subnormal and huge values, and values that are not finite: their block's scale is NaN until it
    starts anew, and no other block's."""
    def change(c, x):
        x[0:16, 4:] = 0.0                      # sequence 0: a block of zeros
        x[16:32, 4:] *= np.float32(2.0**-140)  # and one of subnormal values
        x[32:40, 4:] *= np.float32(1e38) / 30
        x[40, 4, 7] = np.inf                   # sequence 1: head 0's keys
        x[42, 6, 0] = np.nan                   # head 0's values
        x[60, 7, 63] = -np.inf                 # a later block, head 1's values
        c.ks[c.table[2, 0], 1, 0] = np.nan     # sequence 2: head 1 was broken before

    c, t, _ = _append_case(qd, 4, 4, 2, 64, 32, fmt, [0, 3, 5], [40, 40, 3], 64, "adjacent", change=change)
    _same_cache(t, c)
    assert np.isnan(c.ks).sum() == 2 and np.isnan(c.vs).sum() == 2 and (c.ks == 0).sum() == 2


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("hd,rot", [(64, 8), (64, 24), (64, 40), (64, 64), (128, 24), (128, 120), (128, 128)])
@pytest.mark.parametrize("tiny", [0, 1])
def test_append_where_the_lanes_of_a_row_part(qd, fmt, hd, rot, tiny):
    """Pairs (i, i + rot / 2): the two lanes of a row read each other's rotated values for their codes.  Here one of them
    has the tiny values, whose rotation takes longer, and the numbers of rotated units differ."""
    def change(c, x):
        i = np.arange(rot // 2)
        i = i[(i // 4) % 2 == tiny]
        x[:, 4:6, np.concatenate([i, i + rot // 2])] *= np.float32(2.0**-90)  # keys

    c, t, args = _append_case(qd, 6, 4, 2, hd, 32, fmt, [0, 5, 16, 31], [40, 3, 16, 1], rot, "half", change=change)
    _same_cache(t, c)
    for _ in range(20):
        qd.paged_append(*args)
    _same_cache(t, c)


@pytest.mark.parametrize("fmt,hd", [("i8", 64), ("e4m3", 128)])
def test_append_one_position_at_a_time(qd, fmt, hd):
    """40 steps of one token: the codes of the step by step reference, so no growing scale loses a code."""
    rng = np.random.default_rng(8)
    hk, c = 3, Cache(np.random.default_rng(9), 2, 3, hd, 32, [60, 45], fmt)
    turns, d_turns, mag = _plan(qd, hd)
    kv, t = _handle(qd, c)
    start = dev(_starts([1, 1]))
    for i in range(40):
        x = (rng.normal(size=(2, 2 * hk, hd)) * (1 + i % 16)).astype(np.float32)
        pos = np.array([20 + i, i], np.int32)
        d = dev(x)
        qd.paged_append(kv, None, d, d[:, hk:], 2 * hk * hd, None, 0, 2, start, dev(pos), 2, hd, "half", d_turns, mag)
        for b in range(2):
            c.put(b, int(pos[b]), rotate(x[b : b + 1, :hk], cos_sin(turns, pos[b : b + 1], mag), hd, "half"), x[b : b + 1, hk:])
    _same_cache(t, c)


# ------------------------------------------------------------------ read back
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("hk,hd,tokens,lens,ctx", [(1, 64, 16, [1], 1), (3, 64, 16, [200, 0, 17], 250), (2, 128, 48, [100, 333], 333),
                                                   (5, 64, 1024, [1500], 1400), (8, 128, 32, [65] * 20, 100)])
def test_read(qd, fmt, f16, hk, hd, tokens, lens, ctx):
    rng = np.random.default_rng([hk, hd, tokens])
    c = Cache(rng, len(lens), hk, hd, tokens, lens, fmt)
    c.ks[c.table[0, 0], 0, 0] = np.nan
    kv, _ = _handle(qd, c)
    kind = torch.float16 if f16 else torch.float32
    k, v = (torch.full((len(lens), hk, ctx, hd), 3.0, dtype=kind, device="cuda") for _ in range(2))
    qd.paged_read(kv, dev(np.array(lens, np.int32)), len(lens), ctx, k, v, out_f16=f16)
    want = np.full((2, len(lens), hk, ctx, hd), 3.0, np.float32)
    for b, n in enumerate(lens):
        for h in range(hk):
            ck, sk, cv, sv = c.values(b, h, n)
            m = min(n, ctx)
            want[0, b, h, :m], want[1, b, h, :m] = (ck * sk[:, None])[:m], (cv * sv[:, None])[:m]
    if f16:
        want = want.astype(np.float16)
    assert np.array_equal(k.cpu().numpy(), want[0], equal_nan=True) and np.array_equal(v.cpu().numpy(), want[1])


def test_read_without_pages(qd):
    c = Cache(np.random.default_rng(1), 2, 2, 64, 16, [40, 20], "i8")
    c.table[0, 1], c.table[1, 0] = -1, len(c.k)
    kv, _ = _handle(qd, c)
    k, v = (torch.full((2, 2, 60, 64), 3.0, device="cuda") for _ in range(2))
    qd.paged_read(kv, dev(np.array([40, -3], np.int32)), 2, 60, k, v)
    for x in (k, v):
        assert x[0, :, 16:32].isnan().all() and x[0, :, :16].isfinite().all() and x[0, :, 32:40].isfinite().all()
        assert (x[0, :, 40:] == 3).all() and (x[1] == 3).all()
    qd.paged_read(kv, dev(np.array([1000, 20], np.int32)), 2, 60, k, v)  # more than the table holds: 3 pages
    assert k[0, :, 32:48].isfinite().all() and (k[0, :, 48:] == 3).all() and k[1, :, :16].isnan().all()


# ------------------------------------------------------------------ attention
def _attn(qd, kv, q, start, pos, n_heads, scale, window, out=None, ws=None, stride=None, n=None):
    n = len(q) if n is None else n
    out = torch.full((n, n_heads, kv.head_dim), 9.0, device="cuda") if out is None else out
    if ws is None:
        ws = torch.empty(qd.paged_attn_workspace(kv, n_heads, n, len(pos)), dtype=torch.uint8, device="cuda")
    qd.paged_attn(kv, q, stride or n_heads * kv.head_dim, out, n_heads, n, start, pos, len(pos), scale, window, ws)
    return out


def _check(got, ref, tol):
    got = got.cpu().numpy().astype(np.float64)
    none = np.isnan(ref).all((1, 2))
    assert np.all(got[none] == 9.0)
    off, tol = np.abs(got - ref)[~none], tol[~none]
    assert np.all(off[tol == 0] == 0)  # one position whose code is zero
    worst = np.max(off[tol > 0] / tol[tol > 0], initial=0.0)
    assert worst <= 1.0, f"{worst:.2f} of the bound"
    return worst


SHAPES = [
    # heads, hk, hd, tokens, total positions, rows, window
    (1, 1, 64, 16, [1], [1], 0),
    (9, 3, 64, 16, [200], [1], 0),
    (9, 3, 64, 16, [15, 16, 17, 1, 33, 2], [1, 1, 1, 1, 1, 1], 0),
    (32, 32, 64, 64, [300, 5, 700], [1, 1, 1], 0),
    (32, 8, 128, 32, [500, 129, 64], [1, 1, 1], 0),
    (40, 8, 128, 64, [333, 1000], [1, 1], 100),
    (16, 1, 64, 16, [100, 47], [1, 2], 0),
    (16, 1, 128, 48, [500], [9], 17),
    (8, 1, 64, 16, [1100, 40, 200, 7, 64], [1, 40, 0, 7, 13], 0),
    (8, 1, 64, 16, [1100, 40, 200, 7, 64], [1, 40, 0, 7, 13], 1),
    (8, 2, 128, 1024, [1500, 300], [33, 64], 16),
    (6, 2, 64, 16, [129, 128, 127], [129, 128, 127], 0),
    (5, 5, 64, 32, [400], [300], 0),
    (4, 1, 128, 64, [700], [257], 250),
    (12, 3, 64, 16, [2500], [140], 0),
    (2, 2, 128, 16, [3000, 2], [2, 1], 5000),
    (4, 2, 64, 16, [300, 90], [70, 2], 2**31 - 1),
    # no more rows than sequences: blocks of 8, though a sequence has several
    (8, 2, 64, 16, [100, 20, 50], [3, 0, 0], 0),
    (32, 8, 128, 32, [200, 7, 90, 300], [0, 4, 0, 0], 5),
    (24, 8, 64, 48, [1000, 31, 32, 33, 500], [1, 0, 2, 1, 1], 40),
    (8, 1, 128, 16, [700, 64], [1, 1], 0),
]


WIDE = 1 << 22  # positions that a table has room for: with many rows, the work that it allows takes blocks of 128


@pytest.mark.parametrize("room", [None, WIDE])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("heads,hk,hd,tokens,total,rows,window", SHAPES)
def test_attention(qd, fmt, heads, hk, hd, tokens, total, rows, window, room):
    if room and max(rows) * heads // hk <= 48:
        pytest.skip("few rows take the same kernel whatever the room")
    rng = np.random.default_rng([heads, hd, tokens, len(total), total[0]])
    c = Cache(rng, len(total), hk, hd, tokens, total, fmt, width=room and room // tokens)
    kv, _ = _handle(qd, c)
    start = _starts(rows)
    pos = np.array(total, np.int32) - np.array(rows, np.int32)
    n = int(start[-1])
    gap = 8
    q = (rng.normal(size=(n + 3, heads, hd)) * 1.5).astype(np.float32)
    wide = torch.zeros(n + 3, heads * hd + gap, device="cuda")
    wide[:, : heads * hd] = dev(q).view(n + 3, -1)
    scale = 1 / math.sqrt(hd)
    got = _attn(qd, kv, wide, dev(start), dev(pos), heads, scale, window, stride=heads * hd + gap)
    ref, tol = attn_all(c, q, start, pos, heads // hk, scale, window)
    _check(got, ref, tol)
    again = _attn(qd, kv, wide, dev(start), dev(pos), heads, scale, window, stride=heads * hd + gap)
    assert torch.equal(got, again)
    # without rows behind the last sequence: blocks of 8 where no more rows than sequences are left
    _check(_attn(qd, kv, wide[:n], dev(start), dev(pos), heads, scale, window, stride=heads * hd + gap), ref[:n], tol[:n])


@pytest.mark.parametrize("heads,hk,hd,total,rows", [(12, 3, 64, [2500], [140]), (32, 8, 128, [1500] * 9, [1] * 9),
                                                    (16, 1, 128, [3000, 500], [30, 3]), (9, 3, 64, [900] * 20, [1] * 20),
                                                    (8, 2, 128, [700, 90, 1300], [600, 1, 900]),
                                                    (32, 32, 64, [400], [300])])
@pytest.mark.parametrize("room", [None, WIDE])
def test_attention_gives_the_same_bits_every_time(qd, heads, hk, hd, total, rows, room):
    """Walks that are cut, and CTAs that go from one to the next: 100 runs, so that warps that run ahead show."""
    rng = np.random.default_rng([25, heads, hd])
    c = Cache(rng, len(total), hk, hd, 32, total, "i8", width=room and room // 32)
    kv, _ = _handle(qd, c)
    start, pos = _starts(rows), np.array(total, np.int32) - np.array(rows, np.int32)
    q = dev((rng.normal(size=(int(start[-1]), heads, hd)) * 1.5).astype(np.float32))
    d_start, d_pos = dev(start), dev(pos)
    outs = [_attn(qd, kv, q, d_start, d_pos, heads, 0.1, 0) for _ in range(100)]
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_attention_of_many_sequences(qd):
    rng = np.random.default_rng(12)
    total = [1 + (b * 29) % 150 for b in range(256)]
    c = Cache(rng, 256, 2, 64, 16, total, "i8")
    kv, _ = _handle(qd, c)
    rows = [1 if b % 5 else min(3, total[b]) for b in range(256)]
    rows[7] = rows[255] = 0
    start, pos = _starts(rows), np.array(total, np.int32) - np.array(rows, np.int32)
    q = rng.normal(size=(int(start[-1]), 4, 64)).astype(np.float32)
    got = _attn(qd, kv, dev(q), dev(start), dev(pos), 4, 0.125, 0)
    _check(got, *attn_all(c, q, start, pos, 2, 0.125, 0))


@pytest.mark.parametrize("hd,rows", [(64, 1), (128, 1), (64, 40), (128, 150), (64, 150)])
def test_attention_over_a_long_walk(qd, hd, rows):
    """20000 positions, some heads and rows of them checked; large scores, and scales of different size."""
    rng = np.random.default_rng([13, hd, rows])
    c = Cache(rng, 1, 2, hd, 64, [20000], "i8")
    c.ks[:] = np.float32(0.02) * 4.0 ** rng.integers(-3, 2, c.ks.shape)
    c.vs[:] = np.float32(0.02) * 10.0 ** rng.integers(-6, 6, c.vs.shape)
    kv, _ = _handle(qd, c)
    q = (rng.normal(size=(rows, 8, hd)) * 2).astype(np.float32)
    start, pos = _starts([rows]), np.array([20000 - rows], np.int32)
    got = _attn(qd, kv, dev(q), dev(start), dev(pos), 8, 1 / math.sqrt(hd), 0).cpu().numpy()
    for r in sorted({0, rows // 2, rows - 1}):
        for h in (0, 5):
            o, tol = attn_ref(q[r, h], *c.values(0, h // 4, 20000), int(pos[0]) + r, 1 / math.sqrt(hd), 0)
            assert np.max(np.abs(got[r, h] - o) / tol) <= 1.0


UNEQUAL = [
    # heads, hk, hd, tokens, total positions, rows, window, room
    (1, 1, 64, 16, [200], [1], 0, None),
    (9, 3, 128, 16, [300, 33, 17], [1, 1, 1], 0, None),
    (8, 2, 64, 32, [3000], [1], 100, None),  # cut walks, whose warps see tiles of their own
    (16, 1, 128, 48, [500], [9], 17, None),
    (4, 2, 64, 64, [150, 90], [100, 90], 0, None),
    (4, 2, 128, 64, [150, 90], [40, 60], 20, None),
    (4, 2, 64, 64, [450, 290], [400, 290], 0, WIDE),
    (4, 2, 128, 64, [450, 290], [400, 290], 20, WIDE),
    (2, 1, 64, 32, [5000], [140], 0, WIDE),
]


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("heads,hk,hd,tokens,total,rows,window,room", UNEQUAL)
def test_attention_of_unequal_scales(qd, fmt, heads, hk, hd, tokens, total, rows, window, room):
    """Scales of values from 2^-60 to 2^60 and weights that differ as much, in any order: a block that weighs nothing, or
    that a row does not see, takes nothing from the others, however large its scale."""
    rng = np.random.default_rng([28, heads, hd, tokens, total[0]])
    c = Cache(rng, len(total), hk, hd, tokens, total, fmt, width=room and room // tokens)
    c.ks *= (4.0 ** rng.integers(-3, 3, c.ks.shape) * (1 if fmt == "i8" else 0.25)).astype(np.float32)
    c.vs[:] = (2.0 ** rng.integers(-60, 61, c.vs.shape)).astype(np.float32)
    kv, _ = _handle(qd, c)
    start, pos = _starts(rows), np.array(total, np.int32) - np.array(rows, np.int32)
    q = (rng.normal(size=(int(start[-1]), heads, hd)) * 2).astype(np.float32)
    got = _attn(qd, kv, dev(q), dev(start), dev(pos), heads, 1 / math.sqrt(hd), window)
    _check(got, *attn_all(c, q, start, pos, heads // hk, 1 / math.sqrt(hd), window))


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("exponent", [110, 117, -95])
@pytest.mark.parametrize("heads,hk,hd,tokens,total,rows,window,room", UNEQUAL)
def test_attention_of_values_near_the_ends_of_f32(qd, fmt, heads, hk, hd, tokens, total, rows, window, room, exponent):
    """Values to 2^124 (and from 2^-95 on): their sums over the positions have no place in f32, their weighted means do."""
    rng = np.random.default_rng([30, heads, hd, tokens, total[0]])
    c = Cache(rng, len(total), hk, hd, tokens, total, fmt, width=room and room // tokens)
    c.vs[:] = (2.0**exponent * rng.uniform(0.1, 1 if fmt == "i8" else 0.25, c.vs.shape)).astype(np.float32)
    kv, _ = _handle(qd, c)
    start, pos = _starts(rows), np.array(total, np.int32) - np.array(rows, np.int32)
    q = rng.normal(size=(int(start[-1]), heads, hd)).astype(np.float32)
    got = _attn(qd, kv, dev(q), dev(start), dev(pos), heads, 0.1, window)
    assert got.isfinite().all()
    _check(got, *attn_all(c, q, start, pos, heads // hk, 0.1, window))


@pytest.mark.parametrize("size", [1e5, 1e8, 1e12])
@pytest.mark.parametrize("heads,hk,hd,tokens,total,rows,window,room", UNEQUAL)
def test_attention_of_huge_scores(qd, heads, hk, hd, tokens, total, rows, window, room, size):
    """Scores so large that one position takes all the weight: its values come out.  A score is off by (hd + 16) 2^-24 of
    sum |q k| (attn_ref); rows whose two largest scores are nearer than four times that say nothing but that they are
    finite.  The weight is 1 in two parts and a sum, 2^-20 with room."""
    rng = np.random.default_rng([31, heads, hd, tokens, total[0]])
    c = Cache(rng, len(total), hk, hd, tokens, total, "i8", width=room and room // tokens)
    kv, _ = _handle(qd, c)
    start, pos = _starts(rows), np.array(total, np.int32) - np.array(rows, np.int32)
    q = (rng.normal(size=(int(start[-1]), heads, hd)) * size).astype(np.float32)
    out = _attn(qd, kv, dev(q), dev(start), dev(pos), heads, 0.5, window)
    assert out.isfinite().all()
    got, clear = out.cpu().numpy(), 0
    for b in range(len(pos)):
        for h in range(heads):
            ck, sk, cv, sv = c.values(b, h // (heads // hk), int(pos[b]) + rows[b])
            for i in range(rows[b]):
                r, p = start[b] + i, int(pos[b]) + i
                lo = max(0, p - window + 1) if window else 0
                x = q[r, h].astype(np.float64)
                s = (ck[lo : p + 1] @ x) * sk[lo : p + 1] * 0.5
                off = (hd + 16) * 2.0**-24 * ((np.abs(ck[lo : p + 1]) @ np.abs(x)) * sk[lo : p + 1] * 0.5).max()
                top = int(s.argmax())
                if len(s) > 1 and s[top] - np.delete(s, top).max() < 4 * off + 40:
                    continue
                clear += 1
                want = cv[lo + top] * sv[lo + top]
                assert np.all(np.abs(got[r, h] - want) <= 2.0**-20 * np.abs(want)), (b, h, i)
    assert clear >= len(q) * heads // 2


@pytest.mark.parametrize("name", ["ks", "vs"])
@pytest.mark.parametrize("hd,rows,window,room", [(64, 1, 20, None), (128, 40, 0, None), (64, 40, 20, None), (64, 300, 0, WIDE),
                                                 (128, 300, 20, WIDE)])
def test_attention_keeps_an_infinite_scale_apart(qd, hd, rows, window, room, name):
    """The scale of positions 160 .. 175 of the first key head is infinite: rows that do not see them are as they would be."""
    rng = np.random.default_rng([29, hd, rows])
    c = Cache(rng, 1, 2, hd, 32, [500], "i8", width=room and room // 32)
    start, pos = _starts([rows]), np.array([190 if rows == 1 else 150], np.int32)
    q = rng.normal(size=(rows, 4, hd)).astype(np.float32)
    ref, tol = attn_all(c, q, start, pos, 2, 0.1, window)
    getattr(c, name)[c.table[0, 5], 0, 0] = np.inf
    kv, _ = _handle(qd, c)
    got = _attn(qd, kv, dev(q), dev(start), dev(pos), 4, 0.1, window)
    at = pos[0] + np.arange(rows)
    sees = (at >= 160) & (at - window + 1 <= 175 if window else True)
    keep = np.repeat(~sees[:, None], 4, 1)
    keep[:, 2:] = True
    ref[~keep], tol[~keep] = 0, np.inf
    if name == "vs":
        assert not got.cpu().numpy()[~keep].any(where=np.isfinite(got.cpu().numpy()[~keep]))
    _check(torch.where(torch.from_numpy(keep).cuda()[..., None], got, 0.0), ref, tol)


@pytest.mark.parametrize("rows", [1, 20, 130])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_keeps_what_is_broken_apart(qd, hd, rows):
    """NaN in one query's head, NaN scales of a block: they reach the rows that see them and no other; what lies
    behind a row's position does not matter."""
    rng = np.random.default_rng([14, hd, rows])
    c = Cache(rng, 2, 2, hd, 16, [300, 300], "e4m3", width=WIDE // 16 if rows == 130 else None)
    q = rng.normal(size=(2 * rows, 4, hd)).astype(np.float32)
    start, pos = _starts([rows, rows]), np.array([150, 150], np.int32)
    kv, t = _handle(qd, c)
    base = _attn(qd, kv, dev(q), dev(start), dev(pos), 4, 0.1, 0)
    end = 150 + rows
    # behind the last position: codes that are NaN, scales that are not numbers
    for b in range(2):
        for p in range(end, 300):
            page, r = int(c.table[b, p // 16]), p % 16
            t["k"][page, :, r] = 127
            t["v"][page, :, r] = 127
            if p % 16 == 0:
                t["ks"][page, :, 0] = float("nan")
                t["vs"][page, :, 0] = float("inf")
    assert torch.equal(_attn(qd, kv, dev(q), dev(start), dev(pos), 4, 0.1, 0), base)
    # a query's head
    bad = q.copy()
    bad[0, 1, 5] = np.nan
    got = _attn(qd, kv, dev(bad), dev(start), dev(pos), 4, 0.1, 0)
    assert got[0, 1].isnan().all()
    got[0, 1] = base[0, 1]
    assert torch.equal(got, base)
    # the scale of positions 144 .. 159 of sequence 1, head 0 (query heads 0, 1), of keys; the same of values
    for name in ("ks", "vs"):
        page = int(c.table[1, 9])
        keep = t[name][page, 0, 0].item()
        t[name][page, 0, 0] = float("nan")
        got = _attn(qd, kv, dev(q), dev(start), dev(pos), 4, 0.1, 0)
        assert got[rows:, :2].isnan().all()
        assert torch.equal(got[:rows], base[:rows]) and torch.equal(got[rows:, 2:], base[rows:, 2:])
        # a window behind the block does not see it, and a row before it neither
        w = _attn(qd, kv, dev(q), dev(start), dev(pos), 4, 0.1, 20)
        sees = torch.arange(rows, device="cuda") + 150 - 19 <= 159
        assert w[rows:][sees][:, :2].isnan().all() and w[rows:][~sees].isfinite().all() and w[:rows].isfinite().all()
        t[name][page, 0, 0] = keep
    # the blocks of 256 .. 271 and of 272 .. 287, seen by rows 106 (122) and later alone, which see 240 .. 255 too
    if rows == 130:
        for block, seen in ((16, 106), (17, 122)):
            page = int(c.table[0, block])
            keep = t["vs"][page, 1, 0].item()
            t["vs"][page, 1, 0] = float("nan")
            got = _attn(qd, kv, dev(q), dev(start), dev(pos), 4, 0.1, 0)
            t["vs"][page, 1, 0] = keep
            assert got[seen:130, 2:].isnan().all() and torch.equal(got[:, :2], base[:, :2])
            # the unit that a tile's scales share goes by the other blocks alone then: rounding may differ
            assert (got[:seen, 2:] - base[:seen, 2:]).abs().max() <= 2.0**-18 * base[:seen, 2:].abs().max()
            assert torch.equal(got[130:], base[130:])


def test_attention_of_sequences_out_of_range(qd):
    """Positions below 0 or behind the table give zeros; an entry that is no page gives NaN."""
    rng = np.random.default_rng(15)
    c = Cache(rng, 5, 1, 64, 16, [48] * 5, "i8")
    c.table[3, 1] = -1
    c.table[4, 0] = len(c.k) + 7
    kv, _ = _handle(qd, c)
    rows = [2, 2, 2, 2, 2]
    start, pos = _starts(rows), np.array([-1, 47, 46, 40, 2**31 - 2], np.int32)
    q = rng.normal(size=(10, 3, 64)).astype(np.float32)
    got = _attn(qd, kv, dev(q), dev(start), dev(pos), 3, 0.125, 0)
    assert (got[:4] == 0).all() and (got[8:] == 0).all() and got[6:8].isnan().all()
    want = np.stack([[attn_ref(q[4 + i, h], *c.values(2, 0, 48), 46 + i, 0.125, 0)[0]
                      for h in range(3)] for i in range(2)])
    assert np.abs(got[4:6].cpu().numpy() - want).max() < 1e-4
    w = _attn(qd, kv, dev(q), dev(start), dev(pos), 3, 0.125, 4)  # the window has left the missing page behind
    assert w[6:8].isfinite().all()


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("heads,hk,hd", [(2, 2, 64), (8, 2, 128)])
def test_attention_of_many_rows_out_of_range(qd, heads, hk, hd, window):
    """Blocks of 128 rows: rows of a sequence that is out of range are zeros whatever their queries hold (an append leaves
    them as they were), and the sequence beside them is what it is alone."""
    rng = np.random.default_rng([27, heads])
    c = Cache(rng, 3, hk, hd, 16, [16, 400, 16], "i8", width=WIDE // 16)
    kv, _ = _handle(qd, c)
    q = rng.normal(size=(900, heads, hd)).astype(np.float32)
    q[:300], q[600:700], q[700:] = np.nan, np.inf, -np.inf
    start, pos = _starts([300, 300, 300]), np.array([-1, 100, WIDE - 299], np.int32)
    got = _attn(qd, kv, dev(q), dev(start), dev(pos), heads, 0.1, window)
    assert (got[:300] == 0).all() and (got[600:] == 0).all()
    ref, tol = attn_all(c, q[300:600], _starts([0, 300, 0]), np.array([0, 100, 0], np.int32), heads // hk, 0.1, window)
    _check(got[300:600], ref, tol)
    for b in (0, 2):  # a sequence alone
        r = slice(300 * b, 300 * b + 300)
        one = qd.PagedKV(*kv.tensors[:4], kv.tensors[4][b : b + 1], fmt=c.fmt)
        assert (_attn(qd, one, dev(q[r]), dev(_starts([300])), dev(pos[b : b + 1]), heads, 0.1, window) == 0).all()


def test_attention_of_shared_pages(qd):
    """Two sequences over the same pages give the same rows."""
    rng = np.random.default_rng(16)
    c = Cache(rng, 2, 2, 64, 16, [100, 100], "i8")
    c.table[1] = c.table[0]
    kv, _ = _handle(qd, c)
    q = rng.normal(size=(1, 4, 64)).astype(np.float32)
    got = _attn(qd, kv, dev(np.concatenate([q, q])), dev(_starts([1, 1])), dev(np.array([99, 99], np.int32)), 4, 0.125, 0)
    assert torch.equal(got[0], got[1])


def test_attention_offsets_behind_32_bits(qd):
    """A pool of more than 2^32 bytes: the pages behind it are the ones read, written and attended to."""
    tokens, hk, hd = 1024, 8, 128
    pages = 2**32 // (tokens * hk * hd) + 3
    codes = [torch.zeros(pages, hk, tokens, hd, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.full((pages, hk, tokens // BLOCK), 0.02, device="cuda") for _ in range(2)]
    table = torch.tensor([[pages - 1, 1], [2, pages - 2]], dtype=torch.int32, device="cuda")
    kv = qd.PagedKV(*codes, *scale, table)
    rng = np.random.default_rng(17)
    turns, d_turns, mag = _plan(qd, hd)
    x = dev(rng.normal(size=(24, 3 * hk, hd)).astype(np.float32))
    start, pos = dev(_starts([4, 20])), dev(np.array([0, 1020], np.int32))
    q = torch.empty(24, hk, hd, device="cuda")
    qd.paged_append(kv, x, x[:, hk:], x[:, 2 * hk :], 3 * hk * hd, q, hk, 24, start, pos, 2, hd, "half", d_turns, mag)
    assert codes[1][pages - 1, :, :4].float().abs().sum() > 0 and codes[1][pages - 2, :, :16].float().abs().sum() > 0
    assert codes[1][0].count_nonzero() == 0 and codes[1][1].count_nonzero() == 0 and codes[0][3:10].count_nonzero() == 0
    out = _attn(qd, kv, q, start, pos, hk, 0.1, 0)
    k, v = (torch.zeros(2, hk, 1040, hd, device="cuda") for _ in range(2))
    qd.paged_read(kv, dev(np.array([4, 1040], np.int32)), 2, 1040, k, v)
    for b, (r0, p0, t) in enumerate(((0, 0, 4), (4, 1020, 20))):
        s = torch.einsum("thd,hjd->thj", q[r0 : r0 + t].double(), k[b, :, : p0 + t].double()) * 0.1
        at = torch.arange(p0 + t, device="cuda")
        s.masked_fill_(at[None, None] > (torch.arange(t, device="cuda") + p0)[:, None, None], -math.inf)
        want = torch.einsum("thj,hjd->thd", s.softmax(-1), v[b, :, : p0 + t].double())
        assert (out[r0 : r0 + t] - want).abs().max() < 2e-5


# ------------------------------------------------------------------ a step's calls together
@pytest.mark.parametrize("fmt,hd,group", [("i8", 64, 3), ("e4m3", 128, 4)])
def test_prompt_then_steps(qd, fmt, hd, group):
    """A packed batch of prompts, then steps of one token each: after every step the cache is the reference's and
    the rows are its attention; then the sequences are read back and the next token's attention over the contiguous
    caches is the same."""
    rng = np.random.default_rng(20)
    hk, tokens = 2, 32
    heads = hk * group
    rows = [37, 1, 64]
    c = Cache(rng, 3, hk, hd, tokens, [n + 20 for n in rows], fmt)
    kv, t = _handle(qd, c)
    turns, d_turns, mag = _plan(qd, 32, "turns", factor=4.0, trained_ctx=64, low=1.0, high=4.0)
    pos = np.zeros(3, np.int32)
    ws = torch.empty(qd.paged_attn_workspace(kv, heads, sum(rows), 3), dtype=torch.uint8, device="cuda")
    for step in range(6):
        start = _starts(rows)
        n = int(start[-1])
        x = rng.normal(size=(n, heads + 2 * hk, hd)).astype(np.float32)
        d, q_out = dev(x), torch.empty(n, heads, hd, device="cuda")
        d_start, d_pos = dev(start), dev(pos)
        qd.paged_append(kv, d, d[:, heads:], d[:, heads + hk :], (heads + 2 * hk) * hd, q_out, heads, n, d_start, d_pos, 3, 32,
                        "half", d_turns, mag)
        out = _attn(qd, kv, q_out, d_start, d_pos, heads, 1 / math.sqrt(hd), 0, ws=ws)
        for b in range(3):
            r = slice(start[b], start[b + 1])
            at = np.arange(pos[b], pos[b] + rows[b])
            y = rotate(x[r, heads : heads + hk], cos_sin(turns, at, mag), 32, "half")
            c.put(b, int(pos[b]), y, x[r, heads + hk :])
        _same_cache(t, c)
        _check(out, *attn_all(c, q_out.cpu().numpy(), start, pos, group, 1 / math.sqrt(hd), 0))
        pos = pos + np.array(rows, np.int32)
        rows = [1, 1, 1]
    if hd == 64:  # the contiguous caches that the decode step's attention takes
        ctx = int(pos.max())
        k, v = (torch.zeros(3, hk, ctx, hd, device="cuda") for _ in range(2))
        qd.paged_read(kv, dev(pos), 3, ctx, k, v)
        q = dev(rng.normal(size=(3, heads, hd)).astype(np.float32))
        at = dev(pos - 1)
        size = qd.gqa_decode_attn_workspace(heads, hd, ctx, 3)
        want = torch.empty(3, heads, hd, device="cuda")
        qd.gqa_decode_attn(q, heads * hd, k, v, want, heads, hk, hd, at, ctx, 3,
                           torch.empty(size, dtype=torch.uint8, device="cuda"), size)
        got = _attn(qd, kv, q, dev(_starts([1, 1, 1])), at, heads, 1 / math.sqrt(hd), 0)
        _, tol = attn_all(c, q.cpu().numpy(), _starts([1, 1, 1]), pos - 1, group, 1 / math.sqrt(hd), 0)
        assert np.all(np.abs((got - want).cpu().numpy()) <= 2 * tol)


def test_the_readme_example_runs(qd):
    """The lines of README.md on the paged cache, over names as it uses them."""
    import os

    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    code = next(c for c in text.split("```python")[1:] if "qd.PagedKV(" in c).split("```")[0]
    heads, kv_heads, head_dim, n_seqs, max_ctx = 8, 2, 64, 2, 200
    c = Cache(np.random.default_rng(26), n_seqs, kv_heads, head_dim, 64, [150, 200], "i8")
    _, t = _handle(qd, c)
    names = dict(qd=qd, torch=torch, k_pages=t["k"], v_pages=t["v"], k_scale=t["ks"], v_scale=t["vs"], page_table=t["table"],
                 heads=heads, kv_heads=kv_heads, head_dim=head_dim, n_seqs=n_seqs, max_ctx=max_ctx, n_tokens=51,
                 qkv=torch.randn(51, heads + 2 * kv_heads, head_dim, device="cuda"),
                 q=torch.zeros(51, heads, head_dim, device="cuda"), out=torch.full((51, heads, head_dim), 9.0, device="cuda"),
                 row_start=dev(_starts([50, 1])), pos=dev(np.array([100, 199], np.int32)),
                 lengths=dev(np.array([150, 200], np.int32)),
                 k_cache=torch.zeros(n_seqs, kv_heads, max_ctx, head_dim, device="cuda"),
                 v_cache=torch.zeros(n_seqs, kv_heads, max_ctx, head_dim, device="cuda"))
    exec(code, names)
    k, v, q = names["k_cache"], names["v_cache"], names["q"]
    w = (q[50].view(2, 4, 64).double() @ k[1].double().transpose(1, 2) / 8).softmax(-1)
    assert (names["out"][50].view(2, 4, 64) - w @ v[1].double()).abs().max() < 1e-4
    assert names["out"].isfinite().all()


def test_a_captured_step_replays_over_new_positions(qd):
    """Append and attention in one graph: each replay takes what pos and the rows hold then."""
    rng = np.random.default_rng(21)
    heads, hk, hd = 8, 2, 64
    c = Cache(rng, 2, hk, hd, 16, [200, 200], "i8")
    kv, t = _handle(qd, c)
    kv2, t2 = _handle(qd, c)
    turns, d_turns, mag = _plan(qd, hd)
    start, pos = dev(_starts([1, 1])), dev(np.array([30, 3], np.int32))
    x = torch.zeros(2, heads + 2 * hk, hd, device="cuda")
    q_out, out = torch.zeros(2, heads, hd, device="cuda"), torch.zeros(2, heads, hd, device="cuda")
    ws = torch.empty(qd.paged_attn_workspace(kv, heads, 2, 2), dtype=torch.uint8, device="cuda")

    def step(cache, q_out, out, ws):
        qd.paged_append(cache, x, x[:, heads:], x[:, heads + hk :], (heads + 2 * hk) * hd, q_out, heads, 2, start, pos, 2, hd,
                        "adjacent", d_turns, mag)
        qd.paged_attn(cache, q_out, heads * hd, out, heads, 2, start, pos, 2, 0.125, 0, ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(kv, q_out, out, ws)  # warm-up, undone below
    side.synchronize()
    for name in t:
        t[name].copy_(t2[name])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kv, q_out, out, ws)
        pos.add_(1)
    q2, out2 = torch.zeros_like(q_out), torch.zeros_like(out)
    pos.copy_(dev(np.array([30, 3], np.int32)))
    for i in range(40):
        x.copy_(dev(rng.normal(size=x.shape).astype(np.float32)))
        if i == 20:
            pos.copy_(dev(np.array([150, 100], np.int32)))  # further on, over what the pages hold there
        step(kv2, q2, out2, torch.empty_like(ws))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(q_out, q2)
    for name in t:
        assert torch.equal(t[name], t2[name])


def test_two_streams_with_a_workspace_each(qd):
    rng = np.random.default_rng(22)
    c = Cache(rng, 4, 8, 128, 64, [3000] * 4, "i8")
    kv, _ = _handle(qd, c)
    calls = []
    for rows in ([1, 1, 1, 1], [200, 1, 0, 100]):
        start, pos = _starts(rows), np.array([3000 - r for r in rows], np.int32)
        q = dev(rng.normal(size=(int(start[-1]), 32, 128)).astype(np.float32))
        calls.append((q, dev(start), dev(pos)))
    want = [_attn(qd, kv, *call, 32, 0.09, 0) for call in calls]
    ws = [torch.empty(qd.paged_attn_workspace(kv, 32, len(call[0]), 4), dtype=torch.uint8, device="cuda") for call in calls]
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for call, o, w, st in zip(calls, outs, ws, streams):
            with torch.cuda.stream(st):
                _attn(qd, kv, *call, 32, 0.09, 0, out=o, ws=w)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_tensors_that_are_too_small_or_of_another_type(qd):
    """What only the tensors tell is an error before any device work."""
    c = Cache(np.random.default_rng(23), 2, 2, 64, 16, [40, 40], "i8")
    kv, _ = _handle(qd, c)
    start, pos = dev(_starts([1, 1])), dev(np.array([30, 3], np.int32))
    q, out = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 4, 64, device="cuda")
    ws = torch.empty(qd.paged_attn_workspace(kv, 4, 2, 2), dtype=torch.uint8, device="cuda")
    good = dict(q=q, out=out, row_start=start, pos=pos, workspace=ws)

    def call(**c):
        a = {**good, **c}
        qd.paged_attn(kv, a["q"], 256, a["out"], 4, 2, a["row_start"], a["pos"], 2, 0.125, 0, a["workspace"])

    call()
    for bad in (dict(q=q[:1].clone()), dict(q=q.half()), dict(out=out[:1].clone()), dict(row_start=start[:2]), dict(pos=pos[:1]),
                dict(pos=pos.long()), dict(q=q.cpu()), dict(out=out.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(qd.QDError):
        call(workspace=ws[:8])
    k = torch.zeros(2, 2, 40, 64, device="cuda")
    with pytest.raises(ValueError):
        qd.paged_read(kv, pos, 2, 41, k, k)
    with pytest.raises(ValueError):
        qd.paged_read(kv, pos, 2, 40, k, k, out_f16=True)
    x = torch.zeros(2, 4, 64, device="cuda")
    turns = qd.rope_plan(1e4, 64)[0].cuda()
    with pytest.raises(ValueError):
        qd.rope_tokens(x, 256, x, 256, 3, 4, 64, 64, pos, "half", turns)
    with pytest.raises(ValueError):
        qd.rope_tokens(x, 256, x, 256, 2, 4, 64, 64, pos, "half", turns[:31])
