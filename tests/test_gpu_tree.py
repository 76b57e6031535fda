"""Tree verification on the GPU: each operator against 64-bit references, the rows and slots
that must not matter, graphs and streams, and the four operators together against one token
at a time."""
import os
import re

import numpy as np
import pytest
import torch

from gpu_helpers import dev
from tree_helpers import (attn_bound, attn_plain, attn_ref, attn_tol, commit_ref, logprobs_ref, mask_bits, random_tree,
                          rms)

pytestmark = pytest.mark.gpu
HD = 64


def _i32(a):
    return dev(np.asarray(a, np.int32))


def _trees(rng, batch, n):
    t = [random_tree(rng, n) for _ in range(batch)]
    return np.stack([p for p, _ in t]), np.stack([a for _, a in t])


class Attn:
    """Inputs of one tree_attn call: NumPy copies (k, v rounded to the cache's type) and tensors."""

    def __init__(self, qd, seed, hq, hk, n, ctx, pos, cnt=None, f16=False, q_gap=0, kscale=1.0, vscale=1.0):
        rng = np.random.default_rng(seed)
        self.qd, self.hq, self.hk, self.n, self.ctx, self.f16 = qd, hq, hk, n, ctx, f16
        self.b = b = len(pos)
        self.pos, self.cnt = list(pos), list(cnt) if cnt is not None else None
        t = np.float16 if f16 else np.float32
        mk = lambda *s, scale=1.0: (rng.standard_normal(s) * scale).astype(np.float32)  # noqa: E731
        self.q_gap = q_gap
        self.qrow = n * hq * HD + q_gap
        self.q = mk(b, self.qrow, scale=1.5)
        self.k, self.v = mk(b, hk, ctx, HD, scale=kscale).astype(t), mk(b, hk, ctx, HD, scale=vscale).astype(t)
        self.kd, self.vd = mk(b, hk, n, HD, scale=kscale).astype(t), mk(b, hk, n, HD, scale=vscale).astype(t)
        self.parent, self.anc = _trees(rng, b, n)

    def call(self, out=None, ws=None, stream=None):
        out = torch.full((self.b, self.n, self.hq, HD), 7.0, device="cuda") if out is None else out
        if ws is None:
            size = self.qd.tree_attn_workspace(self.hq, self.hk, HD, self.n, self.ctx, self.b)
            ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns: nothing needs to start at zero
        self.dev = [dev(a) for a in (self.q, self.k, self.v, self.kd, self.vd)]
        q, k, v, kd, vd = self.dev
        self.small = (_i32(self.pos), dev(mask_bits(self.anc)), None if self.cnt is None else _i32(self.cnt))
        pos, mask, cnt = self.small
        self.args = (q, self.qrow, k, v, kd, vd, out, self.hq, self.hk, HD, pos, mask, cnt, self.n, self.ctx, self.b,
                     ws)
        self.qd.tree_attn(*self.args, kv_f16=self.f16, stream=stream)
        return out

    def ref(self, b):
        cnt = self.n if self.cnt is None else self.cnt[b]
        q = self.q[b, :self.n * self.hq * HD].reshape(self.n, self.hq, HD)
        return attn_ref(q, self.k[b], self.v[b], self.kd[b], self.vd[b], self.pos[b], self.anc[b], cnt, self.hq,
                        self.hk)

    def check(self, got=None):
        got = (self.call() if got is None else got).cpu().numpy()
        for b in range(self.b):
            cnt = self.n if self.cnt is None else max(0, min(self.n, self.cnt[b]))
            want, smax, vmax = self.ref(b)
            err = np.abs(got[b, :cnt] - want).max() if cnt else 0.0
            assert err <= attn_tol(self.pos[b] + cnt, smax, vmax), (b, err, attn_tol(self.pos[b] + cnt, smax, vmax))
            assert np.all(got[b, cnt:] == 7.0)  # rows behind the sequence's nodes
        return got


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("hq,hk,n,ctx,pos", [
    (1, 1, 1, 1, [0]), (1, 1, 1, 1, [1]), (9, 3, 8, 256, [100]), (9, 3, 1, 70, [64, 63, 65, 1]),
    (32, 32, 16, 200, [130, 0]), (8, 1, 27, 300, [300, 0, 17, 64, 128]), (4, 2, 64, 129, [128, 129]),
    (16, 2, 64, 520, [511]), (7, 1, 33, 96, [95]), (5, 5, 3, 2100, [2049]), (6, 2, 22, 1000, [1000, 1, 999]),
    (10, 2, 13, 64, list(range(48, 64))),
    # 16, 17, 32, 33, 64 rows to a kv head, one and two blocks of 128, walks whole and cut
    (2, 1, 8, 40, [40]), (1, 1, 17, 300, [299, 31]), (4, 1, 8, 1030, [1029, 513]), (3, 1, 11, 640, [640, 127, 129]),
    (2, 2, 64, 1300, [1290, 640]), (4, 1, 33, 2400, [2399, 0, 897, 128]), (8, 1, 64, 1500, [1500])])
def test_attn_matches_64_bits(qd, hq, hk, n, ctx, pos, f16):
    Attn(qd, 1, hq, hk, n, ctx, pos, f16=f16).check()


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("hq,n", [(3, 5), (8, 30)])
def test_attn_long_context_split(qd, hq, n, f16):
    Attn(qd, 2, hq, 1, n, 20000, [19990], f16=f16).check()


@pytest.mark.parametrize("f16", [False, True])
def test_attn_ragged_counts_and_row_stride(qd, f16):
    a = Attn(qd, 3, 6, 2, 19, 150, [149, 3, 70, 0, 150], cnt=[19, 7, 0, 1, 18], f16=f16, q_gap=36)
    a.check()
    a = Attn(qd, 3, 6, 2, 19, 150, [149, 3], cnt=[19, 19], f16=f16)
    want = a.call().clone()
    a.cnt = [40, -3]  # taken as n_nodes and as 0
    got = a.call()
    assert torch.equal(got[0], want[0]) and torch.all(got[1] == 7.0)


@pytest.mark.parametrize("f16", [False, True])
def test_attn_rows_that_see_nothing_and_bad_positions(qd, f16):
    a = Attn(qd, 4, 4, 2, 10, 80, [0, 80, 81, -1], f16=f16)
    a.anc[0, 3] = False
    a.anc[0, 9] = False
    got = a.call().cpu().numpy()
    assert np.all(got[0, [3, 9]] == 0) and np.all(got[2:] == 0)
    for b in (0, 1):
        want, smax, vmax = a.ref(b)
        assert np.abs(got[b] - want).max() <= attn_tol(90, smax, vmax)


def test_attn_mask_bits_behind_the_nodes_do_not_count(qd):
    a = Attn(qd, 5, 4, 2, 10, 80, [33, 5], cnt=[10, 4])
    want = a.call().clone()
    a.small[1].bitwise_or_(torch.tensor(-1 << 10, device="cuda"))
    out = torch.full_like(want, 7.0)
    a.qd.tree_attn(*a.args[:6], out, *a.args[7:])
    assert torch.equal(out, want)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("hq,hk,ctx,pos", [(6, 2, 140, [70, 128]), (3, 3, 140, [70, 128]), (6, 2, 2300, [2201, 1000]),
                                           (2, 2, 2500, [2201, 1000])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attn_unseen_values_do_not_reach_a_row(qd, bad, hq, hk, ctx, pos, f16):
    """Slots that a node does not see, positions behind pos and slots behind n_valid hold `bad`."""
    a = Attn(qd, 6, hq, hk, 24, ctx, pos, cnt=[24, 20], f16=f16)
    want = a.check(a.call())
    for b in range(2):
        a.k[b, :, a.pos[b]:] = bad
        a.v[b, :, a.pos[b]:] = bad
        a.kd[b, :, a.cnt[b]:] = bad
        a.vd[b, :, a.cnt[b]:] = bad
    assert np.array_equal(a.call().cpu().numpy(), want)
    a.kd[:, :, 5] = bad  # seen by node 5 and those below it alone
    a.vd[:, :, 5, 3] = bad
    got = a.call().cpu().numpy()
    for b in range(2):
        sees = a.anc[b, :a.cnt[b], 5]
        assert np.array_equal(got[b, :a.cnt[b]][~sees], want[b, :a.cnt[b]][~sees])
        assert np.all(~np.isfinite(got[b, :a.cnt[b]][sees][..., 3]))


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("hk", [2, 6])
def test_attn_infinite_value_in_the_cache_stays_in_its_dim(qd, hk, f16):
    a = Attn(qd, 16, 6, hk, 24, 300, [290], f16=f16)
    a.v[0, :, 100, 3] = np.inf
    a.v[0, :, 17, 60] = np.nan
    got = a.call().cpu().numpy()
    dims = [d for d in range(HD) if d not in (3, 60)]
    assert np.all(~np.isfinite(got[..., [3, 60]]))
    a.v[0, :, 100, 3] = a.v[0, :, 17, 60] = 0
    want, smax, vmax = a.ref(0)
    assert np.abs(got[0] - want)[..., dims].max() <= attn_tol(314, smax, vmax)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("hk", [2, 6])
def test_attn_unseen_large_values_keep_the_others_digits(qd, hk, f16):
    """A draft that a row does not see may hold the type's largest value."""
    a = Attn(qd, 17, 6, hk, 24, 100, [90], f16=f16)
    want = a.call().cpu().numpy()
    big = 65504.0 if f16 else np.finfo(np.float32).max
    a.kd[:, :, 7] = big
    a.vd[:, :, 7] = -big
    got = a.call().cpu().numpy()
    sees = a.anc[0, :, 7]
    assert np.array_equal(got[0][~sees], want[0][~sees]) and not sees.all()


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("hk", [2, 6])
def test_attn_non_finite_query_stays_in_its_row(qd, hk, f16):
    a = Attn(qd, 7, 6, hk, 24, 140, [70], f16=f16)
    want = a.call().cpu().numpy()
    a.q.reshape(1, 24, 6, HD)[0, 4, 1, 9] = np.nan
    a.q.reshape(1, 24, 6, HD)[0, 20, 5, 0] = np.inf
    got = a.call().cpu().numpy()
    hit = np.zeros((24, 6), bool)
    hit[4, 1] = hit[20, 5] = True
    assert np.all(np.isnan(got[0][hit])) and np.array_equal(got[0][~hit], want[0][~hit])


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("n", [9, 20])
@pytest.mark.parametrize("kscale,vscale", [(1e-3, 1e-4), (8.0, 300.0)])
def test_attn_small_and_large_values(qd, f16, n, kscale, vscale):
    Attn(qd, 8, 6, 2, n, 400, [390], f16=f16, kscale=kscale, vscale=vscale).check()


@pytest.mark.parametrize("n", [9, 20])
def test_attn_values_beyond_binary16_in_an_f32_cache(qd, n):
    a = Attn(qd, 9, 6, 2, n, 400, [390], kscale=1e-6, vscale=1e9)
    a.k[0, 0, 40] *= 1e12  # one row far larger than its neighbours: 1e6
    a.q[:] *= 1e-6
    a.check()


def test_attn_peaked_rows(qd):
    """Scores of hundreds: one position takes nearly all the weight."""
    a = Attn(qd, 10, 4, 1, 12, 700, [690], kscale=6.0)
    a.q *= 6.0
    a.check()


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("n", [5, 40])
def test_attn_two_calls_at_once_with_their_own_workspaces(qd, n, f16):
    pair = [Attn(qd, 18 + i, 9, 3, n, 5000, [4990, 3000 - 900 * i], f16=f16) for i in range(2)]
    want = [a.call().clone() for a in pair]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pair]
    outs = [torch.full_like(w, 7.0) for w in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for a, st, out in zip(pair, streams, outs):
            qd.tree_attn(*a.args[:6], out, *a.args[7:], kv_f16=f16, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_attn_same_bits_again_and_on_another_stream(qd):
    a = Attn(qd, 11, 9, 3, 40, 3000, [2999, 1500, 7], f16=True)
    want = a.call().clone()
    for _ in range(5):
        assert torch.equal(a.call(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        a.qd.tree_attn(*a.args[:6], out, *a.args[7:], kv_f16=True)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("n,ctx", [(8, 600), (8, 3000), (30, 600), (30, 3000)])
def test_attn_captured_replays_follow_the_device_positions(qd, n, ctx, f16):
    a = Attn(qd, 12, 9, 3, n, ctx, [100, ctx - 10], f16=f16)
    out = a.call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.qd.tree_attn(*a.args, kv_f16=f16)
    for pos in ([0, ctx], [ctx - 1, 1], [64, 65]):
        a.small[0].copy_(_i32(pos))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        a.pos = pos
        a.check(out)


@pytest.mark.parametrize("hq", [32, 128])
def test_attn_offsets_past_32_bits(qd, hq):
    """A binary16 cache of more than 2^32 elements: the last sequence's rows are the ones read."""
    hk = 32
    ctx, b, n, p = 140000, 16, 9, 130
    need = b * hk * ctx * HD
    assert need > 2**32
    if torch.cuda.mem_get_info()[0] < 5 * need:
        pytest.skip("not enough free memory")
    a = Attn(qd, 13, hq, hk, n, p, [p] * b, f16=True)
    k = torch.zeros(b, hk, ctx, HD, dtype=torch.float16, device="cuda")
    v = torch.zeros(b, hk, ctx, HD, dtype=torch.float16, device="cuda")
    want = a.call()
    k[:, :, :p], v[:, :, :p] = a.dev[1], a.dev[2]
    ws = torch.empty(qd.tree_attn_workspace(hq, hk, HD, n, ctx, b), dtype=torch.uint8, device="cuda")
    out = torch.full_like(want, 7.0)
    pos, mask, _ = a.small
    qd.tree_attn(a.dev[0], a.qrow, k, v, a.dev[3], a.dev[4], out, hq, hk, HD, pos, mask, None, n, ctx, b, ws,
                 kv_f16=True)
    for x in (0, b - 1):
        w, smax, vmax = a.ref(x)
        assert np.abs(out[x].cpu().numpy() - w).max() <= attn_tol(p + n, smax, vmax)


# Blocks of 128 rows take over where a call's work (in positions of 16-row blocks) passes a bound,
# which most sizes above stay below: a head with many rows and a cache with room for many positions
# (16 blocks' worth more than 1100000 binary16 or 300000 f32 ones), or many short walks.
def _wide(qd, seed, pos, f16, hq=8, n=64, **kw):
    return Attn(qd, seed, hq, 1, n, (17600000 if f16 else 4800000) // (hq * n), pos, f16=f16, **kw)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("hq,n", [(8, 64), (7, 31)])
def test_attn_128_lengths(qd, hq, n, f16):
    ctx = (1100000 if f16 else 300000) // (6 * ((hq * n + 15) // 16))
    Attn(qd, 40, hq, 1, n, ctx, [0, 1, 127, 129, 1030, ctx], f16=f16).check()


@pytest.mark.parametrize("f16", [False, True])
def test_attn_128_long_walk_cut_over_all_ctas(qd, f16):
    _wide(qd, 41, [12000 if f16 else 6000], f16, hq=7, n=37).check()


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("ctx", [128, 300])
def test_attn_128_many_short_walks(qd, ctx, f16):
    """16 sequences, whole walks (of at most four tiles) and cut ones."""
    hk = 3
    a = Attn(qd, 42, 8 * hk, hk, 64, ctx, [ctx - 7 * i for i in range(16)], f16=f16,
             cnt=[64 - 3 * i for i in range(16)], q_gap=12)
    a.check()


@pytest.mark.parametrize("f16", [False, True])
def test_attn_128_rows_that_see_nothing_and_bad_positions(qd, f16):
    a = _wide(qd, 43, [0, 300, 10**6, -1], f16)
    a.anc[0, 3] = a.anc[0, 60] = False
    got = a.call().cpu().numpy()
    assert np.all(got[0, [3, 60]] == 0) and np.all(got[2:] == 0)
    for b in range(2):
        want, smax, vmax = a.ref(b)
        assert np.abs(got[b] - want).max() <= attn_tol(a.pos[b] + 64, smax, vmax)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attn_128_unseen_values_do_not_reach_a_row(qd, bad, f16):
    a = _wide(qd, 44, [70, 2000], f16, cnt=[64, 50])
    want = a.check(a.call())
    for b in range(2):
        a.k[b, :, a.pos[b]:] = bad
        a.v[b, :, a.pos[b]:] = bad
        a.kd[b, :, a.cnt[b]:] = bad
        a.vd[b, :, a.cnt[b]:] = bad
    assert np.array_equal(a.call().cpu().numpy(), want)
    a.kd[:, :, 5] = bad
    a.vd[:, :, 5, 3] = bad
    got = a.call().cpu().numpy()
    for b in range(2):
        sees = a.anc[b, :a.cnt[b], 5]
        assert np.array_equal(got[b, :a.cnt[b]][~sees], want[b, :a.cnt[b]][~sees])
        assert np.all(~np.isfinite(got[b, :a.cnt[b]][sees][..., 3]))


@pytest.mark.parametrize("f16", [False, True])
def test_attn_128_infinite_values_and_queries_stay_where_they_are(qd, f16):
    a = _wide(qd, 45, [290], f16)
    want = a.check()
    _, smax, vmax = a.ref(0)
    a.v[0, :, 100, 3] = np.inf
    a.v[0, :, 17, 60] = np.nan
    a.q.reshape(1, 64, 8, HD)[0, 4, 1, 9] = np.nan
    a.q.reshape(1, 64, 8, HD)[0, 20, 5, 0] = np.inf
    got = a.call().cpu().numpy()
    assert np.isnan(got[0, 4, 1]).all() and np.isnan(got[0, 20, 5]).all()
    keep = np.ones((64, 8), bool)
    keep[4, 1] = keep[20, 5] = False
    dims = [d for d in range(HD) if d not in (3, 60)]
    assert not np.isfinite(got[0][keep][:, [3, 60]]).any()
    # the scale of a position's values may change with them: as exact as before, not the same bits
    assert np.abs(got[0][keep][:, dims] - want[0][keep][:, dims]).max() <= 2 * attn_tol(354, smax, vmax)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("kscale,vscale", [(1e-3, 1e-4), (8.0, 300.0)])
def test_attn_128_small_and_large_values(qd, f16, kscale, vscale):
    _wide(qd, 46, [390, 1500], f16, kscale=kscale, vscale=vscale).check()


def test_attn_128_values_beyond_binary16_in_an_f32_cache(qd):
    a = _wide(qd, 47, [390], False, kscale=1e-6, vscale=1e9)
    a.k[0, 0, 40] *= 1e12
    a.q[:] *= 1e-6
    a.check()


@pytest.mark.parametrize("f16", [False, True])
def test_attn_128_two_calls_at_once_and_captured(qd, f16):
    pair = [_wide(qd, 48 + i, [4000 - 900 * i, 33], f16) for i in range(2)]
    want = [a.call().clone() for a in pair]
    torch.cuda.synchronize()
    outs = [torch.full_like(w, 7.0) for w in want]
    streams, graphs = [torch.cuda.Stream() for _ in pair], []
    for a, o, s in zip(pair, outs, streams):
        ws = torch.empty_like(a.args[16])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(4):
                qd.tree_attn(*a.args[:6], o, *a.args[7:16], ws, kv_f16=f16)
        graphs.append((g, ws))
    for (g, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


# What a value's own size asks for: each output against a bound that does not grow with the other
# dimensions of the rows, or with rows that have no weight (attn_bound).  (hq, hk, n) below the
# bound of the 128-row blocks and above it (_wide).
def _close(a, b=0):
    got = a.call()[b].cpu().numpy()
    q = a.q[b, :a.n * a.hq * HD].reshape(a.n, a.hq, HD)
    want, tol = attn_bound(q, a.k[b], a.v[b], a.kd[b], a.vd[b], a.pos[b], a.anc[b], a.n, a.hq, a.hk, a.f16)
    off = np.abs(got - want) / tol
    assert off.max() <= 1, (off.max(), np.unravel_index(off.argmax(), off.shape))


def _either(qd, wide, seed, pos, f16):
    return _wide(qd, seed, [pos], f16) if wide else Attn(qd, seed, 6, 2, 9, pos + 10, [pos], f16=f16)


def _rows(a):
    return a.q.reshape(a.b, -1, HD)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ratio", [2.0**10, 2.0**14])
def test_attn_large_dimension_of_the_values_leaves_the_others_their_digits(qd, ratio, wide):
    a = _either(qd, wide, 60, 390, False)
    a.v[..., 11] *= ratio
    a.vd[..., 11] *= ratio
    _close(a)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ratio", [2.0**10, 2.0**14])
def test_attn_large_dimension_of_the_keys_leaves_the_others_their_digits(qd, ratio, wide):
    a = _either(qd, wide, 61, 390, False)
    a.k[..., 11] *= ratio
    a.kd[..., 11] *= ratio
    _rows(a)[..., 11] /= ratio
    _close(a)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ratio", [2.0**10, 2.0**14])
def test_attn_large_dimension_of_the_queries_leaves_the_others_their_digits(qd, ratio, wide):
    a = _either(qd, wide, 62, 390, False)
    _rows(a)[..., 11] *= np.float32(ratio)
    a.k[..., 11] /= ratio
    a.kd[..., 11] /= ratio
    _close(a)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("score,big", [(-300.0, 1e9), (-300.0, 1e30), (-100.0, 1e20), (-18.0, 1e6)])
def test_attn_large_value_row_of_little_weight_leaves_the_others_their_digits(qd, score, big, wide, f16):
    """A cached row whose values are far larger than the others', behind a score far below theirs."""
    a = _either(qd, wide, 63, 390, f16)
    _rows(a)[..., 5] = 16.0
    a.k[..., 5] = a.kd[..., 5] = 0
    a.k[0, :, 200] = 0
    a.k[0, :, 200, 5] = score / 2
    a.v[0, :, 200] *= min(big, 8192.0) if f16 else big
    _close(a)


@pytest.mark.parametrize("f16", [False, True])
def test_attn_128_unseen_large_values_keep_the_others_digits(qd, f16):
    """A draft that a row does not see may hold the type's largest value."""
    a = _wide(qd, 65, [90], f16)
    want = a.call().cpu().numpy()
    a.kd[:, :, 7] = 65504.0 if f16 else np.finfo(np.float32).max
    a.vd[:, :, 7] = -a.kd[:, :, 7]
    got = a.call().cpu().numpy()
    sees = a.anc[0, :, 7]
    assert np.array_equal(got[0][~sees], want[0][~sees]) and not sees.all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("f16", [False, True])
def test_attn_infinite_draft_value_over_a_cache_of_zeros(qd, wide, f16):
    """The other dimensions of such a draft count with their own size, whatever the other values are."""
    a = _either(qd, wide, 66, 120, f16)
    a.v[:] = 0
    a.vd[:] = 0
    a.vd[0, :, 2] = 100.0 if f16 else 1e9
    a.vd[0, :, 2, 3] = np.inf
    got = a.call()[0].cpu().numpy()
    sees = a.anc[0, :, 2]
    assert np.all(got[~sees] == 0) and np.all(~np.isfinite(got[sees][..., 3]))
    a.vd[0, :, 2, 3] = 0
    q = a.q[0, :a.n * a.hq * HD].reshape(a.n, a.hq, HD)
    want, tol = attn_bound(q, a.k[0], a.v[0], a.kd[0], a.vd[0], 120, a.anc[0], a.n, a.hq, a.hk, f16)
    dims = [d for d in range(HD) if d != 3]
    assert np.all(np.abs(got - want)[sees][..., dims] <= tol[sees][..., dims])

@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ratio", [2.0**10, 2.0**14])
def test_attn_large_dimension_of_the_queries_over_a_binary16_cache(qd, ratio, wide):
    a = _either(qd, wide, 67, 390, True)
    _rows(a)[..., 11] *= np.float32(ratio)
    a.k[..., 11] /= ratio
    a.kd[..., 11] /= ratio
    _close(a)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("score", [-18.0, -20.0, -24.0])
def test_attn_small_weights_of_large_values_over_a_binary16_cache(qd, score, wide):
    """A row of values near the type's largest behind a small weight, the other values small."""
    a = _either(qd, wide, 68, 390, True)
    _rows(a)[..., 5] = 16.0
    a.k[..., 5] = a.kd[..., 5] = 0
    a.k[0, :, 200] = 0
    a.k[0, :, 200, 5] = score / 2
    a.v *= np.float16(1e-5)
    a.vd *= np.float16(1e-5)
    a.v[0, :, 200] = np.where(a.v[0, :, 200] < 0, -60000.0, 60000.0)
    _close(a)

@pytest.mark.parametrize("wide", [False, True])
def test_attn_infinite_key_of_a_binary16_cache(qd, wide):
    """A row is NaN, or, where the score is -infinity, what it is without that position."""
    a = _either(qd, wide, 69, 120, True)
    a.k[0, :, 7, 9] = -np.inf
    got = a.call()[0].cpu().numpy()
    nan = np.isnan(got).any(-1)
    assert np.array_equal(nan, np.isnan(got).all(-1)) and nan.any()
    up = a.q[0, :a.n * a.hq * HD].reshape(a.n, a.hq, HD)[..., 9] < 0  # a score of +infinity
    assert nan[up].all()
    q = a.q[0, :a.n * a.hq * HD].reshape(a.n, a.hq, HD)
    without = [np.delete(x, 7, axis=1) for x in (a.k[0], a.v[0])]
    want, tol = attn_bound(q, *without, a.kd[0], a.vd[0], 119, a.anc[0], a.n, a.hq, a.hk, True)
    assert np.all(np.abs(got - want)[~nan] <= tol[~nan])

@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("wide,pos", [(False, 40), (False, 700), (False, 9000), (True, 40), (True, 700), (True, 6000)])
def test_attn_error_is_about_that_of_f32_arithmetic(qd, wide, pos, f16):
    """RMS error against 64 bits beside that of a plain f32 computation of the same inputs.  The
    roundings are f32's own and operands 2^-21 off at most, so it is of f32's size; an operand that
    lost its low part is 2^-9 to 2^-12 off, hundreds of times that (test_tree_cpu.py)."""
    a = _either(qd, wide, 64, pos, f16)
    got = a.call()[0].cpu().numpy()
    args = (a.q[0, :a.n * a.hq * HD].reshape(a.n, a.hq, HD), a.k[0], a.v[0], a.kd[0], a.vd[0], pos, a.anc[0], a.n, a.hq,
            a.hk)
    want = attn_plain(*args, dtype=np.float64)
    plain = rms(attn_plain(*args) - want)
    assert rms(got - want) <= 3 * plain, (rms(got - want), plain)


def test_attn_workspace_serves_both_cache_types(qd):
    """Between the bounds an f32 cache takes blocks of 128 rows and a binary16 one blocks of 16."""
    for f16 in (False, True):
        Attn(qd, 50, 16, 2, 64, 6000, [1990, 700], f16=f16).check()


def test_attn_workspace_does_not_fall_with_the_sizes(qd):
    rng = np.random.default_rng(51)
    for _ in range(2000):
        hk, g, n, b = (int(rng.integers(1, x)) for x in (40, 9, 64, 16))
        ctx = int(np.exp(rng.uniform(0, 12)))
        need = qd.tree_attn_workspace(g * hk, hk, HD, n, ctx, b)
        more = (n + 1, ctx, b), (n, ctx + int(rng.integers(1, 500)), b), (n, ctx, b + 1)
        assert need > 0 and all(qd.tree_attn_workspace(g * hk, hk, HD, *m) >= need for m in more), (hk, g, n, ctx, b)


# ------------------------------------------------------------------------------ append
def _table(ctx, hd, theta=1e4):
    a = np.arange(ctx)[:, None] * theta ** (-2.0 * np.arange(hd // 2) / hd)[None]
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("pairing", ["adjacent", "half"])
@pytest.mark.parametrize("h,hk,hd,n,pos,cnt", [(9, 3, 64, 8, [100], None), (4, 4, 64, 64, [0, 190, 3], [64, 5, 0]),
                                               (3, 1, 8, 1, [7], None), (2, 2, 128, 17, [5, 60], None),
                                               (5, 1, 24, 6, [-1, 200, 10], [6, 6, 9])])
def test_append(qd, h, hk, hd, n, pos, cnt, pairing, f16):
    b, ctx = len(pos), 200
    rng = np.random.default_rng(20)
    width = h + 2 * hk + 1  # a gap between the rows, as in a padded projection
    x = rng.standard_normal((b, n, width, hd)).astype(np.float32)
    parent, anc = _trees(rng, b, n)
    depth = (anc.sum(-1) - 1).astype(np.int32)
    if n == 6:
        depth[2, 1], depth[2, 2] = -11, 190  # outside the table: those nodes write nothing
    kv = torch.float16 if f16 else torch.float32
    q_out = torch.full((b, n, h, hd), 7.0, device="cuda")
    kd, vd = (torch.full((b, hk, n, hd), 7.0, dtype=kv, device="cuda") for _ in range(2))
    tab = _table(ctx, hd)
    xd = dev(x)
    qd.tree_append(xd, xd[:, :, h:], xd[:, :, h + hk:], n * width * hd, width * hd, q_out, kd, vd, h, hk, hd, _i32(pos),
                   dev(depth), None if cnt is None else _i32(cnt), n, pairing, dev(tab), ctx, b, kv_f16=f16)
    q, k, v = q_out.cpu().numpy(), kd.cpu().numpy(), vd.cpu().numpy()
    for i in range(b):
        for j in range(n):
            p = pos[i] + depth[i, j]
            live = (cnt is None or j < cnt[i]) and 0 <= pos[i] < ctx and depth[i, j] >= 0 and p < ctx
            if not live:
                assert np.all(q[i, j] == 7) and np.all(k[i, :, j] == 7) and np.all(v[i, :, j] == 7)
                continue
            r = x[i, j, :h + hk].astype(np.float64)
            c, s = tab[p, :, 0].astype(np.float64), tab[p, :, 1].astype(np.float64)
            e = np.empty_like(r)
            lo, hi = (slice(0, hd, 2), slice(1, hd, 2)) if pairing == "adjacent" else (slice(0, hd // 2), slice(hd // 2, hd))
            e[:, lo], e[:, hi] = r[:, lo] * c - r[:, hi] * s, r[:, lo] * s + r[:, hi] * c
            # two products and their sum, each off by half a step of at most |x0| + |x1|
            size = np.empty_like(r)
            size[:, lo] = size[:, hi] = np.abs(r[:, lo]) + np.abs(r[:, hi])
            tol = 2 * 2.0**-24 * size
            assert np.all(np.abs(q[i, j] - e[:h]) <= tol[:h])
            half = (2.0**-11 * np.abs(e[h:]) + 2.0**-25) if f16 else 0.0
            assert np.all(np.abs(k[i, :, j].astype(np.float64) - e[h:]) <= tol[h:] * 1.001 + half)
            want = x[i, j, h + hk:h + 2 * hk]
            assert np.array_equal(v[i, :, j], want.astype(np.float16) if f16 else want)
    assert np.array_equal(xd.cpu().numpy(), x)


# ------------------------------------------------------------------------------ log probabilities
def _logprob_rows(rng, rows, vocab):
    x = (rng.standard_normal((rows, vocab)) * 2).astype(np.float32)
    for r in range(rows):
        x[r, rng.integers(0, vocab, 5)] += np.float32(8)
    return x


def _run_logprobs(qd, x, tokens, top_k, stride=None, entropy=True):
    rows, vocab = x.shape
    stride = stride or vocab
    buf = np.full((rows - 1) * stride + vocab, np.float32(1e30))
    for r in range(rows):
        buf[r * stride:r * stride + vocab] = x[r]
    nt = tokens.shape[1]
    lp, h = torch.full((rows, nt), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    ti = torch.full((rows, top_k), -7, dtype=torch.int32, device="cuda")
    tl = torch.full((rows, top_k), 7.0, device="cuda")
    qd.token_logprobs(dev(buf), stride, vocab, rows, _i32(tokens), nt, lp, h if entropy else None, top_k, ti, tl)
    return lp.cpu().numpy(), h.cpu().numpy(), ti.cpu().numpy(), tl.cpu().numpy()


def _check_logprobs(x, tokens, top_k, got):
    lp, h, ti, tl = got
    for r in range(x.shape[0]):
        wlp, wh, wti, wtl = logprobs_ref(x[r], tokens[r], top_k)
        assert np.array_equal(ti[r], wti), (r, ti[r], wti)
        fin = x[r][np.isfinite(x[r])].astype(np.float64)
        spread = float(fin.max() - fin.min()) if len(fin) else 0.0
        # r is a sum of positive terms: at most 100 additions one after the other (a thread's run,
        # then the tree), each term off by the rounding of x - m (as much as |x - m| half steps)
        # and of exp (2 steps); a term with |x - m| > 100 is zero
        rel = (100 + min(spread, 100.0) + 8 + x.shape[1] / 4096) * 2.0**-24
        for g, w, near in ((lp[r], wlp, tokens[r]), (tl[r], wtl, wti)):
            assert np.array_equal(np.isnan(g), np.isnan(w))
            ok = np.isfinite(w)
            assert np.array_equal(g[~ok & ~np.isnan(w)], w[~ok & ~np.isnan(w)])
            if ok.any():
                top = np.fmax.reduce(x[r].astype(np.float64))
                # without the largest itself: 1 + r - 1 is 0 for r below 2^-53
                lse = np.log1p(np.exp(np.delete(x[r].astype(np.float64), wti[0] if top_k else np.argmax(x[r])) - top).sum())
                d = np.abs(x[r].astype(np.float64)[np.asarray(near)[ok]] - top)
                tol = rel * min(lse, 1.0) + 2.0**-24 * (d + 3 * lse + np.abs(w[ok]))
                assert np.all(np.abs(g[ok] - w[ok]) <= tol), (r, np.abs(g[ok] - w[ok]) / tol)
        assert np.isnan(h[r]) == np.isnan(wh)
        if np.isfinite(wh):
            # both terms of the entropy are positive and as exact as r, each to a few steps
            assert abs(h[r] - wh) <= (3 * rel + 8 * 2.0**-24) * wh + 1e-37, (r, h[r], wh)


@pytest.mark.parametrize("rows,vocab,nt,top_k,gap", [
    (1, 1, 1, 1, 0), (1, 49152, 1, 8, 0), (3, 2, 2, 2, 1), (2, 31, 3, 31, 0), (5, 1000, 64, 32, 3), (37, 50257, 4, 20, 0),
    (2, 152064, 2, 32, 0), (300, 321, 1, 5, 0), (4, 33, 0, 32, 7), (3, 4097, 2, 0, 2), (2, 300001, 2, 10, 1),
    (1, 2100000, 3, 32, 0)])
def test_logprobs(qd, rows, vocab, nt, top_k, gap):
    rng = np.random.default_rng(30)
    x = _logprob_rows(rng, rows, vocab)
    tokens = rng.integers(0, vocab, (rows, nt)).astype(np.int32)
    _check_logprobs(x, tokens, top_k, _run_logprobs(qd, x, tokens, top_k, vocab + gap))


def test_logprobs_ruled_out_padding_and_ties(qd):
    rng = np.random.default_rng(31)
    v = 5003
    x = _logprob_rows(rng, 9, v)
    x[0, rng.random(v) < 0.99] = -np.inf
    x[1] = -np.inf
    x[1, [17, 4000, 4001]] = [1.0, 2.0, 2.0]       # fewer finite values than top_k
    x[2] = 0.25                                      # all equal
    x[3] = np.round(x[3])                            # many equal values
    x[4] = np.float32(-3.4028235e38)                 # the type's lowest value nearly everywhere
    x[4, 77] = 3.0
    x[5] = np.where(np.arange(v) % 2, np.float32(0.0), np.float32(-0.0))  # equal as numbers
    x[6] = np.sort(x[6])
    x[7] = np.sort(x[7])[::-1]
    x[8, :40] = x[8].max() + 1                       # more equal largest values than top_k
    tokens = np.tile(np.array([0, v - 1, -1, v, 4000, 2**31 - 1], np.int32), (9, 1))
    _check_logprobs(x, tokens, 32, _run_logprobs(qd, x, tokens, 32))


def test_logprobs_rows_without_a_softmax(qd):
    v = 3000
    x = _logprob_rows(np.random.default_rng(32), 6, v)
    x[0] = -np.inf
    x[1, 50] = np.nan
    x[2, [9, 8]] = np.inf
    x[3] = np.nan
    x[4, v - 30:] = np.nan
    x[4, :v - 31] = -np.inf
    tokens = np.tile(np.array([3, 50, -1], np.int32), (6, 1))
    got = _run_logprobs(qd, x, tokens, 32)
    _check_logprobs(x, tokens, 32, got)
    assert np.all(np.isfinite(got[0][5, :2]))  # the sound row beside them


def test_logprobs_nearly_certain_rows_keep_their_digits(qd):
    """One token far above the rest: log p and the entropy are small numbers, not zero."""
    v = 49152
    x = np.zeros((4, v), np.float32)
    for r, top in enumerate([20.0, 30.0, 60.0, 85.0]):
        x[r, 1000 * r] = top
    tokens = np.array([[1000 * r, 5] for r in range(4)], np.int32)
    got = _run_logprobs(qd, x, tokens, 3)
    _check_logprobs(x, tokens, 3, got)
    assert np.all(got[0][:, 0] < 0) and np.all(got[1] > 0)


def test_logprobs_without_entropy_and_outputs_beside(qd):
    x = _logprob_rows(np.random.default_rng(33), 4, 777)
    tokens = np.zeros((4, 1), np.int32)
    lp, h, ti, tl = _run_logprobs(qd, x, tokens, 2, entropy=False)
    assert np.all(h == 7.0)
    full = _run_logprobs(qd, x, tokens, 2)
    assert np.array_equal(lp, full[0]) and np.array_equal(ti, full[2]) and np.array_equal(tl, full[3])


def test_logprobs_many_rows_same_bits_and_captured(qd):
    rows, vocab = 1500, 4099
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 3
    tok = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda", dtype=torch.int32)
    out = [torch.zeros(rows, 1, device="cuda"), torch.zeros(rows, device="cuda"),
           torch.zeros(rows, 6, dtype=torch.int32, device="cuda"), torch.zeros(rows, 6, device="cuda")]
    call = lambda: qd.token_logprobs(x, vocab, vocab, rows, tok, 1, out[0], out[1], 6, out[2], out[3])  # noqa: E731
    call()
    first = [o.clone() for o in out]
    d = x.double().log_softmax(1)
    # as in _check_logprobs with |x - m| <= 30 and a log sum of at most 12: 138 + 30 + 36 + 42 half steps
    assert (out[0] - d.gather(1, tok.long())).abs().max() <= 246 * 2.0**-24
    assert torch.equal(out[2], x.sort(dim=1, descending=True, stable=True).indices[:, :6].int())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, first))


# ------------------------------------------------------------------------------ commit
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("layers,hk,hd,n,ctx,pos,cnt", [
    (1, 1, 64, 1, 4, [0], None), (30, 3, 64, 16, 64, [40], None), (3, 2, 64, 64, 100, [30, 0, 99, 100, 101, -1], None),
    (2, 5, 128, 33, 64, [20, 31, 7], [33, 0, 5]), (2, 1, 8, 40, 50, [45, 3], [99, -1])])
def test_commit(qd, layers, hk, hd, n, ctx, pos, cnt, f16):
    rng = np.random.default_rng(40)
    b = len(pos)
    t = np.float16 if f16 else np.float32
    gap = 64  # elements between the layers
    stride = b * hk * ctx * hd + gap
    k, v = (rng.standard_normal((layers, stride)).astype(t) for _ in range(2))
    kd, vd = (rng.standard_normal((layers, b, hk, n, hd)).astype(t) for _ in range(2))
    parent, _ = _trees(rng, b, n)
    parent[:, 2:] = np.maximum(parent[:, 2:], np.arange(n)[2:] - 3)  # deeper trees
    tokens = rng.integers(0, 2, (b, n)).astype(np.int32)             # repeated children are common
    chosen = rng.integers(0, 2, (b, n, 3)).astype(np.int32)
    outs = [torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((b, n), (b,), (b,), (b,))]
    kc, vc = dev(k), dev(v)
    qd.tree_commit(_i32(tokens), _i32(parent), _i32(chosen), 3, None if cnt is None else _i32(cnt), n, dev(kd), dev(vd),
                   kc, vc, layers, stride, hk, hd, _i32(pos), ctx, b, *outs, kv_f16=f16)
    path, na, nx, po = (o.cpu().numpy() for o in outs)
    longest = 0
    for i in range(b):
        c = n if cnt is None else max(0, min(n, cnt[i]))
        want, nxt = commit_ref(tokens[i], parent[i], chosen[i, :, 0], c, pos[i], ctx)
        longest = max(longest, len(want))
        assert list(path[i]) == want + [-1] * (n - len(want))
        assert (na[i], nx[i], po[i]) == (len(want), nxt, pos[i] + len(want))
        for a, d in ((k, kd), (v, vd)):
            rows = a[:, :stride - gap].reshape(layers, b, hk, ctx, hd)
            for j, node in enumerate(want):
                rows[:, i, :, pos[i] + j] = d[:, i, :, node]
    assert np.array_equal(kc.cpu().numpy(), k) and np.array_equal(vc.cpu().numpy(), v)
    assert n == 1 or longest > 1


def test_commit_ignores_parents_that_are_not_smaller(qd):
    """Cycles and forward parents end the walk instead of turning in it."""
    n = 64
    parent = np.arange(n, dtype=np.int32)[None] + 1
    parent[0, 1] = 0
    tokens = np.zeros((1, n), np.int32)
    kd = torch.ones(1, 1, 1, n, HD, device="cuda")
    kc, vc = torch.zeros(1, 1, 80, HD, device="cuda"), torch.zeros(1, 1, 80, HD, device="cuda")
    outs = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, n), (1,), (1,), (1,))]
    qd.tree_commit(_i32(tokens), _i32(parent), _i32(tokens), 1, None, n, kd, kd, kc, vc, 1, 0, 1, HD, _i32([3]), 80, 1,
                   *outs)
    assert outs[0][0, :3].tolist() == [0, 1, -1] and outs[1].item() == 2 and outs[3].item() == 5
    assert kc[0, 0, :, 0].nonzero().flatten().tolist() == [3, 4]


def test_binding_refuses_tensors_that_are_too_small(qd):
    a = Attn(qd, 14, 4, 2, 6, 50, [20])
    a.call()
    for i, small in ((0, a.args[0][:, :-4].clone()), (2, a.args[2][:, :1]), (4, a.args[4][:, :, :5]), (5, a.args[5].double()),
                     (6, a.args[6][:, :, :3]), (10, a.args[10].long()), (11, a.args[11][:, :5]), (2, a.args[2].cpu()),
                     (2, a.args[2].transpose(1, 2))):
        bad = list(a.args)
        bad[i] = small.contiguous() if i != 2 or small.is_contiguous() else small
        with pytest.raises(ValueError):
            qd.tree_attn(*bad)
    x = torch.zeros(4, 100, device="cuda")
    with pytest.raises(ValueError):
        qd.token_logprobs(x, 101, 101, 4, None, 0, None, torch.zeros(4, device="cuda"), 0, None, None)


def test_commit_refuses_a_cache_in_another_order(qd):
    n, ctx, L, hk = 4, 10, 2, 3
    one = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    d = torch.ones(L, 1, hk, n, HD, device="cuda")
    call = lambda k, v, chosen: qd.tree_commit(  # noqa: E731
        one(1, n), one(1, n), chosen, 1, None, n, d, d, k, v, L, hk * ctx * HD, hk, HD, one(1), ctx, 1, one(1, n), one(1),
        one(1), one(1))
    k, turned = torch.zeros(L, 1, hk, ctx, HD, device="cuda"), torch.zeros(L, 1, ctx, hk, HD, device="cuda").transpose(2, 3)
    for args in ((turned, k, one(1, n)), (k, turned, one(1, n)), (k, k.clone(), one(n, 2)[:, 0])):
        with pytest.raises(ValueError, match="strides"):
            call(*args)
    assert not k.any() and not turned.any()
    a = Attn(qd, 15, 4, 2, 6, 50, [20])
    a.call()
    q = a.args[0].reshape(1, a.n, a.hq, HD).transpose(1, 2)
    with pytest.raises(ValueError, match="strides"):
        qd.tree_attn(q, *a.args[1:])

# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("f16", [False, True])
def test_a_tree_is_verified_as_one_token_at_a_time(qd, f16):
    """Two layers of a small model without feed-forward: x -> qkv -> attention -> x + Wo a, head.
    One pass over a tree, scores, acceptance and commit, against the walk that runs one token
    at a time in 64 bits; then a second tree on the committed cache."""
    rng = np.random.default_rng(50)
    H, HK, D, V, n, ctx, b, L = 4, 2, 64, 97, 12, 64, 2, 2
    width = (H + 2 * HK) * HD
    emb = rng.standard_normal((V, D)).astype(np.float32)
    wqkv = (rng.standard_normal((L, width, D)) / np.sqrt(D)).astype(np.float32)
    wo = (rng.standard_normal((L, D, H * HD)) / np.sqrt(H * HD)).astype(np.float32)
    head = (rng.standard_normal((V, D)) / 2).astype(np.float32)
    tab = _table(ctx, HD)
    t = torch.float16 if f16 else torch.float32
    kc, vc = (torch.zeros(L, b, HK, ctx, HD, dtype=t, device="cuda") for _ in range(2))
    kd, vd = (torch.zeros(L, b, HK, n, HD, dtype=t, device="cuda") for _ in range(2))
    ws = torch.empty(qd.tree_attn_workspace(H, HK, HD, n, ctx, b), dtype=torch.uint8, device="cuda")
    q_out, att = (torch.zeros(b, n, H, HD, device="cuda") for _ in range(2))
    pos = _i32([0, 0])
    dtab, dqkv, dwo, dhead, demb = dev(tab), dev(wqkv), dev(wo), dev(head), dev(emb)

    # one token at a time, in 64 bits: the cache of each sequence as lists of (k, v) rows per layer
    hist = [[([], []) for _ in range(L)] for _ in range(b)]

    def turn(x, p):
        c, s = tab[p, :, 0].astype(np.float64), tab[p, :, 1].astype(np.float64)
        lo, hi = x[..., :HD // 2], x[..., HD // 2:]
        return np.concatenate([lo * c - hi * s, lo * s + hi * c], -1)

    def step(i, token, keep):
        """Logits after `token`; keep: append its rows for good."""
        x = emb[token].astype(np.float64)
        p = len(hist[i][0][0])
        for la in range(L):
            y = (wqkv[la].astype(np.float64) @ x).reshape(-1, HD)
            qq, kk, vv = turn(y[:H], p), turn(y[H:H + HK], p), y[H + HK:]
            if f16:
                kk, vv = (a.astype(np.float16).astype(np.float64) for a in (kk, vv))
            ks, vs = hist[i][la][0] + [kk], hist[i][la][1] + [vv]
            a = np.zeros((H, HD))
            for h in range(H):
                g = h // (H // HK)
                sc = np.array([k[g] @ qq[h] for k in ks]) / 8
                w = np.exp(sc - sc.max())
                a[h] = (w[:, None] * np.array([v[g] for v in vs])).sum(0) / w.sum()
            x = x + wo[la].astype(np.float64) @ a.reshape(-1)
            if keep:
                hist[i][la] = (ks, vs)
        return head.astype(np.float64) @ x

    root = [5, 60]
    for _ in range(3):
        parent, anc = _trees(rng, b, n)
        parent[:, 2:] = np.maximum(parent[:, 2:], np.arange(n)[2:] - 2)
        tokens = rng.integers(0, V, (b, n)).astype(np.int32)
        tokens[:, 0] = root
        # the draft is right along one path: the greedy tokens that the one-by-one model gives
        depth = np.zeros((b, n), np.int32)
        masks = np.zeros((b, n), np.int64)
        saved = [[(list(k), list(v)) for k, v in hist[i]] for i in range(b)]
        for i in range(b):
            m, d = qd.tree_plan(parent[i])
            masks[i], depth[i] = m.numpy(), d.numpy()
            cur, tok = 0, root[i]
            for _ in range(4):
                tok = int(np.argmax(step(i, tok, True)))
                kids = [c for c in range(cur + 1, n) if parent[i, c] == cur]
                if not kids:
                    break
                cur = kids[-1]
                tokens[i, cur] = tok
            hist[i] = saved[i]
        # one pass over the tree
        x = demb[dev(tokens).long()].reshape(b * n, D)
        for la in range(L):
            qkv = (x @ dqkv[la].t()).reshape(b, n, H + 2 * HK, HD)
            qd.tree_append(qkv, qkv[:, :, H:], qkv[:, :, H + HK:], n * width, width, q_out, kd[la], vd[la], H, HK, HD,
                           pos, dev(depth), None, n, "half", dtab, ctx, b, kv_f16=f16)
            qd.tree_attn(q_out, n * H * HD, kc[la], vc[la], kd[la], vd[la], att, H, HK, HD, pos, dev(masks), None, n,
                         ctx, b, ws, kv_f16=f16)
            x = x + att.reshape(b * n, H * HD) @ dwo[la].t()
        logits = x @ dhead.t()
        lp, ent = torch.zeros(b * n, 1, device="cuda"), torch.zeros(b * n, device="cuda")
        ti, tl = torch.zeros(b * n, 4, dtype=torch.int32, device="cuda"), torch.zeros(b * n, 4, device="cuda")
        qd.token_logprobs(logits, V, V, b * n, dev(tokens).reshape(-1, 1), 1, lp, ent, 4, ti, tl)
        outs = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((b, n), (b,), (b,), (b,))]
        qd.tree_commit(dev(tokens), dev(parent), ti, 4, None, n, kd, vd, kc, vc, L, b * HK * ctx * HD, HK, HD, pos, ctx,
                       b, *outs, kv_f16=f16)
        path, na, nx, po = (o.cpu().numpy() for o in outs)
        top, got = ti.reshape(b, n, 4).cpu().numpy(), logits.reshape(b, n, V).cpu().numpy()
        for i in range(b):
            assert na[i] >= 2 and path[i, 0] == 0
            for j in range(na[i]):
                node = path[i, j]
                want = step(i, int(tokens[i, node]), True)
                assert np.abs(got[i, node] - want).max() <= 1e-3 * np.abs(want).max()
                g = int(top[i, node, 0])
                assert want[g] >= want.max() - 1e-3 * np.abs(want).max()
                if j + 1 < na[i]:
                    assert tokens[i, path[i, j + 1]] == g and parent[i, path[i, j + 1]] == node
                else:
                    assert nx[i] == g
            for la in range(L):
                k = kc[la, i, :, :po[i]].float().cpu().numpy()
                want = np.array(hist[i][la][0]).transpose(1, 0, 2)
                assert np.abs(k - want).max() <= 2e-3 * np.abs(want).max()
        pos = outs[3].clone()
        root = [int(t) for t in nx]


def test_the_readme_calls_run_as_they_stand(qd):
    """The drafted-token calls of README.md on two chains of three tokens, the second one drafted wrong."""
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        code = [c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "qd.tree_append" in c]
    assert len(code) == 1
    heads, kv_heads, nodes, batch, layers, vocab, max_ctx = 4, 2, 3, 2, 1, 11, 16
    f32 = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    width = (heads + 2 * kv_heads) * HD
    qkv = f32(batch, nodes, heads + 2 * kv_heads, HD)
    v = dict(
        qd=qd, torch=torch, heads=heads, kv_heads=kv_heads, nodes=nodes, batch=batch, layers=layers, vocab=vocab,
        max_ctx=max_ctx, batch_stride=nodes * width, node_stride=width, layer_stride=batch * kv_heads * max_ctx * HD,
        parents=[[-1, 0, 1], [-1, 0, 1]], q=qkv, k=qkv[:, :, heads:], v=qkv[:, :, heads + kv_heads:],
        q_out=f32(batch, nodes, heads, HD), out=f32(batch, nodes, heads, HD), pos=_i32([4, 9]),
        cos_sin=dev(_table(max_ctx, HD)), logits=f32(batch * nodes, vocab), tokens=_i32([[3, 5, 7], [3, 5, 8]]),
        logprob=f32(batch * nodes, 1), entropy=f32(batch * nodes), top_idx=i32(batch * nodes, 4),
        top_logprob=f32(batch * nodes, 4), path=i32(batch, nodes), accepted=i32(batch), next_token=i32(batch),
        new_pos=i32(batch))
    for name in ("k_drafts", "v_drafts"):
        v[name] = f32(layers, batch, kv_heads, nodes, HD)
        v[name[:-1]] = v[name][0]
    for name in ("k_caches", "v_caches"):
        v[name] = f32(layers, batch, kv_heads, max_ctx, HD)
        v[name[:-1]] = v[name][0]
    v["logits"][torch.arange(6), torch.tensor([5, 7, 9, 5, 7, 9])] = 20.0  # chosen after each node
    exec(code[0], v)
    assert v["path"].tolist() == [[0, 1, 2], [0, 1, -1]] and v["accepted"].tolist() == [3, 2]
    assert v["next_token"].tolist() == [9, 7] and v["new_pos"].tolist() == [7, 11]
    assert torch.equal(v["v_caches"][0, 0, :, 4:7], qkv[0, :, heads + kv_heads:].transpose(0, 1))
    assert v["logprob"].isfinite().all() and v["out"].isfinite().all()
