"""Tree verification without a GPU: the plan of a tree, and the refusals, which come before
any device work."""
import os

import numpy as np
import pytest
import torch

import quantized_decode_gemv_gb300 as qd
from tree_helpers import attn_bound, attn_plain, attn_ref, commit_ref, logprobs_ref, mask_bits, random_tree, rms


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qd.LIB_PATH):
        qd.build()
    return qd.load()


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64])
def test_plan_matches_the_ancestor_relation(lib, n):
    parent, anc = random_tree(np.random.default_rng(n), n)
    parent[0] = -7  # not read
    mask, depth = qd.tree_plan(parent)
    assert np.array_equal(mask.numpy(), mask_bits(anc))
    assert np.array_equal(depth.numpy(), anc.sum(1) - 1)


def test_plan_refusals(lib):
    for bad in ([], [0] * 65):
        with pytest.raises(qd.QDError) as e:
            qd.tree_plan(bad)
        assert e.value.status == 2
    for bad in ([-1, 1], [-1, 0, 3, 0], [-1, -1]):
        with pytest.raises(qd.QDError) as e:
            qd.tree_plan(bad)
        assert e.value.status == 1
    assert lib.qd_tree_plan(None, 1, 16, 16) == 1


def test_plan_takes_one_tree(lib):
    """Parents of several trees in rows are not one tree of all their nodes."""
    two = [[0, 0, 1], [0, 0, 0]]
    for bad in (two, torch.tensor(two), 0):
        with pytest.raises(ValueError, match="one tree"):
            qd.tree_plan(bad)
    for bad in ([-1, 0, 0.5], [-1, 0, 2**32]):
        with pytest.raises(ValueError, match="whole numbers"):
            qd.tree_plan(bad)
    mask, depth = qd.tree_plan(torch.tensor([-1, 0, 1]))
    assert mask.tolist() == [1, 3, 7] and depth.tolist() == [0, 1, 2]

def _call(fn, order, base, **change):
    return fn(*[{**base, **change}[k] for k in order])


G = 4096  # a 16-byte aligned "device" address: never dereferenced on the refused paths


def test_append_refusals(lib):
    order = ("q k v bs ns qo kd vd f16 h hk hd pos depth nv n pairing cs ctx b st").split()
    base = dict(q=G, k=G, v=G, bs=4096, ns=512, qo=G, kd=G, vd=G, f16=0, h=4, hk=2, hd=64, pos=G, depth=G, nv=None,
                n=8, pairing=1, cs=G, ctx=32, b=2, st=None)
    bad = lambda **c: _call(lib.qd_tree_append, order, base, **c)  # noqa: E731
    for k in "q k v qo kd vd pos depth cs".split():
        assert bad(**{k: None}) == 1
    for k in "q k v qo kd vd cs".split():
        assert bad(**{k: G + 4}) == 3
    for k in "pos depth nv".split():
        assert bad(**{k: G + 2}) == 3
    assert bad(f16=2) == 1 and bad(pairing=2) == 4
    assert bad(n=0) == 2 and bad(n=65) == 2 and bad(b=0) == 2 and bad(b=17) == 2 and bad(ctx=0) == 2
    assert bad(hd=4) == 2 and bad(hd=68) == 2 and bad(hd=1032) == 2 and bad(h=0) == 2 and bad(hk=0) == 2
    assert bad(ns=255) == 2 and bad(ns=-512) == 2 and bad(bs=3839) == 2 and bad(ns=514, bs=8192) == 3 and bad(bs=4098) == 3


def test_attn_refusals(lib):
    need = qd.tree_attn_workspace(8, 4, 64, 16, 100, 2)
    assert need > 0
    for bad in ((8, 3, 64, 16, 100, 2), (9, 1, 64, 16, 100, 2), (8, 4, 128, 16, 100, 2), (8, 4, 64, 0, 100, 2),
                (8, 4, 64, 65, 100, 2), (8, 4, 64, 16, 0, 2), (8, 4, 64, 16, 100, 0), (8, 4, 64, 16, 100, 17),
                (0, 4, 64, 16, 100, 2), (8, 0, 64, 16, 100, 2)):
        assert qd.tree_attn_workspace(*bad) == 0
    order = "q qs k v kd vd f16 out h hk hd pos mask nv n ctx b ws wb st".split()
    base = dict(q=G, qs=16 * 8 * 64, k=G, v=G, kd=G, vd=G, f16=0, out=G, h=8, hk=4, hd=64, pos=G, mask=G, nv=None, n=16,
                ctx=100, b=2, ws=G, wb=need, st=None)
    bad = lambda **c: _call(lib.qd_tree_attn, order, base, **c)  # noqa: E731
    for k in "q k v kd vd out pos mask ws".split():
        assert bad(**{k: None}) == 1
    for k in "q k v kd vd out ws".split():
        assert bad(**{k: G + 8}) == 3
    assert bad(mask=G + 4) == 3 and bad(pos=G + 2) == 3 and bad(nv=G + 1) == 3 and bad(qs=16 * 8 * 64 + 2) == 3
    assert bad(f16=-1) == 1 and bad(hd=128) == 4 and bad(h=9) == 2 and bad(n=65) == 2 and bad(b=17) == 2
    assert bad(qs=16 * 8 * 64 - 4) == 2 and bad(wb=need - 1) == 6


def test_logprobs_refusals(lib):
    order = "x rs v rows t nt lp h k ti tl st".split()
    base = dict(x=G, rs=1000, v=1000, rows=3, t=G, nt=2, lp=G, h=G, k=5, ti=G, tl=G, st=None)
    bad = lambda **c: _call(lib.qd_token_logprobs, order, base, **c)  # noqa: E731
    for k in "x t lp ti tl".split():
        assert bad(**{k: None}) == 1
    assert bad(nt=0, k=0, h=None) == 1
    assert bad(x=G + 4) == 3
    for c in (dict(v=0), dict(v=(1 << 24) + 1), dict(rows=0), dict(rows=65537), dict(nt=-1), dict(nt=65), dict(k=-1),
              dict(k=33), dict(v=4), dict(rs=999)):
        assert bad(**c) == 2, c


def test_logprobs_refuses_small_arrays_off_their_type(lib):
    order = "x rs v rows t nt lp h k ti tl st".split()
    base = dict(x=G, rs=1000, v=1000, rows=3, t=G, nt=2, lp=G, h=G, k=5, ti=G, tl=G, st=None)
    for k in "t lp h ti tl".split():
        assert _call(lib.qd_token_logprobs, order, base, **{k: G + 2}) == 3, k


def test_commit_refusals(lib):
    order = "t par ch cs nv n kd vd k v f16 la ls hk hd pos ctx b path na nx po st".split()
    base = dict(t=G, par=G, ch=G, cs=1, nv=None, n=8, kd=G, vd=G, k=G, v=G, f16=1, la=3, ls=2 * 2 * 32 * 64, hk=2, hd=64,
                pos=G, ctx=32, b=2, path=G, na=G, nx=G, po=G + 16, st=None)
    bad = lambda **c: _call(lib.qd_tree_commit, order, base, **c)  # noqa: E731
    for k in "t par ch kd vd k v pos path na nx po".split():
        assert bad(**{k: None}) == 1
    for k in "kd vd k v".split():
        assert bad(**{k: G + 8}) == 3
    for k in "t par ch nv pos path na nx po".split():
        assert bad(**{k: G + 1}) == 3
    assert bad(cs=0) == 1 and bad(f16=2) == 1 and bad(po=G) == 1
    assert bad(ls=2 * 2 * 32 * 64 - 8) == 2 and bad(ls=2 * 2 * 32 * 64 + 4) == 3
    for c in (dict(la=0), dict(hk=0), dict(hd=4), dict(hd=12), dict(ctx=0), dict(b=0), dict(b=17), dict(n=0), dict(n=65)):
        assert bad(**c) == 2, c


def test_binding_refuses_tensors_that_do_not_hold_the_call():
    room = qd._room
    a = torch.zeros(8)
    with pytest.raises(ValueError, match="has type"):
        room("f", "a", a, torch.int32, -1, 8)
    with pytest.raises(ValueError, match="current device"):
        room("f", "a", a, torch.float32, 0, 8)
    with pytest.raises(ValueError, match="contiguous"):
        room("f", "a", torch.zeros(2, 8).t(), torch.float32, -1, 8)
    with pytest.raises(ValueError, match="holds 8 elements"):
        room("f", "a", a, torch.float32, -1, 9)
    b = torch.zeros(4, 6)[:, 2:]  # a view with gaps: 22 elements from its pointer on
    with pytest.raises(ValueError, match="holds 22 elements"):
        room("f", "b", b, torch.float32, -1, 23, True)
    assert room("f", "b", b, torch.float32, -1, 22, True) == b.data_ptr()
    assert room("f", "a", a, torch.float32, -1, 8) == a.data_ptr()
    assert room("f", "a", None, torch.float32, 0, 8) is None and room("f", "a", 64, torch.float32, 0, 8) == 64


def test_binding_refuses_views_in_another_order_than_the_call_takes():
    """Only the strides that a call is given may leave gaps; what lies inside them is dense."""
    f = torch.float32
    cache = torch.zeros(3, 2, 4, 10, 64)  # [layers][batch][kv head][ctx][64]
    layer, n = cache.stride(0), cache.numel()
    room = lambda t, *steps: qd._room("f", "t", t, f, -1, 1, True, steps)  # noqa: E731
    for bad in (cache.transpose(2, 3), cache.transpose(1, 2), cache.transpose(3, 4), cache[:, :, :, :9], cache[:, :, :3],
                cache[..., :32], cache[..., ::2], cache[:, :1].expand(3, 2, 4, 10, 64), cache.permute(4, 3, 2, 1, 0)):
        with pytest.raises(ValueError, match="strides"):
            room(bad, layer)
    padded = torch.zeros(3, layer + 64)[:, :layer]
    for good, step in ((cache, layer), (cache[::2], 2 * layer), (padded, layer + 64), (padded.view(3, 2, 4, 10, 64), layer + 64),
                       (cache[:, 1:], layer), (cache[1:, :1], layer)):
        assert room(good, step) == good.data_ptr()
    assert qd._room("f", "t", cache[1:], f, -1, 2 * layer, True, (layer,)) == cache[1:].data_ptr()
    with pytest.raises(ValueError, match=f"holds {n - layer} elements"):
        qd._room("f", "t", cache[1:], f, -1, n, True, (layer,))
    # the parts of a fused projection, whole and a head short, nodes before sequences, padded rows
    qkv = torch.zeros(2, 5, 8, 64)
    for good in (qkv[:, :, 4:], qkv[:, :, 4:6], qkv[:, :, 1:].transpose(0, 1), qkv.view(10, 512)[:, 128:], qkv[:, :3, 2:]):
        assert room(good, 5 * 512, 512) == good.data_ptr()
    for bad in (qkv[:, :, 4:].transpose(2, 3), qkv[:, :, 4:].transpose(1, 2), qkv[..., :32], qkv[:, ::2, 4:]):
        with pytest.raises(ValueError, match="strides"):
            room(bad, 5 * 512, 512)
    # one column of the largest logits' indices; logits inside padded rows
    top = torch.zeros(2, 5, 4, dtype=torch.int32)
    assert qd._room("f", "t", top[..., 1], torch.int32, -1, 37, True, (4,)) == top[..., 1].data_ptr()
    with pytest.raises(ValueError, match="strides"):
        qd._room("f", "t", top[..., 0].t(), torch.int32, -1, 37, True, (4,))
    rows = torch.zeros(6, 104)[:, :97]
    assert room(rows, 104) == rows.data_ptr() and room(rows.view(2, 3, 97), 104) == rows.data_ptr()

def test_references_on_hand_values():
    """The references themselves: a two-token softmax, ties, and a walk with a repeated child."""
    lp, h, idx, tl = logprobs_ref([0.0, np.log(3.0), -np.inf], [1, 2, 5, -1], 3)
    assert np.allclose(lp, [np.log(0.75), -np.inf, -np.inf, -np.inf])
    assert np.isclose(h, -(0.75 * np.log(0.75) + 0.25 * np.log(0.25)))
    assert list(idx) == [1, 0, 2] and np.allclose(tl[:2], np.log([0.75, 0.25]))
    assert list(logprobs_ref([1.0, 2.0, 2.0, 1.0], [], 4)[2]) == [1, 2, 0, 3]
    assert list(logprobs_ref([np.nan, 2.0, -np.inf], [], 3)[2]) == [1, 2, 0]
    # 0 -> {1: a, 2: b, 3: b}, 3 -> {4: c}; the first child with the token is taken, which has no child
    toks, par = [9, 1, 2, 2, 3], [-1, 0, 0, 0, 3]
    assert commit_ref(toks, par, [2, 0, 3, 3, 7], 5, 10, 100) == ([0, 2], 3)
    assert commit_ref(toks, par, [2, 0, 3, 3, 7], 2, 10, 100) == ([0], 2)
    assert commit_ref(toks, par, [1, 0, 3, 3, 7], 5, 10, 11) == ([0], 1)
    assert commit_ref(toks, par, [1, 0, 3, 3, 7], 5, 11, 11) == ([], -1)


def _tree_rows(seed, pos, n=9, hq=6, hk=2):
    rng = np.random.default_rng(seed)
    mk = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    q, k, v, kd, vd = 1.5 * mk(n, hq, 64), mk(hk, pos, 64), mk(hk, pos, 64), mk(hk, n, 64), mk(hk, n, 64)
    return q, k, v, kd, vd, pos, random_tree(rng, n)[1], n, hq, hk


def test_attention_references_agree():
    for pos in (0, 3, 200):
        args = _tree_rows(pos, pos)
        want = attn_ref(*args)[0]
        out, tol = attn_bound(*args, False)
        assert np.abs(out - want).max() < 1e-13 and np.abs(attn_plain(*args, dtype=np.float64) - want).max() < 1e-13
        assert np.all(np.abs(attn_plain(*args) - want) <= tol)


def _bits(a, n):
    """a rounded to n significant bits."""
    m, e = np.frexp(np.asarray(a, np.float64))
    return np.ldexp(np.round(np.ldexp(m, n)), e - n)


@pytest.mark.parametrize("pos", [40, 700, 6000])
@pytest.mark.parametrize("operand", ["q", "k", "v", "p"])
def test_an_operand_without_its_low_part_is_far_from_f32(pos, operand):
    """What the comparison with plain f32 arithmetic on the GPU would see: operands of 22 bits pass
    it, one of 11 (a single TF32 or binary16 part) or 16 (two of the three bfloat16 parts) does not."""
    args = _tree_rows(pos, pos)
    want = attn_plain(*args, dtype=np.float64)
    plain = rms(attn_plain(*args) - want)

    def error(bits, only=None):
        cut = lambda name, a: _bits(a, bits) if only in (None, name) else a  # noqa: E731
        return rms(attn_plain(*args, dtype=np.float64, part=cut) - want)

    assert error(22) <= 3 * plain
    assert error(11, operand) > 30 * plain and error(16, operand) > 3 * plain
