"""The paged 8-bit cache without a GPU: the plan of a rotation, the refusals, which come before any
device work, and the references that the GPU tests go by."""
import ctypes
import os

import numpy as np
import pytest
import torch

import quantized_decode_gemv_gb300 as qd
from paged_helpers import E4M3, Cache, attn_ref, decode, encode, frequencies

G = 4096  # a 16-byte aligned "device" address: never dereferenced on the refused paths
SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
            ("turns", dict(factor=8.0, trained_ctx=4096, low=1.0, high=4.0)),
            ("pairs", dict(factor=16.0, trained_ctx=4096, low=1.0, high=32.0))]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qd.LIB_PATH):
        qd.build()
    return qd.load()


def _turns(t):
    return t.numpy().view(np.uint64)


@pytest.mark.parametrize("rot", [8, 32, 64, 128, 1024])
@pytest.mark.parametrize("scaling,more", SCALINGS)
def test_plan_matches_the_formulas(lib, rot, scaling, more):
    turns, mag = qd.rope_plan(1e4, rot, scaling, **more)
    f, want = frequencies(1e4, rot, scaling, more.get("factor", 1.0), more.get("trained_ctx", 0), more.get("low", 1.0),
                          more.get("high", 32.0))
    assert mag == want
    # f in 64 bits by two libraries' pow (a few 2^-53) and blends; the turns themselves end at 2^-64
    assert np.all(np.abs(_turns(turns) / 2.0**64 * 2 * np.pi - f) <= f * 2.0**-49 + 2.0**-61)


def test_plan_is_exact_to_the_last_place(lib):
    """theta 4 and 8 dimensions: f = 1, 2^-0.5, 1/2, 2^-1.5; the even ones are 2^64 / (2 pi) to the nearest."""
    turns, _ = qd.rope_plan(4.0, 8)
    inv = 2935890503282001226  # 2^64 / (2 pi) = 2935890503282001226.38...
    assert _turns(turns)[0] == inv and _turns(turns)[2] == inv // 2


def test_plan_refusals(lib):
    base = dict(theta=1e4, rot=64, kind=0, factor=2.0, ctx=4096, low=1.0, high=32.0)

    def call(out=None, **c):
        a = {**base, **c}
        t, m = (ctypes.c_uint64 * 512)(), ctypes.c_double()
        return lib.qd_rope_plan(a["theta"], a["rot"], a["kind"], a["factor"], a["ctx"], a["low"], a["high"],
                                None if out == "t" else t, None if out == "m" else ctypes.addressof(m))

    assert call() == 0 and call(kind=4) == 0
    assert call("t") == 1 and call("m") == 1
    assert call(kind=5) == 4 and call(kind=-1) == 4
    for rot in (0, 4, 12, -8, 1032):
        assert call(rot=rot) == 2
    for theta in (1.0, 0.0, -3.0, float("inf"), float("nan")):
        assert call(theta=theta) == 1
    for kind in (1, 2, 3, 4):
        assert call(kind=kind, factor=0.5) == 1 and call(kind=kind, factor=float("nan")) == 1
    for kind in (3, 4):
        assert call(kind=kind, ctx=0) == 1 and call(kind=kind, low=0.0) == 1 and call(kind=kind, high=1.0) == 1
        assert call(kind=kind, high=float("inf")) == 1 and call(kind=kind, low=float("nan")) == 1
    assert call(kind=2, theta=1e300, factor=1e300) == 1
    assert call(factor=0.0, ctx=-1, low=-1.0) == 0  # not looked at


def _call(fn, order, base, **change):
    return fn(*[{**base, **change}[k] for k in order])


def _kv(**c):
    a = dict(k_pages=G, v_pages=G, k_scale=G, v_scale=G, page_table=G, n_pages=10, page_tokens=32, n_kv_heads=2,
             head_dim=64, max_seqs=4, max_pages=5, fmt=0)
    a.update(c)
    return qd.PagedKVStruct(*[a[k] for k, _ in qd.PagedKVStruct._fields_])


def _cache_refusals(call, reads_scale_alignment=True):
    """What every entry point refuses of a cache's description; call(struct or None) -> status."""
    assert call(None) == 1
    for k in ("k_pages", "v_pages", "k_scale", "v_scale", "page_table"):
        assert call(_kv(**{k: None})) == 1
    for k in ("k_pages", "v_pages"):
        assert call(_kv(**{k: G + 8})) == 3
    for k in ("k_scale", "v_scale", "page_table"):
        assert call(_kv(**{k: G + 2})) == 3
    for hd in (32, 96, 256, 0):
        assert call(_kv(head_dim=hd)) == 4
    assert call(_kv(fmt=2)) == 4 and call(_kv(fmt=-1)) == 4
    for c in (dict(n_pages=0), dict(page_tokens=8), dict(page_tokens=24), dict(page_tokens=1040), dict(page_tokens=0),
              dict(n_kv_heads=0), dict(n_kv_heads=4097), dict(max_pages=0), dict(max_seqs=0), dict(max_seqs=257),
              dict(max_seqs=2), dict(max_pages=2**26), dict(n_pages=2**30)):
        assert call(_kv(**c)) == 2, c


def _ref(kv):
    return None if kv is None else ctypes.addressof(kv)


def test_rope_tokens_refusals(lib):
    order = "x xs o os n h hd rot pos pairing turns mag st".split()
    base = dict(x=G, xs=512, o=2 * G, os=512, n=7, h=8, hd=64, rot=32, pos=G, pairing=1, turns=G, mag=1.0, st=None)
    bad = lambda **c: _call(lib.qd_rope_tokens, order, base, **c)  # noqa: E731
    for k in "x o pos turns".split():
        assert bad(**{k: None}) == 1
    for k in "x o".split():
        assert bad(**{k: G + 4}) == 3
    assert bad(pos=G + 2) == 3 and bad(turns=G + 4) == 3 and bad(xs=514) == 3 and bad(os=513) == 3
    assert bad(pairing=2) == 4 and bad(mag=float("nan")) == 1 and bad(mag=1e300) == 1
    for c in (dict(n=0), dict(n=65537), dict(h=0), dict(h=65537), dict(hd=4), dict(hd=68), dict(hd=1032), dict(rot=0),
              dict(rot=12), dict(rot=72), dict(xs=508), dict(os=508), dict(xs=-512)):
        assert bad(**c) == 2, c
    assert bad(o=G, os=516) == 1  # in place, but another stride


def test_append_refusals(lib):
    order = "kv q k v ts qo h n rs pos b rot pairing turns mag st".split()
    kv = _kv()
    base = dict(kv=_ref(kv), q=G, k=G, v=G, ts=512, qo=G, h=8, n=7, rs=G, pos=G, b=3, rot=64, pairing=0, turns=G, mag=1.0,
                st=None)
    bad = lambda **c: _call(lib.qd_paged_append, order, base, **c)  # noqa: E731
    _cache_refusals(lambda s: bad(kv=_ref(s)))
    for k in "k v qo rs pos turns".split():
        assert bad(**{k: None}) == 1
    for k in "q k v qo".split():
        assert bad(**{k: G + 4}) == 3
    assert bad(rs=G + 2) == 3 and bad(pos=G + 2) == 3 and bad(turns=G + 4) == 3 and bad(ts=514) == 3
    assert bad(pairing=-1) == 4 and bad(mag=float("inf")) == 1
    for c in (dict(n=0), dict(n=65537), dict(h=0), dict(b=0), dict(b=5), dict(rot=4), dict(rot=72), dict(ts=508)):
        assert bad(**c) == 2, c


def test_attn_refusals(lib):
    kv = _kv()
    need = lib.qd_paged_attn_workspace(_ref(kv), 8, 7, 3)
    assert need > 0
    for c in ((None, 8, 7, 3), (_ref(kv), 7, 7, 3), (_ref(kv), 34, 7, 3), (_ref(kv), 0, 7, 3), (_ref(kv), 8, 0, 3),
              (_ref(kv), 8, 65537, 3), (_ref(kv), 8, 7, 0), (_ref(kv), 8, 7, 5)):
        assert lib.qd_paged_attn_workspace(*c) == 0, c
    for more in ((9, 3), (7, 4), (300, 4)):  # one of the largest serves them all
        assert lib.qd_paged_attn_workspace(_ref(kv), 8, *more) >= need
    order = "kv q qs o h n rs pos b scale win ws wb st".split()
    base = dict(kv=_ref(kv), q=G, qs=512, o=G, h=8, n=7, rs=G, pos=G, b=3, scale=0.125, win=0, ws=G, wb=need, st=None)
    bad = lambda **c: _call(lib.qd_paged_attn, order, base, **c)  # noqa: E731
    _cache_refusals(lambda s: bad(kv=_ref(s)))
    for k in "q o rs pos ws".split():
        assert bad(**{k: None}) == 1
    for k in "q o ws".split():
        assert bad(**{k: G + 8}) == 3
    assert bad(rs=G + 1) == 3 and bad(pos=G + 2) == 3 and bad(qs=514) == 3
    assert bad(scale=float("nan")) == 1 and bad(win=-1) == 1 and bad(wb=need - 1) == 6
    for c in (dict(h=9), dict(h=34), dict(n=0), dict(b=0), dict(b=5), dict(qs=508)):
        assert bad(**c) == 2, c


def test_attn_refuses_a_scale_beyond_f32(lib):
    """Scores are taken in powers of two: the scale times log2 e has to be a finite f32 too."""
    kv = _kv()
    need = lib.qd_paged_attn_workspace(_ref(kv), 8, 7, 3)
    call = lambda scale: lib.qd_paged_attn(_ref(kv), G, 512, G, 8, 7, G, G, 3, scale, 0, G, need, None)  # noqa: E731
    for scale in (2.4e38, -2.4e38, 3.4e38, float("inf"), float("-inf")):
        assert call(scale) == 1, scale


def test_read_refusals(lib):
    order = "kv len b ctx k v f16 st".split()
    kv = _kv()
    base = dict(kv=_ref(kv), len=G, b=3, ctx=100, k=G, v=G, f16=0, st=None)
    bad = lambda **c: _call(lib.qd_paged_read, order, base, **c)  # noqa: E731
    _cache_refusals(lambda s: bad(kv=_ref(s)))
    for k in "len k v".split():
        assert bad(**{k: None}) == 1
    assert bad(f16=2) == 1 and bad(k=G + 4) == 3 and bad(v=G + 8) == 3 and bad(len=G + 2) == 3
    assert bad(ctx=0) == 2 and bad(b=5) == 2


def test_handle_takes_tensors_that_fit_together():
    pages = torch.zeros(4, 2, 32, 64, dtype=torch.int8)
    scale = torch.zeros(4, 2, 2)
    table = torch.zeros(3, 2, dtype=torch.int32)
    kv = qd.PagedKV(pages, pages, scale, scale, table)
    assert (kv.struct.n_pages, kv.struct.page_tokens, kv.struct.n_kv_heads, kv.struct.head_dim) == (4, 32, 2, 64)
    assert (kv.max_seqs, kv.max_pages) == (3, 2)
    qd.PagedKV(pages.view(torch.float8_e4m3fn), pages.view(torch.uint8), scale, scale, table, fmt="e4m3")
    for bad in ((pages.view(torch.float8_e4m3fn), pages, scale, scale, table), (pages.float(), pages, scale, scale, table),
                (pages, pages[:3], scale, scale, table), (pages, pages, scale[:, :, :1], scale, table),
                (pages, pages, scale, scale.double(), table), (pages, pages, scale, scale, table.long()),
                (pages, pages, scale, scale, table[0]), (pages[:, :, ::2], pages[:, :, ::2], scale, scale, table),
                (pages, pages.transpose(0, 1).contiguous().transpose(0, 1), scale, scale, table)):
        with pytest.raises(ValueError):
            qd.PagedKV(*bad)
    with pytest.raises(KeyError):
        qd.PagedKV(pages, pages, scale, scale, table, fmt="e5m2")


def test_reference_codes():
    """The references' codes against torch's 8-bit float and hand-worked ties."""
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.nan_to_num(t, nan=1e9), np.nan_to_num(E4M3, nan=1e9))
    x = np.random.default_rng(1).uniform(-460, 460, 20000).astype(np.float32)
    x[:2000] *= 2.0**-15
    x[2000:2512] = np.clip(np.repeat((E4M3[:126] + E4M3[1:127]) / 2, 5)[:512], -448, 448)  # ties
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(decode(encode(x, "e4m3"), "e4m3"), decode(want, "e4m3"))
    got = encode(np.float32([0.5, -0.5, 1.5, 2.5, -2.5, 126.5, 127.4, 200, 0.49999997]), "i8").view(np.int8)
    assert got.tolist() == [1, -1, 2, 3, -3, 127, 127, 127, 0]


def test_reference_append_keeps_what_it_stands_for():
    """One position at a time: every value within one step of the last scale of what went in (half a step of
    rounding, and half a step of a smaller scale for each time that the scale grew)."""
    rng = np.random.default_rng(2)
    c = Cache(rng, 1, 2, 64, 16, [40], "i8")
    k, v = rng.normal(size=(40, 2, 64)).astype(np.float32), rng.normal(size=(40, 2, 64)).astype(np.float32)
    for i in range(40):
        c.put(0, i, k[i : i + 1], v[i : i + 1])
    for h in range(2):
        ck, sk, cv, sv = c.values(0, h, 40)
        assert np.abs(ck * sk[:, None] - k[:, h]).max() <= 2.0 * sk.max()
        assert np.all(np.abs(cv).reshape(-1, 8, 64).max() <= 127)


def test_reference_attention_of_a_single_position():
    rng = np.random.default_rng(3)
    c = Cache(rng, 1, 1, 64, 16, [5], "e4m3")
    ck, sk, cv, sv = c.values(0, 0, 5)
    o, tol = attn_ref(rng.normal(size=64).astype(np.float32), ck, sk, cv, sv, 0, 0.125, 0)
    assert np.allclose(o, cv[0] * sv[0]) and np.all(tol > 0)
    o3, _ = attn_ref(rng.normal(size=64).astype(np.float32), ck, sk, cv, sv, 3, 0.125, 1)
    assert np.allclose(o3, cv[3] * sv[3])
