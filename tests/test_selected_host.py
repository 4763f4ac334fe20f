"""Serving with selected pages without a GPU: every entry point's host checks, and the
frequencies of pkv_rope_init."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_decode_16_gb300 as pkv
import selected_ref as ref

OK, INVALID, UNSUPPORTED, ALIAS, OUT_OF_PAGES, WORKSPACE, CUDA = range(7)
F16, BF16 = 0, 1
A = 1 << 20  # fake device addresses, 1 MiB apart: the checks never dereference them
V, D, L, F = ctypes.c_void_p, ctypes.c_double, ctypes.c_int64, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    return pkv.load_library()


@pytest.fixture(scope="module")
def pool(lib):
    h = V()
    assert lib.kv_pool_create(8, 16, 2, 128, BF16, V(A), V(A * 2), ctypes.byref(h)) == OK
    yield h
    lib.kv_pool_destroy(h)


def _tables(lib, **kw):
    a = dict(cached=A, new=A * 2, batch=4, free=A * 3, n_free=16, begin=A * 4, end=A * 5, page=16,
             pages=64, table=A * 6, cols=8, lens=A * 7, starts=A * 8, tokens=100, pos=A * 9,
             seq=A * 10, slots=A * 11)
    a.update(kw)
    return lib.paged_tables_build(V(a["cached"]), V(a["new"]), a["batch"], V(a["free"]),
                                  a["n_free"], V(a["begin"]), V(a["end"]), a["page"], a["pages"],
                                  V(a["table"]), a["cols"], V(a["lens"]), V(a["starts"]),
                                  a["tokens"], V(a["pos"]), V(a["seq"]), V(a["slots"]), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID),
    (dict(n_free=-1), INVALID),
    (dict(page=0), INVALID),
    (dict(pages=0), INVALID),
    (dict(cols=0), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(page=24), UNSUPPORTED),
    (dict(page=512), UNSUPPORTED),
    (dict(batch=16385), UNSUPPORTED),
    (dict(cached=0), INVALID),
    (dict(new=0), INVALID),
    (dict(free=0), INVALID),
    (dict(end=0), INVALID),
    (dict(table=0), INVALID),
    (dict(lens=0), INVALID),
    (dict(starts=0), INVALID),
    (dict(pos=0), INVALID),
    (dict(seq=0), INVALID),
    (dict(slots=0), INVALID),
    (dict(slots=A * 11 + 4), INVALID),
    (dict(pos=A * 9 + 2), INVALID),
    (dict(begin=A * 5), ALIAS),            # the next call's start over this one's
    (dict(lens=A), ALIAS),                 # lengths over an input
    (dict(table=A * 3 + 8), ALIAS),        # the table over the free list
    (dict(seq=A * 9 + 16), ALIAS),         # two outputs
    (dict(slots=A * 6), ALIAS),
])
def test_tables_checks(lib, kw, code):
    assert _tables(lib, **kw) == code


def _rope(rdim=128, theta=1e4, inter=0, mag=1.0, scaling=0, factor=8.0, low=1.0, high=4.0,
          ctx=8192.0):
    s = pkv._RopeStruct()
    return pkv.load_library().pkv_rope_init(ctypes.addressof(s), rdim, theta, inter, mag, scaling,
                                            factor, low, high, ctx), s


@pytest.mark.parametrize("kw,code", [
    (dict(), OK),
    (dict(rdim=0), INVALID),
    (dict(rdim=24), INVALID),
    (dict(rdim=144), INVALID),
    (dict(theta=0.0), INVALID),
    (dict(theta=math.inf), INVALID),
    (dict(theta=math.nan), INVALID),
    (dict(mag=0.0), INVALID),
    (dict(mag=1e300), INVALID),
    (dict(scaling=4), INVALID),
    (dict(scaling=-1), INVALID),
    (dict(factor=0.0), OK),                # not read
    (dict(scaling=1, factor=0.0), INVALID),
    (dict(scaling=1, low=0.0), OK),        # not read
    (dict(scaling=2, low=4.0), INVALID),
    (dict(scaling=2, ctx=0.0), INVALID),
    (dict(scaling=3, high=math.nan), INVALID),
    (dict(scaling=3, theta=1.0), INVALID),
])
def test_rope_init_checks(kw, code):
    assert _rope(**kw)[0] == code


def test_rope_init_refuses_null(lib):
    assert lib.pkv_rope_init(None, 128, 1e4, 0, 1.0, 0, 1.0, 1.0, 4.0, 8192.0) == INVALID
    with pytest.raises(ValueError, match="scaling"):
        pkv.Rope(64, scaling="ntk")
    with pytest.raises(pkv.PagedKVError, match="INVALID"):
        pkv.Rope(40)


@pytest.mark.parametrize("scaling", ["none", "linear", "turns", "index"])
@pytest.mark.parametrize("rdim,theta,factor,low,high,ctx", [
    (128, 500000.0, 8.0, 1.0, 4.0, 8192.0), (64, 10000.0, 2.5, 1.0, 32.0, 4096.0),
    (16, 10000.0, 32.0, 0.5, 7.0, 100.0), (128, 0.5, 4.0, 1.0, 32.0, 4096.0)])
def test_rope_frequencies(scaling, rdim, theta, factor, low, high, ctx):
    r = pkv.Rope(rdim, theta, scaling=scaling, factor=factor, low_turns=low, high_turns=high,
                 original_context=ctx)
    want = ref.frequencies(rdim, theta, scaling, factor, low, high, ctx) / (2 * math.pi)
    got = np.array(r.turns())
    # a few roundings of 2^-53 relative each, whole turns dropped
    d = (got - want) % 1.0
    assert np.all(np.minimum(d, 1 - d) <= 16 * 2.0 ** -53 * np.maximum(want, 2.0 ** -11))


def test_rope_scalings_keep_the_ends():
    """Pairs of many turns keep their frequency, those of few are divided by the factor."""
    plain = np.array(pkv.Rope(128, 500000.0).turns())
    for scaling, high in (("turns", 4.0), ("index", 32.0)):
        x = np.array(pkv.Rope(128, 500000.0, scaling=scaling, factor=8.0, high_turns=high).turns())
        assert x[0] == plain[0] and abs(x[-1] * 8 / plain[-1] - 1) < 1e-12
        assert np.all(np.diff(x) < 0)
        assert np.all(x <= plain) and np.all(x >= plain / 8 * (1 - 1e-12))


def _append(lib, pool, rope=True, rdim=128, **kw):
    a = dict(k=A * 3, ks=256, v=A * 4, vs=256, slots=A * 5, tokens=4, q=A * 6, qs=1024, hq=8,
             pos=A * 7, qw=0, kw=0, eps=1e-6, out=A * 8, os=1024)
    if not rope:
        a.update(q=0, hq=0, pos=0, out=0, qs=0, os=0)
    a.update(kw)
    s = _rope(rdim)[1]
    if "mag" in a:
        s.magnitude = a["mag"]
    if "reserved" in a:
        s.reserved = a["reserved"]
    return lib.kv_append_tokens(pool, V(a["k"]), L(a["ks"]), V(a["v"]), L(a["vs"]), V(a["slots"]),
                                a["tokens"], V(a["q"]), L(a["qs"]), a["hq"], V(a["pos"]),
                                V(ctypes.addressof(s)) if rope else None, V(a["qw"]), V(a["kw"]),
                                F(a["eps"]), V(a["out"]), L(a["os"]), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID),
    (dict(hq=-1), INVALID),
    (dict(k=0), INVALID),
    (dict(v=0), INVALID),
    (dict(slots=0), INVALID),
    (dict(pos=0), INVALID),
    (dict(q=0), INVALID),                   # heads without queries
    (dict(out=0), INVALID),
    (dict(hq=0), INVALID),                  # queries without heads
    (dict(q=0, hq=0), INVALID),             # an output without queries
    (dict(q=0, hq=0, out=0, qw=A * 9), INVALID),
    (dict(k=A * 3 + 8), INVALID),
    (dict(qw=A * 9 + 8), INVALID),
    (dict(slots=A * 5 + 4), INVALID),
    (dict(ks=248), INVALID),                # less than a token's heads
    (dict(vs=260), INVALID),                # not whole 16-byte vectors
    (dict(qs=1016), INVALID),
    (dict(os=0), INVALID),
    (dict(qw=A * 9, eps=-1.0), INVALID),
    (dict(kw=A * 9, eps=math.nan), INVALID),
    (dict(mag=math.inf), INVALID),
    (dict(reserved=1), INVALID),
    (dict(out=A * 6 + 512), ALIAS),         # partly over q
    (dict(out=A * 6, os=2048), ALIAS),      # q's address with other strides
    (dict(out=A * 3), ALIAS),               # over k_new
    (dict(k=A + 256), ALIAS),               # inside the K pool
    (dict(out=A * 2 + 512), ALIAS),         # inside the V pool
    (dict(slots=A * 8 + 64), ALIAS),
    (dict(rope=False, q=A * 6), INVALID),
    (dict(rope=False, pos=A * 7), INVALID),
    (dict(rope=False, kw=A * 9), INVALID),
    (dict(tokens=0), OK),
    (dict(tokens=0, q=0, out=0, k=0, v=0, slots=0, pos=0), OK),
    (dict(rope=False, tokens=0), OK),
])
def test_append_checks(lib, pool, kw, code):
    assert _append(lib, pool, **kw) == code


def test_append_alias_of_interleaved_rows(lib, pool):
    """Rows of one fused projection: q turns in place between k's and v's rows; a row
    that reaches into k's is refused."""
    row = 8 * 128 + 2 * 256
    base = dict(q=A * 6, qs=row, k=A * 6 + 2048, ks=row, v=A * 6 + 2048 + 512, vs=row, os=row)
    assert _append(lib, pool, **base, out=A * 6 + 16) == ALIAS
    assert _append(lib, pool, **base, out=A * 6 + 2048) == ALIAS
    assert _append(lib, pool, **base, out=A * 6 + 2048 + 1024 - 16) == ALIAS


def test_append_rotary_dim_beyond_the_head(lib):
    h = V()
    assert lib.kv_pool_create(8, 16, 2, 64, F16, V(A), V(A * 2), ctypes.byref(h)) == OK
    try:
        assert _append(lib, h, rdim=128) == UNSUPPORTED
    finally:
        lib.kv_pool_destroy(h)


def test_append_and_bounds_refuse_an_8_bit_pool(lib):
    h = V()
    assert lib.kv8_pool_create(8, 16, 2, 128, V(A), V(A * 2), V(A * 13), ctypes.byref(h)) == OK
    try:
        assert _append(lib, h) == UNSUPPORTED
        assert lib.kv_page_bounds(h, V(A * 5), 4, V(A * 6), None, None) == UNSUPPORTED
    finally:
        lib.kv_pool_destroy(h)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID), (dict(slots=0), INVALID), (dict(bounds=0), INVALID),
    (dict(bounds=A * 6 + 8), INVALID), (dict(slots=A * 5 + 4), INVALID),
    (dict(bounds=A + 512), ALIAS), (dict(bounds=A * 2), ALIAS), (dict(bounds=A * 5), ALIAS),
    (dict(tokens=0, slots=0), OK)])
def test_bounds_checks(lib, pool, kw, code):
    a = dict(slots=A * 5, tokens=4, bounds=A * 6)
    a.update(kw)
    assert lib.kv_page_bounds(pool, V(a["slots"]), a["tokens"], V(a["bounds"]), None,
                              None) == code


def _select(lib, **kw):
    a = dict(q=A, bounds=A * 2, table=A * 3, cols=64, lens=A * 4, batch=2, hq=8, hkv=2, d=128,
             page=16, pages=32, dt=BF16, first=1, last=2, keep=8, sel=A * 5, ws=A * 6,
             ws_bytes=1 << 19)
    a.update(kw)
    return lib.paged_select_pages(V(a["q"]), V(a["bounds"]), V(a["table"]), a["cols"],
                                  V(a["lens"]), a["batch"], a["hq"], a["hkv"], a["d"], a["page"],
                                  a["pages"], a["dt"], a["first"], a["last"], a["keep"],
                                  V(a["sel"]), V(a["ws"]), a["ws_bytes"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(hq=6, hkv=4), INVALID),
    (dict(batch=-1), INVALID), (dict(cols=0), INVALID), (dict(pages=0), INVALID),
    (dict(dt=2), INVALID), (dict(keep=0), INVALID), (dict(first=-1), INVALID),
    (dict(last=-1), INVALID), (dict(first=5, last=4), INVALID),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID),
    (dict(cols=131073), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED),
    (dict(hq=514, hkv=2), UNSUPPORTED), (dict(batch=0, q=0, ws=0), OK),
    (dict(q=0), INVALID), (dict(bounds=0), INVALID), (dict(table=0), INVALID),
    (dict(lens=0), INVALID), (dict(sel=0), INVALID), (dict(q=A + 8), INVALID),
    (dict(sel=A * 5 + 2), INVALID), (dict(ws=0), WORKSPACE), (dict(ws=A * 6 + 64), WORKSPACE),
    (dict(ws_bytes=1024), WORKSPACE), (dict(sel=A), ALIAS), (dict(sel=A * 2 + 64), ALIAS),
    (dict(sel=A * 6 + 256), ALIAS), (dict(ws=A * 3), ALIAS)])
def test_select_checks(lib, kw, code):
    assert _select(lib, **kw) == code


def test_select_workspace_size(lib):
    n = ctypes.c_size_t(7)
    assert lib.paged_select_workspace_size(2, 8, 100, None) == INVALID
    assert lib.paged_select_workspace_size(2, 0, 100, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.paged_select_workspace_size(2, 8, 131073, ctypes.byref(n)) == UNSUPPORTED
    assert pkv.paged_select_workspace_size(2, 8, 1000) >= 2 * 8 * 1000 * 12
    assert pkv.paged_select_workspace_size(0, 8, 1000) == 0


def _attend(lib, **kw):
    a = dict(q=A, k=A * 2, v=A * 4, table=A * 6, cols=64, lens=A * 7, sel=A * 8, keep=8, batch=2,
             hq=8, hkv=2, d=128, page=16, pages=32, dt=BF16, scale=0.1, out=A * 9)
    a.update(kw)
    return lib.paged_decode_attention_selected(
        V(a["q"]), V(a["k"]), V(a["v"]), V(a["table"]), a["cols"], V(a["lens"]), V(a["sel"]),
        a["keep"], a["batch"], a["hq"], a["hkv"], a["d"], a["page"], a["pages"], a["dt"],
        F(a["scale"]), V(a["out"]), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=32), UNSUPPORTED), (dict(page=20), UNSUPPORTED), (dict(hq=6, hkv=4), INVALID),
    (dict(batch=-1), INVALID), (dict(cols=0), INVALID), (dict(pages=0), INVALID),
    (dict(dt=2), INVALID), (dict(keep=0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(pages=2 ** 27), UNSUPPORTED),
    (dict(keep=2 ** 31 - 1, page=32, pages=4), UNSUPPORTED), (dict(batch=0, q=0, out=0), OK),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(table=0), INVALID),
    (dict(lens=0), INVALID), (dict(sel=0), INVALID), (dict(out=0), INVALID),
    (dict(out=A * 9 + 8), INVALID), (dict(sel=A * 8 + 1), INVALID), (dict(out=A), ALIAS),
    (dict(out=A * 2 + 512), ALIAS), (dict(out=A * 4), ALIAS), (dict(out=A * 6), ALIAS),
    (dict(out=A * 8), ALIAS)])
def test_attend_checks(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_native_binding_checks_its_arguments():
    """The native part of the binding has the five calls; each wants its own number of
    arguments and, without a GPU, raises instead of calling anything."""
    calls = pkv.load_binding()
    for name, n in (("paged_tables_build", 15), ("kv_append_tokens", 14), ("kv_page_bounds", 6),
                    ("paged_select_pages", 11), ("paged_decode_attention_selected", 10)):
        fn = getattr(calls, name)
        with pytest.raises(TypeError, match=f"expected {n} arguments"):
            fn(None)
        with pytest.raises((RuntimeError, TypeError, ValueError)):
            fn(*[None] * n)


def test_reference_table_builder_by_hand():
    """The reference of the GPU tests on a case worked out by hand: P 16, request 0 with 15
    + 2 tokens (old page 7, new page 3), 1 idle, 2 refused (no room in its row), 3 new."""
    t = [[7, -1], [5, -1], [1, -1], [-1, -1]]
    got = ref.tables([15, 3, 30, 0], [2, 0, 5, 1], [9, 3, 4, 8], 1, t, 16, 16, 10)
    table, lens, starts, pos, seq, slots, end, status = got
    assert table == [[7, 3], [5, -1], [1, -1], [4, -1]]
    assert lens == [17, 3, 30, 1] and starts == [0, 2, 2, 7, 8]
    assert pos == [15, 16, -1, -1, -1, -1, -1, 0, -1, -1]
    assert seq == [0, 0, 2, 2, 2, 2, 2, 3, -1, -1]
    assert slots == [7 * 16 + 15, 3 * 16] + [-1] * 5 + [4 * 16] + [-1] * 2
    assert end == 3 and status == ref.BAD_LEN
