"""The 8-bit cache without a GPU: pool handle and allocator, refusals of every
entry point before anything is launched, and the plain forms' own ground."""
import ctypes

import numpy as np
import pytest

import kv8_ref
import paged_kv_decode_16_gb300 as pkv

OK, INVALID, UNSUPPORTED, ALIAS, OUT_OF_PAGES, WORKSPACE, CUDA, DEVCHECK, REFCOUNT = range(9)
F16, BF16, E4M3 = 0, 1, 2
A = 1 << 24  # fake, 256-byte aligned "device" addresses; validation never dereferences them
V = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return pkv.load_library()


def _pool(lib, np_=8, p=16, h=2, d=128, k=A, v=A * 2, s=A * 3):
    out = V()
    code = lib.kv8_pool_create(np_, p, h, d, V(k), V(v), V(s), ctypes.byref(out))
    return code, out


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), UNSUPPORTED), (dict(p=24), UNSUPPORTED), (dict(p=512), UNSUPPORTED),
    (dict(np_=0), INVALID), (dict(h=0), INVALID),
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(s=0), INVALID),
    (dict(k=A + 8), INVALID), (dict(s=A * 3 + 2), INVALID),
])
def test_pool_create_refuses(lib, kw, code):
    assert _pool(lib, **kw)[0] == code


def test_pool_handle_and_allocator(lib):
    code, h = _pool(lib)
    assert code == OK
    dt, d = ctypes.c_int(), ctypes.c_int()
    assert lib.kv_pool_info(h, None, None, None, ctypes.byref(d), ctypes.byref(dt)) == OK
    assert (dt.value, d.value) == (E4M3, 128)
    assert lib.kv8_pool_scales(h) == A * 3 and lib.kv8_pool_scales(None) is None
    ids = (ctypes.c_int32 * 3)()
    assert lib.kv_pool_alloc_pages(h, 3, ids) == OK and lib.kv_pool_free_count(h) == 5
    assert lib.kv_pool_release_pages(h, ids, 3) == OK
    # the 16-bit calls refuse it
    assert lib.kv_append(h, V(A * 4), V(A * 5), V(A * 6), 4, V(A * 7), 2, None,
                         None) == UNSUPPORTED
    assert lib.kv_append_rope(h, V(A * 4), V(A * 5), V(A * 6), V(A * 7), 4, V(A * 8), 2, 8,
                              ctypes.c_double(1e4), None, None, ctypes.c_float(0), V(A * 9), None,
                              None) == UNSUPPORTED
    assert lib.kv_gather(h, V(A * 5), 4, V(A * 6), 2, 64, V(A * 8), V(A * 9), None,
                         None) == UNSUPPORTED
    assert lib.kv_pool_destroy(h) == OK
    # a 16-bit pool has no scales
    assert lib.kv_pool_create(8, 16, 2, 128, BF16, V(A), V(A * 2), ctypes.byref(h)) == OK
    assert lib.kv8_pool_scales(h) is None
    assert lib.kv8_append(h, V(A * 4), V(A * 5), BF16, V(A * 6), 4, 2, V(A * 7), None, 2, None,
                          None) == UNSUPPORTED
    assert lib.kv_pool_destroy(h) == OK
    # e4m3 is no 16-bit pool's type
    assert lib.kv_pool_create(8, 16, 2, 128, E4M3, V(A), V(A * 2), ctypes.byref(h)) == INVALID


def test_prefix_cache_over_an_8_bit_pool(lib):
    code, h = _pool(lib, np_=6)
    assert code == OK
    c = pkv.PrefixCache(h)
    ids = (ctypes.c_int32 * 2)()
    assert lib.kv_pool_alloc_pages(h, 2, ids) == OK
    tokens = list(range(32))
    assert c.insert(tokens, list(ids)) == 2
    assert c.match(tokens + [5]) == list(ids)
    c.destroy()
    assert lib.kv_pool_destroy(h) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), OK), (dict(n=-1), INVALID), (dict(dt=5), INVALID), (dict(dt=E4M3), INVALID),
    (dict(stride=0), INVALID), (dict(seqs=-1), INVALID),
    (dict(n=5), INVALID),                      # more tokens than table rows, no seq_ids
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(pos=0), INVALID), (dict(table=0), INVALID),
    (dict(k=A * 4 + 2), INVALID),
    (dict(k=A + 256), ALIAS), (dict(v=A * 2 + 256), ALIAS), (dict(pos=A * 3), ALIAS),
    (dict(table=A), ALIAS), (dict(seq=A * 3 + 16, n=2), ALIAS),
    (dict(theta=0.0), INVALID), (dict(theta=float("nan")), INVALID),
    (dict(theta=float("inf")), INVALID), (dict(theta=1e4, hq=0), INVALID),
    (dict(theta=1e4, q=0), INVALID), (dict(theta=1e4, qo=0), INVALID),
    (dict(theta=1e4, qo=A * 9 + 64), ALIAS),   # q_out inside q, not q itself
    (dict(theta=1e4, qo=A * 4), ALIAS), (dict(theta=1e4, qo=A * 2), ALIAS),
    (dict(theta=1e4, qw=A * 11 + 1), INVALID),
    (dict(theta=1e4, qw=A * 11, eps=-1.0), INVALID),
    (dict(theta=1e4, qw=A * 11, eps=float("nan")), INVALID),
])
def test_append_refuses(lib, kw, code):
    a = dict(k=A * 4, v=A * 5, dt=BF16, table=A * 6, stride=4, seqs=4, pos=A * 7, seq=0, n=2,
             q=A * 9, qo=A * 10, hq=8, theta=None, qw=0, kw=0, eps=1e-6)
    a.update(kw)
    st, h = _pool(lib)
    assert st == OK
    if a["theta"] is None:
        got = lib.kv8_append(h, V(a["k"]), V(a["v"]), a["dt"], V(a["table"]), a["stride"],
                             a["seqs"], V(a["pos"]), V(a["seq"]), a["n"], None, None)
    else:
        got = lib.kv8_append_rope(h, V(a["q"]), V(a["k"]), V(a["v"]), a["dt"], V(a["table"]),
                                  a["stride"], a["seqs"], V(a["pos"]), V(a["seq"]), a["n"],
                                  a["hq"], ctypes.c_double(a["theta"]), V(a["qw"]), V(a["kw"]),
                                  ctypes.c_float(a["eps"]), V(a["qo"]), None, None)
    assert got == code
    assert lib.kv_pool_destroy(h) == OK


_ARGS = dict(q=A, k=A * 2, v=A * 3, s=A * 4, table=A * 5, stride=4, lens=A * 6, batch=2, nq=1,
             hq=8, hkv=2, d=128, p=16, np_=8, dt=BF16, scale=0.088, out=A * 7, ws=A * 8,
             ws_bytes=1 << 20, workers=0, kn=A * 9, vn=A * 10, pos=A * 11, theta=0.0, qw=0)


def _call(lib, which, kw):
    a = dict(_ARGS, **kw)
    if which == "step":
        return lib.paged_decode_step_kv8(
            V(a["kn"]), V(a["vn"]), V(a["pos"]), V(a["q"]), V(a["k"]), V(a["v"]), V(a["s"]),
            V(a["table"]), a["stride"], V(a["lens"]), a["batch"], a["hq"], a["hkv"], a["d"],
            a["p"], a["np_"], a["dt"], ctypes.c_float(a["scale"]), ctypes.c_double(a["theta"]),
            V(a["qw"]), None, ctypes.c_float(1e-6), V(a["out"]), V(a["ws"]), a["ws_bytes"],
            a["workers"], None)
    head = (V(a["q"]), V(a["k"]), V(a["v"]), V(a["s"]), V(a["table"]), a["stride"], V(a["lens"]),
            a["batch"])
    tail = (a["hq"], a["hkv"], a["d"], a["p"], a["np_"], a["dt"], ctypes.c_float(a["scale"]),
            V(a["out"]), V(a["ws"]), a["ws_bytes"], a["workers"], None)
    if which == "multi":
        return lib.paged_decode_attention_multi_kv8(*head, a["nq"], *tail)
    return lib.paged_decode_attention_kv8(*head, *tail)


@pytest.mark.parametrize("which", ["decode", "multi", "step"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=0, q=0, out=0, ws=0), OK),
    (dict(d=96), UNSUPPORTED), (dict(p=8), UNSUPPORTED), (dict(p=272), UNSUPPORTED),
    (dict(hq=6, hkv=4), INVALID), (dict(batch=-1), INVALID), (dict(np_=0), INVALID),
    (dict(stride=0), INVALID), (dict(dt=E4M3), INVALID), (dict(dt=7), INVALID),
    (dict(workers=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(s=0), INVALID), (dict(lens=0), INVALID),
    (dict(q=A + 8), INVALID), (dict(s=A * 4 + 2), INVALID), (dict(out=A * 7 + 4), INVALID),
    (dict(ws=0), WORKSPACE), (dict(ws=A * 8 + 64), WORKSPACE),
    (dict(np_=1 << 27), UNSUPPORTED),          # rows beyond a 32-bit coordinate
    (dict(out=A), ALIAS), (dict(out=A * 2 + 4096), ALIAS), (dict(out=A * 4), ALIAS),
    (dict(out=A * 5), ALIAS), (dict(out=A * 6), ALIAS), (dict(out=A * 8 + 1024), ALIAS),
])
def test_attention_refuses(lib, which, kw, code):
    assert _call(lib, which, kw) == code


@pytest.mark.parametrize("nq,code", [(0, INVALID), (-3, INVALID), (65, UNSUPPORTED)])
def test_multi_refuses_query_counts(lib, nq, code):
    assert _call(lib, "multi", dict(nq=nq)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(kn=0), INVALID), (dict(vn=0), INVALID), (dict(pos=0), INVALID),
    (dict(kn=A * 9 + 2), INVALID), (dict(theta=-1.0), INVALID),
    (dict(theta=float("inf")), INVALID),
    (dict(qw=A * 12), INVALID),                # a norm without the rotation
    (dict(theta=1e4, qw=A * 12 + 1), INVALID),
    (dict(kn=A * 7), ALIAS), (dict(pos=A * 7), ALIAS), (dict(theta=1e4, vn=A * 7), ALIAS),
    (dict(kn=A * 2), ALIAS), (dict(v=A * 2), ALIAS), (dict(s=A * 3 + 4096), ALIAS),
])
def test_step_refuses(lib, kw, code):
    assert _call(lib, "step", kw) == code


def test_workspace_size_refuses(lib):
    n = ctypes.c_size_t()
    f = lib.paged_decode_kv8_workspace_size
    assert f(2, 1, 8, 2, 128, 0, None) == INVALID
    assert f(2, 0, 8, 2, 128, 0, ctypes.byref(n)) == INVALID
    assert f(2, 65, 8, 2, 128, 0, ctypes.byref(n)) == UNSUPPORTED
    assert f(2, 1, 8, 3, 128, 0, ctypes.byref(n)) == INVALID
    assert f(2, 1, 8, 2, 80, 0, ctypes.byref(n)) == UNSUPPORTED


def test_plain_encoding_against_the_format():
    torch = pytest.importorskip("torch")
    # every byte's value, and the nearest byte of many values, as torch has them
    b = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(kv8_ref.VALUES, b.view(torch.float8_e4m3fn).double().numpy(),
                          equal_nan=True)
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 30
    x = torch.cat([x, x * 2.0 ** -12, torch.tensor([0.0, 448.0, 2.0 ** -10, 3 * 2.0 ** -10])])
    got = kv8_ref.encode(x.double().numpy())
    assert np.array_equal(got, x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert kv8_ref.encode(np.array([1e9, -1e9])).tolist() == [0x7E, 0xFE]
    assert kv8_ref.encode(np.array([np.inf, np.nan])).tolist() == [0x7F, 0x7F]


def test_plain_scale_is_the_smallest():
    for e in range(-60, 41):
        top = 448.0 * 2.0 ** e
        assert kv8_ref.need_exp(top) == e
        assert kv8_ref.need_exp(np.nextafter(top, np.inf)) == min(e + 1, 40)
