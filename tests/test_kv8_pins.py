"""Pins of the 8-bit caches' oracle against facts fixed independently of it, and
the refusals of the 8-bit caches' and the shared rows' calls, which need no GPU."""

import ctypes as C
import os

import numpy as np
import pytest
import torch

from draft_tree_construction_depth_amd import _lib
from oracle import kv8 as K
from oracle import verify as O


# ---- codes ----------------------------------------------------------------------
def test_codes_stand_for_the_formats_values():
    bytes_ = torch.arange(256).to(torch.uint8)
    for kind, dtype in (("e4m3", torch.float8_e4m3fn), ("i8", torch.int8)):
        want = bytes_.view(dtype).to(torch.float64).numpy()
        assert np.array_equal(K.decode(kind), want, equal_nan=True)
    assert K.decode("e4m3")[[0x38, 0x01, 0x7E, 0xB8]].tolist() == [1.0, 2.0 ** -9, 448.0, -1.0]


def test_nearest_code():
    """Every code's own value, midpoints (to the even code) and points just beside them."""
    for kind in ("e4m3", "i8"):
        v = K.decode(kind)
        codes = [c for c in range(256) if abs(v[c]) <= K.MOST[kind]]
        back = K.decode(kind)[K.nearest(v[codes], kind)]
        assert np.array_equal(back, v[codes]) and np.array_equal(np.signbit(back), np.signbit(v[codes]))
        grid = sorted({v[c] for c in codes})
        code = {v[c]: c for c in codes}
        for a, b in zip(grid, grid[1:]):
            mid = (a + b) / 2
            got = v[K.nearest(np.array([mid, np.nextafter(mid, a), np.nextafter(mid, b)]), kind)]
            assert got[0] == (a if code[a] % 2 == 0 else b) and got[1] == a and got[2] == b
        assert v[K.nearest(np.array([1e9, -1e9]), kind)].tolist() == [K.MOST[kind], -K.MOST[kind]]
    y = np.random.default_rng(0).uniform(-460, 460, 20000).astype(np.float32)
    e4m3 = torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(K.nearest(y, "e4m3"), e4m3)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_quantised_rows(kind):
    """The largest element has the largest code, and what is read back is off by half a step of the
    format and the float32 roundings of scale, 1 / scale and product."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((500, 40)) * 10.0 ** rng.uniform(-20, 20, (500, 1))).astype(np.float32)
    codes, scale = K.quantise(x, kind)
    back = K.values(codes, scale, kind)
    top = np.abs(x).max(-1)
    assert np.array_equal(np.abs(K.decode(kind)[codes]).max(-1), np.full(500, K.MOST[kind]))
    assert np.all(np.abs(scale * K.MOST[kind] / top - 1) <= 2.0 ** -22)
    if kind == "i8":
        step = np.broadcast_to(scale[:, None] / 2, x.shape)
    else:
        step = np.maximum(np.abs(x) * 2.0 ** -4, scale[:, None] * 2.0 ** -10)
    assert np.all(np.abs(back - x) <= step + 2.0 ** -22 * top[:, None])
    # small, zero and non-finite rows
    odd = np.zeros((6, 8), np.float32)
    odd[1, 3], odd[2, 2], odd[3, 5], odd[4, 7], odd[5, 0] = 1e-40, np.nan, np.inf, -np.inf, -0.0
    codes, scale = K.quantise(odd, kind)
    assert scale[0] == scale[1] == scale[5] == np.float32(2.0 ** -126) and np.isnan(scale[2:5]).all()
    assert not codes[2:5].any() and not K.values(codes, scale, kind)[[0, 5]].any()
    assert np.isnan(K.values(codes, scale, kind)[2:5]).all()


def test_append_places_and_turns_rows():
    """As the 16-bit append does, up to the rows' quantisation."""
    rng = np.random.default_rng(2)
    batch, T, H, dh, ps = 3, 5, 2, 16, 4
    k, v = (rng.standard_normal((batch, T, H, dh)).astype(np.float32) for _ in range(2))
    a = np.arange(40)[:, None] * np.linspace(1, 0.1, dh // 2)
    rope = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    table = np.array([[3, 0, 9], [1, -1, 4], [2, 5, 6]], np.int32)  # 7 pages: 9 is none
    past, nn = np.array([2, 3, -1], np.int32), np.array([4, 2, 4], np.int32)
    dep = np.array([[1, 1, 2, 3]] * 3, np.int32)
    for inter in (False, True):
        zero, none = np.zeros((7, H, ps, dh), np.uint8), np.zeros((7, H, ps), np.float32)
        kc, vc, ks, vs = K.append(k, v, zero, zero, none, none, "i8", past, rope, inter, table, dep, nn)
        _, ke, ve = O.append(k.astype(float), k.astype(float), v.astype(float), np.zeros(zero.shape),
                             np.zeros(zero.shape), past, rope.astype(float), inter, table, dep, nn)
        for c, s, want in ((kc, ks, ke), (vc, vs, ve)):
            assert np.all(np.abs(K.values(c, s, "i8") - want) <= s[..., None] * 0.501)
            assert np.array_equal(s > 0, np.abs(want).max(-1) > 0)


def test_reading_back():
    codes = np.arange(2 * 1 * 4 * 8, dtype=np.uint8).reshape(2, 1, 4, 8)
    scales = np.arange(1.0, 9.0, dtype=np.float32).reshape(2, 1, 4)
    got = K.read(codes, scales, "i8", [2, 0], [3, 9], 4, np.array([[1, -1], [0, 1]]))
    assert np.array_equal(got[0, :2, 0], np.array([np.arange(48, 56) * 7.0, np.arange(56, 64) * 8.0]))
    assert not got[0, 2:].any()  # an unmapped page, then the count
    assert np.array_equal(got[1, :, 0], np.arange(32).reshape(4, 8) * np.arange(1.0, 5.0)[:, None])


def test_shared_rows_are_the_requests_own():
    """Attention through a table whose requests share pages is that over caches of their own."""
    rng = np.random.default_rng(3)
    T, ps, past = 2, 4, np.array([9, 11], np.int32)
    table = np.array([[5, 2, 0, 6], [5, 2, 1, 3]])
    kc, vc = rng.standard_normal((7, 1, ps, 8)), rng.standard_normal((7, 1, ps, 8))
    q = rng.standard_normal((2, T, 2, 8))
    got = O.attend(q, kc, vc, past, table)
    for b in range(2):
        k1 = kc[table[b]].transpose(1, 0, 2, 3).reshape(1, 1, 16, 8)
        v1 = vc[table[b]].transpose(1, 0, 2, 3).reshape(1, 1, 16, 8)
        want = O.attend(q[b:b + 1], k1, v1, past[b:b + 1])
        assert all(np.allclose(g[b], w[0], rtol=1e-13) for g, w in zip(got, want))


# ---- refusals: nothing is enqueued, so any pointer will do ------------------------
FAKE, ODD, TORN = C.c_void_p(0x100000), C.c_void_p(0x100008), C.c_void_p(0x100002)  # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from draft_tree_construction_depth_amd import _build
        _build.build_library()
    return _lib.lib()


def test_append_refusals(L):
    def call(q=FAKE, k=FAKE, dtype=0, batch=2, T=9, Hq=8, Hkv=2, dh=128, qs=1024, ks=256, vs=256, rope=FAKE,
             rl=100, rot=128, inter=0, past=FAKE, table=FAKE, width=4, pages=16, ps=16, code=3, kc=FAKE, vc=FAKE,
             ksc=FAKE, vsc=FAKE, qo=FAKE):
        return L.ddtree_append_kv8(q, k, FAKE, dtype, batch, T, Hq, Hkv, dh, qs, ks, vs, rope, rl, rot, inter, past,
                                   None, None, table, width, pages, ps, code, kc, vc, ksc, vsc, qo, None)
    for bad in (dict(k=None), dict(q=None), dict(qo=None), dict(kc=None), dict(vc=None), dict(ksc=None), dict(vsc=None),
                dict(past=None), dict(rope=None), dict(dtype=1), dict(dtype=3), dict(code=0), dict(code=2), dict(code=5),
                dict(T=0), dict(Hkv=0), dict(Hq=7), dict(dh=0), dict(rot=-16), dict(rot=256), dict(rl=-1),
                dict(inter=2), dict(qs=1016), dict(ks=128), dict(vs=128), dict(k=ODD), dict(kc=ODD), dict(qo=ODD),
                dict(rope=ODD), dict(ksc=TORN), dict(vsc=TORN), dict(pages=0), dict(ps=0), dict(width=0),
                dict(table=None), dict(batch=-1)):
        assert call(**bad) == -1, bad
    for bad in (dict(T=514), dict(dh=516, qs=4128, ks=1032, vs=1032), dict(dh=1024, qs=8192, ks=2048, vs=2048),
                dict(rot=120), dict(ps=24), dict(qs=1028), dict(ks=260), dict(batch=1 << 31), dict(batch=1 << 24, T=1)):
        assert call(**bad) == -2, bad
    assert call(batch=0) == 0


def attention_call(L, name):
    """A call of one of the two attentions with one thing wrong, as a function of that thing."""
    def call(q=FAKE, dtype=0, batch=2, T=9, Hq=8, Hkv=2, dh=128, code=4, kc=FAKE, ksc=FAKE, vsc=FAKE, table=FAKE,
             width=4, pages=16, ps=16, past=FAKE, shared=FAKE, scale=0.1, out=FAKE, ws=FAKE, n=1 << 40):
        if name == "kv8":
            return L.ddtree_attention_kv8(q, dtype, batch, T, Hq, Hkv, dh, code, kc, FAKE, ksc, vsc, table, width,
                                          pages, ps, past, None, None, shared, scale, out, None, ws, n, None)
        return L.ddtree_attention_shared(q, dtype, batch, T, Hq, Hkv, dh, kc, FAKE, table, width, pages, ps, past,
                                         None, None, shared, scale, out, None, ws, n, None)
    return call


@pytest.mark.parametrize("name", ["kv8", "shared"])
def test_attention_refusals(L, name):
    call = attention_call(L, name)
    for T, width in ((9, 4), (9, 1 << 16), (40, 1 << 16)):  # rows shared apart in the second alone
        for bad in (dict(q=None), dict(kc=None), dict(past=None), dict(out=None), dict(ws=None), dict(q=ODD),
                    dict(kc=ODD), dict(out=ODD), dict(ws=ODD), dict(dtype=1), dict(dtype=3), dict(Hq=0), dict(Hq=7),
                    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                    dict(scale=3.4e38), dict(table=None), dict(pages=0), dict(width=0), dict(batch=-1)):
            assert call(**{"T": T, "width": width, **bad}) == -1, bad
        for bad in (dict(dh=96), dict(dh=512), dict(ps=24), dict(batch=1 << 31), dict(width=1 << 24)):
            assert call(**{"T": T, "width": width, **bad}) == -2, bad
        assert call(T=T, width=width, n=0) == -3
        assert call(T=T, width=width, batch=0) == 0
    assert call(T=0) == -1 and call(T=514) == -2
    if name == "kv8":
        for bad in (dict(code=0), dict(code=2), dict(code=5), dict(ksc=None), dict(vsc=None), dict(ksc=TORN)):
            assert call(**bad) == -1, bad
        # a contiguous cache has nothing to share, and is fine without
        assert call(table=None, pages=2, width=1) == -1
        assert call(table=None, pages=2, width=1, shared=None, n=0) == -3
    else:
        assert call(shared=None) == -1


def test_attention_workspaces(L):
    plain, kv8 = L.ddtree_attention_workspace_size, L.ddtree_attention_kv8_workspace_size
    shared = L.ddtree_attention_shared_workspace_size
    size = (6, 9, 8, 2, 128, 1 << 14, 16)
    assert kv8(*size, 0) == plain(*size) > 0
    # the shared rows' part: a float32 row for each row of q, beside the larger of the two passes' needs
    assert kv8(*size, 1) == shared(*size) >= 6 * 9 * 8 * (128 + 2) * 4 + plain(*size)
    # one request; 84 rows a head; caches that hold too few rows for sharing to pay: 192 MiB
    for alone in ((1, 9, 8, 2, 128, 1 << 14, 16), (6, 21, 8, 2, 128, 1 << 14, 16), (6, 9, 8, 2, 128, 40, 16)):
        assert kv8(*alone, 1) == shared(*alone) == plain(*alone) > 0
    rows = (192 << 20) // (5 * 2 * 2 * 128)  # of 8 bits, for five requests beside the first
    assert kv8(6, 9, 8, 2, 128, rows // 16 + 1, 16, 1) > plain(6, 9, 8, 2, 128, rows // 16 + 1, 16)
    assert kv8(6, 9, 8, 2, 128, rows // 16 - 1, 16, 1) == plain(6, 9, 8, 2, 128, rows // 16 - 1, 16)
    for bad in ((0, 9, 8, 2, 128, 4, 16), (2, 9, 8, 2, 96, 4, 16), (2, 514, 8, 2, 128, 4, 16)):
        assert kv8(*bad, 0) == kv8(*bad, 1) == shared(*bad) == 0


def test_attentions_of_more_than_a_launch_are_refused(L):
    for batch, T, Hq, Hkv in ((1 << 24, 1, 1, 1), (1 << 21, 1, 8, 8), (1 << 26, 1, 8, 8)):
        for s in (0, 1):
            assert L.ddtree_attention_kv8_workspace_size(batch, T, Hq, Hkv, 64, 1, 16, s) == 0
        for name in ("kv8", "shared"):
            assert attention_call(L, name)(batch=batch, T=T, Hq=Hq, Hkv=Hkv, dh=64, width=1, n=1 << 60) == -2


def test_compaction_refusals(L):
    def call(k=FAKE, ksc=FAKE, vsc=FAKE, layers=2, pages=16, heads=4, ps=16, dh=128, table=FAKE, width=4, batch=3,
             past=FAKE, depth=15):
        return L.ddtree_compact_kv8(k, FAKE, ksc, vsc, layers, pages, heads, ps, dh, table, width, batch, past, FAKE,
                                    FAKE, depth, FAKE, None)
    for bad in (dict(k=None), dict(k=ODD), dict(ksc=None), dict(vsc=TORN), dict(table=None), dict(past=None),
                dict(layers=-1), dict(pages=0), dict(ps=0), dict(width=0), dict(dh=0), dict(depth=0)):
        assert call(**bad) == -1, bad
    for bad in (dict(dh=100), dict(dh=520), dict(depth=33), dict(ps=24), dict(layers=1 << 40), dict(batch=1 << 30)):
        assert call(**bad) == -2, bad
    assert call(batch=0) == call(layers=0) == call(heads=0) == 0


def test_reading_refusals(L):
    def call(code=3, k=FAKE, ksc=FAKE, vsc=FAKE, heads=4, dh=128, table=FAKE, width=4, pages=16, ps=16, batch=2,
             first=FAKE, n=10, dtype=0, ko=FAKE, vo=FAKE):
        return L.ddtree_read_kv8(code, k, FAKE, ksc, vsc, heads, dh, table, width, pages, ps, batch, first, None, n,
                                 dtype, ko, vo, None)
    for bad in (dict(code=1), dict(dtype=3), dict(k=None), dict(k=ODD), dict(ksc=None), dict(vsc=TORN), dict(heads=0),
                dict(dh=0), dict(table=None), dict(pages=0), dict(ps=0), dict(width=0), dict(batch=-1),
                dict(first=None), dict(n=-1), dict(ko=None), dict(vo=ODD)):
        assert call(**bad) == -1, bad
    for bad in (dict(dh=100), dict(dh=520), dict(ps=24), dict(batch=1 << 30), dict(heads=1 << 16)):
        assert call(**bad) == -2, bad
    assert call(batch=0) == call(n=0) == 0
