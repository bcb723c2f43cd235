"""GPU tests of caches of 8-bit rows (ddtree_append_kv8, ddtree_attention_kv8,
ddtree_compact_kv8, ddtree_read_kv8) and of attention over shared rows
(ddtree_attention_shared, shared_len) against the oracles.

Tolerances. Append: codes and scales are float32 steps that the oracle does
alike: equal. Reading back: one float32 product and one rounding to the output
type. Attention: as for 16-bit caches (tests/test_gpu_verify_cache.py), with
what a row stands for in the place of the cache's values; a key's scale adds two
float32 roundings to a score, a value's two to a weight, both within 2^-21; in
float16 a weight is held in units of at most twice the largest scale s seen with
steps of 2^-38 of the largest weight (twice that, since the maximum in use may
be half of the true one), which n keys put off by n 2^-37 s M at most, M the
largest code. The shared rows' part is joined by two more exponentials and
products, within another 2^-20 of spread.
"""

import threading

import numpy as np
import pytest
import torch

import draft_tree_construction_depth_amd as pkg
from oracle import kv8 as K
from oracle import oracle as OR
from oracle import verify as O
from test_gpu_verify_cache import ATTEND, BF, DEV, HF, TILES, dev, f64, paging, rounded, trees

pytestmark = pytest.mark.gpu
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
KINDS = ["e4m3", "i8"]


def codes_on(a, kind):
    """uint8 codes as a device tensor of their type."""
    return dev(a).view(CODES[kind])


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def random_cache(rng, shape, kind, spread=4.0):
    """Codes and scales of normal rows, magnitudes `spread` apart: (codes uint8, scales float32)."""
    codes, scales = np.empty(shape, np.uint8), np.empty(shape[:-1], np.float32)
    for p in range(shape[0]):
        x = rng.standard_normal(shape[1:]) * spread ** rng.uniform(-1, 1, shape[1:-1])[..., None]
        codes[p], scales[p] = K.quantise(x.astype(np.float32), kind)
    return codes, scales


# ---- append -----------------------------------------------------------------------
APPEND = [
    # batch, T, Hq, Hkv, dh, rot, inter, page, dtype, tree
    (1, 1, 4, 2, 128, 128, False, 16, BF, False),
    (3, 9, 6, 2, 64, 32, True, 1, HF, True),
    (2, 33, 5, 5, 40, 16, False, 8, BF, True),
    (5, 2, 8, 1, 256, 256, True, 64, BF, False),
    (2, 7, 3, 3, 72, 0, False, 4, HF, True),
    (2, 513, 2, 1, 64, 64, False, 128, BF, True),
    (2, 5, 2, 2, 512, 512, False, None, HF, True),
    (2, 3, 8, 2, 512, 0, False, 16, BF, False),
    (2, 4, 13, 13, 8, 0, False, 2, BF, True),
    (1, 6, 9, 3, 96, 80, True, 32, HF, False),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", APPEND, ids=[f"b{c[0]}T{c[1]}dh{c[4]}rot{c[5]}p{c[7]}" for c in APPEND])
def test_append(case, kind):
    batch, T, Hq, Hkv, dh, rot, inter, ps, dtype, tree = case
    rng = np.random.default_rng(T * dh)
    past = rng.integers(0, 200, batch).astype(np.int32)
    if batch > 2:
        past[1] = -1  # a request taken out
    if ps is None:
        ps, table, pool = int(past.max()) + T + 3, None, batch
    else:
        table, pool = paging(rng, batch, np.maximum(past, 0) + T, ps)
        table[0, (past[0] + T - 1) // ps] = pool  # the last row's page is no page of the pool
    qkv = rounded(rng, (batch, T, Hq + 2 * Hkv, dh), dtype)
    qkv[:, :, Hq:] *= torch.from_numpy(8.0 ** rng.uniform(-2, 2, (batch, T, 2 * Hkv, 1))).to(dtype)
    qkv[0, 0, Hq], qkv[-1, -1, -1] = 0.0, 2.0 ** -24  # a zero key, a tiny value
    if batch > 1:
        qkv[1, 0, Hq + Hkv, 3], qkv[-1, 1, Hq, dh - 1] = float("nan"), float("inf")
    kc, vc = (rng.integers(0, 256, (pool, Hkv, ps, dh)).astype(np.uint8) for _ in range(2))
    ks, vs = (rng.random((pool, Hkv, ps), dtype=np.float32) for _ in range(2))
    dep = trees(rng, batch, T - 1)[1] if tree and T > 1 else None
    nn = rng.integers(0, T, batch).astype(np.int32)
    nn[0] = T + 5  # clamped
    rope = None
    if rot:
        # one position short: the last row of the request that reaches furthest has no angle
        far = int(past.max()) + (int(dep.max()) if dep is not None else T - 1)
        a = np.arange(max(far, 1))[:, None] * 1e4 ** -(np.arange(rot // 2) / (rot / 2))
        rope = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    q0 = rounded(rng, (batch, T, Hq, dh), dtype)
    q, k, v = qkv.to(DEV).split([Hq, Hkv, Hkv], 2)
    kd, vd, ksd, vsd, qo = codes_on(kc, kind), codes_on(vc, kind), dev(ks), dev(vs), q0.to(DEV)
    args = dict(rope=dev(rope), interleaved=inter, page_table=dev(table), depths=dev(dep), num_nodes=dev(nn))
    got = pkg.ddtree_append_kv8(q, k, v, kd, vd, ksd, vsd, dev(past), **args, q_out=qo)
    assert got is qo
    x = qkv.float().numpy()
    want = K.append(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], kc, vc, ks, vs, kind, past, rope, inter, table, dep, nn)
    for g, w in zip((codes_of(kd), codes_of(vd), ksd.cpu().numpy(), vsd.cpu().numpy()), want):
        assert np.array_equal(g, w, equal_nan=g.dtype == np.float32)
    # the queries are the 16-bit append's
    wide = [torch.zeros((pool, Hkv, ps, dh), dtype=dtype, device=DEV) for _ in range(2)]
    same = pkg.ddtree_append_kv(q, k, v, *wide, dev(past), **args, q_out=q0.to(DEV))
    assert torch.equal(qo.view(torch.int16), same.view(torch.int16))
    # no queries, in place
    more = [codes_on(kc, kind), codes_on(vc, kind), dev(ks), dev(vs)]
    assert pkg.ddtree_append_kv8(None, k, v, *more, dev(past), **args) is None
    assert torch.equal(more[0].view(torch.uint8), kd.view(torch.uint8))
    assert torch.equal(more[3].view(torch.int32), vsd.view(torch.int32))


@pytest.mark.parametrize("kind", KINDS)
def test_codes_of_values_at_every_border(kind):
    """Every midpoint of two codes, its float32-wide neighbours in bf16 and the largest values: a
    row of 448 (127) has the scale 1 up to a rounding, so the elements are the codes' own axis."""
    most = K.MOST[kind]
    v = np.sort(K.decode(kind)[np.isfinite(K.decode(kind)) & (np.abs(K.decode(kind)) <= most)])
    mids = np.unique(np.concatenate([(v[:-1] + v[1:]) / 2, v]))
    rows = -(-len(mids) // 63)
    x = np.full((rows, 64), most)
    x[:, 1:].reshape(-1)[:len(mids)] = np.nan
    flat = np.pad(mids, (0, rows * 63 - len(mids))).reshape(rows, 63)
    x[:, 1:] = flat
    for e in range(-3, 4):  # scales that are powers of two times 1's, exactly alike
        t = torch.from_numpy((x * 2.0 ** (9 * e)).astype(np.float32)).to(BF).view(rows, 1, 1, 64)
        kc, vc = (torch.zeros((rows, 1, 1, 64), dtype=CODES[kind], device=DEV) for _ in range(2))
        ks, vs = (torch.zeros((rows, 1, 1), device=DEV) for _ in range(2))
        pkg.ddtree_append_kv8(None, t.to(DEV), -t.to(DEV), kc, vc, ks, vs, dev(np.zeros(rows, np.int32)))
        codes, scale = K.quantise(t.float().numpy()[:, 0, 0], kind)
        assert np.array_equal(codes_of(kc)[:, 0, 0], codes) and np.array_equal(ks.cpu().numpy()[:, 0, 0], scale)
        assert np.array_equal(codes_of(vc)[:, 0, 0], K.quantise(-t.float().numpy()[:, 0, 0], kind)[0])


# ---- attention ----------------------------------------------------------------------
def check(q, cache, kind, past, table, nn, mask, scale=None, clean=None, **kw):
    """One call against the oracle. cache: (k, v, k scales, v scales) as uint8 and float32 arrays;
    `clean`: the cache to give the oracle."""
    on = [codes_on(cache[0], kind), codes_on(cache[1], kind), dev(cache[2]), dev(cache[3])]
    got = pkg.ddtree_attention_kv8(q.to(DEV), *on, dev(past), page_table=dev(table), num_nodes=dev(nn), mask=dev(mask),
                                   scale=scale, with_lse=True, **kw)
    kc, vc, ks, vs = clean or cache
    vo = K.values(vc, vs, kind)
    with np.errstate(invalid="ignore"):
        oracle = O.attend(f64(q), K.values(kc, ks, kind), vo, past, table, nn, mask, scale)
        compare(got, q, oracle, np.nanmax(np.abs(vo)), past, kind)
    return got


def compare(got, q, oracle, most, past, kind):
    """most: the largest magnitude of a value in the cache."""
    T, dh = q.shape[1], q.shape[3]
    out, lse, spread, score = oracle
    g, gl = f64(got["out"]), f64(got["lse"])
    n = int(np.max(past)) + T
    half = torch.finfo(q.dtype).eps / 2
    off = ((dh + 4) * 2.0 ** -24 * score + 2.0 ** -20)[..., None]
    tiny = 0.0
    if q.dtype == HF:
        tiny = 2.0 ** -25  # half a step of the smallest float16s
        if kind:
            tiny += n * 2.0 ** -37 * most
    tol = half * np.abs(out) + spread * (1 + half) * (half + 2 * off + (n + 16) * 2.0 ** -24) + tiny
    assert np.all(np.abs(g - out) <= tol * 1.01), np.max(np.abs(g - out) / np.maximum(tol, 1e-30))
    assert np.array_equal(np.isinf(gl), np.isinf(lse))
    f = np.isfinite(lse)
    tol = ((dh + 4) * 2.0 ** -24 + 2.0 ** -21) * score[f] + (n + 16) * 2.0 ** -24 + 2.0 ** -20 * (np.abs(lse[f]) + 1)
    assert np.all(np.abs(gl[f] - lse[f]) <= tol)


def make_attention(rng, case, kind):
    batch, T, Hq, Hkv, dh, past, ps, dtype, tree = case
    past = np.array(past, np.int32)
    if ps is None:
        ps, table, pool = int(past.max()) + T + 9, None, batch
    else:
        table, pool = paging(rng, batch, past + T, ps)
    q = rounded(rng, (batch, T, Hq, dh), dtype, 2.0)
    (kc, ks), (vc, vs) = (random_cache(rng, (pool, Hkv, ps, dh), kind) for _ in range(2))
    nn = np.where(np.arange(batch) % 2 == 0, T - 1, T // 2).astype(np.int32)
    mask = OR.mask(trees(rng, batch, T - 1)[0], nn, T - 1).view(np.int64) if tree else None
    return q, (kc, vc, ks, vs), past, table, nn, mask


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", ATTEND, ids=[f"b{c[0]}T{c[1]}H{c[2]}-{c[3]}dh{c[4]}past{c[5][0]}p{c[6]}" for c in ATTEND])
def test_attention(case, kind):
    rng = np.random.default_rng(case[1] + case[4] + case[5][0])
    q, cache, past, table, nn, mask = make_attention(rng, case, kind)
    check(q, cache, kind, past, table, nn, mask)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("T,G", TILES, ids=[f"{t * g}rows" for t, g in TILES])
def test_every_arrangement_over_short_and_long_caches(T, G, dh, dtype, kind):
    """Each arrangement of waves in each type and head size: trees and chains, a cache that ends in
    its first tile beside one that is cut over many workgroups and merged; pages of one row (below
    what a load takes at once) and of many."""
    rng = np.random.default_rng(T * dh + 1)
    for past, ps in (([5, 4200, 0], 16), ([130, 3, 77], 1), ([900, 260, 0], 128)):
        past = np.array(past, np.int32)
        table, pool = paging(rng, 3, past + T, ps)
        q = rounded(rng, (3, T, 2 * G, dh), dtype, 2.0)
        (kc, ks), (vc, vs) = (random_cache(rng, (pool, 2, ps, dh), kind) for _ in range(2))
        nn = np.array([T - 1, T // 2, T - 1], np.int32)
        mask = OR.mask(trees(rng, 3, T - 1)[0], nn, T - 1).view(np.int64) if T > 1 else None
        check(q, (kc, vc, ks, vs), kind, past, table, nn, mask)
        if ps == 16:
            check(q, (kc, vc, ks, vs), kind, past, table, None, None)


def garbage(rng, pool, Hkv, ps, dh, kind):
    """What memory that nothing was written to may hold: any codes (e4m3 NaN among them), NaN,
    infinite, huge and negative scales."""
    codes = rng.integers(0, 256, (pool, Hkv, ps, dh)).astype(np.uint8)
    codes[..., :2] = rng.choice([0x7F, 0xFF], codes[..., :2].shape)
    return codes, rng.choice([np.nan, np.inf, -np.inf, 3e38, -1e30, 0.0], (pool, Hkv, ps)).astype(np.float32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(5, 2), (9, 3), (12, 4), (40, 3)], ids=["10rows", "27rows", "48rows", "120rows"])
def test_garbage_in_every_arrangement(T, G, dh, dtype, kind):
    """Garbage behind the block, on an unmapped page, on others' pages and in a sibling's row reaches
    only the rows that see it, whose heads' outputs are NaN."""
    rng = np.random.default_rng(T * dh + 2)
    ps = 16
    past = np.array([61, 130], np.int32)
    nn = np.array([T - 1, T // 2], np.int32)
    mask = OR.mask(np.zeros((2, T - 1), np.int32), nn, T - 1).view(np.int64)  # all nodes are siblings
    table, pool = paging(rng, 2, past + T, ps)
    table[1, 2] = -1  # rows 32..47 of request 1 are on no page
    q = rounded(rng, (2, T, 2 * G, dh), dtype)
    (kc, ks), (vc, vs) = (random_cache(rng, (pool, 2, ps, dh), kind) for _ in range(2))
    used = np.zeros((pool, ps), bool)
    for b in range(2):
        for r in range(int(past[b]) + int(nn[b]) + 1):
            at = O.slot(table, pool, ps, b, r)
            if at is not None:
                used[at] = True
    keep = used[:, None, :]
    (jk, jks), (jv, jvs) = (garbage(rng, pool, 2, ps, dh, kind) for _ in range(2))
    kg, vg = np.where(keep[..., None], kc, jk), np.where(keep[..., None], vc, jv)
    kgs, vgs = np.where(keep, ks, jks), np.where(keep, vs, jvs)
    got = check(q, (kg, vg, kgs, vgs), kind, past, table, nn, mask, clean=(kc, vc, ks, vs))
    page, row = O.slot(table, pool, ps, 0, 61 + 4)  # node 4 of request 0
    rest = [i for i in range(T) if i != 4]
    for bad in (np.nan, np.inf, 3e38, -3e38):
        for name in ("k", "v"):
            k2, v2 = kgs.copy(), vgs.copy()
            (k2 if name == "k" else v2)[page, 0, row] = bad
            o = pkg.ddtree_attention_kv8(q.to(DEV), codes_on(kg, kind), codes_on(vg, kind), dev(k2), dev(v2), dev(past),
                                         page_table=dev(table), num_nodes=dev(nn), mask=dev(mask))["out"]
            assert torch.equal(o[0, rest], got["out"][0, rest]) and torch.equal(o[1], got["out"][1])
            assert torch.equal(o[0, 4, G:], got["out"][0, 4, G:])  # the other key/value head
            if np.isnan(bad):
                assert o[0, 4, :G].isnan().all()
    if kind == "e4m3":  # one NaN code
        v2 = vg.copy()
        v2[page, 0, row, 3] = 0x7F
        o = pkg.ddtree_attention_kv8(q.to(DEV), codes_on(kg, kind), codes_on(v2, kind), dev(kgs), dev(vgs), dev(past),
                                     page_table=dev(table), num_nodes=dev(nn), mask=dev(mask))["out"]
        assert torch.equal(o[0, rest], got["out"][0, rest]) and o[0, 4, :G, 3].isnan().all()
        others = [e for e in range(dh) if e != 3]
        assert torch.equal(o[0, 4][:, others], got["out"][0, 4][:, others])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,G", TILES, ids=[f"{t * g}rows" for t, g in TILES])
def test_float16_values_of_very_different_sizes(T, G, kind):
    """Scales that grow by 2^24 along the cache, and scales far beyond float16 in rows that only some
    see: the outputs of those that see small values alone keep their precision."""
    rng = np.random.default_rng(T)
    dh, past = 64, np.array([700, 300], np.int32)
    n = int(past.max()) + T
    q = rounded(rng, (2, T, 2 * G, dh), HF)
    (kc, ks), (vc, vs) = (random_cache(rng, (2, 2, n, dh), kind) for _ in range(2))
    vs = (vs * np.float32(2.0) ** np.linspace(-20, 4, n).astype(np.float32)).astype(np.float32)
    cache = (kc, vc, ks, vs)
    check(q, cache, kind, past, None, None, None)
    if T > 1:
        mask = OR.mask(np.zeros((2, T - 1), np.int32), np.full(2, T - 1, np.int32), T - 1).view(np.int64)
        far = vs.copy()
        far[:, :, :700] = vs[:, :, :700] * np.float32(2.0 ** -10)
        far[1] = vs[1]
        far[0, :, 700 + 2] = 1e30  # node 2 of request 0: seen by itself alone
        got = pkg.ddtree_attention_kv8(q.to(DEV), codes_on(kc, kind), codes_on(vc, kind), dev(ks), dev(far), dev(past),
                                       mask=dev(mask), with_lse=True)
        small = far.copy()
        small[0, :, 700 + 2] = 0
        rest = [i for i in range(T) if i != 2]
        out, lse, spread, score = O.attend(f64(q), K.values(kc, ks, kind), K.values(vc, small, kind), past, None, None, mask)
        half = 2.0 ** -11
        off = ((dh + 4) * 2.0 ** -24 * score + 2.0 ** -20)[..., None]
        tol = half * np.abs(out) + spread * (1 + half) * (half + 2 * off + (n + 16) * 2.0 ** -24) + 2.0 ** -25 + \
            n * 2.0 ** -37 * np.abs(K.values(vc, small, kind)).max()
        assert np.all(np.abs(f64(got["out"])[:, rest] - out[:, rest]) <= tol[:, rest] * 1.01)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("size", [2.0 ** 21, 2.0 ** 25], ids=["2p21", "2p25"])
@pytest.mark.parametrize("T,G", TILES, ids=[f"{t * g}rows" for t, g in TILES])
def test_attention_of_small_differences_between_large_scores(T, G, size, dtype, kind):
    """Scores that share a large part and differ by a few float32 steps of it at most: no weight
    leaves its range, and the differences come through to three steps of the score."""
    rng = np.random.default_rng(T)
    dh, n, past = 64, 200 + T, np.array([200], np.int32)
    q = torch.zeros((1, T, 2 * G, dh), dtype=dtype)
    q[..., 0], q[..., 1] = size / 2.0 ** 11, 1.0
    kc, ks = np.zeros((1, 2, n, dh), np.uint8), np.full((1, 2, n), 2.0 ** 5, np.float32)
    kc[..., 0] = K.nearest(np.array(64.0), kind)
    step = max(size / 2.0 ** 23, 0.5)
    kc[..., 1] = K.nearest(rng.integers(-12, 13, (1, 2, n)) * step / 32, kind)
    vc, vs = random_cache(rng, (1, 2, n, dh), kind)
    got = pkg.ddtree_attention_kv8(q.to(DEV), codes_on(kc, kind), codes_on(vc, kind), dev(ks), dev(vs), dev(past),
                                   scale=1.0, with_lse=True)
    assert got["out"].isfinite().all()
    out, lse, spread, _ = O.attend(f64(q), K.values(kc, ks, kind), K.values(vc, vs, kind), past, None, None, None, 1.0)
    half = torch.finfo(dtype).eps / 2
    # a score in powers of two: the product's rounding and scale * log2(e)'s, for the weight and for
    # the others: three steps at most
    off = np.expm1(3 * np.spacing(np.float32(1.45 * size)) * np.log(2))
    tol = half * np.abs(out) + spread * (1 + half) * (half + 2 * off + 2.0 ** -14) + 2.0 ** -25
    assert np.all(np.abs(f64(got["out"]) - out) <= tol + n * 2.0 ** -37 * np.abs(K.values(vc, vs, kind)).max())
    assert np.all(np.abs(f64(got["lse"]) - lse) <= 2.0 ** -20 * np.abs(lse))


@pytest.mark.parametrize("kind", KINDS)
def test_attention_of_a_padded_batch_and_rows_without_room(kind):
    """Requests taken out, node counts outside the range; past + block beyond the table's rows."""
    rng = np.random.default_rng(10)
    past = np.array([-1, 30, -5, 7], np.int32)
    q = rounded(rng, (4, 6, 2, 64), HF)
    (kc, ks), (vc, vs) = (random_cache(rng, (4, 1, 50, 64), kind) for _ in range(2))
    for nn in (None, np.array([3, -2, 0, 99], np.int32)):
        check(q, (kc, vc, ks, vs), kind, past, None, nn, None)
    T, ps = 9, 8
    past = np.array([20, 27, 40, 500], np.int32)  # room for 32 rows
    table = rng.permutation(16).astype(np.int32).reshape(4, 4)
    q = rounded(rng, (4, T, 2, 64), BF)
    (kc, ks), (vc, vs) = (random_cache(rng, (16, 1, ps, 64), kind) for _ in range(2))
    check(q, (kc, vc, ks, vs), kind, past, table, None, None)
    k = rounded(rng, (4, T, 1, 64), BF)
    on = [codes_on(kc, kind), codes_on(vc, kind), dev(ks), dev(vs)]
    pkg.ddtree_append_kv8(None, k.to(DEV), k.to(DEV), *on, dev(past), page_table=dev(table))
    x = k.float().numpy()
    want = K.append(x, x, kc, vc, ks, vs, kind, past, table=table)
    assert np.array_equal(codes_of(on[0]), want[0]) and np.array_equal(on[3].cpu().numpy(), want[3])


# ---- shared rows ----------------------------------------------------------------------
ENOUGH = 192 << 20  # bytes that sharing has to save before rows are shared


def shared_pages(rng, batch, past, T, ps, shared):
    """A table whose requests share the pages of their first `shared` rows, -1 behind their own."""
    same = shared // ps
    own, pool = paging(rng, batch, np.maximum(past + T - same * ps, 1), ps)
    table = np.concatenate([np.tile(np.arange(pool, pool + same, dtype=np.int32), (batch, 1)), own], 1)
    table[:, :same] = rng.permutation(table[0, :same])
    return table, pool + same


def one(n):
    return torch.tensor([n], dtype=torch.int32, device=DEV)


def make_cache(g, shape, kind, dtype):
    """Device caches of normal rows: (k, v), or (k, v, k scales, v scales) of a kind of codes."""
    if not kind:
        return tuple(torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g) for _ in range(2))
    codes, scales = [], []
    for _ in range(2):
        c, s = torch.empty(shape, dtype=CODES[kind], device=DEV), torch.empty(shape[:-1], device=DEV)
        for p in range(0, shape[0], 4096):
            x = torch.randn(c[p:p + 4096].shape, device=DEV, generator=g)
            most = x.abs().amax(-1, keepdim=True)
            x = x / most * K.MOST[kind]
            c[p:p + 4096] = x.round().to(torch.int8) if kind == "i8" else x.to(CODES[kind])
            s[p:p + 4096] = most[..., 0] / K.MOST[kind] * 4.0 ** torch.empty_like(most[..., 0]).uniform_(-1, 1, generator=g)
        codes.append(c)
        scales.append(s)
    return (*codes, *scales)


def attend64(q, cache, kind, past, table, nn, mask, scale=None):
    """O.attend on the device, in float64, for caches too long for it."""
    batch, T, Hq, dh = q.shape
    ps, Hkv = cache[0].shape[2], cache[0].shape[1]
    G, scale = Hq // Hkv, dh ** -0.5 if scale is None else scale
    out, spread = (torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.full((batch, T, Hq), -float("inf"), dtype=torch.float64, device=DEV)
    score, most = torch.zeros((batch, T, Hq), dtype=torch.float64, device=DEV), 0.0
    bits = None if mask is None else O.mask_bits(mask, T)
    for b in range(batch):
        n = T - 1 if nn is None else min(max(int(nn[b]), 0), T - 1)
        if past[b] < 0:
            continue
        rows = np.arange(min(int(past[b]) + n + 1, table.shape[1] * ps))
        page = table[b, rows // ps]
        held = (page >= 0) & (page < cache[0].shape[0])
        sees = np.tile(held, (n + 1, 1))
        own = np.tril(np.ones((n + 1, n + 1), bool)) if bits is None else bits[b, :n + 1, :n + 1]
        sees[:, past[b]:] &= own[:, :max(len(rows) - int(past[b]), 0)]
        sees = dev(sees)[None]
        at = (dev(np.where(held, page, 0)).long(), slice(None), dev(rows % ps).long())
        k, v = (c.view(torch.int8)[at].view(c.dtype).double() * s[at].double()[..., None] if kind else c[at].double()
                for c, s in zip(cache[:2], cache[2:] or (None, None)))
        most = max(most, float(v.abs().max()))
        for h in range(Hkv):
            x = q[b, :n + 1, h * G:(h + 1) * G].to(DEV).double().transpose(0, 1).reshape(-1, dh)
            kt, vh = k[:, h].t().contiguous(), v[:, h].contiguous()
            y = torch.where(sees, (x @ kt * scale).view(G, n + 1, -1), -float("inf"))
            z = torch.logsumexp(y, -1)
            a = torch.where(sees, (y - z[..., None]).exp(), 0.0).view(G * (n + 1), -1)
            put = lambda t: t.view(G, n + 1, dh).transpose(0, 1)  # noqa: E731
            out[b, :n + 1, h * G:(h + 1) * G], spread[b, :n + 1, h * G:(h + 1) * G] = put(a @ vh), put(a @ vh.abs())
            lse[b, :n + 1, h * G:(h + 1) * G] = z.t()
            size = torch.where(sees, (x.abs() @ kt.abs() * scale).view(G, n + 1, -1), 0.0).amax(-1)
            score[b, :n + 1, h * G:(h + 1) * G] = size.t()
    return tuple(t.cpu().numpy() for t in (out, lse, spread, score)), most


def check_shared(q, cache, kind, past, table, nn, mask, shared, used):
    """One call on device caches against the oracle; used: the rows that it takes as shared, None
    where it makes no pass over them."""
    batch, T, Hq, dh = q.shape
    Hkv, ps = cache[0].shape[1:3]
    args = (batch, T, Hq, Hkv, dh, table.shape[1], ps)
    size = pkg.lib().ddtree_attention_kv8_workspace_size(*args, 1) if kind else \
        pkg.lib().ddtree_attention_shared_workspace_size(*args)
    assert (size > pkg.lib().ddtree_attention_workspace_size(*args)) == (used is not None)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    call = pkg.ddtree_attention_kv8 if kind else pkg.ddtree_attention_shared
    got = call(q.to(DEV), *cache, dev(past), page_table=dev(table), num_nodes=dev(nn), mask=dev(mask), shared_len=one(shared),
               with_lse=True, ws=ws)
    if used is not None:
        assert int(ws[:4].view(torch.int32)) == used  # the pass leaves them at the workspace's start
    oracle, most = attend64(q, cache, kind, past, table, nn, mask)
    compare(got, q, oracle, most, past, kind)
    return got


LENGTHS = {"cut": [2600, 1531, 64], "one": [3001], "whole": [700, 0, 450, 699, 31, 512] * 7,
           "uneven": [3000] + [40] * 30, "many": [130, 7, -1] * 100}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 8), (9, 3), (12, 4), (40, 3)], ids=["8rows", "27rows", "48rows", "120rows"])
def test_units_cut_and_whole(T, G, dh, dtype, kind):
    """Batches whose work is cut into even stretches and merged, is dealt out as whole requests, and
    is planned for more requests than a workgroup has threads; every one twice, with the same bits."""
    rng, g = np.random.default_rng(T * dh + 3), torch.Generator(device=DEV)
    g.manual_seed(T * dh + 3)
    ps = 16
    for past in LENGTHS.values():
        past = np.array(past, np.int32)
        batch = len(past)
        table, pool = paging(rng, batch, past + T, ps)
        q = rounded(rng, (batch, T, 2 * G, dh), dtype, 2.0)
        cache = make_cache(g, (pool, 2, ps, dh), kind, dtype)
        nn = rng.integers(0, T, batch).astype(np.int32)
        mask = OR.mask(trees(rng, batch, T - 1)[0], nn, T - 1).view(np.int64) if T > 1 else None
        got, again = (pkg.ddtree_attention_kv8(q.to(DEV), *cache, dev(past), page_table=dev(table), num_nodes=dev(nn),
                                               mask=dev(mask), with_lse=True) for _ in range(2))
        assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])
        compare(got, q, *attend64(q, cache, kind, past, table, nn, mask), past, kind)


# T * G rows of a key/value head: with batch requests, all arrangements of both passes
SHARED = [(3, 1, 1), (2, 1, 8), (5, 3, 8), (3, 9, 6), (40, 5, 4), (6, 16, 4), (4, 26, 3)]


@pytest.mark.parametrize("kind", ["", "e4m3", "i8"])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("batch,T,G", SHARED, ids=[f"{b}x{t * g}rows" for b, t, g in SHARED])
def test_shared_rows(batch, T, G, dh, dtype, kind):
    """Trees behind a prefix that is just long enough to be shared, in every arrangement, type and
    head size, with requests that have nothing but the prefix."""
    rng, g = np.random.default_rng(batch * T * dh), torch.Generator(device=DEV)
    g.manual_seed(batch * T * dh)
    Hkv, ps = 2, 128
    rows = -(-ENOUGH // ((batch - 1) * 2 * Hkv * dh * (1 if kind else 2)))
    used = -(-rows // 128) * 128
    past = (used + rng.integers(0, 200, batch)).astype(np.int32)
    past[0] = used
    table, pool = shared_pages(rng, batch, past, T, ps, used)
    q = rounded(rng, (batch, T, Hkv * G, dh), dtype, 2.0)
    cache = make_cache(g, (pool, Hkv, ps, dh), kind, dtype)
    nn = rng.integers(0, T, batch).astype(np.int32)
    mask = OR.mask(trees(rng, batch, T - 1)[0], nn, T - 1).view(np.int64) if T > 1 else None
    check_shared(q, cache, kind, past, table, nn, mask, used, used)


@pytest.mark.parametrize("kind", ["", "e4m3"])
def test_shared_lengths_of_every_kind(kind):
    """None, negative ones, odd ones, too short ones, more than the shortest request has committed;
    requests taken out (whose table rows are not used), all of them, full caches; pages of one row."""
    rng, g = np.random.default_rng(20), torch.Generator(device=DEV)
    g.manual_seed(20)
    batch, T, G, dh, ps, Hkv = 6, 3, 2, 256, 16, 8
    least = -(-ENOUGH // (3 * 2 * Hkv * dh * (1 if kind else 2)))  # four take part
    least = -(-least // 128) * 128
    most = least + 1280
    past = np.array([-1, most + 60, most, most + 50, -7, most + 300], np.int32)
    table, pool = shared_pages(rng, batch, past, T, ps, most)
    table[[0, 4]] = -1
    q = rounded(rng, (batch, T, Hkv * G, dh), BF, 2.0)
    cache = make_cache(g, (pool, Hkv, ps, dh), kind, BF)
    for shared, used in ((0, 0), (-5, 0), (-2 ** 31, 0), (least - 1, 0), (least, least), (least + 127, least),
                         (least + 129, least + 128), (most, most)):
        got = check_shared(q, cache, kind, past, table, None, None, shared, used)
        assert not got["out"][[0, 4]].any()
    # pages that are alike further than the shortest request reaches: what it has committed is shared
    alike = table.copy()
    alike[:] = table[5]
    short = np.array([-1, most + 60, least + 130, most + 300, -7, most + 300], np.int32)
    for shared in (most, 10 ** 6, 2 ** 31 - 1):
        check_shared(q, cache, kind, short, alike, None, None, shared, least + 128)
    short[2] = 5
    check_shared(q, cache, kind, short, alike, None, None, most, 0)
    none = np.full(batch, -1, np.int32)
    assert not check_shared(q, cache, kind, none, table, None, None, most, 0)["out"].any()
    # a cache that ends inside or at the end of the shared rows (for it, six take part)
    for rows, used in ((least + 640, least + 640), (least + 656, least + 640), (least, least)):
        cut = np.ascontiguousarray(alike[:, :rows // ps])
        full = np.array([rows + 7, rows, rows + 5, rows, -7, rows], np.int32)
        check_shared(q, cache, kind, full, cut, None, None, rows, used)


@pytest.mark.parametrize("kind", ["", "i8"])
def test_shared_rows_on_no_page(kind):
    """Entries of the prefix outside the pool; more requests than a workgroup has threads."""
    rng, g = np.random.default_rng(21), torch.Generator(device=DEV)
    g.manual_seed(21)
    batch, T, dh, ps, Hkv = 300, 1, 64, 16, 2
    used = -(-ENOUGH // (296 * 2 * Hkv * dh * (1 if kind else 2)) // 128) * 128 + 128
    past = (used + rng.integers(0, 300, batch)).astype(np.int32)
    past[[0, 17, 290]] = -1
    table, pool = shared_pages(rng, batch, past, T, ps, used)
    table[:, 3], table[:, 20] = -1, pool
    q = rounded(rng, (batch, T, 8, dh), BF)
    cache = make_cache(g, (pool, Hkv, ps, dh), kind, BF)
    check_shared(q, cache, kind, past, table, None, None, used, used)


@pytest.mark.parametrize("kind", ["", "e4m3"])
def test_poison_in_shared_rows_reaches_everybody(kind):
    rng, g = np.random.default_rng(22), torch.Generator(device=DEV)
    g.manual_seed(22)
    batch, T, G, dh, ps, used = 40, 2, 2, 128, 16, 10240
    past = np.full(batch, used + 44, np.int32)
    table, pool = shared_pages(rng, batch, past, T, ps, used)
    q = rounded(rng, (batch, T, 2 * G, dh), BF).to(DEV)
    on = make_cache(g, (pool, 2, ps, dh), kind, BF)
    (on[3] if kind else on[1])[int(table[0, 5]), 1, 7] = float("nan")  # a value of head 1
    call = pkg.ddtree_attention_kv8 if kind else pkg.ddtree_attention_shared
    got = call(q, *on, dev(past), page_table=dev(table), shared_len=one(used), with_lse=True)
    assert got["out"][:, :, G:].isnan().all() and got["out"][:, :, :G].isfinite().all()
    assert got["lse"].isfinite().all()


@pytest.mark.parametrize("kind", ["", "e4m3"])
def test_shared_calls_are_deterministic_and_keep_apart(kind):
    """Two streams and several host threads on one, with the binding's own workspaces."""
    rng, g = np.random.default_rng(23), torch.Generator(device=DEV)
    g.manual_seed(23)
    batch, T, ps, shared = 5, 3, 32, 53248
    past = (shared + np.array([0, 100, 1100, 50, 1])).astype(np.int32)
    table, pool = shared_pages(rng, batch, past, T, ps, shared)
    call = pkg.ddtree_attention_kv8 if kind else pkg.ddtree_attention_shared
    kw = dict(page_table=dev(table), shared_len=one(shared))
    at, sets = dev(past), []
    for _ in range(4):
        sets.append((rounded(rng, (batch, T, 16, 128), BF).to(DEV), *make_cache(g, (pool, 4, ps, 128), kind, BF)))
    run = lambda s: call(*s, at, **kw)["out"]  # noqa: E731
    ref = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[] for _ in sets]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run(sets[i]))
    torch.cuda.synchronize()

    def calls(i):
        for _ in range(20):
            got[i].append(run(sets[i]))
    threads = [threading.Thread(target=calls, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for want, outs in zip(ref, got):
        assert len(outs) >= 20 and all(torch.equal(o, want) for o in outs)


# ---- compaction and reading back --------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("paged", [True, False], ids=["paged", "contiguous"])
@pytest.mark.parametrize("case", [(3, 5, 4, 128, 16, 15, 64), (2, 3, 1, 8, 1, 32, 40), (1, 2, 2, 512, 64, 32, 255),
                                  (4, 7, 8, 64, 32, 4, 6), (40, 64, 4, 72, 8, 7, 20)], ids=str)
def test_compact(case, paged, kind):
    layers, batch, heads, dh, ps, L, B = case
    rng = np.random.default_rng(sum(case))
    past = rng.integers(0, 100, batch).astype(np.int32)
    past[-1] = -1 if batch > 4 else past[-1]
    n = rng.integers(0, min(L, B) + 1, batch).astype(np.int32)
    n[0] = min(L, B)
    acc = np.full((batch, L), -1, np.int32)
    for b in range(batch):
        acc[b, :n[b]] = np.sort(rng.choice(np.arange(1, B + 1), n[b], replace=False))
    if paged:
        table, pool = paging(rng, batch, np.maximum(past, 0) + B + 1, ps)
        table[1, (past[1] + B // 2) // ps] = -1  # a page that is none: its rows neither come nor go
    else:
        table, pool, ps = None, batch, int(past.max()) + B // 2  # the last rows have no room
    if batch > 2:
        n[2] = 99  # limited to L; its nodes end with -1
    shape = (layers, pool, heads, ps, dh)
    k, v = (rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))
    ks, vs = (rng.random(shape[:-1], dtype=np.float32) for _ in range(2))
    on = [codes_on(k, kind), codes_on(v, kind), dev(ks), dev(vs)]
    nl = pkg.ddtree_compact_kv8(*on, dev(table), dev(past), dev(acc), dev(n))
    wide = np.zeros((1, 1)) if table is None else table
    if table is None:  # the paged oracle on one page a request
        size = 1 << (ps - 1).bit_length()
        pad = [(0, 0), (0, 0), (0, 0), (0, size - ps)]
        wide = np.arange(batch, dtype=np.int32)[:, None]
        grow = lambda a: np.pad(a, pad + [(0, 0)] * (a.ndim - 4))  # noqa: E731
        acc = np.where((past[:, None] + acc < ps) & (past[:, None] + np.arange(1, L + 1) < ps), acc, -1)
    else:
        grow, size = (lambda a: a), ps
    ke, ve, ne = O.compact_paged(grow(k), grow(v), wide, past, acc, n)
    kse, vse, _ = O.compact_paged(grow(ks)[..., None], grow(vs)[..., None], wide, past, acc, n)
    assert np.array_equal(codes_of(on[0]), ke[..., :ps, :]) and np.array_equal(codes_of(on[1]), ve[..., :ps, :])
    assert np.array_equal(on[2].cpu().numpy(), kse[..., :ps, 0]) and np.array_equal(on[3].cpu().numpy(), vse[..., :ps, 0])
    assert np.array_equal(nl.cpu().numpy(), ne)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case,each", [((13, 400, 5, 8, 4, 7, 12), 3), ((41, 500, 7, 16, 4, 4, 6), 16),
                                       ((13, 400, 5, 128, 4, 15, 20), 3), ((6, 1000, 3, 256, 2, 9, 12), 2)], ids=str)
def test_compact_of_many_slices(case, each, kind):
    """So many slices (a layer's head of a request) that a wave moves `each` of them: over the end of
    a layer, in groups of loads that hold several slices or a part of one, with a shorter last part."""
    layers, batch, heads, dh, ps, L, B = case
    slices = layers * heads
    assert min(slices * batch // 8192, 16) == each and (slices % each or heads % each)
    rng = np.random.default_rng(sum(case))
    past = rng.integers(0, 7, batch).astype(np.int32)
    past[5] = -1
    n = rng.integers(0, L + 1, batch).astype(np.int32)
    n[0] = L
    acc = np.full((batch, L), -1, np.int32)
    for b in range(batch):
        acc[b, :n[b]] = np.sort(rng.choice(np.arange(1, B + 1), n[b], replace=False))
    table, pool = paging(rng, batch, np.maximum(past, 0) + B + 1, ps)
    table[1, 1] = -1
    shape = (layers, pool, heads, ps, dh)
    k, v = (rng.integers(0, 256, shape, np.uint8) for _ in range(2))
    ks, vs = (rng.random(shape[:-1], dtype=np.float32) for _ in range(2))
    on = [codes_on(k, kind), codes_on(v, kind), dev(ks), dev(vs)]
    nl = pkg.ddtree_compact_kv8(*on, dev(table), dev(past), dev(acc), dev(n))
    ke, ve, ne = O.compact_paged(k, v, table, past, acc, n)
    kse, vse, _ = O.compact_paged(ks[..., None], vs[..., None], table, past, acc, n)
    assert np.array_equal(codes_of(on[0]), ke) and np.array_equal(codes_of(on[1]), ve)
    assert np.array_equal(on[2].cpu().numpy(), kse[..., 0]) and np.array_equal(on[3].cpu().numpy(), vse[..., 0])
    assert np.array_equal(nl.cpu().numpy(), ne)


READ = [(1, 1, 1, 128, 16), (3, 40, 2, 64, 8), (2, 129, 8, 128, 64), (4, 7, 3, 40, 1), (2, 300, 1, 512, 32),
        (2, 33, 5, 256, None), (3, 2, 200, 24, 4)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, HF, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", READ, ids=str)
def test_read(case, dtype, kind):
    batch, n, heads, dh, ps = case
    rng = np.random.default_rng(n * dh)
    rows = rng.integers(n, 2 * n + 5, batch)
    if ps is None:
        ps, table, pool = int(rows.max()), None, batch
    else:
        table, pool = paging(rng, batch, rows, ps)
        table[0, 0] = pool + 3  # no page
    (kc, ks), (vc, vs) = (random_cache(rng, (pool, heads, ps, dh), kind) for _ in range(2))
    first = rng.integers(0, n + 1, batch).astype(np.int32)
    first[-1] = -2  # rows before the first do not exist
    count = rng.integers(0, n + 2, batch).astype(np.int32)
    count[0] = 2 * n  # no more than n
    on = [codes_on(kc, kind), codes_on(vc, kind), dev(ks), dev(vs)]
    for c in (count, None):
        got = pkg.ddtree_read_kv8(*on, dev(first), dev(c), n, dtype=dtype, page_table=dev(table))
        for g, codes, scales in ((got["k"], kc, ks), (got["v"], vc, vs)):
            want = K.read(codes, scales, kind, first, c, n, table)
            assert g.dtype == dtype
            # the product in float32, then one rounding (below the smallest normal, half a step)
            tol = np.abs(want) * (2.0 ** -24 + (0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2 * 1.001))
            assert np.all(np.abs(f64(g) - want) <= tol + (2.0 ** -25 if dtype == HF else 2.0 ** -133))
            assert np.array_equal(f64(g) == 0, np.abs(want) < (2.0 ** -24 if dtype == HF else 1e-40)) or dtype == HF
    # NaN scales read as NaN
    on[2].fill_(float("nan"))
    got = pkg.ddtree_read_kv8(*on, dev(np.zeros(batch, np.int32)), None, 1, dtype=dtype)["k"] if table is None else None
    assert got is None or got.isnan().all()


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes: the last pages are written and read, not wrapped ones."""
    ps, Hkv, dh = 128, 8, 128
    pages = (1 << 32) // (ps * Hkv * dh) + 3
    on = [torch.zeros((pages, Hkv, ps, dh), dtype=torch.int8, device=DEV) for _ in range(2)]
    on += [torch.zeros((pages, Hkv, ps), device=DEV) for _ in range(2)]
    rng = np.random.default_rng(12)
    last = pages - 1
    k, v, q = (rounded(rng, (1, 60, Hkv, dh), BF).to(DEV) for _ in range(3))
    past, table, zero = dev(np.array([0], np.int32)), dev(np.array([[last]], np.int32)), dev(np.zeros((1, 1), np.int32))
    small = [t[:1].clone() for t in on]
    pkg.ddtree_append_kv8(None, k, v, *on, past, page_table=table)
    pkg.ddtree_append_kv8(None, k, v, *small, past, page_table=zero)
    for t, s in zip(on, small):
        assert torch.equal(t[last], s[0]) and s.any() and not t[:last].any()
    past.fill_(40)
    a, b = (pkg.ddtree_attention_kv8(q[:, :20].contiguous(), *c, past, page_table=t)["out"]
            for c, t in ((on, table), (small, zero)))
    assert torch.equal(a, b)
    a, b = (pkg.ddtree_read_kv8(*c, past, None, 10, page_table=t) for c, t in ((on, table), (small, zero)))
    assert torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"]) and a["k"].any()
    acc, n = dev(np.array([[3, 7, 11]], np.int32)), dev(np.array([3], np.int32))
    for c, t in ((on, table), (small, zero)):
        pkg.ddtree_compact_kv8(*(x[None] for x in c), t, past, acc, n)
    for t, s in zip(on, small):
        assert torch.equal(t[last], s[0])


# ---- together ---------------------------------------------------------------------------
def make_round(seed, kind, L=6, B=14, V=2000, layers=2):
    """A verification round's inputs: drafter rows, 8-bit caches whose requests share a prompt."""
    from test_gpu_sampled import make_round as plain
    rng = np.random.default_rng(seed)
    r = plain(seed, batch=3, L=L, B=B, V=V, layers=layers)
    Hq, Hkv, dh = r["dims"]
    batch, ps, shared = 3, 16, 256
    past = np.array([shared, shared + 41, shared + 150], np.int32)
    table, pool = shared_pages(rng, batch, past, B + 1, ps, shared)
    r["past"], r["table"], r["shared"] = dev(past), dev(table), one(shared)
    caches = [random_cache(rng, (layers * pool, Hkv, ps, dh), kind) for _ in range(2)]
    for x, (codes, scales) in zip("kv", caches):
        r[x] = codes_on(codes.reshape(layers, pool, Hkv, ps, dh), kind)
        r[x + "s"] = dev(scales.reshape(layers, pool, Hkv, ps))
    a = np.arange(600)[:, None] * 1e4 ** -(np.arange(dh // 2) / (dh / 2))
    r["rope"] = dev(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))
    r["n"] = 6
    return r


def play_round(r):
    """Tree, append, attention per layer, acceptance, compaction, the newest rows read back."""
    Hq, Hkv, dh = r["dims"]
    t = pkg.ddtree_build(r["draft"], r["B"])
    batch, T = r["past"].shape[0], r["B"] + 1
    x, outs = 0, []
    for layer, qkv in enumerate(r["qkv"]):
        q, k, v = qkv.split([Hq, Hkv, Hkv], 2)
        cache = (r["k"][layer], r["v"][layer], r["ks"][layer], r["vs"][layer])
        q = pkg.ddtree_append_kv8(q, k, v, *cache, r["past"], rope=r["rope"], page_table=r["table"],
                                  depths=t["depths"], num_nodes=t["num_nodes"])
        o = pkg.ddtree_attention_kv8(q, *cache, r["past"], page_table=r["table"], num_nodes=t["num_nodes"],
                                     mask=t["mask"], shared_len=r["shared"], with_lse=True)
        outs.append((q, o))
        x = x + o["out"].float().view(batch * T, -1)
    logits = (x @ r["head"]).view(batch, T, -1)
    depth = torch.nn.functional.pad(t["depths"].clamp(min=0), (1, 0)).long().clamp(max=r["L"] - 1)
    logits += r["draft"].gather(1, depth[..., None].expand(-1, -1, logits.shape[-1]))
    a = pkg.ddtree_accept_sampled(t["tree_tokens"], t["parents"], t["num_nodes"], logits, r["heat"], r["u"])
    n = pkg.ddtree_compact_kv8(r["k"], r["v"], r["ks"], r["vs"], r["table"], r["past"], a["accepted_nodes"],
                               a["accept_len"])
    first = n - r["n"]
    back = pkg.ddtree_read_kv8(r["k"][0], r["v"][0], r["ks"][0], r["vs"][0], first, None, r["n"], page_table=r["table"])
    return {**t, **a, "new_len": n, "back_k": back["k"], "back_v": back["v"]}, outs


@pytest.mark.parametrize("kind", KINDS)
def test_a_round(kind):
    """The operators in the order of a verification round, each step against the oracle on the
    device's own inputs of that step."""
    r = make_round(1, kind)
    Hq, Hkv, dh = r["dims"]
    before = [codes_of(r["k"]), codes_of(r["v"]), r["ks"].cpu().numpy(), r["vs"].cpu().numpy()]
    got, outs = play_round(r)
    g = {k: v.cpu() for k, v in got.items()}
    past, table, rope = r["past"].cpu().numpy(), r["table"].cpu().numpy(), r["rope"].cpu().numpy()
    dep, nn = g["depths"].numpy(), g["num_nodes"].numpy()
    after = [codes_of(r["k"]), codes_of(r["v"]), r["ks"].cpu().numpy(), r["vs"].cpu().numpy()]
    assert g["accept_len"].max() > 0
    for layer in range(2):
        x = r["qkv"][layer].float().cpu().numpy()
        kc, vc, ks, vs = K.append(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], *(a[layer] for a in before), kind, past,
                                  rope, False, table, dep, nn)
        q, o = outs[layer]
        vo = K.values(vc, vs, kind)
        compare(o, q.cpu(), O.attend(f64(q), K.values(kc, ks, kind), vo, past, table, nn, g["mask"].numpy()), np.abs(vo).max(),
                past, kind)
        acc, n = g["accepted_nodes"].numpy(), g["accept_len"].numpy()
        k2, v2, nl = O.compact_paged(kc[None], vc[None], table, past, acc, n)
        ks2, vs2, _ = O.compact_paged(ks[None, ..., None], vs[None, ..., None], table, past, acc, n)
        for a, w in zip(after, (k2, v2, ks2[..., 0], vs2[..., 0])):
            assert np.array_equal(a[layer], w[0])
        if layer == 0:
            for name, c, s in (("back_k", k2, ks2), ("back_v", v2, vs2)):
                want = K.read(c[0], s[0, ..., 0], kind, nl - r["n"], None, r["n"], table)
                assert np.all(np.abs(f64(g[name]) - want) <= np.abs(want) * (2.0 ** -8 * 1.001))
    assert np.array_equal(g["new_len"].numpy(), nl)


def test_captured_rounds_replay_and_keep_apart():
    """Two rounds captured into two graphs, replayed in turn with eager work between: each
    replay equals the eager round on the same inputs, also after the lengths have changed."""
    rounds, names = [make_round(s, k) for s, k in ((2, "e4m3"), (3, "i8"))], ("k", "v", "ks", "vs")
    keeps = [{x: r[x].clone() for x in (*names, "past", "shared")} for r in rounds]

    def reset(r, keep, short):
        for x in (*names, "past", "shared"):
            r[x].copy_(keep[x])
        if short:  # another prompt length, other contexts
            r["past"].sub_(100)
            r["shared"].fill_(140)

    fresh = {}
    for i, r in enumerate(rounds):
        for short in (False, True):
            reset(r, keeps[i], short)
            want, _ = play_round(r)
            fresh[i, short] = ({k: v.clone() for k, v in want.items()}, [r[x].clone() for x in names])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r, keep in zip(rounds, keeps):
        reset(r, keep, False)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(play_round(r))
        graphs.append(g)
    for turn in range(4):
        for i, (r, g, (o, _)) in enumerate(zip(rounds, graphs, outs)):
            reset(r, keeps[i], turn % 2 == 1)
            g.replay()
            play_round(make_round(4 + turn, "i8"))  # eager work between the replays
            torch.cuda.synchronize()
            want, cache = fresh[i, turn % 2 == 1]
            for name in ("tree_tokens", "accepted_nodes", "accept_len", "next_token", "logp", "new_len", "back_k", "back_v"):
                assert torch.equal(o[name], want[name]), name
            for x, w in zip(names, cache):
                assert torch.equal(r[x].view(torch.uint8), w.view(torch.uint8)), x


# ---- refusals of the binding ------------------------------------------------------------
def test_binding_refusals():
    q = torch.zeros((2, 3, 4, 64), dtype=BF, device=DEV)
    kv = torch.zeros((2, 3, 2, 64), dtype=BF, device=DEV)
    c = torch.zeros((2, 2, 16, 64), dtype=torch.int8, device=DEV)
    s = torch.ones((2, 2, 16), device=DEV)
    past = torch.zeros(2, dtype=torch.int32, device=DEV)
    table = torch.zeros((2, 1), dtype=torch.int32, device=DEV)
    cache = dict(k_cache=c, v_cache=c.clone(), k_scale=s, v_scale=s.clone())
    att = lambda **k: pkg.ddtree_attention_kv8(**{**dict(q=q, **cache, past_len=past), **k})  # noqa: E731
    app = lambda **k: pkg.ddtree_append_kv8(**{**dict(q=q, k=kv, v=kv, **cache, past_len=past), **k})  # noqa: E731
    red = lambda **k: pkg.ddtree_read_kv8(**{**dict(**cache, first=past, count=None, n=2), **k})  # noqa: E731
    five = {k: v[None] for k, v in cache.items()}
    acc = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    com = lambda **k: pkg.ddtree_compact_kv8(**{**dict(**five, page_table=table, past_len=past, accepted_nodes=acc, accept_len=past), **k})  # noqa: E731
    att(), app(), red(), com()
    for call in (att, app, red):
        for bad in (dict(k_scale=s[:, :1]), dict(v_scale=s.cpu()), dict(v_cache=c[:1]), dict(page_table=table[:1])):
            with pytest.raises(ValueError):
                call(**bad)
        for bad in (dict(k_cache=c.view(torch.uint8)), dict(k_scale=s.double()),
                    dict(v_cache=c.view(torch.float8_e4m3fn)), dict(k_cache=kv.view(torch.int8))):
            with pytest.raises((TypeError, ValueError)):
                call(**bad)
    for bad in (dict(shared_len=past[:1]), dict(page_table=table, shared_len=past), dict(q=q.transpose(1, 2)),
                dict(past_len=past[:1]), dict(q=q[..., :32].contiguous())):
        with pytest.raises(ValueError):
            att(**bad)
    with pytest.raises(TypeError):
        att(q=q.float())
    for bad in (dict(scale=0.0), dict(q=q[:, :, :3].contiguous())):
        with pytest.raises(pkg.DDTreeError):
            att(**bad)
    for bad in (dict(k=kv[:, :2]), dict(v=kv[:, :, :1]), dict(q_out=q[:, :2]), dict(depths=past)):
        with pytest.raises(ValueError):
            app(**bad)
    for bad in (dict(count=past[:1]), dict(first=past[:1]), dict(out={"k": kv, "v": kv})):
        with pytest.raises(ValueError):
            red(**bad)
    for bad in (dict(dtype=torch.float64), dict(count=past.long())):
        with pytest.raises(TypeError):
            red(**bad)
    for bad in (dict(accepted_nodes=acc[:1]), dict(accept_len=past[:1]), dict(k_scale=s), dict(k_cache=c)):
        with pytest.raises(ValueError):
            com(**bad)
    half = torch.zeros((2, 2, 16, 64), dtype=BF, device=DEV)
    sha = lambda **k: pkg.ddtree_attention_shared(**{**dict(q=q, k_cache=half, v_cache=half, past_len=past, shared_len=past[:1], page_table=table), **k})  # noqa: E731
    sha()
    for bad in (dict(page_table=None), dict(shared_len=past), dict(mask=acc), dict(q=q[..., :32].contiguous())):
        with pytest.raises((ValueError, TypeError)):
            sha(**bad)
    with pytest.raises(TypeError):
        sha(q=q.half())
