"""GPU tests of the verification pass's cache and attention (ddtree_append_kv,
ddtree_attention, ddtree_compact_kv_paged) against the float64 oracle.

Tolerances. A rounding to type t is off by at most eps/2 of the value, eps =
torch.finfo(t).eps. Append: two float32 products and a sum (2^-22 of the
terms) and one rounding. Attention: a score is a float32 sum of dh exact
products, off by at most dh 2^-24 of its terms' size s (the oracle's `score`),
so a weight by that fraction; the weight may be rounded to t once (eps/2), its
exponential costs 2^-21, the sums n 2^-24; all act on spread = sum a |V|, and
the output is rounded once. lse: the score's error, the sum's, and 2^-22 of
its value and of the largest exponent argument's.
"""

import threading

import numpy as np
import pytest
import torch

import draft_tree_construction_depth_amd as pkg
from oracle import oracle as OR
from oracle import verify as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def rounded(rng, shape, dtype, scale=1.0):
    """Normal values held in dtype, on the CPU."""
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype)


def trees(rng, batch, B, depth=15):
    par, dep = np.zeros((batch, B), np.int32), np.zeros((batch, B), np.int32)
    for b in range(batch):
        d = [0]
        for j in range(B):
            p = int(rng.integers(max(0, j - 6), j + 1))
            while d[p] >= depth:
                p = int(rng.integers(0, j + 1))
            par[b, j], dep[b, j] = p, d[p] + 1
            d.append(d[p] + 1)
    return par, dep


def paging(rng, batch, rows, ps, spare=2):
    """A table of random pages with room for `rows` rows per request, -1 behind a request's own."""
    need = [-(-r // ps) for r in rows]
    pool = sum(need) + spare
    order = rng.permutation(pool).astype(np.int32)
    table, at = np.full((batch, max(need) + 1), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


# ---- append -------------------------------------------------------------------
APPEND = [
    # batch, T, Hq, Hkv, dh, rot, inter, page, dtype, tree
    (1, 1, 4, 2, 128, 128, False, 16, BF, False),
    (3, 9, 6, 2, 64, 32, True, 1, HF, True),
    (2, 33, 5, 5, 40, 16, False, 8, BF, True),
    (5, 2, 8, 1, 256, 256, True, 64, BF, False),
    (2, 7, 3, 3, 72, 0, False, 4, HF, True),
    (2, 513, 2, 1, 64, 64, False, 128, BF, True),
    (2, 5, 2, 2, 512, 512, False, None, HF, True),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"b{c[0]}T{c[1]}dh{c[4]}rot{c[5]}p{c[7]}" for c in APPEND])
def test_append(case):
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
    kc, vc = rounded(rng, (pool, Hkv, ps, dh), dtype), rounded(rng, (pool, Hkv, ps, dh), dtype)
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
    kd, vd, qo = kc.to(DEV), vc.to(DEV), q0.to(DEV)
    got = pkg.ddtree_append_kv(q, k, v, kd, vd, dev(past), rope=dev(rope), interleaved=inter, page_table=dev(table),
                               depths=dev(dep), num_nodes=dev(nn), q_out=qo)
    assert got is qo
    x = f64(qkv)
    qe, ke, ve = O.append(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], f64(kc), f64(vc), past,
                          None if rope is None else rope.astype(np.float64), inter, table, dep, nn, f64(q0))
    assert np.array_equal(f64(vd), ve)
    for g, e, old in ((f64(qo), qe, f64(q0)), (f64(kd), ke, f64(kc))):
        assert np.array_equal(g[e == old], e[e == old])
        size = np.abs(x).max()
        assert np.all(np.abs(g - e) <= torch.finfo(dtype).eps / 2 * np.abs(e) + 2 ** -22 * size + 2.0 ** -25)


def test_append_in_place_and_without_queries():
    rng = np.random.default_rng(3)
    k, v = rounded(rng, (2, 4, 2, 64), BF), rounded(rng, (2, 4, 2, 64), BF)
    q = rounded(rng, (2, 4, 4, 64), BF)
    a = np.arange(50)[:, None] * np.linspace(1, 0.01, 32)
    rope = dev(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))
    past = dev(np.array([3, 20], np.int32))
    c = [torch.zeros((2, 2, 40, 64), dtype=BF, device=DEV) for _ in range(4)]
    qd = q.to(DEV)
    apart = pkg.ddtree_append_kv(qd, k.to(DEV), v.to(DEV), c[0], c[1], past, rope=rope)
    assert torch.equal(qd.cpu(), q)
    assert pkg.ddtree_append_kv(qd, k.to(DEV), v.to(DEV), c[0], c[1], past, rope=rope, q_out=qd) is qd
    assert torch.equal(qd, apart)
    assert pkg.ddtree_append_kv(None, k.to(DEV), v.to(DEV), c[2], c[3], past, rope=rope) is None
    assert torch.equal(c[0], c[2]) and torch.equal(c[1], c[3])


# ---- attention ------------------------------------------------------------------
def check_attention(q, kc, vc, past, table, nn, mask, scale=None, clean=None, **kw):
    """One call against the oracle; `clean`: the caches to give the oracle (garbage taken out)."""
    batch, T, Hq, dh = q.shape
    got = pkg.ddtree_attention(q.to(DEV), kc.to(DEV), vc.to(DEV), dev(past), page_table=dev(table),
                               num_nodes=dev(nn), mask=dev(mask), scale=scale, with_lse=True, **kw)
    ko, vo = clean or (kc, vc)
    out, lse, spread, score = O.attend(f64(q), f64(ko), f64(vo), past, table, nn, mask, scale)
    g, gl = f64(got["out"]), f64(got["lse"])
    n = int(np.max(past)) + T
    half = torch.finfo(q.dtype).eps / 2
    off = (dh * 2.0 ** -24 * score + 2.0 ** -21)[..., None]
    tiny = 2.0 ** -25 if q.dtype == HF else 0.0  # half a step of the smallest float16s
    tol = half * np.abs(out) + spread * (1 + half) * (half + 2 * off + (n + 8) * 2.0 ** -24) + tiny
    assert np.all(np.abs(g - out) <= tol * 1.01), np.max(np.abs(g - out) / np.maximum(tol, 1e-30))
    assert np.array_equal(np.isinf(gl), np.isinf(lse))
    f = np.isfinite(lse)
    tol = (dh * 2.0 ** -24 + 2.0 ** -21) * score[f] + (n + 8) * 2.0 ** -24 + 2.0 ** -21 * (np.abs(lse[f]) + 1)
    assert np.all(np.abs(gl[f] - lse[f]) <= tol)
    return got


ATTEND = [
    # batch, T, Hq, Hkv, dh, pasts, page, dtype, tree
    (1, 1, 4, 2, 128, [0], 16, BF, False),
    (1, 1, 8, 1, 64, [1], 1, HF, False),
    (3, 1, 8, 2, 128, [5, 63, 300], 16, BF, False),
    (2, 1, 5, 5, 256, [64, 127], 64, HF, False),
    (2, 5, 6, 2, 64, [0, 31], 8, BF, True),
    (2, 17, 5, 1, 128, [700, 33], 32, HF, False),
    (3, 33, 4, 2, 128, [100, 0, 1029], 64, BF, True),
    (2, 65, 8, 2, 128, [257, 64], 16, BF, True),
    (1, 129, 3, 3, 64, [95], 128, HF, True),
    (1, 65, 6, 1, 256, [200], 16, BF, True),
    (1, 513, 2, 2, 64, [40], 32, BF, True),
    (1, 1, 16, 1, 128, [5000], 16, BF, False),
    (1, 3, 32, 1, 64, [2500], 128, HF, True),
    (2, 9, 12, 2, 128, [40, 77], None, BF, True),
]


@pytest.mark.parametrize("case", ATTEND, ids=[f"b{c[0]}T{c[1]}H{c[2]}-{c[3]}dh{c[4]}past{c[5][0]}p{c[6]}" for c in ATTEND])
def test_attention(case):
    batch, T, Hq, Hkv, dh, past, ps, dtype, tree = case
    rng = np.random.default_rng(T + dh + past[0])
    past = np.array(past, np.int32)
    if ps is None:
        ps, table, pool = int(past.max()) + T + 9, None, batch
    else:
        table, pool = paging(rng, batch, past + T, ps)
    q = rounded(rng, (batch, T, Hq, dh), dtype, 2.0)
    kc, vc = rounded(rng, (pool, Hkv, ps, dh), dtype), rounded(rng, (pool, Hkv, ps, dh), dtype)
    nn = np.where(np.arange(batch) % 2 == 0, T - 1, T // 2).astype(np.int32)
    mask = OR.mask(trees(rng, batch, T - 1)[0], nn, T - 1).view(np.int64) if tree else None
    check_attention(q, kc, vc, past, table, nn, mask)


def test_attention_of_a_strongly_peaked_softmax():
    """Scores of hundreds: the running maximum moves by large steps; one weight dominates."""
    rng = np.random.default_rng(8)
    q, kc = rounded(rng, (1, 9, 4, 128), BF, 8.0), rounded(rng, (1, 2, 400, 128), BF, 6.0)
    vc = rounded(rng, (1, 2, 400, 128), BF)
    got = check_attention(q, kc, vc, np.array([391], np.int32), None, None, None)
    assert torch.isfinite(got["lse"]).all()


# T * Hq / Hkv rows share a key/value head: one size for each arrangement of waves
TILES = [(1, 2), (3, 8), (9, 6), (33, 3)]


@pytest.mark.parametrize("every", [False, True], ids=["one", "many"])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("T,G", TILES, ids=[f"{t * g}rows" for t, g in TILES])
def test_attention_of_float16_keys_far_below_one_that_adds_nothing(T, G, dh, every):
    """One key whose value is 0 (or one in every 32), thousands 16 to 18 nats below it with values:
    all of the output comes from weights of 1e-7 to 1e-8 of the largest, which float16 would hold as
    0 or with a few bits if the largest were held as 1."""
    rng = np.random.default_rng(T * dh)
    past = np.array([4991, 300], np.int32)
    n = int(past.max()) + T
    q = torch.zeros((2, T, 2 * G, dh), dtype=HF)
    q[..., 0] = 1.0
    kc, vc = torch.zeros((2, 2, n, dh), dtype=HF), torch.ones((2, 2, n, dh), dtype=HF)
    kc[..., 0] = torch.from_numpy(rng.uniform(2.0, 4.0, (2, 2, n))).to(HF)
    if every:
        vc *= 256.0
        kc[:, :, 3::32, 0], vc[:, :, 3::32] = 20.0, 0.0
    kc[:, :, 70, 0], vc[:, :, 70] = 20.0, 0.0
    got = check_attention(q, kc, vc, past, None, None, None, scale=1.0)
    assert (got["out"][0] > 5e-5).all()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,G", TILES, ids=[f"{t * g}rows" for t, g in TILES])
def test_attention_of_scores_beyond_what_float32_steps_resolve(T, G, dtype):
    """Scores near 2^36, where a float32 step is 4096: the largest takes all the weight, equal ones
    share it, however scale and score are multiplied."""
    rng = np.random.default_rng(T)
    dh, n, past = 128, 200 + T, np.array([200, 9], np.int32)
    big = 2.0 ** 15
    q = torch.zeros((2, T, 2 * G, dh), dtype=dtype)
    q[..., 0] = big
    kc, vc = torch.zeros((2, 2, n, dh), dtype=dtype), rounded(rng, (2, 2, n, dh), dtype)
    # 128 values that both types hold, each a part in 128 or more from the next
    kc[..., 0] = torch.from_numpy(rng.integers(128, 255, (2, 2, n)) * big / 256).to(dtype)
    top = big * 255 / 256
    kc[0, :, 5, 0] = kc[0, :, 190, 0] = kc[1, :, 0, 0] = top
    scale = 77.7  # no power of two: scores are not held as they are
    got = pkg.ddtree_attention(q.to(DEV), kc.to(DEV), vc.to(DEV), dev(past), scale=scale, with_lse=True)
    vd = vc.to(DEV)
    mean = (vd[0, :, 5].double() + vd[0, :, 190].double()) / 2
    want = torch.stack([mean, vd[1, :, 0].double()])[:, None, :, None].expand(2, T, 2, G, dh)
    out = got["out"].double().view(2, T, 2, G, dh)
    # weights of 1 and 1/2 are exact: the output is rounded once
    assert ((out - want).abs() <= torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -25).all()
    lse = scale * big * top
    assert ((got["lse"].double() - lse).abs() <= 2.0 ** -21 * lse).all()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("size", [2.0 ** 21, 2.0 ** 23, 2.0 ** 25], ids=["2p21", "2p23", "2p25"])
@pytest.mark.parametrize("T,G", TILES, ids=[f"{t * g}rows" for t, g in TILES])
def test_attention_of_small_differences_between_large_scores(T, G, size, dtype):
    """Scores that share a large part and differ by a few: float32 holds each of them exactly, so up
    to 2^24 powers of two the differences come through; beyond, to a float32 step of the score."""
    rng = np.random.default_rng(T)
    dh, n, past = 64, 200 + T, np.array([200], np.int32)
    q, kc = torch.zeros((1, T, 2 * G, dh), dtype=dtype), torch.zeros((1, 2, n, dh), dtype=dtype)
    q[..., 0], q[..., 1] = size / 2.0 ** 11, 1.0
    kc[..., 0] = 2.0 ** 11
    step = max(size / 2.0 ** 23, 0.5)  # float32's at the size (half of it below), which the sum keeps
    kc[..., 1] = torch.from_numpy(rng.integers(-12, 13, (1, 2, n)) * step).to(dtype)
    vc = rounded(rng, (1, 2, n, dh), dtype)
    got = pkg.ddtree_attention(q.to(DEV), kc.to(DEV), vc.to(DEV), dev(past), scale=1.0, with_lse=True)
    out, lse, spread, _ = O.attend(f64(q), f64(kc), f64(vc), past, None, None, None, 1.0)
    half = torch.finfo(dtype).eps / 2
    # a weight's exponent is off by 2^-23 of at most 20 powers of two, or by a step of the score
    off = 2.0 ** -18 if 1.4427 * size + 32 < 2.0 ** 24 else np.expm1(np.spacing(np.float32(1.45 * size)) * np.log(2))
    tol = half * np.abs(out) + spread * (1 + half) * (half + 2 * off + 2.0 ** -14)
    assert np.all(np.abs(f64(got["out"]) - out) <= tol + 2.0 ** -25)
    assert np.all(np.abs(f64(got["lse"]) - lse) <= 2.0 ** -21 * np.abs(lse))


@pytest.mark.parametrize("T,G", TILES, ids=[f"{t * g}rows" for t, g in TILES])
def test_attention_of_one_query_with_large_scores_among_others(T, G):
    """Large scores of one query change nothing for those beside it, nor for rows that see nothing."""
    rng = np.random.default_rng(T + 5)
    dh, past = 64, np.array([0, 90], np.int32)
    q = rounded(rng, (2, T, 2 * G, dh), BF)
    kc, vc = rounded(rng, (2, 2, 100 + T, dh), BF), rounded(rng, (2, 2, 100 + T, dh), BF)
    q[:, 0, 1] *= 2.0 ** 40
    mask = None
    if T > 1:
        mask = OR.mask(np.zeros((2, T - 1), np.int32), np.full(2, T - 1, np.int32), T - 1).view(np.int64)
        mask[0, -1] = 0  # sees nothing: no past, no bit
    got = check_attention(q, kc, vc, past, None, None, mask)
    assert got["out"].isfinite().all()


def test_attention_with_garbage_where_nothing_is_seen():
    """NaN and infinities in rows behind the block, on unmapped pages, in pages of
    others, and in a sibling's row do not reach the rows that do not see them."""
    rng = np.random.default_rng(9)
    T, ps = 9, 16
    past = np.array([21, 64, -1, 0], np.int32)
    par = np.zeros((4, T - 1), np.int32)  # all nodes are siblings
    nn = np.array([8, 5, 8, 8], np.int32)
    mask = OR.mask(par, nn, T - 1).view(np.int64)
    mask[3, 0] = 0  # a row that sees nothing at all: no past, no bit
    table, pool = paging(rng, 4, np.maximum(past, 0) + T, ps)
    table[1, 1] = -1  # rows 16..31 of request 1 are on no page
    table[0, -1] = pool + 7
    q = rounded(rng, (4, T, 4, 64), BF)
    kc, vc = rounded(rng, (pool, 2, ps, 64), BF), rounded(rng, (pool, 2, ps, 64), BF)
    used = np.zeros((pool, ps), bool)
    for b in range(4):
        for r in range(max(int(past[b]), 0) + int(nn[b]) + 1):
            at = O.slot(table, pool, ps, b, r)
            if at is not None and past[b] >= 0:
                used[at] = True
    kg, vg = kc.clone(), vc.clone()
    junk = torch.from_numpy(~used)
    kg.permute(0, 2, 1, 3)[junk] = float("nan")
    vg.permute(0, 2, 1, 3)[junk] = float("inf")
    got = check_attention(q, kg, vg, past, table, nn, mask, clean=(kc, vc))
    assert not got["out"][2].any() and not got["out"][1, 6:].any() and not got["out"][3, 0].any()
    # node 3 of request 0: its own row alone may turn
    page, row = O.slot(table, pool, ps, 0, 21 + 3)
    for bad in (float("nan"), float("inf"), -float("inf")):
        vb = vg.clone()
        vb[page, :, row] = bad
        kb = kg.clone()
        kb[page, :, row] = bad
        for k2, v2 in ((kg, vb), (kb, vg)):
            o = pkg.ddtree_attention(q.to(DEV), k2.to(DEV), v2.to(DEV), dev(past), page_table=dev(table),
                                     num_nodes=dev(nn), mask=dev(mask))["out"]
            rest = [i for i in range(T) if i != 3]
            assert torch.equal(o[0, rest], got["out"][0, rest]) and torch.equal(o[1:], got["out"][1:])


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("T,G", TILES, ids=[f"{t * g}rows" for t, g in TILES])
def test_every_arrangement_over_short_and_long_caches(T, G, dh, dtype):
    """Each arrangement of waves in each type and head size: trees and chains, a cache that ends in
    its first tile beside one that is cut over many workgroups and merged."""
    rng = np.random.default_rng(T * dh + 1)
    past, ps = np.array([5, 4200, 0], np.int32), 16
    table, pool = paging(rng, 3, past + T, ps)
    q = rounded(rng, (3, T, 2 * G, dh), dtype, 2.0)
    kc, vc = rounded(rng, (pool, 2, ps, dh), dtype), rounded(rng, (pool, 2, ps, dh), dtype)
    nn = np.array([T - 1, T // 2, T - 1], np.int32)
    mask = OR.mask(trees(rng, 3, T - 1)[0], nn, T - 1).view(np.int64) if T > 1 else None
    check_attention(q, kc, vc, past, table, nn, mask)
    check_attention(q, kc, vc, past, table, None, None)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(5, 2), (9, 3), (12, 4), (40, 3)], ids=["10rows", "27rows", "48rows", "120rows"])
def test_garbage_in_every_arrangement(T, G, dh, dtype):
    """As above for each arrangement of waves: NaN and infinities behind the block, on an unmapped
    page, on others' pages and in a sibling's row reach only the rows that see them."""
    rng = np.random.default_rng(T * dh + 2)
    ps = 16
    past = np.array([61, 130], np.int32)
    nn = np.array([T - 1, T // 2], np.int32)
    mask = OR.mask(np.zeros((2, T - 1), np.int32), nn, T - 1).view(np.int64)  # all nodes are siblings
    table, pool = paging(rng, 2, past + T, ps)
    table[1, 2] = -1  # rows 32..47 of request 1 are on no page
    q = rounded(rng, (2, T, 2 * G, dh), dtype)
    kc, vc = rounded(rng, (pool, 2, ps, dh), dtype), rounded(rng, (pool, 2, ps, dh), dtype)
    used = np.zeros((pool, ps), bool)
    for b in range(2):
        for r in range(int(past[b]) + int(nn[b]) + 1):
            at = O.slot(table, pool, ps, b, r)
            if at is not None:
                used[at] = True
    kg, vg = kc.clone(), vc.clone()
    junk = torch.from_numpy(~used)
    kg.permute(0, 2, 1, 3)[junk] = float("nan")
    vg.permute(0, 2, 1, 3)[junk] = torch.from_numpy(rng.choice([np.nan, np.inf, -np.inf, 1.0], (int(junk.sum()), 2, dh))).to(dtype)
    got = check_attention(q, kg, vg, past, table, nn, mask, clean=(kc, vc))
    page, row = O.slot(table, pool, ps, 0, 61 + 4)  # node 4 of request 0
    rest = [i for i in range(T) if i != 4]
    for bad in (float("nan"), float("inf"), -float("inf")):
        vb, kb = vg.clone(), kg.clone()
        vb[page, :, row, 3] = bad  # one element of a head
        kb[page, :, row] = bad
        for k2, v2 in ((kg, vb), (kb, vg)):
            o = pkg.ddtree_attention(q.to(DEV), k2.to(DEV), v2.to(DEV), dev(past), page_table=dev(table),
                                     num_nodes=dev(nn), mask=dev(mask))["out"]
            assert torch.equal(o[0, rest], got["out"][0, rest]) and torch.equal(o[1], got["out"][1])
            if v2 is vb:
                own, was = o[0, 4].float(), got["out"][0, 4]
                assert torch.equal(own[:, 3].isnan(), torch.full_like(own[:, 3], bad, device=DEV).isnan())
                assert not own[:, 3].isfinite().any() and (own[:, 3] != -bad).all()
                keep = [e for e in range(dh) if e != 3]
                assert torch.equal(o[0, 4][:, keep], was[:, keep])


def test_attention_of_a_round_of_the_operators():
    """The attention in a verification round, on the tree, mask and caches that the operators before
    it left on the device."""
    from test_gpu_sampled import make_round
    r = make_round(7)
    Hq, Hkv, dh = r["dims"]
    t = pkg.ddtree_build(r["draft"], r["B"])
    for layer, qkv in enumerate(r["qkv"]):
        q, k, v = qkv.split([Hq, Hkv, Hkv], 2)
        q = pkg.ddtree_append_kv(q, k, v, r["k"][layer], r["v"][layer], r["past"], rope=r["rope"],
                                 page_table=r["table"], depths=t["depths"], num_nodes=t["num_nodes"])
        check_attention(q.cpu(), r["k"][layer].cpu(), r["v"][layer].cpu(), r["past"].cpu().numpy(),
                        r["table"].cpu().numpy(), t["num_nodes"].cpu().numpy(), t["mask"].cpu().numpy())


def test_attention_of_a_padded_batch_and_node_counts():
    """Requests taken out, node counts outside the range, and no counts at all."""
    rng = np.random.default_rng(10)
    past = np.array([-1, 30, -5, 7], np.int32)
    q = rounded(rng, (4, 6, 2, 64), HF)
    kc, vc = rounded(rng, (4, 1, 50, 64), HF), rounded(rng, (4, 1, 50, 64), HF)
    for nn in (None, np.array([3, -2, 0, 99], np.int32)):
        check_attention(q, kc, vc, past, None, nn, None)


@pytest.mark.parametrize("longest", [300, 6000])
def test_attention_of_many_requests(longest):
    """More requests than a workgroup has threads: units dealt out whole, or (one of them far
    longer than the others) cut; a workspace full of garbage."""
    rng = np.random.default_rng(longest)
    batch, ps = 300, 16
    past = rng.integers(0, 301, batch).astype(np.int32)
    past[[17, 290]] = -1
    past[299] = longest
    table, pool = paging(rng, batch, np.maximum(past, 0) + 1, ps)
    q = rounded(rng, (batch, 1, 4, 64), BF)
    kc, vc = rounded(rng, (pool, 4, ps, 64), BF), rounded(rng, (pool, 4, ps, 64), BF)
    size = pkg.lib().ddtree_attention_workspace_size(batch, 1, 4, 4, 64, table.shape[1], ps)
    check_attention(q, kc, vc, past, table, None, None,
                    ws=torch.full((size,), 255, dtype=torch.uint8, device=DEV))


def test_rows_that_the_cache_has_no_room_for():
    """past + block beyond the table's rows: those rows are neither written nor seen."""
    rng = np.random.default_rng(13)
    T, ps = 9, 8
    past = np.array([20, 27, 40, 500], np.int32)  # room for 32 rows
    table = rng.permutation(16).astype(np.int32).reshape(4, 4)
    q = rounded(rng, (4, T, 2, 64), BF)
    kc, vc = rounded(rng, (16, 1, ps, 64), BF), rounded(rng, (16, 1, ps, 64), BF)
    check_attention(q, kc, vc, past, table, None, None)
    k = rounded(rng, (4, T, 1, 64), BF)
    kd, vd = kc.to(DEV), vc.to(DEV)
    pkg.ddtree_append_kv(None, k.to(DEV), k.to(DEV), kd, vd, dev(past), page_table=dev(table))
    _, ke, ve = O.append(f64(k), f64(k), f64(k), f64(kc), f64(vc), past, table=table)
    assert np.array_equal(f64(kd), ke) and np.array_equal(f64(vd), ve)


def test_attention_is_deterministic_and_streams_keep_apart():
    rng = np.random.default_rng(11)
    past = np.array([900, 33, 2000], np.int32)
    table, pool = paging(rng, 3, past + 5, 32)
    sets = [[rounded(rng, s, BF).to(DEV) for s in ((3, 5, 8, 128), (pool, 2, 32, 128), (pool, 2, 32, 128))]
            for _ in range(2)]
    run = lambda s: pkg.ddtree_attention(*s, dev(past), page_table=dev(table))["out"]  # noqa: E731
    ref = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, (s, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                got[i].append(run(s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, ref[i]) for o in got[i])


def test_threads_on_one_stream_keep_apart():
    """Several host threads on the default stream at once, attention and acceptance with the
    binding's own workspaces: every result is that of the call made alone."""
    rng = np.random.default_rng(14)
    sets = []
    for i in range(4):
        past = np.array([700 + 400 * i, 2000 - 300 * i, 33], np.int32)
        table, pool = paging(rng, 3, past + 5, 32)
        att = [rounded(rng, s, BF).to(DEV) for s in ((3, 5, 8, 128), (pool, 2, 32, 128), (pool, 2, 32, 128))]
        par = dev(np.array([[0, 0, 1, 2, 2, 4]] * 3, np.int32))
        tok = dev(rng.permutation(5000)[:18].astype(np.int32).reshape(3, 6))
        sets.append((att, dev(past), dev(table), tok, par,
                     dev(rng.standard_normal((3, 7, 20000), dtype=np.float32)), dev(rng.random((3, 5), dtype=np.float32))))

    def run(s):
        att, past, table, tok, par, x, u = s
        return (pkg.ddtree_attention(*att, past, page_table=table)["out"],
                *pkg.ddtree_accept_sampled(tok, par, None, x, None, u).values())
    ref = [run(s) for s in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]

    def calls(i):
        for _ in range(30):
            got[i].append(run(sets[i]))
    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for want, outs in zip(ref, got):
        assert len(outs) == 30
        assert all(torch.equal(g, w) for out in outs for g, w in zip(out, want))


def test_attention_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes and elements: the last pages are read, not wrapped ones."""
    ps, Hkv, dh = 128, 8, 128
    pages = (1 << 32) // (ps * Hkv * dh) + 3
    kc = torch.zeros((pages, Hkv, ps, dh), dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    rng = np.random.default_rng(12)
    last = pages - 1
    small = [rounded(rng, (1, Hkv, ps, dh), BF) for _ in range(2)]
    k, v = rounded(rng, (1, 2, Hkv, dh), BF), rounded(rng, (1, 2, Hkv, dh), BF)
    q = rounded(rng, (1, 2, Hkv, dh), BF)
    kc[last], vc[last] = small[0][0].to(DEV), small[1][0].to(DEV)
    past, table = np.array([50], np.int32), np.array([[last]], np.int32)
    pkg.ddtree_append_kv(None, k.to(DEV), v.to(DEV), kc, vc, dev(past), page_table=dev(table))
    out = pkg.ddtree_attention(q.to(DEV), kc, vc, dev(past), page_table=dev(table))["out"]
    a, b = small[0].to(DEV), small[1].to(DEV)
    zero = dev(np.zeros((1, 1), np.int32))
    pkg.ddtree_append_kv(None, k.to(DEV), v.to(DEV), a, b, dev(past), page_table=zero)
    assert torch.equal(kc[last], a[0]) and torch.equal(vc[last], b[0]) and not kc[:last].any()
    assert torch.equal(out, pkg.ddtree_attention(q.to(DEV), a, b, dev(past), page_table=zero)["out"])


# ---- compaction -----------------------------------------------------------------
@pytest.mark.parametrize("case", [(3, 5, 4, 128, 16, 15, 64), (2, 3, 1, 8, 1, 32, 40), (1, 2, 2, 512, 64, 32, 255),
                                  (4, 7, 8, 64, 32, 4, 6)], ids=str)
def test_compact_paged(case):
    layers, batch, heads, dh, ps, L, B = case
    rng = np.random.default_rng(sum(case))
    past = rng.integers(0, 100, batch).astype(np.int32)
    past[-1] = -1 if batch > 4 else past[-1]
    n = rng.integers(0, min(L, B) + 1, batch).astype(np.int32)
    n[0] = min(L, B)
    acc = np.full((batch, L), -1, np.int32)
    for b in range(batch):
        acc[b, :n[b]] = np.sort(rng.choice(np.arange(1, B + 1), n[b], replace=False))
    table, pool = paging(rng, batch, np.maximum(past, 0) + B + 1, ps)
    table[1, (past[1] + B // 2) // ps] = -1  # a page that is none: its rows neither come nor go
    shape = (layers, pool, heads, ps, dh)
    k, v = (rng.integers(-30000, 30000, shape).astype(np.int16) for _ in range(2))
    kd, vd = dev(k), dev(v)
    nl = pkg.ddtree_compact_kv_paged(kd, vd, dev(table), dev(past), dev(acc), dev(n))
    ke, ve, ne = O.compact_paged(k, v, table, past, acc, n)
    assert np.array_equal(kd.cpu().numpy(), ke) and np.array_equal(vd.cpu().numpy(), ve)
    assert np.array_equal(nl.cpu().numpy(), ne)


def test_a_request_taken_out_stays_out_from_round_to_round():
    """Two rounds of append and compaction, each from the lengths that the one before gave: a
    request taken out, whatever its accept_len, keeps its length and its old pages' rows."""
    rng = np.random.default_rng(15)
    T, ps, dh, batch = 5, 8, 64, 4
    past = np.array([6, -1, 11, -3], np.int32)
    table = rng.permutation(batch * 4).astype(np.int32).reshape(batch, 4)
    kc, vc = (rounded(rng, (1, batch * 4, 2, ps, dh), BF) for _ in range(2))
    kd, vd, pd = kc.to(DEV), vc.to(DEV), dev(past)
    acc = np.tile(np.array([1, 3, 4], np.int32), (batch, 1))
    for n in (np.array([2, 0, 3, 2], np.int32), np.array([0, 3, 1, 99], np.int32)):
        k, v = rounded(rng, (batch, T, 2, dh), BF), rounded(rng, (batch, T, 2, dh), BF)
        pkg.ddtree_append_kv(None, k.to(DEV), v.to(DEV), kd[0], vd[0], pd, page_table=dev(table))
        pd = pkg.ddtree_compact_kv_paged(kd, vd, dev(table), pd, dev(acc), dev(n))
        past = np.where(past < 0, past, past + np.minimum(n, 3) + 1)
        assert np.array_equal(pd.cpu().numpy(), past)
    for b in (1, 3):
        assert torch.equal(kd[0, table[b]].cpu(), kc[0, table[b]]) and torch.equal(vd[0, table[b]].cpu(), vc[0, table[b]])


# ---- refusals of the binding ------------------------------------------------------
def test_binding_refusals():
    q = torch.zeros((2, 3, 4, 64), dtype=BF, device=DEV)
    kv = torch.zeros((2, 3, 2, 64), dtype=BF, device=DEV)
    c = torch.zeros((2, 2, 16, 64), dtype=BF, device=DEV)
    past = torch.zeros(2, dtype=torch.int32, device=DEV)
    table = torch.zeros((2, 1), dtype=torch.int32, device=DEV)
    att = lambda **k: pkg.ddtree_attention(**{**dict(q=q, k_cache=c, v_cache=c, past_len=past), **k})  # noqa: E731
    app = lambda **k: pkg.ddtree_append_kv(**{**dict(q=q, k=kv, v=kv, k_cache=c, v_cache=c.clone(), past_len=past), **k})  # noqa: E731
    att(), app()
    for bad in (dict(q=q.cpu()), dict(past_len=past[:1]), dict(k_cache=c[:1], v_cache=c[:1]),
                dict(page_table=table[:1]), dict(q=q.transpose(1, 2)), dict(v_cache=c[:, :1]),
                dict(mask=torch.zeros((2, 3, 2), dtype=torch.int64, device=DEV)), dict(q=q[..., :32].contiguous())):
        with pytest.raises(ValueError):
            att(**bad)
    for bad in (dict(q=q.float()), dict(q=q.half()), dict(past_len=past.long())):
        with pytest.raises(TypeError):
            att(**bad)
    for bad in (dict(scale=0.0), dict(q=q[:, :, :3].contiguous())):
        with pytest.raises(pkg.DDTreeError):
            att(**bad)
    for bad in (dict(k=kv[:, :2]), dict(v=kv[:, :, :1]), dict(k=kv.transpose(1, 2)), dict(q_out=q[:, :2]),
                dict(depths=past), dict(num_nodes=past[:1]), dict(rope=torch.zeros(3, device=DEV))):
        with pytest.raises(ValueError):
            app(**bad)
    with pytest.raises(TypeError):
        app(k=kv.half())
    with pytest.raises(ValueError):
        pkg.ddtree_compact_kv_paged(c[None], c[None], None, past, torch.zeros((2, 3), dtype=torch.int32, device=DEV), past)
