"""GPU tests of attention over shared rows (ddtree_attention_shared, and shared_len of
ddtree_attention_kv8) where the pass over them runs: as many query rows as 32-bit products do not
hold, captured graphs, garbage, small pages, large scores. Tolerances as in
tests/test_gpu_kv8.py."""

import numpy as np
import pytest
import torch

import draft_tree_construction_depth_amd as pkg
from oracle import verify as O
from test_gpu_kv8 import ENOUGH, attend64, compare, make_cache, one, shared_pages
from test_gpu_verify_cache import BF, DEV, HF, dev, f64, paging, rounded

pytestmark = pytest.mark.gpu
NAN = float("nan")


def call(kind):
    return pkg.ddtree_attention_kv8 if kind else pkg.ddtree_attention_shared


def workspace(kind, *sizes):
    """A workspace that ends exactly where the call may write last; its first number is the rows
    that the pass takes as shared."""
    size = pkg.lib().ddtree_attention_kv8_workspace_size(*sizes, 1) if kind else \
        pkg.lib().ddtree_attention_shared_workspace_size(*sizes)
    assert size > pkg.lib().ddtree_attention_workspace_size(*sizes)  # it has the shared rows' part
    return torch.full((size,), 255, dtype=torch.uint8, device=DEV)


def used_by(ws):
    return int(ws[:4].view(torch.int32))


def least_rows(sharing, Hkv, dh, kind):
    """Shared rows that `sharing` requests beside the first need for a pass of their own."""
    return -(-ENOUGH // (sharing * 2 * Hkv * dh * (1 if kind else 2)) // 128) * 128


# ---- many query rows ----------------------------------------------------------------------
@pytest.mark.parametrize("batch,dh,kind", [(40000, 64, "e4m3"), (20000, 256, "")], ids=["64", "256"])
def test_query_rows_beyond_32_bit_products(batch, dh, kind):
    """One pass over the shared rows for 3.2 or 1.6 million query rows, whose query tiles times waves
    pass 2^31: every row is written, and those of 300 requests from end to end are the oracle's."""
    T, ps, past = 80, 128, np.full(batch, 128, np.int32)
    g = torch.Generator(device=DEV)
    g.manual_seed(dh)
    table = np.stack([np.zeros(batch, np.int32), np.arange(1, batch + 1, dtype=np.int32)], 1)
    cache = make_cache(g, (batch + 1, 1, ps, dh), kind, BF)
    q = torch.empty((batch, T, 1, dh), dtype=BF, device=DEV).normal_(generator=g)
    past[7] = -1
    ws = workspace(kind, batch, T, 1, 1, dh, 2, ps)
    out = {"out": torch.full_like(q, NAN), "lse": torch.full(q.shape[:3], NAN, device=DEV)}
    call(kind)(q, *cache, dev(past), page_table=dev(table), shared_len=one(128), out=out, ws=ws)
    assert used_by(ws) == 128
    assert not out["out"].isnan().any() and not out["lse"].isnan().any()
    nq = 16 if dh == 256 else 32  # query rows of a wave, four to a tile
    border = (1 << 31) // (batch * T // nq) * nq * 4 // T  # the request where tile * waves passes 2^31
    assert 0 < border < batch
    some = np.unique(np.concatenate([np.linspace(0, batch - 1, 280).astype(int), np.arange(6, 10),
                                     border + np.arange(-8, 8)]))
    some = some[(some >= 0) & (some < batch)]
    qs = q[dev(some)].cpu()
    oracle, most = attend64(qs, cache, kind, past[some], table[some], None, None)
    compare({x: v[dev(some)] for x, v in out.items()}, qs, oracle, most, past[some], kind)


# ---- few heads -----------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("batch,T,G,Hkv,dh", [(1, 513, 64, 1, 256), (1, 513, 24, 3, 256), (1, 200, 659, 1, 64),
                                              (3, 513, 24, 1, 256), (5, 300, 40, 1, 256), (1, 513, 8, 1, 128)], ids=str)
def test_whole_units_of_few_heads(batch, T, G, Hkv, dh, kind):
    """More query tiles than the card holds at once, of heads that do not fill the XCDs alike."""
    rng, g = np.random.default_rng(batch * G), torch.Generator(device=DEV)
    g.manual_seed(batch * G)
    past = rng.integers(150, 400, batch).astype(np.int32)
    table, pool = paging(rng, batch, past + T, 32)
    q = rounded(rng, (batch, T, Hkv * G, dh), BF)
    cache = make_cache(g, (pool, Hkv, 32, dh), kind, BF)
    nn = np.array([T - 1, T // 2, T - 1, 0, T - 9][:batch], np.int32)
    out = {"out": torch.full(q.shape, NAN, dtype=BF, device=DEV), "lse": torch.full(q.shape[:3], NAN, device=DEV)}
    got = pkg.ddtree_attention_kv8(q.to(DEV), *cache, dev(past), page_table=dev(table), num_nodes=dev(nn), out=out)
    oracle, most = attend64(q, cache, kind, past, table, nn, None)
    compare(got, q, oracle, most, past, kind)


@pytest.mark.parametrize("kind", ["", "e4m3"])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_shared_rows_of_few_heads(Hkv, kind):
    rng, g = np.random.default_rng(Hkv), torch.Generator(device=DEV)
    g.manual_seed(Hkv)
    batch, T, dh, ps = 420 // Hkv, 80, 256, 64
    shared = least_rows(batch - 1, Hkv, dh, kind)
    past = (shared + rng.integers(0, 90, batch)).astype(np.int32)
    table, pool = shared_pages(rng, batch, past, T, ps, shared)
    q = rounded(rng, (batch, T, Hkv, dh), BF)
    cache = make_cache(g, (pool, Hkv, ps, dh), kind, BF)
    ws = workspace(kind, batch, T, Hkv, Hkv, dh, table.shape[1], ps)
    got = call(kind)(q.to(DEV), *cache, dev(past), page_table=dev(table), shared_len=one(shared), with_lse=True, ws=ws)
    assert used_by(ws) == shared
    oracle, most = attend64(q, cache, kind, past, table, None, None)
    compare(got, q, oracle, most, past, kind)


# ---- captured ------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["", "e4m3"])
def test_captured_calls_replay_and_keep_apart(kind):
    """Calls whose pass over the shared rows runs, in two graphs, replayed in turn with eager work
    between, after the shared rows, the contexts and the requests that take part have changed: the
    device takes all rows, fewer and none, and each replay equals the eager call."""
    rng, g = np.random.default_rng(31), torch.Generator(device=DEV)
    g.manual_seed(31)
    batch, T, G, Hkv, dh, ps = 5, 3, 4, 4, 128, 32
    least = least_rows(batch - 1, Hkv, dh, kind)
    shared = least + 4096
    long = (shared + np.array([0, 100, 1100, 50, 1])).astype(np.int32)
    table, pool = shared_pages(rng, batch, long, T, ps, shared)
    less, out, gone = long.copy(), long.copy(), np.full(batch, -1, np.int32)
    less[3] = least + 129  # one request has less
    out[[0, 4]] = -1  # three take part: too few, but for the row counts below
    lens = [(shared, long, shared), (least + 200, long, least + 128), (shared, less, least + 128), (shared, out, 0),
            (least - 1, long, 0), (shared, gone, 0), (-3, long, 0), (shared, long, shared)]
    where, sizes = dev(table), (batch, T, Hkv * G, Hkv, dh, table.shape[1], ps)
    at, count, nn = dev(long), one(shared), dev(np.array([2, 0, 2, 1, 2], np.int32))
    sets, spaces, eager = [], [], {}
    for i in range(2):
        sets.append((rounded(rng, (batch, T, Hkv * G, dh), (BF, HF)[i]).to(DEV),
                     *make_cache(g, (pool, Hkv, ps, dh), kind, (BF, HF)[i])))
        spaces.append(workspace(kind, *sizes))
    run = lambda i, ws=None: call(kind)(*sets[i], at, page_table=where, num_nodes=nn, shared_len=count, with_lse=True, ws=ws)  # noqa: E731

    def set_lengths(n):
        count.fill_(lens[n][0])
        at.copy_(torch.from_numpy(lens[n][1]))

    for n, (_, past, used) in enumerate(lens):
        set_lengths(n)
        for i in range(2):
            ws = workspace(kind, *sizes)
            eager[n, i] = run(i, ws)
            assert used_by(ws) == used
            if n in (1, 2, 3):  # (the tests of test_gpu_kv8.py have the others)
                oracle, most = attend64(sets[i][0].cpu(), sets[i][1:], kind, past, table, nn.cpu().numpy(), None)
                compare(eager[n, i], sets[i][0].cpu(), oracle, most, past, kind)
    set_lengths(0)
    torch.cuda.synchronize()
    graphs, got = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # one workspace of the caller's, one of the graph's own
            got.append((run(i, spaces[i]), run(i)))
        graphs.append(graph)
    for n in [0, 3, 1, 5, 2, 4, 7, 6, 1, 0]:
        set_lengths(n)
        for i in range(2):
            for o in got[i]:
                o["out"].fill_(NAN)
            graphs[i].replay()
            run(1 - i)  # eager work between the replays
        torch.cuda.synchronize()
        for i in range(2):
            assert used_by(spaces[i]) == lens[n][2], n
            for o in got[i]:
                assert torch.equal(o["out"], eager[n, i]["out"]) and torch.equal(o["lse"], eager[n, i]["lse"]), (n, i)


# ---- garbage ---------------------------------------------------------------------------------
def spoil(g, cache, kind, keep):
    """The cache with garbage in every row but those of `keep` [pages, page_size]: NaN, infinities,
    the largest numbers, in codes e4m3 NaN and in their scales the same."""
    junk = dev(~keep)
    bad = torch.tensor([NAN, float("inf"), -float("inf"), 3e38, -3e38], device=DEV)
    pick = lambda n: bad[torch.randint(0, 5, n, device=DEV, generator=g)]  # noqa: E731
    got = [c.clone() for c in cache]
    n = int(junk.sum())
    for c in got[:2]:
        heads, dh = c.shape[1], c.shape[3]
        rows = c.view(torch.uint8).permute(0, 2, 1, 3) if kind else c.permute(0, 2, 1, 3)
        if kind:
            codes = torch.randint(0, 256, (n, heads, dh), device=DEV, generator=g).to(torch.uint8)
            codes[..., :2] = 0x7F
            rows[junk] = codes
        else:
            values = torch.randn((n, heads, dh), device=DEV, generator=g)
            values[..., ::3] = pick(values[..., ::3].shape)
            rows[junk] = values.to(c.dtype)
    for s in got[2:]:
        s.permute(0, 2, 1)[junk] = pick((n, s.shape[1]))
    return tuple(got)


# query rows of a key/value head: all of the batch's, a request's: every arrangement of both passes
ARRANGED = [(2, 5, 1), (3, 5, 2), (2, 9, 3), (4, 10, 4), (3, 26, 3)]


@pytest.mark.parametrize("kind", ["", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("batch,T,G", ARRANGED, ids=[f"{b}x{t * g}rows" for b, t, g in ARRANGED])
def test_garbage(batch, T, G, dh, dtype, kind):
    """Garbage behind the block, on entries of the shared rows and of a request's own that are no
    page, on others' pages and in a sibling's row reaches only the rows that see it; so does that
    in queries of rows that take no part."""
    rng, g = np.random.default_rng(batch * T * dh + 5), torch.Generator(device=DEV)
    g.manual_seed(batch * T * dh + 5)
    Hkv, ps = 2, 16
    shared = least_rows(batch - 1, Hkv, dh, kind) + 128
    past = (shared + rng.integers(40, 90, batch)).astype(np.int32)
    past[0] = shared + 61
    nn = np.array([T - 1, T // 2, T - 1, T - 2][:batch], np.int32)
    # all nodes are siblings: a row sees the root and itself
    bits = np.zeros((batch, T, 64 * ((T + 63) // 64)), np.uint8)
    bits[:, :, 0] = 1
    bits[:, np.arange(T), np.arange(T)] = 1
    mask = np.packbits(bits, axis=2, bitorder="little").view(np.int64)
    table, pool = shared_pages(rng, batch, past, T, ps, shared)
    table[:, 5], table[:, 9] = -1, pool + 3  # of the shared rows
    table[1, shared // ps + 1] = -1  # rows of request 1 alone
    q = rounded(rng, (batch, T, Hkv * G, dh), dtype)
    q[1, T // 2 + 1:] = NAN
    clean = make_cache(g, (pool, Hkv, ps, dh), kind, dtype)
    keep = np.zeros((pool, ps), bool)
    for b in range(batch):
        rows = np.arange(past[b] + nn[b] + 1)
        page = table[b, rows // ps]
        on = (page >= 0) & (page < pool)
        keep[page[on], rows[on] % ps] = True
    cache = spoil(g, clean, kind, keep)
    sizes = (batch, T, Hkv * G, Hkv, dh, table.shape[1], ps)
    ws, qd = workspace(kind, *sizes), q.to(DEV)
    args = dict(page_table=dev(table), num_nodes=dev(nn), mask=dev(mask), shared_len=one(shared))
    got = call(kind)(qd, *cache, dev(past), with_lse=True, ws=ws, **args)
    assert used_by(ws) == shared
    known = torch.nan_to_num(q)
    oracle, most = attend64(known, clean, kind, past, table, nn, mask)
    compare(got, known, oracle, most, past, kind)
    assert not got["out"][1, T // 2 + 1:].any()
    # node 4 of request 0: its row reaches itself alone, and the other key/value head not at all
    page, row = O.slot(table, pool, ps, 0, int(past[0]) + 4)
    rest = [i for i in range(T) if i != 4]
    for bad in (NAN, float("inf"), -float("inf")):
        for x in range(2):
            worse = [c.clone() for c in cache]
            worse[x + 2 if kind else x][page, 0, row] = bad
            o = call(kind)(qd, *worse, dev(past), **args)["out"]
            assert torch.equal(o[0, rest], got["out"][0, rest]) and torch.equal(o[1:], got["out"][1:])
            assert torch.equal(o[0, 4, G:], got["out"][0, 4, G:])
            if np.isnan(bad):
                assert o[0, 4, :G].isnan().all()


# ---- small pages, large scores ---------------------------------------------------------------
@pytest.mark.parametrize("kind", ["", "e4m3", "i8"])
@pytest.mark.parametrize("ps", [1, 4])
@pytest.mark.parametrize("T,G", [(1, 4), (5, 5), (21, 3)], ids=["4rows", "25rows", "63rows"])
def test_pages_smaller_than_a_load(T, G, ps, kind):
    rng, g = np.random.default_rng(T + ps), torch.Generator(device=DEV)
    g.manual_seed(T + ps)
    batch, Hkv, dh = 4, 4, (64, 128, 256)[T % 3]
    shared = least_rows(batch - 1, Hkv, dh, kind) + 128
    past = (shared + np.array([0, 33, 7, 150])).astype(np.int32)
    table, pool = shared_pages(rng, batch, past, T, ps, shared)
    q = rounded(rng, (batch, T, Hkv * G, dh), BF, 2.0)
    cache = make_cache(g, (pool, Hkv, ps, dh), kind, BF)
    ws = workspace(kind, batch, T, Hkv * G, Hkv, dh, table.shape[1], ps)
    got = call(kind)(q.to(DEV), *cache, dev(past), page_table=dev(table), shared_len=one(shared + 5), with_lse=True, ws=ws)
    assert used_by(ws) == shared
    oracle, most = attend64(q, cache, kind, past, table, None, None)
    compare(got, q, oracle, most, past, kind)


@pytest.mark.parametrize("kind", ["", "e4m3", "i8"])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("size", [2.0 ** 21, 2.0 ** 25], ids=["2p21", "2p25"])
@pytest.mark.parametrize("T,G", [(1, 2), (5, 5), (21, 3)], ids=["2rows", "25rows", "63rows"])
def test_small_differences_between_large_scores(T, G, size, dtype, kind):
    """Scores that share a large part, the same in the shared rows and in a request's own, and
    differ by a few float32 steps of it at most: the two parts are joined as one."""
    rng, g = np.random.default_rng(T), torch.Generator(device=DEV)
    g.manual_seed(T)
    batch, Hkv, dh, ps = 5, 4, 64, 64
    shared = least_rows(batch - 1, Hkv, dh, kind)
    past = (shared + np.array([0, 70, 300, 11, 1])).astype(np.int32)
    table, pool = shared_pages(rng, batch, past, T, ps, shared)
    q = torch.zeros((batch, T, Hkv * G, dh), dtype=dtype)
    q[..., 0], q[..., 1] = size / 2.0 ** 11, 1.0
    step = max(size / 2.0 ** 23, 0.5)
    small = torch.from_numpy(rng.integers(-12, 13, (pool, Hkv, ps)) * step)
    cache = list(make_cache(g, (pool, Hkv, ps, dh), kind, dtype))
    if kind:  # codes of scale 2^5: 64 and the small part, which both kinds have exactly up to a rounding
        cache[0].zero_()
        as_code = lambda x: x.round().to(torch.int8) if kind == "i8" else x.float().to(cache[0].dtype)  # noqa: E731
        cache[0][..., 0] = as_code(torch.tensor(64.0)).to(DEV)
        cache[0][..., 1] = as_code(small / 32).to(DEV)
        cache[2].fill_(2.0 ** 5)
    else:
        cache[0].zero_()
        cache[0][..., 0] = 2.0 ** 11
        cache[0][..., 1] = small.to(dtype).to(DEV)
    ws = workspace(kind, batch, T, Hkv * G, Hkv, dh, table.shape[1], ps)
    got = call(kind)(q.to(DEV), *cache, dev(past), page_table=dev(table), shared_len=one(shared), scale=1.0, with_lse=True,
                     ws=ws)
    assert used_by(ws) == shared and got["out"].isfinite().all()
    (out, lse, spread, _), most = attend64(q, cache, kind, past, table, None, None, 1.0)
    half, n = torch.finfo(dtype).eps / 2, int(past.max()) + T
    # a score in powers of two: its own product's rounding, scale * log2(e)'s and the maximum's, for
    # the weight and for the others, and the maxima of the two parts once more: four steps at most
    off = np.expm1(4 * np.spacing(np.float32(1.45 * size)) * np.log(2))
    tiny = 2.0 ** -25 + (n * 2.0 ** -37 * most if kind else 0)
    tol = half * np.abs(out) + spread * (1 + half) * (half + 2 * off + 2.0 ** -14 + n * 2.0 ** -24) + tiny
    assert np.all(np.abs(f64(got["out"]) - out) <= tol)
    assert np.all(np.abs(f64(got["lse"]) - lse) <= 2.0 ** -20 * np.abs(lse))
