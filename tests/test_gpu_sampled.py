"""GPU tests of the acceptance at a temperature (ddtree_accept_sampled,
dspark_accept_sampled) against the float64 oracle: paths and tokens equal,
log-probabilities to the float32 rounding (2^-24 of the value; 1e-12 for the
float64 sums), and the verification round as a whole, eager and captured."""

import numpy as np
import pytest
import torch

import draft_tree_construction_depth_amd as pkg
from draft_tree_construction_depth_amd import gen
from oracle import verify as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def held(x, kind):
    """x rounded to the logits' type: (device tensor, its float64 values)."""
    t = torch.from_numpy(x).to(torch.bfloat16 if kind == "bf16" else torch.float32)
    return t.to(DEV), t.double().numpy()


def random_trees(rng, batch, B, V):
    par, tok = np.zeros((batch, B), np.int32), np.zeros((batch, B), np.int32)
    for b in range(batch):
        used = {}
        for j in range(B):
            while True:
                p, x = int(rng.integers(0, j + 1)), int(rng.integers(0, V))
                if x not in used.setdefault(p, set()):
                    break
            par[b, j], tok[b, j] = p, x
            used[p].add(x)
    return par, tok


def favour(x, par, tok, rng, share=2.0):
    """Raise the children's logits so that walks go on: their weight is a few times the row's rest."""
    batch, B = par.shape
    for b in range(batch):
        for j in range(B):
            row = x[b, par[b, j]]
            x[b, par[b, j], tok[b, j]] = np.log(np.exp(row - row.max()).sum()) + row.max() + rng.uniform(-1, share)
    return x


def same(got, want, names):
    for name, w in zip(names, want):
        g = got[name].cpu().numpy()
        if name == "logp":
            assert np.array_equal(np.isinf(g), np.isinf(w))
            f = np.isfinite(w)
            assert np.all(np.abs(g[f] - w[f]) <= 2.0 ** -24 * np.abs(w[f]) + 1e-12)
        else:
            assert np.array_equal(g, w), name


TREE = ("accepted_nodes", "accept_len", "next_token", "logp")
CHAIN = ("accept_len", "next_token", "logp")

TREES = [
    # batch, B, L, V, type
    (1, 1, 1, 2, "f32"),
    (4, 5, 3, 7, "bf16"),
    (3, 64, 15, 1000, "bf16"),
    (5, 20, 6, 4099, "f32"),     # rows that are not a multiple of 16 bytes
    (2, 33, 8, 16385, "bf16"),   # a chunk and one element
    (2, 512, 32, 2048, "f32"),
    (70, 16, 6, 300, "bf16"),
    (1, 64, 15, 151936, "bf16"),
    (40, 64, 15, 40000, "f32"),  # more rows than the path needs
]


@pytest.mark.parametrize("case", TREES, ids=[f"b{c[0]}B{c[1]}V{c[3]}{c[4]}" for c in TREES])
def test_tree_acceptance(case):
    batch, B, L, V, kind = case
    rng = np.random.default_rng(B * V)
    par, tok = random_trees(rng, batch, B, V)
    x = rng.standard_normal((batch, B + 1, V), dtype=np.float32) * rng.uniform(0.5, 3, (batch, B + 1, 1)).astype(np.float32)
    x = favour(x, par, tok, rng)
    xd, xh = held(x, kind)
    heat = rng.uniform(0.4, 1.5, batch).astype(np.float32)
    heat[1::4] = 0.0
    nn = rng.integers(B // 2, B + 1, batch).astype(np.int32)
    u = rng.random((batch, L + 1), dtype=np.float32)
    size = pkg.lib().ddtree_accept_sampled_workspace_size(batch, B, L, V, kind == "f32")
    got = pkg.ddtree_accept_sampled(dev(tok), dev(par), dev(nn), xd, dev(heat), dev(u),
                                    ws=torch.full((size,), 255, dtype=torch.uint8, device=DEV))
    want = O.accept_tree(tok, par, nn, xh, heat, u.astype(np.float64))
    same(got, want, TREE)
    if batch > 2:
        assert want[1].max() > 0  # there are walks that go on


def test_tree_acceptance_of_odd_rows():
    """Masked tokens and rows, NaN, infinities, equal logits, repeated and foreign tokens, a
    child of a later node, numbers and counts outside their range, no counts, no temperatures."""
    inf, nan = np.inf, np.nan
    V, B, L = 24, 6, 3
    rows = np.zeros((12, B + 1, V), np.float32)
    rows[0, :, 3:] = -inf           # three tokens left
    rows[1] = -inf                  # nothing left
    rows[2, :, ::2] = nan
    rows[3, :, 5] = inf
    rows[4, :, 5:7] = inf
    rows[5] = 3e38
    rows[6] = -3e38
    rows[7, :, 9] = 1e4             # a point mass
    rows[8, :, 8:] = np.finfo(np.float32).min  # the type's lowest value as a mask
    tok = np.tile(np.array([2, 5, 5, 9, 1, 7], np.int32), (12, 1))
    par = np.tile(np.array([0, 0, 0, 2, 1, 3], np.int32), (12, 1))
    tok[9] = [V, -1, 3, V + 100, 0, 2]
    par[10] = [5, 0, -3, 2, 9, 0]   # parents that are not earlier nodes
    nn = np.full(12, B, np.int32)
    nn[11] = 99
    u = np.random.default_rng(0).random((12, L + 1), dtype=np.float32)
    for heat in (None, np.full(12, 0.7, np.float32), np.zeros(12, np.float32),
                 np.array([nan, -1, inf, 1e-30, 1, 2, 1e30, 1, 1, 1, 1, 1], np.float32)):
        for uu in (u, np.zeros_like(u), np.full_like(u, 1 - 2.0 ** -24), np.full_like(u, 7.0),
                   np.full_like(u, nan), np.full_like(u, -1.0)):
            for counts in (nn, None, np.zeros(12, np.int32) - 4):
                got = pkg.ddtree_accept_sampled(dev(tok), dev(par), dev(counts), dev(rows), dev(heat), dev(uu))
                same(got, O.accept_tree(tok, par, counts, rows.astype(np.float64), heat, uu.astype(np.float64)), TREE)


@pytest.mark.parametrize("V", [4194303, 4194304])
def test_the_longest_rows(V):
    """Rows whose last chunk holds a few elements or none, the next token their last one."""
    rng = np.random.default_rng(V)
    x = rng.standard_normal((1, 2, V), dtype=np.float32)
    x[0, 0, 77] = x[0, 1, V - 1] = 40.0
    xd, xh = held(x, "f32")
    tok, par, u = np.full((1, 1), 77, np.int32), np.zeros((1, 1), np.int32), np.full((1, 2), 0.5, np.float32)
    got = pkg.ddtree_accept_sampled(dev(tok), dev(par), None, xd, None, dev(u))
    want = O.accept_tree(tok, par, None, xh, None, u.astype(np.float64))
    same(got, want, TREE)
    assert want[1][0] == 1 and want[2][0] == V - 1
    y = x[:, :1].copy()
    yd, yh = held(y, "f32")
    got = pkg.dspark_accept_sampled(dev(tok), xd, yd, None, dev(u))
    same(got, O.accept_chain(tok, None, xh, yh, None, u.astype(np.float64)), CHAIN)
    y[0, 0, 77], y[0, 0, V - 2] = 0.0, 40.0  # the guess falls, what is left is drawn
    yd, yh = held(y, "f32")
    tok[0, 0] = V - 2
    got = pkg.dspark_accept_sampled(dev(tok), xd, yd, None, dev(u))
    same(got, O.accept_chain(tok, None, xh, yh, None, u.astype(np.float64)), CHAIN)


def test_infinite_logits_at_great_temperatures():
    """+inf counts as the largest finite value also where the temperature brings it near the others."""
    rng = np.random.default_rng(8)
    V, P = 5000, 3
    heat = np.array([1e37, 1e38, 3e38, np.inf], np.float32)
    x = (rng.standard_normal((4, P + 1, V)) * 1e37).astype(np.float32)
    y = (rng.standard_normal((4, P, V)) * 1e37).astype(np.float32)
    x[:, :, 11::700], y[:, :, 300::900] = np.inf, np.inf
    x[:, :, 12::700], y[:, :, 301::900] = np.nan, -np.inf
    tok = rng.integers(0, V, (4, P)).astype(np.int32)
    tok[:, 1] = 11
    par = np.array([[0, 0, 1]] * 4, np.int32)
    for kind in ("f32", "bf16"):
        (xd, xh), (yd, yh) = held(x, kind), held(y, kind)
        for share in (0.0, 0.3, 0.7, 0.99):
            u = np.full((4, P + 1), share, np.float32)
            same(pkg.ddtree_accept_sampled(dev(tok), dev(par), None, xd, dev(heat), dev(u)),
                 O.accept_tree(tok, par, None, xh, heat, u.astype(np.float64)), TREE)
            same(pkg.dspark_accept_sampled(dev(tok), xd, yd, dev(heat), dev(u)),
                 O.accept_chain(tok, None, xh, yh, heat, u.astype(np.float64)), CHAIN)


# Eight logits (in steps of 2^-10) and the place among their children of one without weight, such that
# half the row's sum lies between the children's running sums before and behind that place: the float64
# scan over lanes rounds differently from lane to lane, so the latter is a step larger.
BORDERS = [
    (8, [366, 1422, 993, 432, 808, 3269, 3609, 249]),
    (8, [2510, 1047, 1620, 3342, 3550, 123, 3174, 1055]),
    (8, [743, 2201, 1327, 3954, 4, 619, 578, 3046]),
    (8, [3686, 392, 230, 3320, 2637, 3691, 572, 2991]),
    (8, [183, 686, 93, 3085, 3636, 1636, 640, 4006]),
    (8, [3692, 1355, 3318, 577, 146, 874, 61, 2968]),
    (8, [188, 2180, 386, 1589, 1929, 4065, 2830, 3728]),
    (8, [2118, 98, 229, 3710, 4081, 302, 3040, 212]),
]


def test_a_child_without_weight_is_never_accepted():
    """A masked child behind others: however sums round, no number falls on it."""
    batch, B, V = len(BORDERS), 9, 20
    x = np.full((batch, B + 1, V), -np.inf, np.float32)
    tok = np.zeros((batch, B), np.int32)
    for b, (at, steps) in enumerate(BORDERS):
        x[b, :, :8] = x[b, :, 8:16] = np.array(steps) / 1024
        tok[b] = np.insert(np.arange(8), at, 16)
    par, u = np.zeros((batch, B), np.int32), np.full((batch, 2), 0.5, np.float32)
    got = pkg.ddtree_accept_sampled(dev(tok), dev(par), None, dev(x), None, dev(u))
    path, n, last, logp = (got[k].cpu().numpy() for k in TREE)
    taken = np.where(n > 0, tok[np.arange(batch), np.maximum(path[:, 0], 1) - 1], last)
    assert (taken < 16).all() and (last < 16).all() and np.isfinite(logp).all()


def test_tree_acceptance_gives_the_target_distribution():
    """4096 requests with evenly spread numbers: every first token comes out 4096 p(v) times."""
    rng = np.random.default_rng(5)
    N, V = 4096, 50
    x = (rng.standard_normal(V) * 2).astype(np.float32)
    tok = np.tile(np.array([[3, 7, 40, 11]], np.int32), (N, 1))
    par = np.tile(np.array([[0, 0, 0, 1]], np.int32), (N, 1))
    u = np.full((N, 3), 0.5, np.float32)
    u[:, 0] = (np.arange(N) + 0.5) / N
    got = pkg.ddtree_accept_sampled(dev(tok), dev(par), None, dev(np.broadcast_to(x, (N, 5, V))), None, dev(u))
    path, n, last = (got[k].cpu().numpy() for k in TREE[:3])
    first = np.where(n > 0, tok[0, np.maximum(path[:, 0], 1) - 1], last)
    p = np.exp(x.astype(np.float64))
    assert np.abs(np.bincount(first, minlength=V) - N * p / p.sum()).max() <= 1.0


def test_temperature_zero_is_the_greedy_walk():
    rng = np.random.default_rng(6)
    batch, B, L, V = 9, 40, 8, 500
    par, tok = random_trees(rng, batch, B, V)
    x = favour(rng.standard_normal((batch, B + 1, V)).astype(np.float32), par, tok, rng)
    nn = dev(rng.integers(1, B + 1, batch).astype(np.int32))
    got = pkg.ddtree_accept_sampled(dev(tok), dev(par), nn, dev(x), dev(np.zeros(batch, np.float32)),
                                    dev(rng.random((batch, L + 1), dtype=np.float32)))
    want = pkg.ddtree_accept(dev(tok), dev(par), nn, dev(x.argmax(2).astype(np.int32)), L)
    assert all(torch.equal(got[k], want[k]) for k in want) and int(want["accept_len"].max()) > 1


CHAINS = [
    # batch, P, V, type
    (1, 1, 2, "f32"),
    (6, 4, 37, "bf16"),
    (3, 7, 4099, "f32"),
    (2, 16, 16385, "bf16"),
    (33, 5, 1000, "bf16"),
    (4, 32, 2048, "f32"),
    (2, 7, 151936, "bf16"),
    (48, 16, 30000, "f32"),
]


@pytest.mark.parametrize("case", CHAINS, ids=[f"b{c[0]}P{c[1]}V{c[2]}{c[3]}" for c in CHAINS])
def test_chain_acceptance(case):
    batch, P, V, kind = case
    rng = np.random.default_rng(P * V)
    y = rng.standard_normal((batch, P, V), dtype=np.float32) * 2
    x = np.concatenate([y + 0.6 * rng.standard_normal(y.shape, dtype=np.float32),
                        rng.standard_normal((batch, 1, V), dtype=np.float32)], 1)
    xd, xh = held(x, kind)
    yd, yh = held(y, kind)
    heat = rng.uniform(0.4, 1.5, batch).astype(np.float32)
    heat[1::4] = 0.0
    noise = rng.gumbel(size=yh.shape)
    tok = (yh + heat[:, None, None] * noise).argmax(2).astype(np.int32)
    keep = rng.integers(0, P + 1, batch).astype(np.int32)
    u = rng.random((batch, P + 1), dtype=np.float32)
    size = pkg.lib().dspark_accept_sampled_workspace_size(batch, P, V, kind == "f32")
    for k in (keep, None):
        got = pkg.dspark_accept_sampled(dev(tok), xd, yd, dev(heat), dev(u), keep=dev(k),
                                        ws=torch.full((size,), 255, dtype=torch.uint8, device=DEV))
        want = O.accept_chain(tok, k, xh, yh, heat, u.astype(np.float64))
        same(got, want, CHAIN)
    if batch * P > 8:
        assert want[0].max() > 0


@pytest.mark.parametrize("batch,L,V", [(60, 1, 60000), (24, 2, 60003), (40, 4, 40001), (40, 15, 40001)])
def test_many_long_walks(batch, L, V):
    """Many rows, walks of every length: ended before the first depths are over, there, behind
    them and at the last; chains of as many guesses the same."""
    rng = np.random.default_rng(L * V)
    B = 4 * L
    par, tok = random_trees(rng, batch, B, V)
    par[::2, :L] = np.arange(L)  # some chains as deep as can be
    x = rng.standard_normal((batch, B + 1, V), dtype=np.float32)
    x = favour(favour(x, par, tok, rng, 5.0), par[:, :L], tok[:, :L], rng, 9.0)
    xd, xh = held(x, "f32")
    heat = np.where(np.arange(batch) % 5 == 3, 0.0, 1.0).astype(np.float32)
    nn = rng.integers(0, B + 1, batch).astype(np.int32)
    u = rng.random((batch, L + 1), dtype=np.float32)
    for counts in (nn, None):
        got = pkg.ddtree_accept_sampled(dev(tok), dev(par), dev(counts), xd, dev(heat), dev(u))
        want = O.accept_tree(tok, par, counts, xh, heat, u.astype(np.float64))
        same(got, want, TREE)
    assert want[1].max() == L
    del x, xd, xh
    y = rng.standard_normal((batch, L, V), dtype=np.float32)
    x = np.concatenate([y + rng.uniform(0.05, 0.4, (batch, 1, 1)).astype(np.float32) * rng.standard_normal(y.shape, dtype=np.float32),
                        rng.standard_normal((batch, 1, V), dtype=np.float32)], 1)
    (xd, xh), (yd, yh) = held(x, "f32"), held(y, "f32")
    tok = (yh + heat[:, None, None] * rng.gumbel(size=yh.shape)).argmax(2).astype(np.int32)
    keep = rng.integers(0, L + 1, batch).astype(np.int32)
    for k in (keep, None):
        got = pkg.dspark_accept_sampled(dev(tok), xd, yd, dev(heat), dev(u), keep=dev(k))
        want = O.accept_chain(tok, k, xh, yh, heat, u.astype(np.float64))
        same(got, want, CHAIN)
    assert want[0].max() == L and want[0].min() < L


def test_chain_acceptance_of_odd_rows():
    inf, nan = np.inf, np.nan
    V, P = 24, 3
    x = np.zeros((9, P + 1, V), np.float32)
    y = np.zeros((9, P, V), np.float32)
    x[0, :, 3:] = -inf
    y[1, :, 3:] = -inf               # guesses the drafter could not have drawn stand
    x[2] = -inf
    y[3] = -inf
    x[4, :, ::2], y[4, :, 1::2] = nan, nan  # disjoint: every guess falls
    x[5, :, 5] = inf
    y[6, :, 1] = 1e4
    tok = np.tile(np.array([1, 5, 20], np.int32), (9, 1))
    tok[7] = [-1, V, 3]
    u = np.random.default_rng(1).random((9, P + 1), dtype=np.float32)
    for heat in (None, np.full(9, 0.6, np.float32), np.zeros(9, np.float32)):
        for uu in (u, np.zeros_like(u), np.full_like(u, 1 - 2.0 ** -24), np.full_like(u, nan)):
            for keep in (None, np.array([-1, 0, 1, 2, 3, 99, 3, 3, 3], np.int32)):
                got = pkg.dspark_accept_sampled(dev(tok), dev(x), dev(y), dev(heat), dev(uu), keep=dev(keep))
                same(got, O.accept_chain(tok, keep, x.astype(np.float64), y.astype(np.float64), heat,
                                         uu.astype(np.float64)), CHAIN)


def test_drafter_equal_to_target_keeps_every_guess():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((8, 6, 999)).astype(np.float32)
    tok = x[:, :5].argmax(2).astype(np.int32)
    u = np.full((8, 6), 1 - 2.0 ** -24, np.float32)
    got = pkg.dspark_accept_sampled(dev(tok), dev(x), dev(x[:, :5]), None, dev(u))
    assert (got["accept_len"] == 5).all()


def test_sampled_refusals():
    i32 = dict(dtype=torch.int32, device=DEV)
    tok, x = torch.zeros((2, 4), **i32), torch.zeros((2, 5, 30), device=DEV)
    u, heat = torch.zeros((2, 4), device=DEV), torch.ones(2, device=DEV)
    call = lambda **k: pkg.ddtree_accept_sampled(**{**dict(tree_tokens=tok, parents=tok, num_nodes=None,  # noqa: E731
                                                          target_logits=x, temperature=heat, u=u), **k})
    call()
    for bad in (dict(parents=tok[:1]), dict(target_logits=x[:, :4]), dict(u=u[:1]), dict(temperature=heat[:1]),
                dict(u=u.cpu()), dict(target_logits=x.transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(target_logits=x.half()), dict(u=u.double()), dict(tree_tokens=tok.long())):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(pkg.DDTreeError):
        call(u=u[:, :1].contiguous())  # L = 0
    with pytest.raises(pkg.DDTreeError):
        call(ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        pkg.dspark_accept_sampled(tok, x, x, heat, torch.zeros((2, 5), device=DEV))


# ---- a round of them together -------------------------------------------------------
def make_round(seed, batch=3, L=6, B=20, V=2000, Hq=4, Hkv=2, dh=64, ps=16, layers=2):
    """One verification round's inputs: drafter rows, paged caches of `layers` layers and
    projections that stand in for the model's."""
    rng = np.random.default_rng(seed)
    r = {"L": L, "B": B, "dims": (Hq, Hkv, dh)}
    # peaked rows: deep trees
    r["draft"] = dev(np.stack([gen.request_rows(90, seed, b, L=L, V=V, sigma=(2.0, 4.0), peak=True,
                                                dtype=gen.DTYPE_F32) for b in range(batch)]))
    past = np.array([37, 0, 101], np.int32)[:batch]
    width = (int(past.max()) + B + 1 + ps - 1) // ps
    pool = batch * width
    r["table"], r["past"] = dev(rng.permutation(pool).astype(np.int32).reshape(batch, width)), dev(past)
    half = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).to(DEV)  # noqa: E731
    r["k"], r["v"] = half(layers, pool, Hkv, ps, dh), half(layers, pool, Hkv, ps, dh)
    r["qkv"] = [half(batch, B + 1, Hq + 2 * Hkv, dh) for _ in range(layers)]
    a = np.arange(200)[:, None] * 1e4 ** -(np.arange(dh // 2) / (dh / 2))
    r["rope"] = dev(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))
    r["head"] = half(Hq * dh, V).float() / 8
    r["heat"] = dev(np.array([0.8, 0.0, 1.2], np.float32)[:batch])
    r["u"] = dev(rng.random((batch, L + 1), dtype=np.float32))
    return r


def play_round(r):
    """Tree, append and attention per layer, target logits, acceptance, compaction."""
    Hq, Hkv, dh = r["dims"]
    t = pkg.ddtree_build(r["draft"], r["B"])
    batch, T = r["past"].shape[0], r["B"] + 1
    x = 0
    for layer, qkv in enumerate(r["qkv"]):
        q, k, v = qkv.split([Hq, Hkv, Hkv], 2)
        q = pkg.ddtree_append_kv(q, k, v, r["k"][layer], r["v"][layer], r["past"], rope=r["rope"],
                                 page_table=r["table"], depths=t["depths"], num_nodes=t["num_nodes"])
        o = pkg.ddtree_attention(q, r["k"][layer], r["v"][layer], r["past"], page_table=r["table"],
                                 num_nodes=t["num_nodes"], mask=t["mask"])["out"]
        x = x + o.float().view(batch * T, -1)
    logits = (x @ r["head"]).view(batch, T, -1)
    # a target near its drafter: the drafter's row of each node's depth added
    depth = torch.nn.functional.pad(t["depths"].clamp(min=0), (1, 0)).long().clamp(max=r["L"] - 1)
    logits += r["draft"].gather(1, depth[..., None].expand(-1, -1, logits.shape[-1]))
    a = pkg.ddtree_accept_sampled(t["tree_tokens"], t["parents"], t["num_nodes"], logits, r["heat"], r["u"])
    n = pkg.ddtree_compact_kv_paged(r["k"], r["v"], r["table"], r["past"], a["accepted_nodes"], a["accept_len"])
    return {**t, **a, "logits": logits, "new_len": n}


def test_a_round():
    """The operators in the order of a verification round, each step against the oracle on the
    device's own inputs of that step."""
    r = make_round(1)
    Hq, Hkv, dh = r["dims"]
    k0, v0 = r["k"].clone(), r["v"].clone()
    got = {k: v.cpu().numpy() for k, v in play_round(r).items()}
    past, table = r["past"].cpu().numpy(), r["table"].cpu().numpy()
    want = O.accept_tree(got["tree_tokens"], got["parents"], got["num_nodes"], got["logits"].astype(np.float64),
                         r["heat"].cpu().numpy(), r["u"].double().cpu().numpy())
    same({k: torch.from_numpy(got[k]) for k in TREE}, want, TREE)
    assert got["accept_len"].max() > 0
    for layer in range(2):
        x = r["qkv"][layer].double().cpu().numpy()
        _, k1, v1 = O.append(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], k0[layer].double().cpu().numpy(),
                             v0[layer].double().cpu().numpy(), past, r["rope"].double().cpu().numpy(), False, table,
                             got["depths"], got["num_nodes"])
        k2, v2, nl = O.compact_paged(k1[None], v1[None], table, past, got["accepted_nodes"], got["accept_len"])
        assert np.array_equal(r["v"][layer].double().cpu().numpy(), v2[0])
        off = np.abs(r["k"][layer].double().cpu().numpy() - k2[0])
        assert np.all(off <= 2.0 ** -8 * np.abs(k2[0]) + 2.0 ** -22 * np.abs(x).max())
    assert np.array_equal(got["new_len"], nl)


def test_captured_rounds_replay_and_keep_apart():
    """Two rounds captured into two graphs, replayed in turn with eager work between: each
    replay equals the eager round on the same inputs."""
    rounds, fresh = [make_round(s) for s in (2, 3)], []
    for r in rounds:
        keep = (r["k"].clone(), r["v"].clone())
        want = play_round(r)
        fresh.append((keep, {k: v.clone() for k, v in want.items()}, r["k"].clone(), r["v"].clone()))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r, f in zip(rounds, fresh):
        r["k"].copy_(f[0][0])
        r["v"].copy_(f[0][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(play_round(r))
        graphs.append(g)
    for turn in range(4):
        for r, f, g, o in zip(rounds, fresh, graphs, outs):
            r["k"].copy_(f[0][0])
            r["v"].copy_(f[0][1])
            g.replay()
            play_round(make_round(4 + turn))  # eager work between the replays
            torch.cuda.synchronize()
            for name in ("tree_tokens", "accepted_nodes", "accept_len", "next_token", "logp", "new_len"):
                assert torch.equal(o[name], f[1][name]), name
            assert torch.equal(r["k"], f[2]) and torch.equal(r["v"], f[3])
