"""GPU tests of attention over shared rows (ddtree_attention_shared, and shared_len of
ddtree_attention_kv8) where the pass over them runs. Tolerances as in tests/test_gpu_kv8.py."""

import numpy as np
import pytest
import torch

import draft_tree_construction_depth_amd as pkg
from oracle import verify as O
from test_gpu_kv8 import ENOUGH, attend64, compare, make_cache, one, shared_pages
from test_gpu_verify_cache import BF, DEV, dev, paging, rounded

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
