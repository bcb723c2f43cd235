"""CPU oracle of the verification pass: append to a paged cache, attention
under the ancestor mask, paged compaction, acceptance at a temperature.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the product path.
Shares no code with the HIP library. float64 throughout, one request, row and
head at a time.

Readings: the block's row j (0 the root) lies at cache row past + j and stands
at text position past + depth(j); a request's row r lies on page
table[r // page_size] (none where that entry is outside the pool); row i of
the block sees every committed row and the block's rows whose bit is set in
its mask row (no mask: j <= i). A negative past takes the request out, and it
stays out: the compaction's new length is that past.
"""

from __future__ import annotations

import numpy as np


def slot(table, pages: int, page_size: int, b: int, r: int):
    """(page, row in the page) of request b's row r, or None where no page holds it.
    table None: page b holds all of request b's rows."""
    if table is None:
        return (b, r) if 0 <= r < page_size else None
    if r < 0 or r >= table.shape[1] * page_size:
        return None
    page = int(table[b, r // page_size])
    return (page, r % page_size) if 0 <= page < pages else None


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [heads, dh] turned by the angles of one position (rot / 2 of them)."""
    half = len(cos)
    y = x.copy()
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    z = (x[:, a] + 1j * x[:, b]) * (cos + 1j * sin)
    y[:, a], y[:, b] = z.real, z.imag
    return y


def append(q, k, v, k_cache, v_cache, past_len, rope=None, interleaved=False, table=None,
           depths=None, num_nodes=None, q_out=None):
    """Returns (q_out, k_cache, v_cache) in float64; inputs float64 and unchanged.
    q, k, v [batch, T, heads, dh]; caches [pages, heads, page_size, dh]."""
    batch, T = k.shape[:2]
    pages, _, page_size, _ = k_cache.shape
    kc, vc = k_cache.copy(), v_cache.copy()
    qo = np.zeros_like(q) if q_out is None else q_out.copy()
    for b in range(batch):
        past = int(past_len[b])
        n = T - 1 if num_nodes is None else min(max(int(num_nodes[b]), 0), T - 1)
        for j in range(n + 1 if past >= 0 else 0):
            pos = past + (0 if j == 0 else int(depths[b, j - 1]) if depths is not None else j)
            if rope is not None and not 0 <= pos < len(rope):
                continue
            half = 0 if rope is None else rope.shape[1] // 2
            turn = lambda x: x if half == 0 else rotate(x, rope[pos, :half], rope[pos, half:], interleaved)  # noqa: E731
            qo[b, j] = turn(q[b, j])
            at = slot(table, pages, page_size, b, past + j)
            if at is not None:
                kc[at[0], :, at[1]] = turn(k[b, j])
                vc[at[0], :, at[1]] = v[b, j]
    return qo, kc, vc


def mask_bits(mask: np.ndarray, T: int) -> np.ndarray:
    """[batch, T, words] int64 -> bool [batch, T, T]."""
    w = mask.view(np.uint64)
    j = np.arange(T)
    return ((w[:, :, j >> 6] >> (j & 63).astype(np.uint64)) & np.uint64(1)).astype(bool)


def attend(q, k_cache, v_cache, past_len, table=None, num_nodes=None, mask=None, scale=None):
    """Returns (out, lse, spread, score) in float64: out [batch, T, Hq, dh], lse [batch, T, Hq],
    spread = sum_n a_n |V_n| (the size of the terms that out sums), score = the largest
    scale * sum_d |q_d K_nd| of a row (the size of the terms that a score sums)."""
    batch, T, Hq, dh = q.shape
    pages, Hkv, page_size, _ = k_cache.shape
    scale = dh ** -0.5 if scale is None else scale
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    lse, score = np.full((batch, T, Hq), -np.inf), np.zeros((batch, T, Hq))
    bits = None if mask is None else mask_bits(mask, T)
    for b in range(batch):
        past = int(past_len[b])
        if past < 0:
            continue
        n = T - 1 if num_nodes is None else min(max(int(num_nodes[b]), 0), T - 1)
        at = [slot(table, pages, page_size, b, r) for r in range(past + n + 1)]
        held = np.array([a is not None for a in at], bool)
        pg = np.array([a[0] if a else 0 for a in at])
        rw = np.array([a[1] if a else 0 for a in at])
        for i in range(n + 1):
            sees = held.copy()
            own = np.arange(n + 1) <= i if bits is None else bits[b, i, :n + 1]
            sees[past:] &= own
            idx = np.nonzero(sees)[0]
            if len(idx) == 0:
                continue
            for h in range(Hq):
                g = h // (Hq // Hkv)
                K, V = k_cache[pg[idx], g, rw[idx]], v_cache[pg[idx], g, rw[idx]]
                x = scale * (K @ q[b, i, h])
                m = x.max()
                e = np.exp(x - m)
                a = e / e.sum()
                out[b, i, h], spread[b, i, h] = a @ V, a @ np.abs(V)
                lse[b, i, h] = m + np.log(e.sum())
                score[b, i, h] = scale * (np.abs(K) @ np.abs(q[b, i, h])).max()
    return out, lse, spread, score


def compact_paged(k, v, table, past_len, accepted, accept_len):
    """(k', v', new_len) of caches [layers, pages, heads, page_size, dh]; inputs unchanged."""
    k2, v2 = k.copy(), v.copy()
    pages, page_size = k.shape[1], k.shape[3]
    for b in range(len(past_len)):
        past, n = int(past_len[b]), min(max(int(accept_len[b]), 0), accepted.shape[1])
        for i in range(1, n + 1 if past >= 0 else 0):
            node = int(accepted[b, i - 1])
            s = slot(table, pages, page_size, b, past + node) if node >= 0 else None
            d = slot(table, pages, page_size, b, past + i)
            if s is not None and d is not None:
                k2[:, d[0], :, d[1]] = k[:, s[0], :, s[1]]
                v2[:, d[0], :, d[1]] = v[:, s[0], :, s[1]]
    n = np.clip(accept_len, 0, accepted.shape[1])
    return k2, v2, np.where(past_len < 0, past_len, past_len + n + 1).astype(np.int32)


# ---- acceptance at a temperature --------------------------------------------
def weights(row: np.ndarray, temperature: float) -> np.ndarray:
    """exp((x - max) / T) of a row of float64 logits; T <= 0 or NaN: 1 at the first
    largest. NaN logits count as -inf, +inf as the largest float32; all zero
    where every logit is -inf."""
    x = np.where(np.isnan(row), -np.inf, np.minimum(row, np.finfo(np.float32).max))
    top = x.max()
    if top == -np.inf:
        return np.zeros_like(x)
    if not temperature > 0:
        w = np.zeros_like(x)
        w[int(np.argmax(x))] = 1.0
        return w
    with np.errstate(invalid="ignore"):
        w = np.exp((x - top) / temperature)
    w[x == -np.inf] = 0.0
    return w


def number(u: float) -> float:
    """u clamped into [0, 1); NaN: 0."""
    return 0.0 if not u >= 0 else min(float(u), 1.0 - 2.0 ** -24)


def line(mass: np.ndarray, t: float) -> int:
    """The first index whose running sum passes t, else the last with any mass, else -1."""
    some = np.nonzero(mass > 0)[0]
    if len(some) == 0:
        return -1
    over = np.nonzero(np.cumsum(mass[some]) > t)[0]
    return int(some[over[0]] if len(over) else some[-1])


def _logp(w: float, Z: float) -> float:
    return float(np.log(w / Z)) if Z > 0 else -np.inf


def accept_tree(tokens, parents, num_nodes, logits, temperature, u):
    """(accepted_nodes, accept_len, next_token, logp) of trees [batch, B]; logits
    [batch, B+1, V] float64, u [batch, L+1]."""
    batch, B = tokens.shape
    V, L = logits.shape[2], u.shape[1] - 1
    path, logp = np.full((batch, L), -1, np.int32), np.zeros((batch, L + 1))
    length, last = np.zeros(batch, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        n = B if num_nodes is None else min(max(int(num_nodes[b]), 0), B)
        heat = 1.0 if temperature is None else float(temperature[b])
        node, d = 0, 0
        while True:
            w = weights(logits[b, node], heat)
            Z = float(w.sum())
            t = number(u[b, d]) * Z
            kids, seen = [], set()
            for j in range(n if d < L else 0):
                x = int(tokens[b, j])
                if parents[b, j] == node and node <= j and 0 <= x < V and x not in seen:
                    kids.append(j)
                    seen.add(x)
            edge, go = 0.0, None
            for j in kids:
                edge += w[tokens[b, j]]
                if t < edge:
                    go = j
                    break
            if go is None:
                rest = w.copy()
                rest[sorted(seen)] = 0.0
                last[b] = line(rest, t - edge)
                logp[b, d] = _logp(w[last[b]], Z) if last[b] >= 0 else -np.inf
                length[b] = d
                break
            logp[b, d], path[b, d] = _logp(w[tokens[b, go]], Z), go + 1
            node, d = go + 1, d + 1
    return path, length, last, logp


def accept_chain(tokens, keep, logits, draft, temperature, u):
    """(accept_len, next_token, logp) of chains [batch, P]; logits [batch, P+1, V] and
    draft [batch, P, V] float64, u [batch, P+1]."""
    batch, P = tokens.shape
    V = logits.shape[2]
    length, last = np.zeros(batch, np.int32), np.zeros(batch, np.int32)
    logp = np.zeros((batch, P + 1))
    for b in range(batch):
        n = P if keep is None else min(max(int(keep[b]), 0), P)
        heat = 1.0 if temperature is None else float(temperature[b])
        for i in range(n + 1):
            w = weights(logits[b, i], heat)
            Z = float(w.sum())
            p = w / Z if Z > 0 else w
            rest = p
            if i < n:
                x = int(tokens[b, i])
                wq = weights(draft[b, i], heat)
                q = wq / wq.sum() if wq.sum() > 0 else wq
                if 0 <= x < V and number(u[b, i]) * q[x] < p[x]:
                    logp[b, i] = _logp(w[x], Z)
                    continue
                if wq.sum() > 0:
                    rest = np.maximum(p - q, 0.0)
                if rest.sum() == 0:
                    rest = p
            last[b] = line(rest, number(u[b, P]) * float(rest.sum()))
            logp[b, i] = _logp(w[last[b]], Z) if last[b] >= 0 else -np.inf
            length[b] = i
            break
    return length, last, logp
