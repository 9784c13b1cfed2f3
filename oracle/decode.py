"""A paged cache's step and the decoding attention, by their definitions (numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this folder: the library and its
binding never import it.

A cache row is a tree node: its tokens in order, in pages of `ps` tokens.

- step: rows go from held to held + added tokens, in row order.  A growing
  row takes page ids from the head of the ring of free ids for the pages it
  lacks; a shrinking row gives the pages it no longer needs to the tail.
- attention: query j of a sample's n newest tokens is token len - n + j of
  the path's last node.  It keeps every token of the path's other nodes and
  that node's tokens up to itself; softmax in fp64 over what it keeps.
"""
from __future__ import annotations

import numpy as np


def step(held, added, start, tables, ring, counters, ps, max_new):
    """(lens, counters, row_ptr, slots, positions, tables, ring) after a step;
    the arguments are left alone.  When the ring runs out, the tokens without
    a page get slot -1 and lens counts the rest."""
    tables, ring = np.array(tables), np.array(ring)
    src = ring.copy()
    head, tail = int(counters[0]), int(counters[1])
    cap = ring.size
    avail = tail - head
    taken = 0
    lens, row_ptr, slots, pos = [], [0], [], []
    for i, (h, a) in enumerate(zip(np.asarray(held).tolist(), np.asarray(added).tolist())):
        p0, p1 = -(-h // ps), -(-(h + a) // ps)
        have = p0
        for k in range(p0, p1):
            if taken < avail:
                tables[i, k] = src[(head + taken) % cap]
                have = k + 1
            taken += 1
        for k in range(p1, p0):
            ring[tail % cap] = tables[i, k]
            tail += 1
        for t in range(h, h + a):
            slots.append(int(tables[i, t // ps]) * ps + t % ps if t // ps < have else -1)
            pos.append(int(start[i]) + t)
        lens.append(min(h + a, have * ps) if a > 0 else h + a)
        row_ptr.append(row_ptr[-1] + max(a, 0))
    pad = max(0, max_new - len(slots))
    return (np.array(lens, np.int32), np.array([head + min(taken, avail), tail], np.int64), np.array(row_ptr, np.int32),
            np.array(slots + [-1] * pad, np.int64)[:max_new], np.array(pos + [0] * pad, np.int64)[:max_new], tables, ring)


def slots_of(table, n, ps):
    """Slots of a row's first n tokens."""
    t = np.arange(n)
    return np.asarray(table, dtype=np.int64)[t // ps] * ps + t % ps


def write(K, V, slots, Kc, Vc):
    """Kc, Vc [n_pages, Hkv, ps, D] with the tokens' rows in their slots."""
    Kc, Vc = np.array(Kc), np.array(Vc)
    ps = Kc.shape[2]
    for t, s in enumerate(np.asarray(slots).tolist()):
        if s >= 0:
            Kc[s // ps, :, s % ps] = K[t]
            Vc[s // ps, :, s % ps] = V[t]
    return Kc, Vc


def attention(Q, Kc, Vc, tables, lens, paths, q_len, q_count=None, scale=None):
    """O [S * q_len, Hq, D] and LSE [Hq, S * q_len] in fp64; rows that are no
    queries are NaN."""
    Q = np.asarray(Q, np.float64)
    Hq, D = Q.shape[1:]
    Kc, Vc = np.asarray(Kc), np.asarray(Vc)
    Hkv, ps = Kc.shape[1], Kc.shape[2]
    g = Hq // Hkv
    scale = scale if scale else 1.0 / np.sqrt(D)
    O = np.full(Q.shape, np.nan)
    L = np.full((Hq, Q.shape[0]), np.nan)

    def rows(cache, node, n):  # [n, Hkv, D]
        s = slots_of(tables[node], n, ps)
        return cache[s // ps, :, s % ps].astype(np.float64)

    for s, path in enumerate(paths):
        n = q_len if q_count is None else int(q_count[s])
        up = [rows(Kc, k, int(lens[k])) for k in path[:-1]], [rows(Vc, k, int(lens[k])) for k in path[:-1]]
        for j in range(n):
            own = max(0, int(lens[path[-1]]) - n + j + 1)
            K = np.concatenate(up[0] + [rows(Kc, path[-1], own)])
            V = np.concatenate(up[1] + [rows(Vc, path[-1], own)])
            r = s * q_len + j
            for h in range(Hq):
                if not K.shape[0]:
                    O[r, h], L[h, r] = 0.0, -np.inf
                    continue
                x = K[:, h // g] @ Q[r, h] * scale
                m = x.max()
                p = np.exp(x - m)
                O[r, h] = p @ V[:, h // g] / p.sum()
                L[h, r] = m + np.log(p.sum())
    return O, L
