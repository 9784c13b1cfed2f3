"""Trees of drafted tokens, rotary positions and log probabilities of tokens, by
their definitions (numpy, fp64).

TEST INFRASTRUCTURE ONLY, like the rest of this folder: the library and its
binding never import it.
"""
from __future__ import annotations

import numpy as np

from .decode import slots_of


def above(parents, j):
    """Draft j and those above it, nearest first."""
    out = []
    while j >= 0:
        out.append(int(j))
        j = int(parents[j])
    return out


def draft_tree(parents, counts, first):
    """mask [S * q, ceil(q / 32)] (int32 bits) and positions [S * q]: parents
    [S, q], drafts counted, first[s] the position of a draft without a parent."""
    parents = np.asarray(parents)
    S, q = parents.shape
    mask, pos = np.zeros((S, q, -(-q // 32)), np.uint32), np.zeros((S, q), np.int64)
    for s in range(S):
        for j in range(int(counts[s])):
            up = above(parents[s], j)
            for i in up:
                mask[s, j, i // 32] |= np.uint32(1 << (i % 32))
            pos[s, j] = int(first[s]) + len(up) - 1
    return mask.view(np.int32).reshape(S * q, -1), pos.reshape(-1)


def attention(Q, Kc, Vc, tables, lens, paths, sees, q_len, counts, scale=None):
    """O [S * q, Hq, D] and LSE [Hq, S * q] in fp64: draft j of sample s (one of
    its counts[s] last tokens) keeps the path's other nodes, its own node's tokens
    before the drafts, and the drafts sees[s][j].  Rows that are no queries: NaN."""
    Q = np.asarray(Q, np.float64)
    Hq, D = Q.shape[1:]
    Hkv, ps = Kc.shape[1], Kc.shape[2]
    scale = scale or 1.0 / np.sqrt(D)
    O, L = np.full(Q.shape, np.nan), np.full((Hq, Q.shape[0]), np.nan)

    def rows(cache, node, toks):
        at = slots_of(tables[node], int(lens[node]), ps)[toks]
        return np.asarray(cache)[at // ps, :, at % ps].astype(np.float64)

    for s, path in enumerate(paths):
        n, leaf = int(counts[s]), path[-1]
        base = int(lens[leaf]) - n
        for j in range(n):
            own = np.array([t for t in range(max(base, 0))] + sorted(base + i for i in sees[s][j] if base + i >= 0), np.int64)
            if base + j < 0:
                own = own[:0]
            K = np.concatenate([rows(Kc, k, np.arange(int(lens[k]))) for k in path[:-1]] + [rows(Kc, leaf, own)])
            V = np.concatenate([rows(Vc, k, np.arange(int(lens[k]))) for k in path[:-1]] + [rows(Vc, leaf, own)])
            r = s * q_len + j
            for h in range(Hq):
                if not K.shape[0]:
                    O[r, h], L[h, r] = 0.0, -np.inf
                    continue
                x = K[:, h // (Hq // Hkv)] @ Q[r, h] * scale
                m = x.max()
                p = np.exp(x - m)
                O[r, h] = p @ V[:, h // (Hq // Hkv)] / p.sum()
                L[h, r] = m + np.log(p.sum())
    return O, L


def keep(kept, counts, lens, leaves, tables, ps, cache):
    """The cache [n_pages, Hkv, ps, D] with each sample's draft kept[s][i] at the
    place of draft i."""
    cache = np.array(cache)
    old = cache.copy()
    for s, leaf in enumerate(leaves):
        at = slots_of(tables[leaf], int(lens[leaf]), ps)
        base = int(lens[leaf]) - int(counts[s])
        for i, j in enumerate(kept[s]):
            if j < 0:
                break
            a, b = at[base + int(j)], at[base + i]
            cache[b // ps, :, b % ps] = old[a // ps, :, a % ps]
    return cache


def rotary(X, positions, inv_freq, sections, interleaved, inverse):
    """X [T, H, D] with pair i turned by positions[axis(i)] * inv_freq[i]."""
    X = np.asarray(X, np.float64)
    f = np.asarray(inv_freq, np.float64)
    positions = np.asarray(positions).reshape(-1, X.shape[0])
    axis = np.repeat(np.arange(len(sections)), sections)
    half = f.size
    Y = X.copy()
    for i in range(half):
        # (the product of a 24-bit and a position of up to 2^31 is exact in the 64 bits of a long double's or, up to
        # 2^29, a double's mantissa: the angle's own error is below 2^-53 of it)
        w = positions[axis[i]].astype(np.longdouble) * np.longdouble(f[i])
        turn = np.longdouble(2) * np.longdouble("3.14159265358979323846264338327950288")
        w = (w - np.rint(w / turn) * turn).astype(np.float64)
        if inverse:
            w = -w
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = np.cos(w)[:, None], np.sin(w)[:, None]
        Y[:, :, a] = X[:, :, a] * c - X[:, :, b] * s
        Y[:, :, b] = X[:, :, b] * c + X[:, :, a] * s
    return Y


def successors(node_lengths, paths):
    """For each flat token the tokens that follow it in some path, ascending;
    and the tokens that follow none."""
    off = np.concatenate([[0], np.cumsum(node_lengths)])
    after = [set() for _ in range(int(off[-1]))]
    first = set(range(int(off[-1])))
    for path in paths:
        flat = [t for n in path for t in range(int(off[n]), int(off[n + 1]))]
        for a, b in zip(flat, flat[1:]):
            after[a].add(b)
            first.discard(b)
    return [sorted(x) for x in after], sorted(first)


def logprobs(x, targets, rows, scale=1.0):
    """logp [N], LSE [R], entropy [R] in fp64: token t is scored by row rows[t]
    (-1: by none); targets below 0 are not scored."""
    z = np.asarray(x, np.float64) * scale
    m, s = _sums(z)
    with np.errstate(divide="ignore"):
        lse, H = m + np.log(s), np.empty(z.shape[0])
    for r in range(z.shape[0]):
        if m[r] == -np.inf:
            lse[r], H[r] = -np.inf, 0.0
            continue
        d = z[r] - m[r]  # (from the maximum: at logits of 1e38 LSE's own rounding is larger than ln S)
        e = np.exp(d)
        H[r] = np.log(s[r]) - (e[e > 0] * d[e > 0]).sum() / s[r] if np.isfinite(lse[r]) else np.nan
    logp = np.zeros(len(targets))
    for t, (v, r) in enumerate(zip(targets, rows)):
        if v >= 0 and r >= 0:
            logp[t] = (z[r, v] - m[r]) - np.log(s[r]) if lse[r] != -np.inf else -np.inf
    return logp, lse, H


def _sums(z):
    """Each row's maximum and sum of exp(z - maximum)."""
    m = z.max(1, initial=-np.inf)
    with np.errstate(invalid="ignore"):
        return m, np.exp(z - np.where(m == -np.inf, 0.0, m)[:, None]).sum(1)


def top(x, k):
    """Ids of the k largest of each row, equal ones by the lower id (NaN as -inf)."""
    x = np.asarray(x, np.float64)
    return np.argsort(-np.where(np.isnan(x), -np.inf, x), axis=1, kind="stable")[:, :k]


def logprobs_grad(x, targets, rows, g, dH=None, scale=1.0):
    """d x of sum g logp + sum dH H in fp64."""
    x = np.asarray(x, np.float64)
    _, _, H = logprobs(x, [], [], scale)
    m, s = _sums(x * scale)
    with np.errstate(invalid="ignore", divide="ignore"):
        l = np.where(np.isneginf(m)[:, None], -np.inf, (x * scale - m[:, None]) - np.log(s)[:, None])
    p = np.exp(l)
    d = np.zeros_like(x)
    for t, (v, r) in enumerate(zip(targets, rows)):
        if v >= 0 and r >= 0:
            d[r, v] += g[t]
            d[r] -= g[t] * p[r]
    if dH is not None:
        d -= np.asarray(dH, np.float64)[:, None] * np.where(p > 0, p * (np.where(p > 0, l, 0.0) + H[:, None]), 0.0)
    return d * scale
