"""Shared by the decoding tests: small cached trees and the tolerances.

Tolerances, set from the arithmetic alone.  u32 = 2^-24, ub = 2^-8 (half a
step of bf16 relative to the value).
- A score is a dot product of D terms accumulated in fp32 in some order and
  multiplied by the scale and log2(e): off by at most (D + 4) u32 times
  sum |q k| scale.  Call the largest over a test ds.
- exp2 is the hardware's, relative error below 2^-22 for the arguments here,
  and the sum of n probabilities adds n u32: a probability is off by a relative
  dp = 2 ds + 2^-21 + (n + 8) u32 (its own score and the normaliser's).
- O in fp32: dp sum p |v|, twice for merging partial results with weights of
  the same form.  On tensor cores each probability is rounded to bf16 for the
  product with V: ub sum p |v| more.  A bf16 O is rounded once: ub |O|.
- LSE: ds + (n + 8) u32 + 2^-21 + 4 u32 |LSE|.
sum p |v| is the oracle's own output for |V|.
"""
import numpy as np
import torch

from oracle import decode as OD

U32, UB = 2.0 ** -24, 2.0 ** -8


def pages_of(lens, ps, rng, spare=3, width=None):
    """tables [n, width] with random distinct pages, and the page count."""
    need = [-(-int(n) // ps) for n in lens]
    n_pages = sum(need) + spare
    ids = rng.permutation(n_pages)
    tables = np.full((len(lens), max([1] + need) if width is None else width), -1, np.int32)
    at = 0
    for i, k in enumerate(need):
        tables[i, :k] = ids[at:at + k]
        at += k
    return tables, n_pages


def cache_of(lens, tables, n_pages, Hkv, ps, D, dtype, seed, poison=float("nan")):
    """Kc, Vc (CPU): N(0, 1) in the rows' tokens, `poison` everywhere else."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        c = torch.full((n_pages, Hkv, ps, D), poison, dtype=dtype)
        for i, n in enumerate(lens):
            if n:
                s = torch.from_numpy(OD.slots_of(tables[i], int(n), ps))
                c[s // ps, :, s % ps] = torch.randn(int(n), Hkv, D, generator=g).to(dtype)
        out.append(c)
    return out


def check(O, L, Q, Kc, Vc, tables, lens, paths, q_len, q_count=None, scale=None, untouched=None):
    """Compare O and LSE (CPU tensors) with the oracle; rows that are no
    queries must equal `untouched` = (O before, LSE before)."""
    bf16 = O.dtype == torch.bfloat16
    q, k, v = (x.to(torch.float32).numpy() for x in (Q, Kc, Vc))
    o, l = O.to(torch.float32).numpy().astype(np.float64), L.numpy().astype(np.float64)
    wo, wl = OD.attention(q, k, v, tables, lens, paths, q_len, q_count, scale)
    av, _ = OD.attention(q, k, np.abs(v), tables, lens, paths, q_len, q_count, scale)
    D = q.shape[2]
    n = max([1] + [sum(int(lens[i]) for i in p) for p in paths])
    kk = np.abs(np.nan_to_num(k, nan=0.0)).max(initial=0.0)
    ds = (D + 4) * U32 * np.abs(q).sum(-1).max(initial=0.0) * kk * (scale or D ** -0.5)
    dp = 2 * ds + 2.0 ** -21 + (n + 8) * U32
    idle = np.isnan(wo)
    tol = 2 * dp * av + (UB * av + UB * np.abs(wo) * (1 + 2 * UB) if bf16 else U32 * np.abs(wo))
    bad = ~idle & ~(np.abs(o - wo) <= tol + 1e-30)
    assert not bad.any(), f"O: {int(bad.sum())} of {bad.size} off, worst {np.nanmax(np.abs(o - wo)[bad])} at {np.argwhere(bad)[0]}"
    idle_l = np.isnan(wl)
    none = np.isneginf(wl)
    assert np.array_equal(np.isneginf(l) & ~idle_l, none)
    fin = ~idle_l & ~none
    tl = ds + (n + 8) * U32 + 2.0 ** -21 + 4 * U32 * np.abs(wl[fin])
    assert (np.abs(l[fin] - wl[fin]) <= tl).all(), f"LSE off by {np.abs(l[fin] - wl[fin]).max()}"
    if untouched is not None:
        t = torch.from_numpy(idle)
        assert torch.equal(O[t], untouched[0][t])
        t = torch.from_numpy(idle_l)
        assert torch.equal(L[t], untouched[1][t])


def csr(paths):
    return np.cumsum([0] + [len(p) for p in paths]).astype(np.int32), np.array([n for p in paths for n in p], np.int32)
