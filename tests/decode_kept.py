"""A cached tree run through pt.attn_decode and compared with the oracle at the
tolerances of decode_cases.check, which scale with the largest key: the cache
that they are taken from holds zeros wherever no row has a token, so what lies
there does not widen them."""
import numpy as np
import torch

import prefix_tree_block_gb300 as pt
from decode_cases import cache_of, check, csr, pages_of
from oracle import decode as OD


def kept(cache, tables, lens):
    """The cache with nothing but the rows' tokens in it."""
    out = torch.zeros_like(cache)
    for i, n in enumerate(lens):
        if n:
            s = torch.from_numpy(OD.slots_of(tables[i], int(n), cache.shape[2]))
            out[s // cache.shape[2], :, s % cache.shape[2]] = cache[s // cache.shape[2], :, s % cache.shape[2]]
    return out


def check_kept(O, L, Q, Kc, Vc, tables, lens, paths, q_len, q_count=None, scale=None, untouched=None):
    check(O, L, Q, kept(Kc, tables, lens), kept(Vc, tables, lens), tables, lens, paths, q_len, q_count, scale, untouched)


def run(lens, paths, Hq, Hkv, D, dtype, ps, q_len=1, q_count=None, seed=0, width=None, poison=float("nan"), kernels=None):
    """One call on the GPU, checked.  kernels: names of pt.profile_read that
    have to have run, or with a leading "-" not."""
    tables, n_pages = pages_of(lens, ps, np.random.default_rng(seed), width=width)
    Kc, Vc = cache_of(lens, tables, n_pages, Hkv, ps, D, dtype, seed, poison)
    Q = torch.randn(len(paths) * q_len, Hq, D, generator=torch.Generator().manual_seed(seed + 1)).to(dtype)
    plan = pt.decode_plan(len(lens), *csr(paths), Hq, Hkv, q_len)
    O = torch.full(Q.shape, 7.0, dtype=dtype, device="cuda")
    L = torch.full((Hq, Q.shape[0]), 7.0, device="cuda")
    cnt = None if q_count is None else torch.tensor(q_count, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    pt.profile_reset()
    pt.profile_enable(True)
    try:
        pt.attn_decode(Q.cuda(), Kc.cuda(), Vc.cuda(), i32(tables), i32(lens), plan, q_count=cnt, O=O, LSE=L)
        pt.sync_status()
        ran = {k: pt.profile_read(k)[0] for k in ("decode_simt", "decode_rows", "decode_tile")}
    finally:
        pt.profile_enable(False)
        pt.profile_reset()
    for k in kernels or ():
        assert (ran[k.lstrip("-")] > 0) == (k[0] != "-"), (k, ran)
    check_kept(O.cpu(), L.cpu(), Q, Kc, Vc, tables, lens, paths, q_len, q_count,
               untouched=(torch.full(Q.shape, 7.0, dtype=dtype), torch.full((Hq, Q.shape[0]), 7.0)))
