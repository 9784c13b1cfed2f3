"""Rows whose largest logit times scale is beyond fp32: a row's results do not
depend on that; LSE is the nearest finite number.

Tolerances, u = 2^-24, n = V / 32 + 64 additions one after another (a row is at
least a warp's): all terms of a row's sum are 1 here, so ln S is off by 2^-22 + n u
of S and 2 u |ln S|, logp and the entropy by two more roundings of ln V; p = 1 / V by
that and exp's 2^-22 and 2 u ln V, the gradient by it for each of its two terms, by
two roundings of the token's own part, and one to the type (u, or 2^-8 in bf16).
"""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U, UB = 2.0 ** -24, 2.0 ** -8
INF = float("inf")
MOST = float(np.finfo(np.float32).max)


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


def near(got, want, tol):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1.25, 0.75, 1.0, 1e30])
@pytest.mark.parametrize("k", [0, 3])
@pytest.mark.parametrize("V,R", [(5, 4), (300, 4), (20001, 4), (131072, 4), (9001, 700)])
def test_scaled_beyond_the_range(dtype, scale, k, V, R):
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = torch.empty(R, V, dtype=dtype)
    x[0::4] = low
    x[1::4] = high
    x[2::4] = low
    x[2::4, 3:] = -INF
    x[3::4] = -INF
    m = np.array([low, high, low, -INF] * (R // 4)) * np.float64(np.float32(scale))
    n = np.log(np.array([V, V, 3, 1] * (R // 4), np.float64))
    x = x.cuda()
    t = torch.full((R,), 1, device="cuda")
    logp, lse, H, top, ids = pt.token_logprobs(x, t, entropy=True, scale=scale, top_k=k)
    none = np.isinf(m)
    tol = 2 * (2.0 ** -22 + (V / 32 + 64) * U + 4 * U * np.log(V))
    near(H, np.where(none, 0.0, n), tol)
    near(logp[torch.from_numpy(~none).cuda()], -n[~none], tol)
    assert (logp[3::4] == -INF).all() and (lse[3::4] == -INF).all()
    near(lse[torch.from_numpy(~none).cuda()], np.clip(m + n, -MOST, MOST)[~none], tol + 4 * U * np.abs(np.clip(m, -MOST, MOST)[~none]))
    if k:
        near(top[torch.from_numpy(~none).cuda()], np.repeat(-n[~none, None], k, 1), tol)
        assert (top[3::4] == -INF).all()
        assert (ids == torch.arange(k, device="cuda")).all()
    g = torch.randn(R, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    d = pt.token_logprobs_bwd(g, x, t, lse, dentropy=torch.ones_like(g), entropy=H, scale=scale)
    pt.sync_status()
    live = np.array([V, V, 3, 0] * (R // 4))
    p = torch.from_numpy(1.0 / np.maximum(live, 1)).cuda()[:, None] * (torch.arange(V, device="cuda")[None] < torch.from_numpy(live).cuda()[:, None])
    want = -g.double()[:, None] * p
    want[:, 1] += g.double()
    tol = (g.double().abs()[:, None] + 1) * p * 8 * tol + want.abs() * ((UB if dtype == BF else U) + 4 * U)
    assert ((d.double() - want * scale).abs() <= tol * scale).all()
