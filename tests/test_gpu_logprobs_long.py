"""Long runs of rows through one CTA's ring and one warp, against torch in 64
bits: every row has its own spread and maximum, so that a row that took
another's elements, statistics or tokens is off by far more than the tolerance.

Tolerances: those of test_gpu_logprobs.py with u = 2^-24, |z| and |LSE| up to 70,
a up to 15, b up to 400 and n = V / 128 + 64 up to 460: tl = (45 + 4 + 460 + 140 + 280) u
< 2^-14, th = (464 * 31 + 1245 + 200) u < 2^-9.9, dp = tl + (140 + 400 + 4) u < 2^-13."""
import pytest
import torch

import prefix_tree_block_gb300 as pt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


@pytest.mark.parametrize("R,V,dtype", [(5000, 40000, BF), (2000, 50001, BF), (4000, 9000, F32), (9001, 1000, BF), (3000, 33000, F32)])
def test_rows_one_after_another(R, V, dtype):
    g = torch.Generator("cuda").manual_seed(R)
    x = torch.randn(R, V, device="cuda", generator=g, dtype=dtype)
    x *= (1 + torch.arange(R, device="cuda") % 7)[:, None].to(dtype)
    x += (torch.arange(R, device="cuda") % 31)[:, None].to(dtype)
    t = torch.randint(0, V, (R,), device="cuda", generator=g)
    w = torch.randn(R, device="cuda", generator=g)
    dh = torch.randn(R, device="cuda", generator=g)
    out = [pt.token_logprobs(x, t, entropy=True, top_k=k, scale=0.9) for k in (0, 10)]
    d = pt.token_logprobs_bwd(w, x, t, out[0][1], dentropy=dh, entropy=out[0][2], scale=0.9)
    pt.sync_status()
    for a in range(0, R, 500):
        rows = slice(a, a + 500)
        z = x[rows].double() * 0.9
        lp = torch.log_softmax(z, 1)
        p = lp.exp()
        H = -(p * lp).sum(1)
        logp = lp.gather(1, t[rows, None])[:, 0]
        for o in out:
            assert (o[0][rows] - logp).abs().max() < 2.0 ** -13  # (tl + 2 u (|z| + |LSE|))
            assert (o[1][rows] - torch.logsumexp(z, 1)).abs().max() < 2.0 ** -14
            assert (o[2][rows] - H).abs().max() < 2.0 ** -9.9
        v, i = x[rows].float().sort(dim=1, descending=True, stable=True)
        assert torch.equal(out[1][4][rows], i[:, :10])
        assert (out[1][3][rows] - lp.gather(1, i[:, :10])).abs().max() < 2.0 ** -13
        want = -p * (w[rows, None].double() + dh[rows, None].double() * (lp + H[:, None]))
        want.scatter_add_(1, t[rows, None], w[rows, None].double())
        want *= 0.9
        # dp and 9 u on the terms, H's error, the token's own three roundings, and one rounding of the result
        terms = p * (w[rows, None].abs() + dh[rows, None].abs() * (lp.abs() + H[:, None]))
        own = torch.zeros_like(p).scatter_(1, t[rows, None], w[rows, None].double().abs())
        r = 2.0 ** -8 if dtype == BF else 2.0 ** -24
        tol = terms * (2.0 ** -13 + 2.0 ** -20) + p * dh[rows, None].abs() * 2.0 ** -9.9 + own * 3 * 2.0 ** -24
        tol = tol * (1 + r) + want.abs() * r + 1e-30
        assert ((d[rows].double() - want).abs() <= tol).all()
