"""Rows of logits far from 0 (masked rows of a large negative number, large
offsets): their gradient is that of the log probabilities that the forward
returned, however large LSE is.

Tolerances, free of the logits' size: u = 2^-24, d = z - m from a row's maximum,
a = E_p|d|, b = E_p d^2, n = V / 32 + 64 additions one after another (a row is
at least a warp's, which takes every 32nd).
- S = sum exp(d): a term is off by 3 u |d| (difference, constant, product) + 2^-22
  (ex2), so S by ts = 3 u a + 2^-22 + n u of it; ln S by ts + 2 u |ln S|.
- l = d - ln S: 2 u |d| (difference, scale), ln S's, u |l|: dl.  Where |LSE| is below 256
  (here up to 257, not to ask the rounding) l = z - LSE may be taken instead: LSE = fl(
  fl(m scale) + ln S) and fl(z - LSE) add u |m scale| + u |LSE|; 2 u of both is allowed.
  p = exp(l): dl + 2 u |l| + 2^-22 of it: dp.
- H = ln S - T / S: (n u + 2^-22)(1 + 2 a) + 3 u (a + b) + 4 u (a + |H|): th.
- The gradient scale (sum g 1[target] - p (G + dH (l + H))), c tokens: dp and (c + 8) u
  of the terms |G| + |dH| (|H| + |l|), |dH| (dl + th) more of p, c + 2 roundings of the
  tokens' own part, one rounding to the type (u, or 2^-8 in bf16).
"""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from oracle import tokens as OT

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U, UB = 2.0 ** -24, 2.0 ** -8
INF = float("inf")


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


class Bounds:
    def __init__(self, x, scale):
        z = x * scale
        m = z.max(1, keepdims=True)
        d = z - np.where(np.isneginf(m), 0.0, m)
        e = np.exp(d)
        s = np.maximum(e.sum(1, keepdims=True), 1.0)  # (a row without weight: 0 p)
        self.p, self.l, self.d = e / s, np.where(e > 0, d - np.log(s), 0.0), np.where(e > 0, -d, 0.0)
        a, b = (self.p * self.d).sum(1, keepdims=True), (self.p * self.d ** 2).sum(1, keepdims=True)
        n = x.shape[1] / 32 + 64
        self.H = np.log(s) + a
        ln_s = np.abs(np.log(s))
        self.dl = 2 * U * self.d + 3 * U * a + 2.0 ** -22 + n * U + 2 * U * ln_s + U * np.abs(self.l)
        lse = np.where(np.isneginf(m), 0.0, m) + np.log(s)
        self.dl = self.dl + np.where(np.abs(lse) < 257, 2 * U * (np.abs(lse) + np.abs(np.where(np.isneginf(m), 0.0, m))), 0.0)
        self.dp = self.dl + 2 * U * np.abs(self.l) + 2.0 ** -22
        self.th = (n * U + 2.0 ** -22) * (1 + 2 * a) + 3 * U * (a + b) + 4 * U * (a + np.abs(self.H))


def near(got, want, tol):
    got = got.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        bad = ~((got == want) | (np.abs(got - want) <= tol))
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def check(x, targets, scale=1.0, row_ptr=None, dH=True, in_place=False):
    """x [R, V] on the GPU; the forward and the gradient against the oracle."""
    R, V = x.shape
    N = len(targets)
    t = torch.tensor(targets, device="cuda")
    ptr = None if row_ptr is None else torch.tensor(row_ptr, dtype=torch.int32, device="cuda")
    rows = np.arange(N) if row_ptr is None else np.repeat(np.arange(R), np.diff(row_ptr))
    logp, lse, H, _, _ = pt.token_logprobs(x, t, row_ptr=ptr, entropy=True, scale=scale)
    xs = x.double().cpu().numpy()
    b = Bounds(xs, scale)
    wp, _, wh = OT.logprobs(xs, targets, rows, scale)
    near(logp, wp, b.dl[rows, targets])
    near(H, wh, b.th[:, 0])
    rng = np.random.default_rng(0)
    g, dh = rng.standard_normal(N).astype(np.float32), rng.standard_normal(R).astype(np.float32)
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    d = pt.token_logprobs_bwd(dev(g), x, t, lse, row_ptr=ptr, dentropy=dev(dh) if dH else None, entropy=H, scale=scale)
    if in_place:
        y = x.clone()
        pt.token_logprobs_bwd(dev(g), y, t, lse, row_ptr=ptr, dentropy=dev(dh) if dH else None, entropy=H, scale=scale, dlogits=y)
        assert torch.equal(y, d)
    pt.sync_status()
    want = OT.logprobs_grad(xs, targets, rows, g.astype(np.float64), dh if dH else None, scale)
    own, all_g, c = np.zeros((R, V)), np.zeros((R, 1)), np.zeros((R, 1))
    for n, (v, r) in enumerate(zip(targets, rows)):
        own[r, v] += abs(g[n])
        all_g[r] += abs(g[n])
        c[r] += 1
    adh = np.abs(dh)[:, None] if dH else np.zeros((R, 1))
    terms = all_g + adh * (np.abs(b.H) + np.abs(b.l))
    tol = scale * (b.p * (terms * (b.dp + (c + 8) * U) + adh * (b.dl + b.th)) + (c + 2) * U * own + 1e-37 * (terms + 105 * adh))
    r = UB if x.dtype == BF else U
    near(d, want, tol * (1 + r) + r * np.abs(want) + 1e-37)


def logits(what, R, V, dtype):
    """x [R, V] and the scale that goes with it."""
    noise = torch.randn(R, V, generator=torch.Generator().manual_seed(V)) * 3
    if what == "lowest":
        return torch.full((R, V), torch.finfo(dtype).min).to(dtype), 1.0
    if what == "-1e9":
        return torch.full((R, V), -1e9).to(dtype), 1.0
    if what == "offset":  # neighbours of 2^20 (bf16: 2^13 apart; fp32: 2^-4) whose z lie a few apart
        step = 2.0 ** 13 if dtype == BF else 2.0 ** -4
        scale = 2.0 ** -12 if dtype == BF else 1.0
        return (2.0 ** 20 + step * (noise if dtype == BF else noise * 16).round()).to(dtype), scale
    if what == "-offset":
        x, scale = logits("offset", R, V, dtype)
        return -x, scale
    x = noise.to(dtype)  # some rows far, some near
    x[1::3] = -1e9
    x[2::3] = logits("lowest", R, V, dtype)[0][2::3]
    x[2, V // 2:] = -INF
    return x, 1.0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["lowest", "-1e9", "offset", "-offset", "some"])
@pytest.mark.parametrize("R,V", [(4, 1), (5, 7), (3, 1000), (40, 6151), (3, 50001), (4, 131072)])
def test_gradient(dtype, what, R, V):
    """A warp a row, four of them, several CTAs a row; in place too."""
    x, scale = logits(what, R, V, dtype)
    t = np.random.default_rng(V).integers(0, max(V // 2, 1), R).tolist()
    check(x.cuda(), t, scale, in_place=True)
    check(x.cuda(), t, scale, dH=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [1, 8])
def test_strides(dtype, pad):
    """Columns of a wider buffer: the gradient starts elsewhere modulo 16 bytes."""
    x, scale = logits("some", 7, 1237, dtype)
    wide = torch.full((7, 1237 + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, :1237] = x.cuda()
    check(wide[:, :1237], [3] * 7, scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [11, 33000])
def test_rows_with_any_number_of_tokens(dtype, V):
    per = [0, 700, 1, 3, 0, 2]
    x, scale = logits("some", len(per), V, dtype)
    t = np.random.default_rng(V).integers(0, max(V // 2, 1), sum(per))
    t[5:9] = t[4]
    check(x.cuda(), t.tolist(), scale, row_ptr=np.concatenate([[0], np.cumsum(per)]).tolist(), in_place=True)


@pytest.mark.parametrize("R,V,dtype", [(2440, 32776, BF), (2440, 16400, F32), (6000, 4096, BF)])
def test_many_masked_rows(R, V, dtype):
    """p = 1 / V and ln p + H = 0 throughout: off by dl + dp + th <= 8 (2^-22 + n u + 4 u
    ln V) of 1 / V, the token's own gradient by two roundings, one rounding to the type."""
    x = torch.full((R, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    t = torch.arange(R, device="cuda") % V
    logp, lse, H, _, _ = pt.token_logprobs(x, t, entropy=True)
    g = torch.randn(R, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    d = pt.token_logprobs_bwd(g, x, t, lse, dentropy=torch.ones_like(g), entropy=H)
    pt.sync_status()
    want = (-g.double() / V)[:, None].repeat(1, V)
    want.scatter_add_(1, t[:, None], g.double()[:, None])
    e = 8 * (2.0 ** -22 + (V / 32 + 64) * U + 4 * U * np.log(V)) / V
    tol = (g.double().abs()[:, None] + 1) * e + want.abs() * ((UB if dtype == BF else U) + 3 * U)
    assert ((d.double() - want).abs() <= tol).all()
