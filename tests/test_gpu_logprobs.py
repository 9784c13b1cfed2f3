"""Log probabilities of tokens, entropy, alternatives and their gradient
(pt_token_logprobs, pt_token_logprobs_bwd) against the fp64 oracle.

Tolerances, set from the arithmetic alone.  u = 2^-24, a = E_p[m - z] and b =
E_p[(m - z)^2] of a row (m its maximum), z = scale * x.
- A term exp(z - m) has a relative error of 3 u |z - m| (the difference, the
  constant and the product) + 2^-22 (ex2), so the sum S one of 3 u a + 2^-22 + n u,
  n = V / 128 + 64 additions and rescalings one after another (a thread of at
  least 128 takes every 128th, then the joins).  ln S takes that, LSE = m scale +
  ln S 2 u |m scale| + 2 u |LSE| more: tl.
- logp = z - LSE: tl + 2 u (|z| + |LSE|).
- H = ln S - T / S, T = sum (m - z) exp: the same terms with one more factor, so
  the errors of a term weigh a and b: (n u + 2^-22)(1 + 2 a) + 3 u (a + b) + 4 u (a + |H|).
- p = exp(l), l = z - LSE with the given LSE (off by tl): a relative tl + 2 u |LSE|
  + 4 u |l| + 2^-22 =: dp.  The gradient's row part is p (ca + cb l) with ca =
  -(G + dH H) scale, cb = -dH scale, G a sum of c tokens' gradients: dp times
  its terms' magnitudes, (c + 8) u of them, and dH times H's error; a token's own
  part is c sums.  Rounded once to the type: u or 2^-8 of the value (and 1 + that
  of the error before).  p below 2^-126 is flushed: 1e-37 of the terms.
"""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from oracle import tokens as OT
from prefix_tree_block_gb300 import workloads as W

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U, UB = 2.0 ** -24, 2.0 ** -8
INF = float("inf")


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


def rows_of(row_ptr, index, R, N):
    """The row that scores each token, -1: none."""
    if row_ptr is None:
        return np.arange(N)
    rows = np.full(N, -1)
    for r in range(R):
        for e in range(row_ptr[r], row_ptr[r + 1]):
            rows[e if index is None else index[e]] = r
    return rows


class Bounds:
    def __init__(self, x, scale):
        z = x * scale
        V = z.shape[1]
        m = z.max(1, initial=-np.inf, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        self.m = np.abs(m[:, 0])
        _, self.lse, self.H = OT.logprobs(x, [], [], scale)
        live = np.isfinite(self.lse)
        lse = np.where(live, self.lse, 0.0)
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            ln_s = np.log(np.exp(z - m).sum(1, keepdims=True))
            p = np.where(live[:, None], np.exp(z - m - ln_s), 0.0)
            d = np.where(p > 0, m - z, 0.0)
        a, b = (p * d).sum(1), (p * d * d).sum(1)
        n = V / 128 + 64
        self.tl = 3 * U * a + 2.0 ** -22 + n * U + 2 * U * self.m + 4 * U * np.abs(lse)
        self.th = (n * U + 2.0 ** -22) * (1 + 2 * a) + 3 * U * (a + b) + 4 * U * (a + np.abs(self.H))
        with np.errstate(invalid="ignore"):
            self.p, self.l = p, np.where(p > 0, z - m - ln_s, 0.0)
        self.alse = np.abs(lse)


def close(got, want, tol):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def check(x, targets, row_ptr=None, index=None, k=0, scale=1.0, seed=0, grad=True, out=None, dH=True):
    """x: a CUDA [R, V] tensor or view; everything against the oracle."""
    R, V = x.shape
    N = len(targets)
    dev = lambda v, t: None if v is None else torch.tensor(np.asarray(v), dtype=t, device="cuda")  # noqa: E731
    t, ptr, idx = dev(targets, torch.int64), dev(row_ptr, torch.int32), dev(index, torch.int32)
    logp, lse, H, top, ids = pt.token_logprobs(x, t, row_ptr=ptr, index=idx, top_k=k, entropy=True, scale=scale)
    bare = pt.token_logprobs(x, t, row_ptr=ptr, index=idx, scale=scale)
    assert bare[2:] == (None, None, None)
    if not k:
        assert torch.equal(bare[0].nan_to_num(7), logp.nan_to_num(7)) and torch.equal(bare[1].nan_to_num(7), lse.nan_to_num(7))
    xs = x.double().cpu().numpy()
    rows = rows_of(row_ptr, index, R, N)
    wp, wl, wh = OT.logprobs(xs, targets, rows, scale)
    b = Bounds(xs, scale)
    close(lse, wl, b.tl)
    close(bare[1], wl, b.tl)  # (with alternatives another kernel than without)
    close(H, wh, b.th)
    z = np.array([abs(xs[r, v]) * scale if r >= 0 and v >= 0 and np.isfinite(xs[r, v]) else 0.0 for v, r in zip(targets, rows)])
    at = np.maximum(rows, 0)
    close(logp, wp, b.tl[at] + 2 * U * (z + b.alse[at]) if N else 0.0)
    close(bare[0], wp, b.tl[at] + 2 * U * (z + b.alse[at]) if N else 0.0)
    if k:
        wi = OT.top(xs, k)
        assert ids.cpu().numpy().tolist() == wi.tolist()
        v = np.take_along_axis(xs, wi, 1) * scale
        with np.errstate(invalid="ignore"):
            w = np.where(np.isneginf(wl)[:, None], -np.inf, np.where(np.isnan(v), -np.inf, v) - wl[:, None])
        close(top, w, b.tl[:, None] + 2 * U * (np.where(np.isfinite(v), np.abs(v), 0) + b.alse[:, None]))
    if not grad:
        pt.sync_status()
        return
    rng = np.random.default_rng(seed)
    g = rng.standard_normal(N).astype(np.float32)
    dh = rng.standard_normal(R).astype(np.float32) if dH else None
    d = pt.token_logprobs_bwd(dev(g, F32), x, t, lse, row_ptr=ptr, index=idx, dentropy=dev(dh, F32), entropy=H, scale=scale, dlogits=out)
    pt.sync_status()
    with np.errstate(invalid="ignore"):
        want = OT.logprobs_grad(xs, targets, rows, g.astype(np.float64), dh, scale)
    own, all_g, c = np.zeros((R, V)), np.zeros(R), np.zeros(R)
    for n, (v, r) in enumerate(zip(targets, rows)):
        if v >= 0 and r >= 0:
            own[r, v] += abs(g[n])
            all_g[r] += abs(g[n])
            c[r] += 1
    dp = b.tl[:, None] + 2 * U * b.alse[:, None] + 4 * U * np.abs(b.l) + 2.0 ** -22
    adh = np.abs(dh) if dH else np.zeros(R)
    terms = all_g[:, None] + adh[:, None] * (np.abs(np.nan_to_num(b.H))[:, None] + np.abs(b.l))
    tol = scale * (b.p * (terms * (dp + (c[:, None] + 8) * U) + adh[:, None] * b.th[:, None]) + (c[:, None] + 2) * U * own + 1e-37 * (terms + 105 * adh[:, None]))
    r = UB if x.dtype == BF else U
    close(d, want, tol * (1 + r) + r * np.abs(want) + 1e-37)


def logits(R, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R, V, generator=g) * spread).to(dtype).cuda()


def targets_of(R, V, seed):
    return np.random.default_rng(seed).integers(0, V, R).tolist()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 16, 63, 65, 255, 1000, 1025, 4099, 8191, 8200, 32768, 50001])
@pytest.mark.parametrize("R", [1, 5])
def test_sizes(dtype, V, R):
    """Odd vocabularies make rows start at every place modulo 16 bytes."""
    check(logits(R, V, dtype, V), targets_of(R, V, 1), k=min(V, 20), scale=1.0 if V % 2 else 0.8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,V", [(1, 131072), (3, 200003), (40, 70001), (300, 9000), (700, 300), (700, 9001), (600, 17000), (3100, 4507), (1, 1048577)])
def test_parts(dtype, R, V):
    """A cluster of two, four or eight CTAs a row; a CTA a row, with a ring or
    without, several rows one after the other; a warp a row."""
    check(logits(R, V, dtype, R), targets_of(R, V, 2), k=7)


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 64])
@pytest.mark.parametrize("V", [64, 100, 5000, 40000])
def test_alternatives(k, V):
    check(logits(3, V, BF, k), targets_of(3, V, 3), k=k, grad=False)
    check(logits(3, V, F32, k), targets_of(3, V, 3), k=k, grad=False)


@pytest.mark.parametrize("V,R", [(64, 2), (1000, 2), (8000, 2), (131072, 2), (40000, 230)])
@pytest.mark.parametrize("what", ["equal", "two values", "zeros of both signs", "rising", "falling", "few threads", "one large"])
def test_equal_and_ordered_logits(V, R, what):
    """The alternatives where values tie, or sit where the search is weakest:
    many large ones among the elements of few threads."""
    v = torch.arange(V)
    x = {"equal": torch.zeros(V), "two values": (v % 3 == 1).float(), "zeros of both signs": torch.where(v % 2 == 0, -0.0, 0.0),
         "rising": v.float() / 256, "falling": -v.float() / 256, "few threads": ((v // 8) % 128 < 63) * 4.0 + ((v * 7) % 11) / 16,
         "one large": torch.where(v == V // 2, 50.0, 0.0)}[what]
    for dtype in (BF, F32):
        check(x.repeat(R, 1).to(dtype).cuda(), targets_of(R, V, 4), k=64, grad=False)


@pytest.mark.parametrize("V", [2, 26, 103, 300, 1001, 4000])
@pytest.mark.parametrize("k", [1, 5, 24])
def test_alternatives_of_many_short_rows(V, k):
    """A warp a row."""
    for dtype in (BF, F32):
        check(logits(1300, V, dtype, V), targets_of(1300, V, 3), k=min(k, V), grad=False)


@pytest.mark.parametrize("V", [31, 150, 301, 512, 513])
@pytest.mark.parametrize("k", [24, 33, 64])
@pytest.mark.parametrize("values", [2, 40, 0])
def test_short_rows_listed_whole(V, k, values):
    """Fewer slots than alternatives: all are listed, and the list cut (few values: equal ones at the cut)."""
    for dtype in (BF, F32):
        x = logits(1300, V, dtype, V)
        check((x * 7).round().remainder(values) if values else x, targets_of(1300, V, 3), k=min(k, V), grad=False)


@pytest.mark.parametrize("V", [30, 999, 4096])
@pytest.mark.parametrize("what", ["equal", "two values", "falling", "few threads", "nothing", "one", "lowest"])
def test_equal_and_masked_logits_in_a_warp(V, what):
    v = torch.arange(V)
    for dtype, slot in ((BF, 8), (F32, 4)):
        x = {"equal": torch.ones(V), "two values": (v % 3 == 1).float(), "falling": -v.float() / 256, "few threads": ((v // slot) % 32 < 20) * 4.0,
             "nothing": torch.full((V,), -INF), "one": torch.where(v == V - 1, 1.0, -INF), "lowest": torch.full((V,), torch.finfo(dtype).min)}[what]
        check(x.repeat(1300, 1).to(dtype).cuda(), targets_of(1300, V, 4), k=24, grad=False)


@pytest.mark.parametrize("threads,V,R", [(128, 4096, 2), (128, 9000, 610), (480, 40000, 230), (480, 131072, 3)])
@pytest.mark.parametrize("ties", [False, True])
def test_large_logits_in_few_threads(threads, V, R, ties):
    """More candidates than the list has room for: every large logit is among the
    elements of 63 threads (of a CTA of 128, or of the 480 that read)."""
    v = torch.arange(V)
    for dtype, slot in ((BF, 8), (F32, 4)):
        x = ((v // slot) % threads < 63) * 4.0 + (0.0 if ties else ((v * 7) % 11) / 16)
        check(x.repeat(R, 1).to(dtype).cuda(), targets_of(R, V, 4), k=64, grad=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [5, 300, 20001])
def test_infinities(dtype, V):
    """Tokens that cannot be chosen, a row of nothing else, the type's lowest
    value as a mask, far apart values."""
    low = torch.finfo(dtype).min
    x = logits(8, V, dtype, 5).cpu()
    x[0, ::2] = -INF
    x[1] = -INF
    x[2] = low
    x[3, 1:] = low
    x[4] = low
    x[4, V // 2] = -INF
    x[5, 0] = torch.finfo(dtype).max
    x[6, 1] = 1e30
    x[7, 1:] = -INF
    t = [1, 0, V - 1, 0, 0, 0, 1, V - 1]
    check(x.cuda(), t, k=min(V, 9))
    check(x.cuda(), t, k=0, dH=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [5, 300, 20001, 131072])
def test_nan_and_positive_infinity(dtype, V):
    """A NaN or +inf makes its row NaN, and no other row."""
    x = logits(6, V, dtype, 6)
    x[1, V // 2] = float("nan")
    x[3, V - 1] = INF
    x[4] = float("nan")
    t = torch.tensor(targets_of(6, V, 5), device="cuda")
    logp, lse, H, top, ids = pt.token_logprobs(x, t, top_k=3, entropy=True)
    d = pt.token_logprobs_bwd(torch.ones(6, device="cuda"), x, t, lse, dentropy=torch.ones(6, device="cuda"), entropy=H)
    pt.sync_status()
    bad = torch.tensor([False, True, False, True, True, False], device="cuda")
    for y in (logp, lse, H, d.isnan().all(1), top.isnan().all(1)):
        got = y if y.dtype == torch.bool else y.isnan()
        assert torch.equal(got, bad)
    assert torch.equal(d.isnan().any(1), bad)
    assert ids.cpu().numpy().tolist() == OT.top(np.nan_to_num(x.double().cpu().numpy(), nan=-np.inf, posinf=np.inf, neginf=-np.inf), 3).tolist()
    keep = ~bad
    check(x[keep].contiguous(), t[keep].tolist(), k=3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [0, 1, 3, 8, 13])
@pytest.mark.parametrize("shift", [0, 1, 5])
def test_strides_and_alignment(dtype, pad, shift):
    """Columns of a wider buffer, what lies beside them poisoned; gradients that
    start as the logits do, elsewhere, and in their place."""
    R, V = 7, 1237
    wide = torch.full((R, V + pad + shift), float("nan"), dtype=dtype, device="cuda")
    x = wide[:, shift:shift + V]
    x.copy_(logits(R, V, dtype, 7))
    t = targets_of(R, V, 6)
    check(x, t, k=5)
    for other in (shift, shift + 1, 0):
        buf = torch.full((R, V + pad + shift + 1), 3.0, dtype=dtype, device="cuda")
        check(x, t, out=buf[:, other:other + V])
        buf[:, other:other + V] = 3.0
        assert torch.equal(buf, torch.full_like(buf, 3.0))
    lse = pt.token_logprobs(x, torch.tensor(t, device="cuda"))[1]
    g = torch.randn(R, device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    want = pt.token_logprobs_bwd(g, x, torch.tensor(t, device="cuda"), lse)
    assert pt.token_logprobs_bwd(g, x, torch.tensor(t, device="cuda"), lse, dlogits=x) is x
    assert torch.equal(x, want)
    x.fill_(float("nan"))
    assert wide.isnan().all()


def test_gradient_beside_the_logits():
    """Columns of one buffer: the logits, then their gradient."""
    both = torch.full((9, 2 * 501 + 3), 7.0, dtype=BF, device="cuda")
    x, d = both[:, 1:502], both[:, 503:1004]
    x.copy_(logits(9, 501, BF, 3))
    check(x, targets_of(9, 501, 3), out=d)
    assert (both[:, [0, 502, 1004]] == 7.0).all()
    with pytest.raises(pt.PTError, match="overlaps"):
        check(x, targets_of(9, 501, 3), out=both[:, 500:1001])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [11, 2000, 33000])
@pytest.mark.parametrize("mixed", [False, True])
def test_rows_with_any_number_of_tokens(dtype, V, mixed):
    """None, one, many, more than a CTA has threads; equal targets in a row;
    tokens not scored; entries of no row; tokens in any order."""
    rng = np.random.default_rng(V)
    per = [0, 1, 0, 7, 1300, 1, 2, 0]
    ptr = np.concatenate([[0], np.cumsum(per)])
    N = int(ptr[-1]) + 5
    t = rng.integers(0, V, N)
    t[rng.random(N) < 0.1] = -100
    t[3:6] = t[2]
    index = rng.permutation(N) if mixed else None
    check(logits(len(per), V, dtype, 8), t.tolist(), row_ptr=ptr.tolist(), index=None if index is None else index.tolist(), k=3)


@pytest.mark.parametrize("V,R", [(50, 4), (50, 2000), (40000, 3)])
@pytest.mark.parametrize("before,behind", [(1, 0), (700, 0), (45, 1300)])
def test_entries_of_no_row(V, R, before, behind):
    ptr = before + np.arange(R + 1)
    N = int(ptr[-1]) + behind
    x, t = logits(R, V, BF, 8), targets_of(N, V, 3)
    check(x, t, row_ptr=ptr.tolist(), k=2)
    check(x, t, row_ptr=ptr.tolist(), index=np.random.default_rng(1).permutation(N).tolist(), grad=False)


def test_nothing():
    x = torch.zeros(0, 9, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    out = pt.token_logprobs(x, none, top_k=2, entropy=True)
    assert [tuple(y.shape) for y in out] == [(0,), (0,), (0,), (0, 2), (0, 2)]
    assert pt.token_logprobs_bwd(torch.zeros(0, device="cuda"), x, none, out[1]).shape == (0, 9)
    check(logits(3, 50, F32, 1), [], row_ptr=[0, 0, 0, 0], k=2)
    check(logits(3, 50, F32, 1), [4, 5], row_ptr=[0, 0, 0, 0])


@pytest.mark.parametrize("spec,V", [([(37, [5, 1, 0, 12]), (0, [4, 9]), (1, [1]), (6, [])], 300), ([(100, [60] * 9)], 1000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_folded_rollouts(spec, V, dtype):
    """A batch as it is used: fold the rollouts, score every flat token under its
    prefix, unfold, take a loss on the rollouts, and bring its gradient back to
    the logits; against the same on the unfolded rollouts, in 64 bits."""
    st = W.grpo_structure(spec)
    L = max(sum(int(st.node_lengths[i]) for i in p) for p in st.paths()) + 2
    plan = pt.fold_plan(st.node_lengths, st.path_ptr, st.path_nodes, L)
    ptr, succ = plan.successors()
    after, first = OT.successors(st.node_lengths, st.paths())
    p, s = ptr.cpu().numpy(), succ.cpu().numpy()
    assert [s[p[i]:p[i + 1]].tolist() for i in range(st.T)] == after and s[p[-1]:].tolist() == first
    rng = np.random.default_rng(0)
    ids = torch.tensor(rng.integers(0, V, st.T), device="cuda")
    x = logits(st.T, V, dtype, 9)
    logp, lse, H, _, _ = pt.token_logprobs(x, ids, row_ptr=ptr, index=succ, entropy=True)
    w = torch.tensor(rng.standard_normal((st.n_samples, L)).astype(np.float32), device="cuda")
    loss = (plan.unfold(logp) * w).double().sum()
    d = pt.token_logprobs_bwd(plan.unfold_grad(w), x, ids, lse, row_ptr=ptr, index=succ)
    pt.sync_status()
    # the rollouts one by one
    off = np.concatenate([[0], np.cumsum(st.node_lengths)])
    y = x.double().cpu().requires_grad_()
    lp = torch.log_softmax(y, 1)
    want, size = 0.0, 0.0
    for k, path in enumerate(st.paths()):
        flat = [t for n in path for t in range(int(off[n]), int(off[n + 1]))]
        for j, (a, b) in enumerate(zip(flat, flat[1:])):
            term = lp[a, ids[b].item()] * w[k, j + 1].item()
            want, size = want + term, size + abs(term.item())
    want.backward()
    # each log probability is off by at most a relative 2^-15 (tl, with |logp| of order one), the sums' rounding is far below
    assert abs(loss.item() - want.item()) <= 2.0 ** -15 * size
    # p and the sums of G weights: dp is below 2^-18 here, then one rounding of the row's own and the tokens' part
    big = torch.zeros_like(y.grad)
    gabs = plan.unfold_grad(w.abs()).double().cpu()
    for a in range(st.T):
        for b in after[a]:
            big[a] += gabs[b] * lp[a].detach().exp()
            big[a, ids[b].item()] += gabs[b]
    tol = big * 2.0 ** -18 + y.grad.abs() * (UB if dtype == BF else U) * 1.01 + 1e-37
    assert ((d.double().cpu() - y.grad).abs() <= tol).all()


def test_far_rows():
    """Rows and gradients whose offsets pass 2^31 elements."""
    stride, V = (1 << 30) + 11, 777
    buf = torch.empty(2 * stride + V, dtype=BF, device="cuda")
    x = torch.as_strided(buf, (3, V), (stride, 1))
    x.copy_(logits(3, V, BF, 10))
    check(x, [1, 2, 776], k=4)
    out = torch.as_strided(torch.empty(2 * stride + V, dtype=BF, device="cuda"), (3, V), (stride, 1))
    check(x, [1, 2, 776], out=out)


def test_many_rows():
    """More rows than the first grid dimension would take in 16 bits."""
    x = logits(70001, 3, F32, 11)
    check(x, targets_of(70001, 3, 7), k=2)


@pytest.mark.parametrize("R", [4, 400])
def test_bad_tokens_are_reported_and_passed_over(R):
    V = 3333
    x = logits(R, V, BF, 12)
    good = targets_of(R, V, 8)
    t = torch.tensor(good, device="cuda")
    want = pt.token_logprobs(x, t)
    pt.sync_status()
    t2 = t.clone()
    t2[1] = V
    t2[2] = 1 << 40
    got = pt.token_logprobs(x, t2)
    with pytest.raises(pt.PTError, match="token log probability"):
        pt.sync_status()
    w = want[0].clone()
    w[1:3] = 0
    assert torch.equal(got[0], w) and torch.equal(got[1], want[1])
    g = torch.randn(R, device="cuda")
    g0 = g.clone()
    g0[1:3] = 0
    d = pt.token_logprobs_bwd(g, x, t2, want[1])
    with pytest.raises(pt.PTError, match="token log probability"):
        pt.sync_status()
    assert torch.equal(d, pt.token_logprobs_bwd(g0, x, t, want[1]))
    ptr = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    for at, value in ((2, -5), (1, R + 9), (R, 1 << 30)):
        bad = ptr.clone()
        bad[at] = value
        got = pt.token_logprobs(x, t, row_ptr=bad)
        pt.token_logprobs_bwd(g, x, t, want[1], row_ptr=bad)
        with pytest.raises(pt.PTError, match="token log probability"):
            pt.sync_status()
        assert torch.equal(got[1], want[1])
    idx = torch.arange(R, dtype=torch.int32, device="cuda")
    idx[0], idx[3] = -1, R
    got = pt.token_logprobs(x, t, row_ptr=ptr, index=idx)
    with pytest.raises(pt.PTError, match="token log probability"):
        pt.sync_status()
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[[0, 3]] = False
    assert torch.equal(got[0][keep], want[0][keep])
    pt.sync_status()


@pytest.mark.parametrize("R,V", [(3, 131072), (500, 5001)])
def test_streams_and_graphs(R, V):
    """On a side stream, two calls at once, and captured and replayed with other
    contents: the same bits as alone."""
    xs = [logits(R, V, BF, 20 + i) for i in range(3)]
    ts = [torch.tensor(targets_of(R, V, 20 + i), device="cuda") for i in range(3)]
    g, dh = torch.randn(R, device="cuda"), torch.randn(R, device="cuda")

    def both(x, t, stream=None):
        out = pt.token_logprobs(x, t, top_k=5, entropy=True, stream=stream)
        return [*out, pt.token_logprobs_bwd(g, x, t, out[1], dentropy=dh, entropy=out[2], stream=stream)]

    want = [both(x, t) for x, t in zip(xs, ts)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = [both(x, t, s) for _ in range(3) for x, t, s in zip(xs, ts, (s1, s2, s1))]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(o, want[i % 3]))
    x, t = xs[0].clone(), ts[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(x, t)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        t.copy_(ts[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    pt.sync_status()


def test_binding_refusals():
    x = torch.zeros(4, 10, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    i = torch.zeros(5, dtype=torch.int32, device="cuda")
    for bad in (lambda: pt.token_logprobs(x.t(), t), lambda: pt.token_logprobs(x, t[:3]), lambda: pt.token_logprobs(x, t, row_ptr=i[:4]),
                lambda: pt.token_logprobs(x, t, index=i), lambda: pt.token_logprobs(x.as_strided((4, 10), (5, 1)), t),
                lambda: pt.token_logprobs_bwd(x[:, 0].contiguous(), x, t, x[:3, 0].contiguous()),
                lambda: pt.token_logprobs_bwd(x[:, 0].contiguous(), x, t, x[:, 0].contiguous(), dentropy=x[:, 0].contiguous())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: pt.token_logprobs(x, t.int()), lambda: pt.token_logprobs(x, t.cpu()), lambda: pt.token_logprobs(x, t, row_ptr=t),
                lambda: pt.token_logprobs_bwd(x[:, 0], x, t, x[:, 0].contiguous()), lambda: pt.token_logprobs(x.double(), t)):
        with pytest.raises(TypeError):
            bad()
    for kw in (dict(top_k=11), dict(top_k=-1), dict(scale=0.0)):
        with pytest.raises(pt.PTError) as e:
            pt.token_logprobs(x, t, **kw)
        assert e.value.status == pt.PT_ERR_INVALID_ARG
    with pytest.raises(pt.PTError) as e:
        pt.token_logprobs(torch.zeros(1, 100, device="cuda"), t[:1], top_k=65)
    assert e.value.status == pt.PT_ERR_UNSUPPORTED
