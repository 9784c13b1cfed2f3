"""Trees of drafted tokens over the cache: pt_draft_tree, pt_attn_decode_drafts and
pt_cache_keep against the oracle, alone and together as a step uses them.  The
attention's tolerances are those of decode_cases.py (the same kernels on other
masks: its derivation counts tokens, not their order)."""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from oracle import decode as OD
from oracle import tokens as OT

from decode_cases import U32, UB, cache_of, csr, pages_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def parents_of(S, q, shape, seed=0):
    rng = np.random.default_rng(seed)
    j = np.arange(q)
    if shape == "chain":
        return np.tile(j - 1, (S, 1))
    if shape == "roots":
        return np.full((S, q), -1)
    if shape == "star":
        return np.tile(np.where(j > 0, 0, -1), (S, 1))
    return np.stack([[int(rng.integers(-1, k)) if k else -1 for k in range(q)] for _ in range(S)])


def counts_of(S, q, seed=0):
    c = np.random.default_rng(seed).integers(0, q + 1, S)
    c[::2] = q
    return c


# ---------------------------------------------------------------------------------------------------------------
# masks and positions

@pytest.mark.parametrize("q", [1, 2, 3, 31, 32, 33, 64, 100, 128, 255, 256])
@pytest.mark.parametrize("shape", ["chain", "roots", "star", "any"])
def test_trees(q, shape):
    S = 7
    up, c = parents_of(S, q, shape, q), counts_of(S, q, q)
    lens = np.random.default_rng(q).integers(q, 1000, S + 1)
    start = np.random.default_rng(q).integers(0, 1000, S + 1)
    plan = pt.decode_plan(S + 1, *csr([[0, 1 + s] for s in range(S)]), 2, 2, q)
    for count, first in ((None, None), (c, None), (c, start)):
        n = np.full(S, q) if count is None else count
        base = lens[1:] - n + (0 if first is None else first[1:])
        want = OT.draft_tree(up, n, base)
        mask, pos = pt.draft_tree(i32(up.reshape(-1)), i32(lens), plan, q_count=None if count is None else i32(count), start=None if first is None else i32(first))
        pt.sync_status()
        np.testing.assert_array_equal(mask.cpu().numpy(), want[0])
        np.testing.assert_array_equal(pos.cpu().numpy(), want[1])


@pytest.mark.parametrize("S", [1, 42, 43, 5000])
def test_many_samples(S):
    q = 3
    up, c = parents_of(S, q, "any", S), counts_of(S, q, S)
    lens = np.random.default_rng(S).integers(q, 1000, S)
    plan = pt.decode_plan(S, *csr([[s] for s in range(S)]), 1, 1, q)
    mask, pos = pt.draft_tree(i32(up.reshape(-1)), i32(lens), plan, q_count=i32(c))
    want = OT.draft_tree(up, c, lens - c)
    np.testing.assert_array_equal(mask.cpu().numpy(), want[0])
    np.testing.assert_array_equal(pos.cpu().numpy(), want[1])


def test_bad_parents_and_counts():
    plan = pt.decode_plan(2, *csr([[0], [1]]), 1, 1, 4)
    lens = i32([10, 20])
    good = [-1, 0, 0, 1, -1, 0, 1, 2]
    for at, value in ((0, 0), (1, 1), (2, 3), (3, -2), (5, 1 << 30), (7, -(1 << 31))):
        up = list(good)
        up[at] = value
        mask, pos = pt.draft_tree(i32(up), lens, plan)
        with pytest.raises(pt.PTError, match="cache") as e:
            pt.sync_status()
        assert e.value.status == pt.PT_ERR_INVALID_ARG
        up[at] = -1
        want = OT.draft_tree(np.array(up).reshape(2, 4), [4, 4], [6, 16])
        np.testing.assert_array_equal(mask.cpu().numpy(), want[0])
        np.testing.assert_array_equal(pos.cpu().numpy(), want[1])
    mask, pos = pt.draft_tree(i32(good), lens, plan, q_count=i32([5, -1]))
    with pytest.raises(pt.PTError, match="cache"):
        pt.sync_status()
    want = OT.draft_tree(np.array(good).reshape(2, 4), [4, 0], [6, 20])
    np.testing.assert_array_equal(mask.cpu().numpy(), want[0])
    # parents behind the count are not looked at
    pt.draft_tree(i32([-1, 0, 99, 99, -1, 99, -7, 99]), lens, plan, q_count=i32([2, 1]))
    pt.sync_status()


# ---------------------------------------------------------------------------------------------------------------
# attention

NODES = {
    "group": ([37, 40, 33, 95, 48], [[0, i] for i in range(1, 5)]),
    "no prompt": ([0, 35, 129], [[0, 1], [0, 2]]),
    "short": ([20, 1, 0, 3, 34], [[0, i] for i in range(1, 5)]),
    "deep": ([130, 31, 0, 64, 2, 33, 250, 40], [[0, 1, 4], [0, 1, 5], [0, 2, 6], [0, 3, 7], [0, 3], [0]]),
    "crowd": ([290] + [33 + 2 * (i % 7) for i in range(70)], [[0, i] for i in range(1, 71)]),
    "shared leaf": ([33, 60], [[0, 1], [0, 1], [1], [0]]),
}


def attend(lens, paths, Hq, Hkv, D, dtype, ps, q, up, c, seed=0, width=None, poison=float("nan"), mask=None, scale=0.0, edit=None):
    rng = np.random.default_rng(seed)
    tables, n_pages = pages_of(lens, ps, rng, width=width)
    Kc, Vc = cache_of(lens, tables, n_pages, Hkv, ps, D, dtype, seed, poison)
    if edit:
        edit(Kc, Vc, tables)
    S = len(paths)
    Q = torch.randn(S * q, Hq, D, generator=torch.Generator().manual_seed(seed + 1)).to(dtype)
    plan = pt.decode_plan(len(lens), *csr(paths), Hq, Hkv, q)
    O = torch.full(Q.shape, 7.0, dtype=dtype, device="cuda")
    L = torch.full((Hq, S * q), 7.0, device="cuda")
    count = None if c is None else i32(c)
    if mask is None:
        mask, _ = pt.draft_tree(i32(up.reshape(-1)), i32(lens), plan, q_count=count)
    pt.attn_decode(Q.cuda(), Kc.cuda(), Vc.cuda(), i32(tables), i32(lens), plan, q_count=count, O=O, LSE=L, draft_mask=mask, scale=scale)
    pt.sync_status()
    return O.cpu(), L.cpu(), Q, Kc, Vc, tables


def compare(O, L, Q, Kc, Vc, tables, lens, paths, q, sees, c, scale=None):
    """As decode_cases.check, with the tree's oracle."""
    bf16 = O.dtype == BF
    qf, k, v = (x.to(F32).numpy() for x in (Q, Kc, Vc))
    o, l = O.double().numpy(), L.double().numpy()
    c = np.full(len(paths), q) if c is None else c
    wo, wl = OT.attention(qf, k, v, tables, lens, paths, sees, q, c, scale)
    av, _ = OT.attention(qf, k, np.abs(v), tables, lens, paths, sees, q, c, scale)
    idle = np.isnan(wl)
    D = qf.shape[2]
    n = max([1] + [sum(int(lens[i]) for i in p) for p in paths])
    kk = np.abs(np.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0)).max(initial=0.0)
    ds = (D + 4) * U32 * np.abs(qf).sum(-1).max(initial=0.0) * kk * (scale or D ** -0.5)
    dp = 2 * ds + 2.0 ** -21 + (n + 8) * U32
    tol = 2 * dp * av + (UB * av + UB * np.abs(wo) * (1 + 2 * UB) if bf16 else U32 * np.abs(wo))
    skip = idle.T[:, :, None]
    bad = ~skip & ~(np.abs(o - wo) <= tol + 1e-30)
    assert not bad.any(), f"O: {int(bad.sum())} of {bad.size} off at {np.argwhere(bad)[0]}"
    none = np.isneginf(wl)
    assert np.array_equal(np.isneginf(l) & ~idle, none)
    fin = ~idle & ~none
    assert (np.abs(l[fin] - wl[fin]) <= ds + (n + 8) * U32 + 2.0 ** -21 + 4 * U32 * np.abs(wl[fin])).all()
    assert (o[np.broadcast_to(skip, o.shape)] == 7.0).all() and (l[idle] == 7.0).all()


def sees_of(up, q):
    return [[OT.above(p, j) for j in range(q)] for p in up]


@pytest.mark.parametrize("nodes", NODES)
@pytest.mark.parametrize("Hq,Hkv,D,dtype,ps", [(14, 2, 64, BF, 16), (16, 4, 128, BF, 32), (8, 2, 256, BF, 64), (2, 1, 512, BF, 16), (2, 2, 32, F32, 16), (3, 1, 80, F32, 7), (6, 2, 96, BF, 24)])
@pytest.mark.parametrize("q", [2, 8, 33])
def test_attention(nodes, Hq, Hkv, D, dtype, ps, q):
    """Every kernel; trees longer than the node, counts of none."""
    lens, paths = NODES[nodes]
    S = len(paths)
    for shape, c in (("any", None), ("roots", counts_of(S, q, q))):
        up = parents_of(S, q, shape, q)
        for width in (None, 65536 // ps) if dtype == BF and D <= 128 else (None,):
            got = attend(lens, paths, Hq, Hkv, D, dtype, ps, q, up, c, seed=q, width=width)
            compare(*got, lens, paths, q, sees_of(up, q), c)


@pytest.mark.parametrize("q", [1, 16, 17, 64, 65, 100])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths_of_drafts(q, dtype):
    """Words of a mask, drafts over several tiles, at every place of the node."""
    paths = [[0, i] for i in range(1, 6)]
    lens = [50] + [q + k for k in (0, 1, 7, 15, 100)]
    up = parents_of(5, q, "any", q)
    for width in (None, 4096):
        got = attend(lens, paths, 4, 2, 64, dtype, 16, q, up, None, seed=q, width=width, scale=0.3)
        compare(*got, lens, paths, q, sees_of(up, q), None, 0.3)


@pytest.mark.parametrize("D,dtype", [(1, F32), (33, F32), (66, F32), (128, F32), (130, F32), (256, F32), (257, F32), (512, F32),
                                     (8, BF), (72, BF), (104, BF), (128, BF), (200, BF), (264, BF), (512, BF)])
def test_head_dims(D, dtype):
    lens, paths = NODES["deep"]
    up = parents_of(len(paths), 7, "any", D)
    for width in (None, 4096) if dtype == BF and D <= 128 else (None,):
        got = attend(lens, paths, 24, 2, D, dtype, 16, 7, up, None, seed=D, width=width)
        compare(*got, lens, paths, 7, sees_of(up, 7), None)


def test_more_drafts_than_trees_have():
    """Masks of the caller's own, of more drafts than pt_draft_tree takes."""
    q, paths, lens = 300, [[0, 1]], [20, 340]
    rng = np.random.default_rng(0)
    sees = np.tril(rng.random((q, q)) < 0.3)
    words = np.zeros((q, 320), np.uint64)
    words[:, :q] = sees
    words = (words.reshape(q, 10, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)
    for dtype, width in ((BF, None), (BF, 65536), (F32, None)):  # (wide: the kernel for many rows)
        got = attend(lens, paths, 2, 1, 64, dtype, 16, q, None, None, mask=torch.from_numpy(words).cuda(), width=width)
        compare(*got, lens, paths, q, [[sorted(set(np.flatnonzero(sees[j])) | {j}) for j in range(q)]], None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks_as_they_are(dtype):
    """A draft sees itself whatever its bit says; bits behind the count are not
    looked at; a mask may show a later draft."""
    lens, paths = [10, 30, 41], [[0, 1], [0, 2]]
    q, c = 6, np.array([6, 4])
    words = torch.tensor([[0]] * 6 + [[-1]] * 6, dtype=torch.int32, device="cuda")
    for width in (None, 4096):
        got = attend(lens, paths, 4, 2, 64, dtype, 16, q, None, c, mask=words, width=width)
        compare(*got, lens, paths, q, [[[j] for j in range(6)], [list(range(4))] * 6], c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq", [4, 40])
def test_a_chain_is_the_causal_call(dtype, Hq):
    """The call without a mask and the one with a chain's agree: bit for bit where
    the nodes are cut alike (with many rows the part of a leaf that all drafts see
    ends in front of the first draft, not behind it, and its pieces' sums are
    others), and each within the tolerance of the oracle."""
    lens, paths = NODES["crowd"]
    q, S = 8, len(paths)
    rng = np.random.default_rng(0)
    tables, n_pages = pages_of(lens, 16, rng)
    Kc, Vc = (x.cuda() for x in cache_of(lens, tables, n_pages, 2, 16, 64, dtype, 0))
    Q = torch.randn(S * q, Hq, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    plan = pt.decode_plan(len(lens), *csr(paths), Hq, 2, q)
    mask, pos = pt.draft_tree(i32(parents_of(S, q, "chain").reshape(-1)), i32(lens), plan)
    want = pt.attn_decode(Q, Kc, Vc, i32(tables), i32(lens), plan)
    got = pt.attn_decode(Q, Kc, Vc, i32(tables), i32(lens), plan, draft_mask=mask)
    pt.sync_status()
    if Hq == 4 or dtype == F32:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for O, L in (got, want):
        compare(O.cpu(), L.cpu(), Q.cpu(), Kc.cpu(), Vc.cpu(), tables, lens, paths, q, sees_of(parents_of(S, q, "chain"), q), None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("what", [0, 1])
@pytest.mark.parametrize("width", [None, 4096])
def test_a_hidden_drafts_values_stay_hidden(dtype, D, value, what, width):
    """A draft whose key (0) or value (1) is not finite reaches the drafts that
    see it only."""
    lens, paths, q = [50, 40, 21], [[0, 1], [0, 2]], 6
    up = np.array([[-1, -1, 0, 1, 2, 3], [-1, 0, 1, 2, 3, 4]])
    sees = sees_of(up, q)

    def edit(Kc, Vc, tables):
        s = OD.slots_of(tables[1], 40, 16)[40 - 6 + 2]  # draft 2 of sample 0: drafts 2 and 4 see it
        (Kc, Vc)[what][s // 16, :, s % 16] = value

    O, L, Q, Kc, Vc, tables = attend(lens, paths, 8, 2, D, dtype, 16, q, up, None, width=width, edit=edit)
    clean = [x.clone() for x in (Kc, Vc)]
    s = OD.slots_of(tables[1], 40, 16)[36]
    for x in clean:
        x[s // 16, :, s % 16] = 0.0
    hit = torch.zeros(12, dtype=torch.bool)
    hit[[2, 4]] = True
    if value != 3e38:  # (a large finite key or value may or may not overflow)
        assert not O[hit].isfinite().all(-1).all() if what else True
    # the rows that do not see it are those of a cache without it
    O2, L2 = O.clone(), L.clone()
    wo, wl = OT.attention(Q.float().numpy(), clean[0].float().numpy(), clean[1].float().numpy(), tables, lens, paths, sees, q, [q, q])
    O2[hit] = torch.from_numpy(wo).to(dtype)[hit]
    L2[:, hit] = torch.from_numpy(wl).float()[:, hit]
    compare(O2, L2, Q, clean[0], clean[1], tables, lens, paths, q, sees, None)


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("Hq,Hkv", [(16, 1), (40, 1), (60, 2)])
@pytest.mark.parametrize("own", [6, 21, 130, 259, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_with_many_rows(D, Hq, Hkv, own, value):
    """In the kernel for nodes that many rows read: one column of some drafts'
    values is not finite.  Only that column, and only of the drafts that see one
    of them, is touched; the rest of those drafts' values counts as it is."""
    lens, paths, q = [150, own, 40], [[0, 1], [0, 2]], 6
    up = np.array([[-1, -1, 0, 1, 2, 3], [-1, 0, 1, 2, 3, 4]])
    sees = sees_of(up, q)
    odd = [2, 5]  # drafts of sample 0

    def slots(tables):
        return OD.slots_of(tables[1], own, 16)[own - 6 + np.array(odd)]

    def edit(Kc, Vc, tables):
        for s in slots(tables):
            Vc[s // 16, :, s % 16, 3] = value

    O, L, Q, Kc, Vc, tables = attend(lens, paths, Hq, Hkv, D, BF, 16, q, up, None, width=4096, edit=edit)
    clean = Vc.clone()
    for s in slots(tables):
        clean[s // 16, :, s % 16, 3] = 0.0
    hit = torch.tensor([any(j in sees[s][i] for j in odd) and s == 0 for s in range(2) for i in range(q)])
    assert not O[hit][:, :, 3].isfinite().any()
    O2 = O.clone()
    wo, _ = OT.attention(Q.float().numpy(), Kc.float().numpy(), clean.float().numpy(), tables, lens, paths, sees, q, [q, q])
    O2[hit, :, 3] = torch.from_numpy(wo).to(BF)[hit, :, 3]
    compare(O2, L, Q, Kc, clean, tables, lens, paths, q, sees, None)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [16, 40])
def test_hidden_keys_with_many_rows(D, Hq):
    """A key that is NaN makes the drafts that see it NaN, and no others."""
    lens, paths, q = [150, 130, 40], [[0, 1], [0, 2]], 6
    up = np.array([[-1, -1, 0, 1, 2, 3], [-1, 0, 1, 2, 3, 4]])
    sees = sees_of(up, q)

    def edit(Kc, Vc, tables):
        s = OD.slots_of(tables[1], 130, 16)[126]
        Kc[s // 16, :, s % 16] = float("nan")

    O, L, Q, Kc, Vc, tables = attend(lens, paths, Hq, 1, D, BF, 16, q, up, None, width=4096, edit=edit)
    hit = torch.tensor([s == 0 and 2 in sees[0][i] for s in range(2) for i in range(q)])
    assert O[hit].isnan().all() and L[:, hit].isnan().all()
    s = OD.slots_of(tables[1], 130, 16)[126]
    clean = Kc.clone()
    clean[s // 16, :, s % 16] = 0.0
    wo, wl = OT.attention(Q.float().numpy(), clean.float().numpy(), Vc.float().numpy(), tables, lens, paths, sees, q, [q, q])
    O[hit], L[:, hit] = torch.from_numpy(wo).to(BF)[hit], torch.from_numpy(wl).float()[:, hit]
    compare(O, L, Q, clean, Vc, tables, lens, paths, q, sees, None)


def test_attention_refuses_bad_masks():
    plan = pt.decode_plan(1, *csr([[0]]), 1, 1, 33)
    Q, c = torch.zeros(33, 1, 64, device="cuda"), torch.zeros(3, 1, 16, 64, device="cuda")
    t, n = i32([[0, 1, 2]]), i32([40])
    for bad in (torch.zeros(33, 1, dtype=torch.int32, device="cuda"), torch.zeros(66, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            pt.attn_decode(Q, c, c, t, n, plan, draft_mask=bad)
    with pytest.raises(TypeError):
        pt.attn_decode(Q, c, c, t, n, plan, draft_mask=torch.zeros(33, 2, dtype=torch.int64, device="cuda"))
    big = pt.decode_plan(1, *csr([[0]]), 1, 1, 257)
    with pytest.raises(pt.PTError) as e:
        pt.draft_tree(i32([-1] * 257), i32([300]), big)
    assert e.value.status == pt.PT_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------------------------------------------
# accepted drafts

def kept_of(S, q, c, seed):
    rng = np.random.default_rng(seed)
    kept = np.full((S, q), -1)
    for s in range(S):
        n = int(rng.integers(0, c[s] + 1))
        kept[s, :n] = np.sort(rng.choice(int(c[s]), n, replace=False))
    return kept


@pytest.mark.parametrize("Hkv,D,dtype,ps", [(2, 64, BF, 16), (8, 128, BF, 16), (1, 8, BF, 1), (3, 5, F32, 7), (3, 5, BF, 7), (2, 6, BF, 3), (2, 256, F32, 64), (24, 128, F32, 16)])
@pytest.mark.parametrize("q", [1, 2, 7, 33, 256])
def test_keep(Hkv, D, dtype, ps, q):
    S = 6
    c = counts_of(S, q, q)
    lens = np.random.default_rng(q).integers(0, 40, S) + c
    lens = np.concatenate([[17], lens])
    leaves = [1 + s for s in range(S)]
    tables, n_pages = pages_of(lens, ps, np.random.default_rng(1))
    Kc, Vc = cache_of(lens, tables, n_pages, Hkv, ps, D, dtype, 2, poison=9.0)
    plan = pt.decode_plan(S + 1, *csr([[0, x] for x in leaves]), Hkv, Hkv, q)
    for kept in (kept_of(S, q, c, q), np.where(np.arange(q) < c[:, None], np.arange(q), -1), np.full((S, q), -1)):
        k, v = Kc.cuda(), Vc.cuda()
        pt.cache_keep(i32(kept), k, v, i32(tables), i32(lens), plan, q_count=i32(c))
        pt.sync_status()
        for got, old in ((k, Kc), (v, Vc)):
            want = OT.keep(kept, c, lens, leaves, tables, ps, old.float().numpy())
            np.testing.assert_array_equal(got.float().cpu().numpy(), want)


def test_keep_of_bad_drafts():
    """A sample with a bad list, length, count or page stays as it is; the others move."""
    q, lens, ps = 4, [20, 20, 20], 16
    tables = np.array([[0, 1], [2, 3], [4, 5]])
    plan = pt.decode_plan(3, *csr([[0], [1], [2]]), 2, 2, q)
    cache = torch.randn(6, 2, ps, 8, generator=torch.Generator().manual_seed(0))
    good = [[1, 3, -1, -1], [0, 2, 3, -1], [3, -1, -1, -1]]
    want = OT.keep(good, [q] * 3, lens, [0, 1, 2], tables, ps, cache.numpy())

    def run(kept=good, lens=lens, tables=tables, count=None):
        k, v = cache.cuda(), cache.cuda()
        pt.cache_keep(i32(kept), k, v, i32(tables), i32(lens), plan, q_count=count)
        with pytest.raises(pt.PTError, match="cache") as e:
            pt.sync_status()
        assert e.value.status == pt.PT_ERR_INVALID_ARG
        for x in (k, v):
            x = x.cpu().numpy()
            np.testing.assert_array_equal(x[2:4], cache.numpy()[2:4])  # sample 1
            np.testing.assert_array_equal(x[[0, 1, 4, 5]], want[[0, 1, 4, 5]])

    for row in ([2, 1, -1, -1], [1, 1, -1, -1], [0, 4, -1, -1], [1 << 30, -1, -1, -1]):
        run(kept=[good[0], row, good[2]])
    for n in (-1, 3, 33, 1 << 30):
        run(lens=[20, n, 20])
    for page in (-1, 6, 1 << 30):
        t = tables.copy()
        t[1] = page
        run(tables=t)
    for n in (-1, 5):
        run(count=i32([4, n, 4]))


def test_keep_refuses_samples_that_share_a_leaf():
    plan = pt.decode_plan(2, *csr([[0, 1], [0, 1]]), 1, 1, 2)
    c = torch.zeros(4, 1, 16, 8, device="cuda")
    with pytest.raises(pt.PTError, match="end at one node"):
        pt.cache_keep(i32([[0, -1], [0, -1]]), c, c.clone(), i32([[0, 1], [2, 3]]), i32([5, 5]), plan)


def test_keep_refuses_caches_that_overlap():
    plan = pt.decode_plan(1, *csr([[0]]), 2, 2, 4)
    c = torch.zeros(7, 2, 16, 8, device="cuda")
    for k, v in ((c[:3], c[:3]), (c[:3], c[2:5]), (c[1:4], c[:3])):
        with pytest.raises(pt.PTError, match="overlap"):
            pt.cache_keep(i32([[0, -1, -1, -1]]), k, v, i32([[0, 1, 2]]), i32([40]), plan)
    pt.cache_keep(i32([[1, -1, -1, -1]]), c[:3], c[3:6], i32([[0, 1, 2]]), i32([40]), plan)
    pt.sync_status()


def test_binding_refusals():
    plan = pt.decode_plan(1, *csr([[0]]), 2, 2, 4)
    c, t, n, k = torch.zeros(3, 2, 16, 8, device="cuda"), i32([[0, 1, 2]]), i32([40]), i32([[0, -1, -1, -1]])
    for bad in (lambda: pt.draft_tree(i32([-1] * 3), n, plan), lambda: pt.draft_tree(i32([-1] * 4), i32([1, 2]), plan),
                lambda: pt.draft_tree(i32([-1] * 4), n, plan, q_count=i32([1, 2])), lambda: pt.draft_tree(i32([-1] * 4), n, plan, start=i32([])),
                lambda: pt.cache_keep(k[0], c, c, t, n, plan), lambda: pt.cache_keep(k, c[:, :1].contiguous(), c[:, :1].contiguous(), t, n, plan),
                lambda: pt.cache_keep(k, c, c[:2], t, n, plan), lambda: pt.cache_keep(k, c, c, t[0], n, plan)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        pt.draft_tree(i32([-1] * 4).long(), n, plan)
    with pytest.raises(TypeError):
        pt.cache_keep(k, c.half(), c.half(), t, n, plan)


# ---------------------------------------------------------------------------------------------------------------
# together

@pytest.mark.parametrize("dtype,ps", [(BF, 16), (F32, 5)])
@pytest.mark.parametrize("captured", [False, True])
def test_a_loop_of_verified_trees(dtype, ps, captured):
    """Steps of rollouts as a user runs them: pages for the drafts, their masks
    and positions, rotated queries and keys, the write, the attention, the scores
    of the drafts, the accepted ones kept, the rest taken back.  In the end the
    cache holds exactly the accepted tokens, rotated at their final positions,
    and every step's attention is the oracle's.  Captured: one graph replayed."""
    Hq, Hkv, D, q, V, steps = 4, 2, 64, 6, 50, 4
    lens = [21, 5, 0, 9]
    paths = [[0, 1], [0, 2], [0, 3]]
    S, width, cap = 3, 16, 64
    rng = np.random.default_rng(0)
    f = torch.tensor(10000.0 ** (-np.arange(32) / 32), dtype=F32, device="cuda")
    plan = pt.decode_plan(4, *csr(paths), Hq, Hkv, q)
    Kc, Vc = torch.zeros(2, cap, Hkv, ps, D, dtype=dtype, device="cuda").unbind(0)
    Kc, Vc = Kc.contiguous(), Vc.contiguous()
    tables, ring = torch.full((4, width), -1, dtype=torch.int32, device="cuda"), i32(rng.permutation(cap))
    counters = torch.tensor([0, cap], device="cuda")
    start = i32([0, 21, 21, 21])
    zero = i32([0, 0, 0, 0])

    def tokens(n, seed):
        return torch.randn(n, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()

    def rope(x, pos):
        pt.rotary(x[:, :Hq + Hkv], pos, f, out=x[:, :Hq + Hkv])

    held, counters, _, slots, pos = pt.cache_tables(zero, i32(lens), tables, ring, counters, ps, sum(lens), start=start)
    x = tokens(sum(lens), 1)
    raw = x.clone()
    rope(x, pos)
    pt.cache_write(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, Kc, Vc)
    off = np.cumsum([0] + lens)
    truth = [[raw[off[i] + t].cpu() for t in range(lens[i])] for i in range(4)]  # each node's tokens, before the rotation

    qkv, up = tokens(S * q, 0), i32(parents_of(S, q, "any").reshape(-1))
    kept, logits = i32(np.full((S, q), -1)), torch.zeros(S * q, V, dtype=dtype, device="cuda")
    drafts = torch.zeros(S * q, dtype=torch.int64, device="cuda")
    ptr, idx = i32(np.zeros(S * q + 1)), i32(np.zeros(S * q))
    grow = i32([0, q, q, q])
    state = dict(held=held, counters=counters)

    def step():
        x = qkv.clone()
        held, counters, _, slots, _ = pt.cache_tables(state["held"], grow, tables, ring, state["counters"], ps, S * q, start=start)
        mask, pos = pt.draft_tree(up, held, plan, start=start)
        rope(x, pos)
        pt.cache_write(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, Kc, Vc)
        O, L = pt.attn_decode(x[:, :Hq], Kc, Vc, tables, held, plan, draft_mask=mask)
        scores = pt.token_logprobs(logits, drafts, row_ptr=ptr, index=idx, top_k=3, entropy=True)
        before = Kc.clone(), Vc.clone(), tables.clone()
        pt.cache_keep(kept, Kc, Vc, tables, held, plan)
        back = torch.cat([zero[:1], ((kept >= 0).sum(1) - q).int()])
        after, counters, _, _, _ = pt.cache_tables(held, back, tables, ring, counters, ps, 0)
        state["held"].copy_(after)
        state["counters"].copy_(counters)
        return O, L, x, held, before, scores

    graph = None
    if captured:
        saved = [t.clone() for t in (Kc, Vc, tables, ring, state["held"], state["counters"])]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for t, o in zip((Kc, Vc, tables, ring, state["held"], state["counters"]), saved):
            t.copy_(o)
    for n in range(steps):
        p = parents_of(S, q, "any", n)
        qkv.copy_(tokens(S * q, 100 + n))
        up.copy_(i32(p.reshape(-1)))
        logits.copy_(tokens(S * q, 200 + n)[:, 0, :V])
        drafts.copy_(torch.tensor(rng.integers(0, V, S * q)))
        # a draft is scored by its parent's row; roots by none here
        rows = np.where(p >= 0, p + np.arange(S)[:, None] * q, -1).reshape(-1)
        order = np.argsort(np.where(rows < 0, S * q, rows), kind="stable")
        ptr.copy_(i32(np.concatenate([[0], np.cumsum(np.bincount(rows[rows >= 0], minlength=S * q))])))
        idx.copy_(i32(order))
        accept = np.full((S, q), -1)
        for s in range(S):
            path = OT.above(p[s], int(rng.integers(0, q)))[::-1]
            accept[s, :len(path)] = path
        kept.copy_(i32(accept))
        if captured:
            graph.replay()
        else:
            out = step()
        pt.sync_status()
        O, L, x, held, (k0, v0, t0), scores = out
        lens_now = held.cpu().numpy()
        compare(O.cpu(), L.cpu(), x[:, :Hq].cpu(), k0.cpu(), v0.cpu(), t0.cpu().numpy(), lens_now, paths, q, sees_of(p, q), None)
        want = OT.logprobs(logits.double().cpu().numpy(), drafts.tolist(), rows)[0]
        # (V = 50 logits of order one: tl of test_gpu_logprobs.py is below 2^-17)
        assert np.abs(scores[0].double().cpu().numpy() - want).max() < 2.0 ** -17
        for s in range(S):
            truth[1 + s] += [qkv[s * q + j].cpu() for j in accept[s] if j >= 0]
    final, t = state["held"].cpu().numpy(), tables.cpu().numpy()
    assert final.tolist() == [len(x) for x in truth]
    u = UB if dtype == BF else U32
    for i in range(4):
        at = OD.slots_of(t[i], int(final[i]), ps)
        got_k, got_v = (c.double().cpu().numpy()[at // ps, :, at % ps] for c in (Kc, Vc))
        x = torch.stack(truth[i]).double().numpy() if truth[i] else np.zeros((0, Hq + 2 * Hkv, D))
        np.testing.assert_array_equal(got_v, x[:, Hq + Hkv:])
        k = x[:, Hq:Hq + Hkv]
        pos = int(start[i]) + np.arange(len(x))
        want = OT.rotary(k, pos, f.cpu().numpy(), [32], False, False)
        size = np.abs(k[..., :32]) + np.abs(k[..., 32:])
        assert (np.abs(got_k - want) <= 12 * U32 * np.concatenate([size, size], -1) + u * 1.01 * np.abs(want)).all()
