"""The decoding attention (pt_attn_decode) against the fp64 oracle: every head
layout, length, page size and mask where it can go wrong; and the cache calls
and the attention run together as a generation loop runs them.  The tolerances
are derived in decode_cases.py."""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from oracle import decode as OD
from prefix_tree_block_gb300 import workloads as W

from decode_cases import cache_of, check, csr, pages_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


# trees: node lengths and paths
TREES = {
    "one token": ([1], [[0]]),
    "empty": ([0], [[0]]),
    "group": ([37, 1, 15, 16, 17, 0], [[0, i] for i in range(1, 6)]),
    "empty prompt": ([0, 5, 129], [[0, 1], [0, 2]]),
    "long": ([700, 300], [[0, 1]]),
    "deep": ([130, 31, 0, 64, 2, 3, 250, 1], [[0, 1, 4], [0, 1, 5], [0, 2, 6], [0, 3, 7], [0, 3], [0]]),
    "crowd": ([290] + [3 + 2 * (i % 7) for i in range(70)], [[0, i] for i in range(1, 71)]),
    "wide": ([1500, 260] + [1 + 9 * (i % 5) for i in range(150)], [[0, i] for i in range(2, 102)] + [[0, 1, i] for i in range(102, 152)]),
    "shared leaf": ([33, 20], [[0, 1], [0, 1], [1], [0]]),
    "unused rows, any order": ([8, 100, 9, 40, 3], [[4, 1], [4, 0]]),
}


def _run(lens, paths, Hq, Hkv, D, dtype, ps, q_len=1, q_count=None, scale=0.0, seed=0, width=None, poison=float("nan")):
    rng = np.random.default_rng(seed)
    tables, n_pages = pages_of(lens, ps, rng, width=width)
    Kc, Vc = cache_of(lens, tables, n_pages, Hkv, ps, D, dtype, seed, poison)
    g = torch.Generator().manual_seed(seed + 1)
    Q = torch.randn(len(paths) * q_len, Hq, D, generator=g).to(dtype)
    plan = pt.decode_plan(len(lens), *csr(paths), Hq, Hkv, q_len)
    O = torch.full(Q.shape, 7.0, dtype=dtype, device="cuda")
    L = torch.full((Hq, Q.shape[0]), 7.0, device="cuda")
    O, L = torch.full_like(O, 7.0), L
    cnt = None if q_count is None else torch.tensor(q_count, dtype=torch.int32, device="cuda")
    pt.attn_decode(Q.cuda(), Kc.cuda(), Vc.cuda(), torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                   plan, q_count=cnt, scale=scale, O=O, LSE=L)
    pt.sync_status()
    check(O.cpu(), L.cpu(), Q, Kc, Vc, tables, lens, paths, q_len, q_count, scale or None,
          untouched=(torch.full(Q.shape, 7.0, dtype=dtype), torch.full((Hq, Q.shape[0]), 7.0)))


@pytest.mark.parametrize("tree", TREES)
@pytest.mark.parametrize("Hq,Hkv,D,dtype,ps", [
    (2, 2, 32, F32, 16), (14, 2, 64, BF, 16), (16, 4, 128, BF, 32), (8, 2, 256, BF, 64), (3, 1, 80, F32, 7), (6, 2, 96, BF, 16),
])
def test_trees(tree, Hq, Hkv, D, dtype, ps):
    lens, paths = TREES[tree]
    _run(lens, paths, Hq, Hkv, D, dtype, ps, seed=3)
    if dtype == BF:  # tables wide enough for nodes that many rows read to take the tile kernel
        _run(lens, paths, Hq, Hkv, D, dtype, ps, seed=3, width=65536 // ps)


@pytest.mark.parametrize("D,dtype", [(1, F32), (31, F32), (33, F32), (66, F32), (128, F32), (130, F32), (256, F32), (257, F32), (512, F32),
                                     (8, BF), (64, BF), (72, BF), (104, BF), (128, BF), (200, BF), (256, BF), (264, BF), (512, BF)])
def test_head_dims(D, dtype):
    lens, paths = TREES["deep"]
    _run(lens, paths, 4, 2, D, dtype, 16, seed=D)


@pytest.mark.parametrize("ps", [1, 3, 8, 16, 48, 128, 256, 1024])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_page_sizes(ps, dtype):
    lens, paths = TREES["crowd"]
    _run(lens, paths, 4, 2, 64, dtype, ps, seed=ps)
    if dtype == BF:
        _run(lens, paths, 4, 2, 64, dtype, ps, seed=ps, width=-(-65536 // ps))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (32, 1), (71, 1), (8, 8), (7, 7), (24, 8), (40, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_head_layouts(Hq, Hkv, dtype):
    lens, paths = TREES["group"]
    _run(lens, paths, Hq, Hkv, 64, dtype, 16, seed=Hq)
    if dtype == BF:
        _run(lens, paths, Hq, Hkv, 64, dtype, 16, seed=Hq, width=4096)


@pytest.mark.parametrize("q_len", [2, 5, 16, 33])
@pytest.mark.parametrize("tree", ["group", "deep", "crowd", "shared leaf"])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 2, 64, BF), (8, 1, 128, BF), (2, 2, 64, F32)])
def test_several_queries(q_len, tree, Hq, Hkv, D, dtype):
    """Rows of a leaf shorter than q_len keep nothing of it at first."""
    lens, paths = TREES[tree]
    _run(lens, paths, Hq, Hkv, D, dtype, 16, q_len=q_len, seed=q_len)
    if dtype == BF:
        _run(lens, paths, Hq, Hkv, D, dtype, 16, q_len=q_len, seed=q_len, width=4096)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_len", [1, 4])
def test_query_counts(dtype, q_len):
    """Samples with fewer queries than q_len, or none: their rows stay."""
    lens, paths = TREES["crowd"]
    _run(lens, paths, 4, 2, 64, dtype, 16, q_len=q_len, q_count=[(i * 7) % (q_len + 1) for i in range(len(paths))], seed=2, width=4096)
    lens, paths = TREES["deep"]
    _run(lens, paths, 4, 2, 64, dtype, 16, q_len=q_len, q_count=[0] * len(paths), seed=2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("poison", [float("inf"), float("-inf"), 3e38])
def test_what_lies_behind_the_rows(dtype, poison):
    lens, paths = TREES["deep"]
    _run(lens, paths, 4, 2, 64, dtype, 16, seed=1, poison=poison)
    _run(lens, paths, 4, 2, 64, dtype, 16, q_len=3, seed=1, poison=poison)
    lens, paths = TREES["wide"]
    _run(lens, paths, 4, 2, 64, dtype, 16, seed=1, poison=poison)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq", [4, 32])
@pytest.mark.parametrize("what", ["K", "V"])
def test_a_later_drafts_nan_stays_with_it(dtype, Hq, what):
    """A token whose key or value is NaN reaches the queries that keep it only."""
    lens, paths, q_len, ps, D = [50, 40, 21], [[0, 1], [0, 2]], 6, 16, 64
    rng = np.random.default_rng(0)
    tables, n_pages = pages_of(lens, ps, rng, width=2048)
    Kc, Vc = cache_of(lens, tables, n_pages, 2, ps, D, dtype, 0)
    s = OD.slots_of(tables[1], 40, ps)[37]  # the third draft token of sample 0
    (Kc if what == "K" else Vc)[s // ps, :, s % ps] = float("nan")
    Q = torch.randn(12, Hq, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    plan = pt.decode_plan(3, *csr(paths), Hq, 2, q_len)
    O, L = pt.attn_decode(Q.cuda(), Kc.cuda(), Vc.cuda(), torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), plan)
    pt.sync_status()
    O = O.cpu().float()
    assert O[3:6].isnan().all() and not O[:3].isnan().any() and not O[6:].isnan().any()
    keep = list(range(3)) + list(range(6, 12))
    clean = [x.clone() for x in (Kc, Vc)]
    for c in clean:
        c[s // ps, :, s % ps] = 0
    o, _ = OD.attention(Q.float().numpy(), *(c.float().numpy() for c in clean), tables, lens, paths, q_len)
    assert np.abs(O.numpy()[keep] - o[keep]).max() < 0.1


def test_scale_and_large_scores():
    lens, paths = TREES["deep"]
    _run(lens, paths, 4, 2, 64, BF, 16, scale=0.01, seed=5)
    _run(lens, paths, 4, 2, 64, F32, 16, scale=2.5, seed=5)
    _run(lens, paths, 4, 2, 64, BF, 16, scale=2.5, seed=5)


def test_fused_query_rows_and_own_buffers():
    """Q inside a wider projection; O, LSE and workspace of the caller's."""
    lens, paths = TREES["group"]
    Hq, Hkv, D, ps = 4, 2, 64, 16
    tables, n_pages = pages_of(lens, ps, np.random.default_rng(1))
    Kc, Vc = cache_of(lens, tables, n_pages, Hkv, ps, D, BF, 1)
    qkv = torch.randn(len(paths), Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    Q = qkv[:, :Hq]
    plan = pt.decode_plan(len(lens), *csr(paths), Hq, Hkv)
    O, L = torch.empty(len(paths), Hq, D, dtype=BF, device="cuda"), torch.empty(Hq, len(paths), device="cuda")
    ws = torch.empty(plan.workspace_bytes(D), dtype=torch.uint8, device="cuda")
    pt.attn_decode(Q, Kc.cuda(), Vc.cuda(), torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), plan, O=O, LSE=L, workspace=ws)
    pt.sync_status()
    check(O.cpu(), L.cpu(), Q.cpu(), Kc, Vc, tables, lens, paths, 1)


@pytest.mark.parametrize("extra", [0, 2, 8])
def test_query_rows_between_16_byte_boundaries(extra):
    """A node that many rows read, with query tokens of every alignment allowed."""
    lens, paths = TREES["crowd"]
    Hq, Hkv, D, ps = 4, 2, 64, 16
    tables, n_pages = pages_of(lens, ps, np.random.default_rng(1), width=4096)
    Kc, Vc = cache_of(lens, tables, n_pages, Hkv, ps, D, BF, 1)
    x = torch.randn(len(paths), Hq * D + extra, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    Q = x.as_strided((len(paths), Hq, D), (Hq * D + extra, D, 1), extra)
    plan = pt.decode_plan(len(lens), *csr(paths), Hq, Hkv)
    O, L = pt.attn_decode(Q, Kc.cuda(), Vc.cuda(), torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), plan)
    pt.sync_status()
    check(O.cpu(), L.cpu(), Q.cpu(), Kc, Vc, tables, lens, paths, 1)


def test_many_rows():
    """Enough query rows that the merge takes several heads to a warp."""
    lens, paths = [300] + [20 + i % 9 for i in range(130)], [[0, i] for i in range(1, 131)]
    for Hq, Hkv, D, dtype in ((32, 4, 64, BF), (40, 4, 128, BF), (36, 12, 64, BF), (32, 8, 32, F32)):
        _run(lens, paths, Hq, Hkv, D, dtype, 16, seed=3)
    _run(lens, paths, 8, 2, 128, BF, 16, q_len=5, seed=3)


def test_far_pages():
    """Element offsets of the cache past 2^31."""
    Hkv, ps, D, n_pages = 8, 64, 128, 70000  # 4.6 G elements
    lens, paths = [70, 5], [[0, 1]]
    Kc = torch.empty(n_pages, Hkv, ps, D, dtype=BF, device="cuda")
    Vc = torch.empty_like(Kc)
    tables = np.array([[69999, 40000], [65000, -1]], np.int32)
    small, places = np.array([[0, 1], [2, -1]], np.int32), [69999, 40000, 65000]
    sk, sv = cache_of(lens, small, 3, Hkv, ps, D, BF, 3)
    for i, p in enumerate(places):
        Kc[p], Vc[p] = sk[i].cuda(), sv[i].cuda()
    Q = torch.randn(1, 16, D, generator=torch.Generator().manual_seed(2)).to(BF)
    plan = pt.decode_plan(2, *csr(paths), 16, Hkv)
    O, L = pt.attn_decode(Q.cuda(), Kc, Vc, torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), plan)
    pt.sync_status()
    check(O.cpu(), L.cpu(), Q, sk, sv, small, lens, paths, 1)


def test_many_nodes():
    """Thousands of segments: their sums span chunks."""
    rng = np.random.default_rng(7)
    lens = [int(x) for x in rng.integers(0, 40, 3000)]
    paths = [[i, 2000 + i % 1000] for i in range(0, 1500)]
    for dtype in (BF, F32):
        _run(lens, paths, 2, 1, 64, dtype, 16, seed=8)


@pytest.mark.parametrize("q_len,D", [(16, 128), (16, 64), (17, 128), (5, 128)])
def test_own_nodes_that_many_rows_read(q_len, D):
    """Continuations of several tiles, ends inside a tile, more of them than
    SMs: the tile kernel goes from one item to the next with its rings full.
    Twice the same."""
    rng = np.random.default_rng(6)
    lens = [1000] + [int(x) for x in rng.integers(130, 900, 40)]
    paths = [[0, i] for i in range(1, 41)]
    Hq, Hkv, ps = 32, 4, 32
    tables, n_pages = pages_of(lens, ps, rng, width=4096)
    Kc, Vc = (c.cuda() for c in cache_of(lens, tables, n_pages, Hkv, ps, D, BF, 1))
    Q = torch.randn(40 * q_len, Hq, D, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    plan = pt.decode_plan(len(lens), *csr(paths), Hq, Hkv, q_len)
    t, n = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    O, L = pt.attn_decode(Q, Kc, Vc, t, n, plan)
    for _ in range(4):
        o, l = pt.attn_decode(Q, Kc, Vc, t, n, plan)
        assert torch.equal(o, O) and torch.equal(l, L)
    pt.sync_status()
    some = [0, 7, 21, 39]  # (the oracle takes its time)
    rows = torch.tensor([s * q_len + j for s in some for j in range(q_len)])
    check(O.cpu()[rows], L.cpu()[:, rows], Q.cpu()[rows], Kc.cpu(), Vc.cpu(), tables, lens, [paths[s] for s in some], q_len)


def test_samples_that_end_at_one_node():
    """Only nodes that many rows read: no work for the other kernel."""
    _run([700], [[0]] * 80, 4, 2, 128, BF, 16, seed=4, width=8192)
    _run([700], [[0]] * 80, 4, 2, 128, BF, 16, q_len=3, seed=4, width=8192)
    _run([300, 5], [[0, 1]] * 300, 2, 1, 64, BF, 16, seed=4, width=32768)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_to_do(dtype):
    """No samples; tables without a column; as many nodes as there may be."""
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    plan = pt.decode_plan(3, [0], [], 4, 2)
    O, L = pt.attn_decode(z(0, 4, 64, t=dtype), z(1, 2, 16, 64, t=dtype), z(1, 2, 16, 64, t=dtype), z(3, 2), z(3), plan)
    assert O.shape == (0, 4, 64) and L.shape == (4, 0)
    plan = pt.decode_plan(2, [0, 2], [0, 1], 4, 2)
    O, L = pt.attn_decode(z(1, 4, 64, t=dtype), z(1, 2, 16, 64, t=dtype), z(1, 2, 16, 64, t=dtype), z(2, 0), z(2), plan)
    pt.sync_status()
    assert not O.any() and torch.isneginf(L).all()
    lens = [0] * (1 << 16)
    lens[5], lens[40000], lens[65535] = 40, 33, 7
    _run(lens, [[5, 40000], [65535], [40000]], 4, 2, 64, dtype, 16, seed=1)


def test_too_much_work_is_refused():
    """Work items times the tiles of a full table row past 2^31."""
    n = 1 << 15
    plan = pt.decode_plan(n, np.arange(n + 1), np.arange(n), 16, 16)
    t = torch.zeros(n, 1 << 4, dtype=torch.int32, device="cuda")
    Kc = torch.zeros(1, 16, 1 << 14, 64, dtype=BF, device="cuda")
    with pytest.raises(pt.PTError) as e:
        pt.attn_decode(torch.zeros(n, 16, 64, dtype=BF, device="cuda"), Kc, Kc, t, torch.zeros(n, dtype=torch.int32, device="cuda"), plan)
    assert e.value.status == pt.PT_ERR_UNSUPPORTED


def test_two_calls_at_once():
    """Two streams, each with its own workspace, over one cache and one plan."""
    lens, paths = [2500] + [40 + i for i in range(40)], [[0, i] for i in range(1, 41)]
    tables, n_pages = pages_of(lens, 64, np.random.default_rng(1), width=2048)
    Kc, Vc = (c.cuda() for c in cache_of(lens, tables, n_pages, 2, 64, 128, BF, 1))
    plan = pt.decode_plan(len(lens), *csr(paths), 16, 2)
    t, n = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    Q = [torch.randn(40, 16, 128, generator=torch.Generator().manual_seed(i)).to(BF).cuda() for i in range(2)]
    want = [pt.attn_decode(q, Kc, Vc, t, n, plan) for q in Q]
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = [pt.attn_decode(q, Kc, Vc, t, n, plan, stream=s) for q, s in zip(Q, side)]
    torch.cuda.synchronize()
    pt.sync_status()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_result_each_time(dtype):
    lens, paths = [3000] + [50 + i for i in range(20)], [[0, i] for i in range(1, 21)]  # (the prompt: 140 rows)
    tables, n_pages = pages_of(lens, 16, np.random.default_rng(1))
    Kc, Vc = (c.cuda() for c in cache_of(lens, tables, n_pages, 2, 16, 64, dtype, 1))
    Q = torch.randn(20, 14, 64, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    plan = pt.decode_plan(len(lens), *csr(paths), 14, 2)
    t, n = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    O, L = pt.attn_decode(Q, Kc, Vc, t, n, plan)
    for _ in range(5):
        o, l = pt.attn_decode(Q, Kc, Vc, t, n, plan)
        assert torch.equal(o, O) and torch.equal(l, L)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, l = pt.attn_decode(Q, Kc, Vc, t, n, plan, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, O) and torch.equal(l, L)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_pages_lengths_and_counts_are_recorded(dtype):
    """The kernels check each page id, length and count before they use it."""
    lens, paths, ps = [40, 20], [[0, 1], [0]], 16
    tables, n_pages = pages_of(lens, ps, np.random.default_rng(1))
    Kc, Vc = (c.cuda() for c in cache_of(lens, tables, n_pages, 2, ps, 64, dtype, 1, poison=0.0))
    Q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    plan = pt.decode_plan(2, *csr(paths), 4, 2)
    good = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def go(t, n, c=None):
        pt.attn_decode(Q, Kc, Vc, t, n, plan, q_count=c)
        with pytest.raises(pt.PTError) as e:
            pt.sync_status()
        assert e.value.status == pt.PT_ERR_INVALID_ARG

    for bad in (-1, n_pages, 1 << 30):
        t = good[0].clone()
        t[1, 0] = bad
        go(t, good[1])
    for bad in (-5, 49, 1 << 30):
        n = good[1].clone()
        n[0] = bad
        if bad > 0:
            go(torch.zeros_like(good[0]), n)
        else:
            go(good[0], n)
    for bad in (-1, 2):
        go(*good, torch.tensor([1, bad], dtype=torch.int32, device="cuda"))
    pt.attn_decode(Q, Kc, Vc, *good, plan)
    pt.sync_status()


def test_binding_refusals():
    lens, paths = TREES["group"]
    plan = pt.decode_plan(len(lens), *csr(paths), 4, 2)
    z = lambda *s, t=BF: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    Q, Kc, tb, n = z(5, 4, 64), z(3, 2, 16, 64), z(6, 3, t=torch.int32), z(6, t=torch.int32)
    for args in [(z(4, 4, 64), Kc, Kc, tb, n), (z(5, 2, 64), Kc, Kc, tb, n), (Q, z(3, 4, 16, 64), z(3, 4, 16, 64), tb, n),
                 (Q, Kc, z(4, 2, 16, 64), tb, n), (Q, Kc, Kc, z(5, 3, t=torch.int32), n), (Q, Kc, Kc, tb, z(5, t=torch.int32))]:
        with pytest.raises(ValueError):
            pt.attn_decode(*args, plan)
    for args in [(Q.float(), Kc, Kc, tb, n), (Q, Kc, Kc, tb.long(), n), (Q, Kc, Kc, tb, n.long()), (Q.half(), Kc.half(), Kc.half(), tb, n)]:
        with pytest.raises(TypeError):
            pt.attn_decode(*args, plan)
    with pytest.raises(pt.PTError) as e:
        pt.attn_decode(Q, Kc, Kc, tb, n, plan, workspace=z(256, t=torch.uint8))
    assert e.value.status == pt.PT_ERR_INVALID_ARG
    with pytest.raises(pt.PTError) as e:
        pt.attn_decode(z(5, 4, 513, t=F32), z(3, 2, 16, 513, t=F32), z(3, 2, 16, 513, t=F32), tb, n, plan)
    assert e.value.status == pt.PT_ERR_UNSUPPORTED
    with pytest.raises(pt.PTError) as e:
        pt.attn_decode(z(5, 4, 60), z(3, 2, 16, 60), z(3, 2, 16, 60), tb, n, plan)
    assert e.value.status == pt.PT_ERR_UNSUPPORTED


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(14, 2, 64, BF), (16, 4, 128, BF), (8, 2, 256, BF), (2, 2, 32, F32)])
def test_agrees_with_the_tree_forward(Hq, Hkv, D, dtype):
    """A flat tree's keys and values put into the cache; the decoding of every
    sample's last token gives the forward's row (each off its exact value by
    its own tolerance, so by both from each other)."""
    st = W.grpo_structure([(300, [40, 1, 129]), (0, [64]), (17, [200, 3])])
    q, k, v, _ = (x.cuda() for x in W.make_tensors(st.T, Hq, Hkv, D, "bf16" if dtype == BF else "f32", seed=4))
    bm = pt.build_blockmap_tree(st.node_lengths, st.path_ptr, st.path_nodes)
    O, L = pt.attn_fwd(q, k, v, bm)
    ps, n = 16, st.n_nodes
    n_pages = int((-(-st.node_lengths // ps)).sum())
    zero = torch.zeros(n, dtype=torch.int32, device="cuda")
    lens = torch.from_numpy(st.node_lengths).cuda()
    tables = torch.full((n, 24), -1, dtype=torch.int32, device="cuda")
    ring = torch.randperm(n_pages, device="cuda").int()
    got, ctr, ptr, slots, pos = pt.cache_tables(zero, lens, tables, ring, torch.tensor([0, n_pages], device="cuda"), ps, st.T)
    Kc, Vc = (torch.full((n_pages, Hkv, ps, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    pt.cache_write(k, v, slots, Kc, Vc)
    paths = st.paths()
    last = torch.tensor([int(st.node_lengths[:p[-1] + 1].sum()) - 1 for p in paths], device="cuda")
    plan = pt.decode_plan(n, st.path_ptr, st.path_nodes, Hq, Hkv)
    o, l = pt.attn_decode(q[last], Kc, Vc, tables, got, plan)
    pt.sync_status()
    assert torch.equal(got, lens) and ctr.tolist() == [n_pages, n_pages]
    tol = 2e-2 if dtype == BF else 1e-5  # the forward's (parity.FWD_ATOL), against which the other is small
    assert float((o.float() - O[last].float()).abs().max()) <= 2 * tol
    assert float((l - L[:, last]).abs().max()) <= (4e-3 if dtype == BF else 2e-5)


@pytest.mark.parametrize("dtype,q_len", [(BF, 1), (BF, 2), (F32, 1)])
def test_a_captured_generation_loop(dtype, q_len):
    """One step (tables, write, attention, the lengths carried over) captured
    once and replayed: completions cross page boundaries, one joins late and one
    ends early.  Two graphs share the workspace and the cache in turn."""
    Hq, Hkv, D, ps, S, steps = 4, 2, 64, 16, 3, 22
    paths = [[0, 1], [0, 2], [0, 3]]
    n, n_pages = 4, 24
    g = torch.Generator().manual_seed(9)
    dev = lambda x: x.cuda()  # noqa: E731
    held = torch.zeros(n, dtype=torch.int32, device="cuda")
    ctr = torch.tensor([0, n_pages], device="cuda")
    ring = torch.randperm(n_pages, generator=g).int().cuda()
    tables = torch.full((n, 6), -1, dtype=torch.int32, device="cuda")
    Kc, Vc = (torch.full((n_pages, Hkv, ps, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    start = torch.tensor([0, 45, 45, 45], dtype=torch.int32, device="cuda")
    # the prompt goes in at once
    K0, V0 = (torch.randn(45, Hkv, D, generator=g).to(dtype).cuda() for _ in range(2))
    lens, ctr, _, slots, _ = pt.cache_tables(held, torch.tensor([45, 0, 0, 0], dtype=torch.int32, device="cuda"), tables, ring, ctr, ps, 45, start=start)
    pt.cache_write(K0, V0, slots, Kc, Vc)
    held.copy_(lens)
    plan = pt.decode_plan(n, *csr(paths), Hq, Hkv, q_len)
    ws = torch.empty(plan.workspace_bytes(D), dtype=torch.uint8, device="cuda")
    added = torch.zeros(n, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(S, dtype=torch.int32, device="cuda")
    M = S * q_len
    Q, K, V = (torch.zeros(M, h, D, dtype=dtype, device="cuda") for h in (Hq, Hkv, Hkv))
    O, L = torch.zeros(M, Hq, D, dtype=dtype, device="cuda"), torch.zeros(Hq, M, device="cuda")
    said = {}

    def step():
        lens, c, ptr, slots, pos = pt.cache_tables(held, added, tables, ring, ctr, ps, M, start=start)
        pt.cache_write(K, V, slots, Kc, Vc)
        pt.attn_decode(Q, Kc, Vc, tables, lens, plan, q_count=cnt, O=O, LSE=L, workspace=ws)
        held.copy_(lens)
        ctr.copy_(c)
        said.update(slots=slots, pos=pos)

    step()  # warm: nothing is added yet
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        graphs.append((gr, dict(said)))
    mirror = [[(K0[t].cpu(), V0[t].cpu()) for t in range(45)], [], [], []]
    for i in range(steps):
        live = [1 if (s != 2 or i >= 5) and (s != 1 or i < 17) else 0 for s in range(S)]
        add = [0] + [q_len * x for x in live]
        if i == 17:
            add[2] = -len(mirror[2])  # sample 1 ends: its pages go back
            mirror[2] = []
        k, v, q = (torch.randn(M, h, D, generator=g).to(dtype) for h in (Hkv, Hkv, Hq))
        at = 0
        for s in range(S):
            for _ in range(q_len * live[s]):
                mirror[s + 1].append((k[at], v[at]))
                at += 1
        for dst, src in ((added, torch.tensor(add, dtype=torch.int32)), (cnt, torch.tensor([q_len * x for x in live], dtype=torch.int32)), (K, k), (V, v), (Q, q)):
            dst.copy_(src)
        O.fill_(7), L.fill_(7)
        gr, out = graphs[i % 2]
        gr.replay()
        pt.sync_status()
        ln = [len(m) for m in mirror]
        assert held.tolist() == ln
        tb = tables.cpu().numpy()
        used = np.concatenate([tb[r, :-(-ln[r] // ps)] for r in range(n)])
        assert len(set(used.tolist())) == used.size
        assert out["slots"].tolist()[at:] == [-1] * (M - at)
        kc, vc = Kc.cpu(), Vc.cpu()
        for r in range(n):
            s = torch.from_numpy(OD.slots_of(tb[r], ln[r], ps))
            if ln[r]:
                assert torch.equal(kc[s // ps, :, s % ps], torch.stack([m[0] for m in mirror[r]]))
        check(O.cpu(), L.cpu(), q, kc, vc, tb, ln, paths, q_len, [q_len * x for x in live],
              untouched=(torch.full(O.shape, 7.0, dtype=dtype), torch.full(L.shape, 7.0)))
    assert int(ctr[1] - ctr[0]) == n_pages - used.size
