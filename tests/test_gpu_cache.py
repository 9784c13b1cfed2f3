"""The paged cache's calls (pt_cache_tables, pt_cache_write) against the oracle,
bit for bit: they only count and copy."""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from oracle import decode as OD

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


def _mix(n, most, ps, seed, kinds=(0.3, 0.3, 0.1, 0.1)):
    """held, added, tables, ring, counters: a step with growing, new, ending
    and shrinking rows (shares of the rows), a ring that wraps."""
    rng = np.random.default_rng(seed)
    held = rng.integers(0, most + 1, n)
    added = np.zeros(n, np.int64)
    u = rng.random(n)
    edges = np.cumsum(kinds)
    for i in range(n):
        if u[i] < edges[0]:
            added[i] = min(int(rng.integers(1, 4)), most - held[i])
        elif u[i] < edges[1]:
            held[i], added[i] = 0, int(rng.integers(0, most + 1))
        elif u[i] < edges[2]:
            added[i] = -held[i]
        elif u[i] < edges[3]:
            added[i] = -int(rng.integers(0, held[i] + 1))
    pages = -(-held // ps)
    width = max(1, -(-most // ps))
    cap = int(pages.sum() + np.maximum(-(-(held + added) // ps) - pages, 0).sum() + 5)
    ids = rng.permutation(cap).astype(np.int32)
    tables = np.full((n, width), -7, np.int32)
    tables[np.arange(width) < pages[:, None]] = ids[:pages.sum()]
    free = ids[pages.sum():]
    head = int(rng.integers(0, 3 * cap)) + (1 << 33)  # the counters run past 32 bits
    ring = np.full(cap, -9, np.int32)
    ring[(head + np.arange(free.size)) % cap] = free
    return held, added, tables, ring, np.array([head, head + free.size], np.int64), rng.integers(0, 100000, n)


def _run(held, added, tables, ring, counters, ps, max_new, start=None):
    c = lambda x, t=torch.int32: torch.from_numpy(np.ascontiguousarray(x)).to("cuda", t)  # noqa: E731
    t, r = c(tables), c(ring)
    out = pt.cache_tables(c(held), c(added), t, r, c(counters, torch.int64), ps, max_new,
                          start=None if start is None else c(start))
    return [x.cpu().numpy() for x in (*out, t, r)]


def _same(got, want):
    for name, g, w in zip(("lens", "counters", "row_ptr", "slots", "positions", "tables", "ring"), got, want):
        np.testing.assert_array_equal(g, w, err_msg=name)


@pytest.mark.parametrize("n,most,ps", [(1, 1, 1), (1, 40, 16), (31, 9, 4), (32, 100, 16), (33, 100, 7), (513, 70, 16), (1500, 300, 32),
                                       (4500, 20, 16), (70, 20000, 64)])
@pytest.mark.parametrize("pad", [0, 1, 3000])
def test_step(n, most, ps, pad):
    held, added, tables, ring, ctr, start = _mix(n, most, ps, seed=n + most + pad)
    new = int(np.maximum(added, 0).sum()) + pad
    _same(_run(held, added, tables, ring, ctr, ps, new, start), OD.step(held, added, start, tables, ring, ctr, ps, new))
    pt.sync_status()
    _same(_run(held, added, tables, ring, ctr, ps, new), OD.step(held, added, start * 0, tables, ring, ctr, ps, new))
    pt.sync_status()


def test_no_rows():
    e = np.zeros(0, np.int32)
    got = _run(e, e, np.zeros((0, 4), np.int32), np.arange(3, dtype=np.int32), np.array([1, 3]), 16, 5)
    assert got[1].tolist() == [1, 3] and got[2].tolist() == [0] and got[3].tolist() == [-1] * 5 and got[4].tolist() == [0] * 5
    pt.sync_status()


def test_many_rows():
    """More rows than 48 KB of chunk sums."""
    n = 140000
    held, added = np.full(n, 5, np.int64), (np.arange(n) % 3 == 0).astype(np.int64) * 12
    tables = np.stack([np.arange(n), np.full(n, -1)], 1).astype(np.int32)
    free = np.arange(n, 2 * n, dtype=np.int32)
    new = int(added.sum())
    got = _run(held, added, tables, free, np.array([0, n]), 16, new)
    _same(got, OD.step(held, added, held * 0, tables, free, [0, n], 16, new))
    pt.sync_status()


@pytest.mark.parametrize("avail", [0, 1, 5, 11])
def test_out_of_pages(avail):
    held, added = np.array([0, 4, 7, 0, 16]), np.array([9, 1, 30, 3, -16])
    tables = np.full((5, 12), -1, np.int32)
    tables[1, 0], tables[2, :2], tables[4, :4] = 50, [51, 52], [53, 54, 55, 56]
    ring = np.full(24, -9, np.int32)
    ring[3:3 + avail] = np.arange(avail)
    want = OD.step(held, added, held * 0, tables, ring, [3, 3 + avail], 4, 50)
    got = _run(held, added, tables, ring, np.array([3, 3 + avail]), 4, 50)
    _same(got, want)
    with pytest.raises(pt.PTError) as e:
        pt.sync_status()
    assert e.value.status == pt.PT_ERR_NOMEM
    pt.sync_status()


def test_bad_rows_stay():
    held, added = np.array([5, -3, 30, 9, 33]), np.array([1, 4, 3, -10, -1])
    tables = np.arange(10, dtype=np.int32).reshape(5, 2)
    got = _run(held, added, tables, np.arange(20, 28, dtype=np.int32), np.array([0, 4]), 16, 9)
    assert got[0].tolist() == [6, 0, 30, 9, 32]  # clamped into the table's range
    assert got[1].tolist() == [0, 4] and got[2].tolist() == [0, 1, 1, 1, 1, 1]
    assert got[3].tolist() == [5] + [-1] * 8
    np.testing.assert_array_equal(got[5], tables)
    with pytest.raises(pt.PTError) as e:
        pt.sync_status()
    assert e.value.status == pt.PT_ERR_INVALID_ARG


@pytest.mark.parametrize("ctr", [(4, 3), (-2, 1), (0, 9)])
def test_bad_counters(ctr):
    got = _run(np.array([0, 5]), np.array([3, 1]), np.full((2, 2), 1, np.int32), np.arange(8, dtype=np.int32), np.array(ctr), 4, 4)
    assert got[1].tolist() == list(ctr) and got[3].tolist()[:3] == [-1] * 3
    with pytest.raises(pt.PTError):
        pt.sync_status()
    pt.sync_status()


def test_more_tokens_than_slots():
    held, added, tables, ring, ctr, start = _mix(40, 50, 16, seed=4)
    new = int(np.maximum(added, 0).sum())
    want = OD.step(held, added, start, tables, ring, ctr, 16, new)
    got = _run(held, added, tables, ring, ctr, 16, new - 7, start)
    _same([got[i] for i in (0, 1, 2, 5, 6)], [want[i] for i in (0, 1, 2, 5, 6)])
    np.testing.assert_array_equal(got[3], want[3][:new - 7])
    np.testing.assert_array_equal(got[4], want[4][:new - 7])
    with pytest.raises(pt.PTError):
        pt.sync_status()


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


@pytest.mark.parametrize("dtype,T,Hkv,D,ps", [
    (torch.bfloat16, 1, 2, 64, 16), (torch.bfloat16, 37, 8, 128, 64), (torch.bfloat16, 1000, 3, 72, 32), (torch.bfloat16, 70, 2, 5, 7),
    (torch.float32, 300, 2, 256, 16), (torch.float32, 65, 1, 33, 1), (torch.bfloat16, 9, 1, 520, 16), (torch.bfloat16, 3000, 16, 256, 16),
])
@pytest.mark.parametrize("fused", [False, True])
def test_write(dtype, T, Hkv, D, ps, fused):
    rng = np.random.default_rng(T)
    n_pages = -(-T // ps) + 4
    slots = rng.permutation(n_pages * ps)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    slots[T - 1] = -(1 << 40)
    if fused:  # the heads of K and V inside one projection's rows
        x = _rand((T, 3 + 2 * Hkv, D), dtype, 1).cuda()
        K, V = x[:, 2:2 + Hkv], x[:, 2 + Hkv:2 + 2 * Hkv]
    else:
        K, V = _rand((T, Hkv, D), dtype, 1).cuda(), _rand((T, Hkv, D), dtype, 2).cuda()
    Kc, Vc = _rand((n_pages, Hkv, ps, D), dtype, 3), _rand((n_pages, Hkv, ps, D), dtype, 4)
    f = lambda x: x.cpu().float().numpy()  # noqa: E731
    wk, wv = OD.write(f(K), f(V), slots, f(Kc), f(Vc))
    kc, vc = Kc.cuda(), Vc.cuda()
    pt.cache_write(K, V, torch.from_numpy(slots).cuda(), kc, vc)
    pt.sync_status()
    np.testing.assert_array_equal(f(kc), wk)
    np.testing.assert_array_equal(f(vc), wv)


def test_write_unaligned_rows():
    """Tokens that start between 16-byte boundaries take narrower copies."""
    x = _rand((20, 2 * 16 + 1), torch.bfloat16, 5).cuda()
    K, V = (x[:, 1:].as_strided((20, 2, 8), (33, 8, 1), o) for o in (1, 17))
    kc = torch.zeros(2, 2, 16, 8, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.arange(5, 25, device="cuda")
    pt.cache_write(K, V, slots, kc, vc)
    pt.sync_status()
    assert torch.equal(kc.transpose(1, 2).reshape(32, 2, 8)[5:25], K) and torch.equal(vc.transpose(1, 2).reshape(32, 2, 8)[5:25], V)


def test_write_beyond_the_cache():
    K = _rand((3, 2, 8), torch.float32, 1).cuda()
    kc = torch.zeros(2, 2, 4, 8, device="cuda")
    vc = torch.zeros_like(kc)
    pt.cache_write(K, K, torch.tensor([8, 1, 1 << 40], device="cuda"), kc, vc)
    with pytest.raises(pt.PTError) as e:
        pt.sync_status()
    assert e.value.status == pt.PT_ERR_INVALID_ARG
    assert torch.equal(kc[0, :, 1], K[1]) and int((kc != 0).sum()) == 16


def test_write_far_slots():
    """Element offsets past 2^31."""
    kc = torch.empty(1, 1, 1 << 17, 1 << 15, dtype=torch.bfloat16, device="cuda")  # 2^32 elements
    vc = torch.empty_like(kc)
    K, V = _rand((2, 1, 1 << 15), torch.bfloat16, 1).cuda(), _rand((2, 1, 1 << 15), torch.bfloat16, 2).cuda()
    pt.cache_write(K, V, torch.tensor([(1 << 17) - 1, 70000], device="cuda"), kc, vc)
    pt.sync_status()
    assert torch.equal(kc[0, 0, -1], K[0, 0]) and torch.equal(vc[0, 0, 70000], V[1, 0])


def test_binding_refusals():
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    c = z(2, t=torch.int64)
    with pytest.raises(ValueError):
        pt.cache_tables(z(4), z(3), z(4, 2), z(8), c, 16, 4)
    with pytest.raises(ValueError):
        pt.cache_tables(z(4), z(4), z(3, 2), z(8), c, 16, 4)
    with pytest.raises(TypeError):
        pt.cache_tables(z(4, t=torch.int64), z(4), z(4, 2), z(8), c, 16, 4)
    with pytest.raises(pt.PTError):
        pt.cache_tables(z(4), z(4), z(4, 2), z(0), c, 16, 4)
    k = z(4, 2, 8, t=torch.float32)
    with pytest.raises(ValueError):
        pt.cache_write(k, k, z(4, t=torch.int64), z(1, 2, 4, 9, t=torch.float32), z(1, 2, 4, 9, t=torch.float32))
    with pytest.raises(ValueError):
        pt.cache_write(k.transpose(1, 2).contiguous().transpose(1, 2), k, z(4, t=torch.int64), z(1, 2, 4, 8, t=torch.float32), z(1, 2, 4, 8, t=torch.float32))
    with pytest.raises(TypeError):
        pt.cache_write(k, k, z(4), z(1, 2, 4, 8, t=torch.float32), z(1, 2, 4, 8, t=torch.float32))
