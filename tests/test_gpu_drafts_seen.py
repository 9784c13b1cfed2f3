"""What the drafts that see a token get of it: keys and values that are not finite
reach all of them, large finite values count; and the calls' streams and masks'
alignment."""
import ctypes

import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from oracle import decode as OD
from oracle import tokens as OT

from decode_cases import cache_of, csr, pages_of
from test_gpu_drafts import BF, F32, attend, compare, counts_of, i32, parents_of, sees_of

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


UP = np.array([[-1, -1, 0, 1, 2, 3], [-1, 0, 1, 2, 3, 4]])
SEEN = [2, 4]  # the rows of the two samples that see draft 2 of the first

# the row kernel and the tile kernel (wide tables; rows for one warpgroup, and for both), CUDA cores
KERNELS = [(BF, 64, 8, 2, None), (BF, 64, 16, 1, 4096), (BF, 128, 40, 1, 4096), (BF, 256, 8, 2, None), (BF, 512, 2, 1, None), (F32, 64, 8, 2, None), (F32, 33, 3, 3, None)]


def run(dtype, D, Hq, Hkv, width, what, value, own=40):
    lens, paths = [50, own, 21], [[0, 1], [0, 2]]

    def edit(Kc, Vc, tables):
        s = OD.slots_of(tables[1], own, 16)[own - 6 + 2]
        (Kc, Vc)[what][s // 16, :, s % 16] = value

    return (lens, paths), attend(lens, paths, Hq, Hkv, D, dtype, 16, 6, UP, None, width=width, edit=edit)


@pytest.mark.parametrize("dtype,D,Hq,Hkv,width", KERNELS)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("own", [6, 40, 259])
def test_keys_that_are_not_finite(dtype, D, Hq, Hkv, width, value, own):
    """Every column and LSE of every row and head that sees the key is NaN (an
    infinite key's products have both signs), and of no other."""
    _, (O, L, *_) = run(dtype, D, Hq, Hkv, width, 0, value, own)
    hit = torch.zeros(12, dtype=torch.bool)
    hit[SEEN] = True
    assert O[hit].isnan().all() and L[:, hit].isnan().all()
    assert O[~hit].isfinite().all() and L[:, ~hit].isfinite().all()


@pytest.mark.parametrize("dtype,D,Hq,Hkv,width", KERNELS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("own", [6, 40, 259])
def test_values_that_are_not_finite(dtype, D, Hq, Hkv, width, value, own):
    _, (O, L, *_) = run(dtype, D, Hq, Hkv, width, 1, value, own)
    hit = torch.zeros(12, dtype=torch.bool)
    hit[SEEN] = True
    assert (O[hit].isnan() if value != value else O[hit] == value).all()
    assert O[~hit].isfinite().all() and L.isfinite().all()


@pytest.mark.parametrize("dtype,D,Hq,Hkv,width", KERNELS)
@pytest.mark.parametrize("own", [6, 40, 259])
def test_large_values(dtype, D, Hq, Hkv, width, own):
    """A value of 1e30 counts by its weight in the rows that see it (tolerances: by the
    magnitudes summed), and not at all in the others."""
    (lens, paths), got = run(dtype, D, Hq, Hkv, width, 1, 1e30, own)
    compare(*got, lens, paths, 6, sees_of(UP, 6), None)


@pytest.mark.parametrize("q", [1, 33, 40, 64])
def test_masks_at_any_word(q):
    """A mask that starts on four bytes, not eight, with two words a row too."""
    S = 9
    up, c = parents_of(S, q, "any", q), counts_of(S, q, q)
    lens = np.random.default_rng(q).integers(q, 1000, S)
    plan = pt.decode_plan(S, *csr([[s] for s in range(S)]), 1, 1, q)
    w = -(-q // 32)
    buf = torch.full((S * q * w + 3,), 77, dtype=torch.int32, device="cuda")
    pos = torch.empty(S * q, dtype=torch.int64, device="cuda")
    mask = buf[1:1 + S * q * w]
    assert mask.data_ptr() % 8 == 4
    keep = i32(up.reshape(-1)), i32(lens), i32(c)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = pt.load_library().pt_draft_tree(p(keep[0]), p(keep[1]), p(keep[2]), None, plan.handle, p(mask), p(pos),
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == pt.PT_OK
    pt.sync_status()
    want = OT.draft_tree(up, c, lens - c)
    np.testing.assert_array_equal(mask.view(S * q, w).cpu().numpy(), want[0])
    np.testing.assert_array_equal(pos.cpu().numpy(), want[1])
    assert buf[[0, -2, -1]].tolist() == [77, 77, 77]


@pytest.mark.parametrize("q", [8, 100])
def test_streams(q):
    """draft_tree and cache_keep on a stream that is given, not the current one: each behind what that
    stream still has to do to its inputs."""
    pt.set_output_allocator(None)  # (it fills its outputs on the current stream)
    S, ps = 6, 16
    up, c = parents_of(S, q, "any", q), np.full(S, q)
    lens = np.random.default_rng(q).integers(q, q + 40, S)
    tables, n_pages = pages_of(lens, ps, np.random.default_rng(1))
    Kc, Vc = cache_of(lens, tables, n_pages, 2, ps, 64, BF, 2, poison=9.0)
    plan = pt.decode_plan(S, *csr([[s] for s in range(S)]), 2, 2, q)
    kept = np.where(np.arange(q) < q // 2, np.arange(q) + q // 2, -1)[None].repeat(S, 0)
    real, real_kept, tab, n = i32(up.reshape(-1)), i32(kept), i32(tables), i32(lens)
    parents, moves, k, v = torch.full_like(real, -1), torch.full_like(real_kept, -1), Kc.cuda(), Vc.cuda()
    busy = torch.randn(4096, 4096, device="cuda", dtype=BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 0.01
        parents.copy_(real)
        moves.copy_(real_kept)
    mask, pos = pt.draft_tree(parents, n, plan, stream=side)
    pt.cache_keep(moves, k, v, tab, n, plan, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    pt.sync_status()
    want = OT.draft_tree(up, c, lens - c)
    np.testing.assert_array_equal(mask.cpu().numpy(), want[0])
    np.testing.assert_array_equal(pos.cpu().numpy(), want[1])
    for got, old in ((k, Kc), (v, Vc)):
        np.testing.assert_array_equal(got.float().cpu().numpy(), OT.keep(kept, c, lens, range(S), tables, ps, old.float().numpy()))
