"""The decoding oracle (oracle/decode.py) against the tree oracle and by hand."""
import numpy as np

from oracle import decode as OD
from oracle import oracle as orc
from prefix_tree_block_gb300 import workloads as W

from decode_cases import cache_of, pages_of
import torch


def test_step_by_hand():
    # pages of 4; row 0 grows 3 -> 5 (one page more), row 1 ends, row 2 starts with 6, row 3 loses 1 of 9
    tables = np.array([[7, -1, -1], [5, 6, -1], [-1, -1, -1], [1, 2, 3]], np.int32)
    ring = np.array([4, 9, 0, 8, 77, 77, 77], np.int32)
    lens, ctr, ptr, slots, pos, t2, r2 = OD.step([3, 6, 0, 9], [2, -6, 6, -1], [10, 0, 0, 0], tables, ring, [7, 11], 4, 10)
    assert lens.tolist() == [5, 0, 6, 8] and ctr.tolist() == [10, 14] and ptr.tolist() == [0, 2, 2, 8, 8]
    assert t2.tolist() == [[7, 4, -1], [5, 6, -1], [9, 0, -1], [1, 2, 3]]
    assert r2.tolist() == [4, 9, 0, 8, 5, 6, 3]
    assert slots.tolist() == [31, 16, 36, 37, 38, 39, 0, 1, -1, -1]
    assert pos.tolist() == [13, 14, 0, 1, 2, 3, 4, 5, 0, 0]


def test_step_out_of_pages():
    lens, ctr, ptr, slots, pos, t2, r2 = OD.step([0, 4], [9, 1], [0, 0], np.full((2, 3), -1, np.int32),
                                                 np.array([5, 6], np.int32), [0, 2], 4, 10)
    assert lens.tolist() == [8, 4] and ctr.tolist() == [2, 2] and ptr.tolist() == [0, 9, 10]
    assert slots.tolist() == [20, 21, 22, 23, 24, 25, 26, 27, -1, -1]


def test_attention_is_the_tree_attention():
    """The newest tokens' rows of the forward over the flat tree."""
    rng = np.random.default_rng(3)
    for case in range(6):
        st = W.random_tree(rng, int(rng.integers(2, 9)), 12, p_zero=0.2)
        Hq, Hkv, D, ps = 4, 2, 8, 4
        q, k, v, _ = W.make_tensors(st.T, Hq, Hkv, D, "f32", seed=case)
        O, L = orc.attn_fwd(q, k, v, orc.structure_labels(st))
        off = np.concatenate([[0], np.cumsum(st.node_lengths)])
        tables, n_pages = pages_of(st.node_lengths, ps, rng)
        Kc, Vc = (c.numpy() for c in cache_of(st.node_lengths, tables, n_pages, Hkv, ps, D, torch.float32, 0))
        for i, n in enumerate(st.node_lengths):
            Kc, Vc = OD.write(k[off[i]:off[i] + n].numpy(), v[off[i]:off[i] + n].numpy(),
                              OD.slots_of(tables[i], int(n), ps), Kc, Vc)
        paths = [p for p in st.paths() if st.node_lengths[p[-1]] >= 2]
        if not paths:
            continue
        last = np.concatenate([off[p[-1] + 1] - 2 + np.arange(2) for p in paths])
        o, l = OD.attention(q[last].numpy(), Kc, Vc, tables, st.node_lengths, paths, 2)
        np.testing.assert_allclose(o, O[last], atol=1e-12)
        np.testing.assert_allclose(l, L[:, last], atol=1e-12)


def test_attention_of_nothing_and_of_few():
    tables, n_pages = pages_of([0, 2], 4, np.random.default_rng(0))
    Kc, Vc = (c.numpy() for c in cache_of([0, 2], tables, n_pages, 1, 4, 4, torch.float32, 1))
    Q = np.ones((4, 1, 4))
    o, l = OD.attention(Q, Kc, Vc, tables, [0, 2], [[0], [0, 1]], 2, [2, 1])
    assert np.array_equal(o[:2], np.zeros((2, 1, 4))) and np.isneginf(l[0, :2]).all()
    assert np.isfinite(o[2]).all() and np.isnan(o[3]).all()
