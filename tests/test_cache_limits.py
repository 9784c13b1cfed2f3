"""Sizes that the cache calls refuse on the host because their indexes would
not fit (no GPU needed)."""
import pytest
import torch

import prefix_tree_block_gb300 as pt
from prefix_tree_block_gb300 import build as ptbuild


@pytest.fixture(scope="module")
def lib():
    ptbuild.build()
    return pt.load_library()


# addresses that no call may follow, far enough apart that nothing overlaps
FAR = {name: (i + 1) << 40 for i, name in enumerate(("held", "added", "tables", "ring", "ctr", "lens", "row_ptr", "slots", "pos", "out"))}


def tables_call(lib, **kw):
    a = dict(held=FAR["held"], added=FAR["added"], start=None, n=4, ps=16, tables=FAR["tables"], mp=4, ring=FAR["ring"], cap=8,
             ctr=FAR["ctr"], lens=FAR["lens"], row_ptr=FAR["row_ptr"], slots=FAR["slots"], pos=FAR["pos"], new=32, out=FAR["out"])
    a.update(kw)
    return lib.pt_cache_tables(*a.values(), None)


@pytest.mark.parametrize("cap", [(1 << 30) + 1, (1 << 31) - 1])
def test_ring_of_more_than_2_30_ids(lib, cap):
    """A page's place is the head's place in the ring plus the pages taken
    before it: two numbers below ring_cap, added in 32 bits."""
    assert tables_call(lib, cap=cap) == pt.PT_ERR_INVALID_ARG
    assert b"ring_cap" in lib.pt_last_error()


def test_binding_refuses_a_ring_whose_size_does_not_fit():
    i = torch.zeros(4, dtype=torch.int32)
    ring = torch.zeros(1, dtype=torch.int32).expand((1 << 32) + 8)  # would reach the library as 8
    with pytest.raises(ValueError, match="ring"):
        pt.cache_tables(i, i, i.view(4, 1), ring, torch.zeros(2, dtype=torch.int64), 16, 4)


OUT = ("tables", "ring", "lens", "row_ptr", "slots", "pos", "out")  # tables and ring change in place


@pytest.mark.parametrize("a,b", [(a, b) for i, a in enumerate(OUT) for b in OUT[i + 1:]])
def test_outputs_over_each_other(lib, a, b):
    assert tables_call(lib, **{a: FAR[b]}) == pt.PT_ERR_INVALID_ARG
    assert b"overlap" in lib.pt_last_error()


def test_an_outputs_last_byte_counts(lib):
    assert tables_call(lib, lens=FAR["slots"] + 32 * 8 - 1) == pt.PT_ERR_INVALID_ARG
    assert b"overlap" in lib.pt_last_error()
    assert tables_call(lib, slots=FAR["ring"] - 32 * 8 + 1) == pt.PT_ERR_INVALID_ARG
    assert b"overlap" in lib.pt_last_error()
