"""What pt_sync_status makes of the units' device status words: the worst kind
is returned whichever unit it comes from, and every one is named."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from prefix_tree_block_gb300 import build as ptbuild

UNITS = ("block map", "forward", "backward", "CUDA-core attention", "fold", "cache", "decoding")
INVALID, NOMEM, TIMEOUT = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    ptbuild.build()
    return pt.load_library()


def status(lib, words):
    w = np.array(words, np.int32)
    return lib.pt_debug_status(w.ctypes.data, w.size), lib.pt_last_error().decode()


def test_nothing(lib):
    assert status(lib, [0] * 7)[0] == pt.PT_OK
    assert lib.pt_debug_status(None, 0) == pt.PT_OK


@pytest.mark.parametrize("i", range(7))
def test_each_unit(lib, i):
    for bit, want in ((INVALID, pt.PT_ERR_INVALID_ARG), (NOMEM, pt.PT_ERR_NOMEM), (TIMEOUT, pt.PT_ERR_TIMEOUT)):
        rc, text = status(lib, [bit if k == i else 0 for k in range(7)])
        assert rc == want and UNITS[i] in text
    assert status(lib, [-1 if k == i else 0 for k in range(7)])[0] == pt.PT_ERR_CUDA


@pytest.mark.parametrize("i,j", list(itertools.permutations(range(7), 2)))
def test_two_units(lib, i, j):
    """A wait that ran out is not hidden by another unit's failed check or by
    a cache without pages, nor a failed check by the latter."""
    for worse, less, want in ((TIMEOUT, INVALID, pt.PT_ERR_TIMEOUT), (TIMEOUT, NOMEM, pt.PT_ERR_TIMEOUT), (INVALID, NOMEM, pt.PT_ERR_INVALID_ARG)):
        words = [0] * 7
        words[i], words[j] = worse, less
        rc, text = status(lib, words)
        assert rc == want and UNITS[i] in text and UNITS[j] in text


def test_several_in_one_unit(lib):
    assert status(lib, [0] * 6 + [INVALID | TIMEOUT])[0] == pt.PT_ERR_TIMEOUT
    assert status(lib, [0] * 5 + [INVALID | NOMEM, 0])[0] == pt.PT_ERR_INVALID_ARG
    rc, text = status(lib, [INVALID | NOMEM | TIMEOUT] * 7)
    assert rc == pt.PT_ERR_TIMEOUT and all(text.count(u) == 3 for u in UNITS if u != "forward")


def test_refusals(lib):
    assert lib.pt_debug_status(None, 1) == pt.PT_ERR_INVALID_ARG
    w = np.zeros(8, np.int32)
    assert lib.pt_debug_status(w.ctypes.data, 8) == pt.PT_ERR_INVALID_ARG
    assert lib.pt_debug_status(w.ctypes.data, -1) == pt.PT_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# the same from kernels

def _out_of_pages():
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pt.cache_tables(i(0, 0), i(9, 9), i(-1, -1, -1, -1).view(2, 2), i(5, 6), torch.tensor([0, 1], device="cuda"), 16, 18)


def _bad_length():
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pt.cache_tables(i(-3), i(1), i(0, 0).view(1, 2), i(5, 6), torch.tensor([0, 1], device="cuda"), 16, 1)


def _bad_page():
    plan = pt.decode_plan(1, [0, 1], [0], 2, 2)
    c = torch.zeros(2, 2, 16, 64, device="cuda")
    pt.attn_decode(torch.zeros(1, 2, 64, device="cuda"), c, c, torch.tensor([[7]], dtype=torch.int32, device="cuda"),
                   torch.tensor([3], dtype=torch.int32, device="cuda"), plan)


def _wait():
    s = torch.cuda.current_stream().cuda_stream
    assert pt.load_library().pt_debug_wait_timeout(ctypes.c_void_p(s)) == pt.PT_OK


@pytest.mark.gpu
@pytest.mark.parametrize("calls,want", [
    ((_out_of_pages,), pt.PT_ERR_NOMEM), ((_bad_length,), pt.PT_ERR_INVALID_ARG), ((_bad_page,), pt.PT_ERR_INVALID_ARG),
    ((_out_of_pages, _bad_length), pt.PT_ERR_INVALID_ARG), ((_bad_length, _out_of_pages), pt.PT_ERR_INVALID_ARG),
    ((_out_of_pages, _bad_page), pt.PT_ERR_INVALID_ARG), ((_out_of_pages, _bad_page, _wait), pt.PT_ERR_TIMEOUT),
])
def test_from_kernels(lib, calls, want):
    pt.sync_status()
    for f in calls:
        f()
    with pytest.raises(pt.PTError) as e:
        pt.sync_status()
    assert e.value.status == want
    for f, text in ((_out_of_pages, "out of free pages"), (_bad_page, "decoding"), (_wait, "wait ran out")):
        assert (text in str(e.value)) == (f in calls)
    pt.sync_status()  # all of them are cleared
