"""pt_decode_plan reads no more of path_nodes than path_ptr's last entry says
there is (no GPU needed: the calls are refused on the host)."""
import ctypes

import numpy as np
import pytest

import prefix_tree_block_gb300 as pt
from prefix_tree_block_gb300 import build as ptbuild


@pytest.fixture(scope="module")
def lib():
    ptbuild.build()
    return pt.load_library()


class _S:
    cuda_stream = 0


@pytest.mark.parametrize("ptr,empty", [([0, 5, 1], 1), ([0, 1, 7, 2], 2), ([0, 3, 3, 1], 1), ([0, 1 << 30, 1], 1), ([0, 2, -1], 1)])
def test_path_ptr_that_turns_back(lib, ptr, empty):
    """Behind the nodes that the last entry counts stands 99, which would be
    named as out of range if it were read."""
    nodes = np.full(16, 99, np.int32)
    nodes[:max(ptr[-1], 0)] = np.arange(max(ptr[-1], 0))
    p = np.array(ptr, np.int32)
    out = ctypes.c_void_p()
    rc = lib.pt_decode_plan(4, p.ctypes.data, nodes.ctypes.data, p.size - 1, 2, 2, 1, None, ctypes.byref(out))
    assert rc == pt.PT_ERR_INVALID_ARG and not out.value
    assert f"sample path {empty} is empty" in lib.pt_last_error().decode()


def test_binding(lib):
    with pytest.raises(pt.PTError) as e:
        pt.decode_plan(4, [0, 3, 1], [0], 2, 2, stream=_S())
    assert e.value.status == pt.PT_ERR_INVALID_ARG and "sample path 1 is empty" in str(e.value)
