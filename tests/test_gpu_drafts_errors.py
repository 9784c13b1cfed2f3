"""Errors of the masked decoding call name it, not the call without masks: those
found where the tensor-core kernels are launched too."""
import ctypes

import pytest
import torch

import prefix_tree_block_gb300 as pt

from decode_cases import csr

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


@pytest.mark.parametrize("masked", [False, True])
def test_errors_name_the_call(masked):
    """2^30 pages of two heads: refused on the host, nothing is launched."""
    plan = pt.decode_plan(1, *csr([[0]]), 2, 2, 4)
    lib = pt.load_library()
    z = torch.zeros(1 << 23, device="cuda")  # (more than the workspace)
    p = ctypes.c_void_p(z.data_ptr())
    args = [p, 2 * 64, p, p, pt.PT_BF16, 64, 1 << 30, 16, p, 1, p, None, *([p] if masked else []), 1.0, plan.handle, p, p,
            p, z.numel() * 4, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)]
    name = "pt_attn_decode_drafts" if masked else "pt_attn_decode"
    assert lib.pt_decode_workspace_bytes(plan.handle, 64) <= z.numel() * 4
    assert getattr(lib, name)(*args) == pt.PT_ERR_INVALID_ARG
    assert lib.pt_last_error().decode() == f"{name}: {1 << 30} pages of 2 heads are out of range"
