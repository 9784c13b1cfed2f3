"""Rotary positions of heads so wide that 256 tokens hold 2^31 elements: the columns
behind the rotated ones are copied, every one of them."""
import pytest
import torch

import prefix_tree_block_gb300 as pt

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


@pytest.mark.parametrize("D,rot", [((1 << 23) + 2, 2), ((1 << 23) + 16, 16)])
def test_wide_heads(D, rot):
    """One rotated pair (elements one by one) and eight (16 bytes at a time); position 0
    turns nothing, half a turn negates: both to one rounding of bf16."""
    pt.set_output_allocator(None)  # (4 GB)
    T = 256
    x = torch.randint(-8, 8, (T, 1, D), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    pos = torch.arange(T, device="cuda") % 2
    f = torch.full((rot // 2,), torch.pi, device="cuda")
    y = pt.rotary(x, pos, f)
    pt.sync_status()
    assert torch.equal(y[:, :, rot:], x[:, :, rot:])
    assert torch.equal(y[0::2], x[0::2])
    # sin(pi rounded to fp32) = -8.7e-8, times 8, beside a multiple of 1: below half a step of bf16, but of a 0
    near = (y[1::2, :, :rot].float() + x[1::2, :, :rot].float()).abs().max()
    assert near <= 8 * 1e-7
