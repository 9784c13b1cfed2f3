"""FoldPlan.successors on a stream that is given: its outputs are marked as used there,
so that their memory is not handed out again while that stream still writes it."""
import pytest
import torch

import prefix_tree_block_gb300 as pt
from oracle import tokens as OT

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


def test_successors_on_a_given_stream(monkeypatch):
    pt.set_output_allocator(None)  # (it fills its outputs on the current stream)
    marked = []
    mark = torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: (marked.append((t.data_ptr(), s)), mark(t, s))[1])
    lens, paths = [4, 3, 0, 2, 5], [[0, 1], [0, 2, 3], [0, 2, 4]]
    plan = pt.fold_plan(lens, [0, 2, 5, 8], [n for p in paths for n in p], 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ptr, succ = plan.successors(stream=side)
    assert marked == [(ptr.data_ptr(), side), (succ.data_ptr(), side)]
    torch.cuda.current_stream().wait_stream(side)
    after, first = OT.successors(lens, paths)
    ptr, succ = ptr.tolist(), succ.tolist()
    assert [succ[a:b] for a, b in zip(ptr, ptr[1:])] == after and succ[ptr[-1]:] == first
