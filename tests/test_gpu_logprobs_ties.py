"""Alternatives of long rows in which many logits tie at the last place: rows of
equal logits, and rows in which fewer tokens than alternatives can be chosen."""
import pytest
import torch

import prefix_tree_block_gb300 as pt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


# a warp a row, four warps, and CTAs of 15 warps, alone and in clusters
SHAPES = [(1300, 4096, BF, 24), (1300, 2048, F32, 17), (700, 30001, BF, 64), (700, 30001, F32, 48), (700, 20000, BF, 20), (230, 40000, BF, 64), (3, 131072, F32, 64)]


def rows(what, R, V, dtype):
    if what == "equal":
        return torch.full((R, V), 0.5, dtype=dtype, device="cuda")
    g = torch.Generator("cuda").manual_seed(V)
    x = torch.randn(R, V, generator=g, device="cuda", dtype=dtype)
    if what == "random":
        return x
    if what == "ten can be chosen":
        keep = torch.randint(0, V, (R, 10), generator=g, device="cuda")
        return torch.full_like(x, -float("inf")).scatter(1, keep, x.gather(1, keep))
    if what == "a step down":  # the first third above, in fewer threads than alternatives each with few
        return torch.where(torch.arange(V, device="cuda") % 977 == 5, 2.0, 1.0).to(dtype).repeat(R, 1)
    return x.clamp(max=0.0)  # half of them are the largest


@pytest.mark.parametrize("R,V,dtype,k", SHAPES)
@pytest.mark.parametrize("what", ["equal", "ten can be chosen", "a step down", "clamped"])
def test_ties(what, R, V, dtype, k):
    x = rows(what, R, V, dtype)
    ids = pt.token_logprobs(x, torch.zeros(R, dtype=torch.int64, device="cuda"), top_k=k)[4]
    pt.sync_status()
    assert torch.equal(ids, x.float().sort(dim=1, descending=True, stable=True)[1][:, :k])


def us(x, k):
    pt.set_output_allocator(None)  # (outputs without guards, which take longer to fill than the call)
    t = torch.zeros(x.shape[0], dtype=torch.int64, device="cuda")
    best = float("inf")
    for i in range(8):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(4):
            pt.token_logprobs(x, t, top_k=k)
        b.record()
        b.synchronize()
        if i >= 3:
            best = min(best, a.elapsed_time(b) * 250)
    return best


@pytest.mark.parametrize("R,V,dtype,k", SHAPES[:6])
@pytest.mark.parametrize("what", ["equal", "ten can be chosen", "clamped"])
def test_ties_take_no_search_for_each_alternative(what, R, V, dtype, k):
    """Searched for one by one, k alternatives would read the row k times (17 to 64
    here); a second look at what ties reads it about once more."""
    plain, tied = us(rows("random", R, V, dtype), k), us(rows(what, R, V, dtype), k)
    print(f"{what}: {tied:.1f} us, random {plain:.1f}")
    assert tied < 5 * plain
