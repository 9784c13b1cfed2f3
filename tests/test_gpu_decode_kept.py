"""What lies behind the rows' tokens in the cache has no part in the decoding
attention, in any of its kernels, at tolerances that it does not widen."""
import pytest
import torch

from decode_kept import run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


TREES = {
    "group": ([37, 1, 15, 16, 17, 0], [[0, i] for i in range(1, 6)]),
    "deep": ([130, 31, 0, 64, 2, 3, 250, 1], [[0, 1, 4], [0, 1, 5], [0, 2, 6], [0, 3, 7], [0, 3], [0]]),
    "crowd": ([290] + [3 + 2 * (i % 7) for i in range(70)], [[0, i] for i in range(1, 71)]),
    "wide": ([1500, 260] + [1 + 9 * (i % 5) for i in range(150)], [[0, i] for i in range(2, 102)] + [[0, 1, i] for i in range(102, 152)]),
}


@pytest.mark.parametrize("poison", [INF, -INF, 3e38])
@pytest.mark.parametrize("tree,q_len", [("group", 1), ("group", 3), ("deep", 1), ("deep", 3), ("crowd", 1), ("crowd", 3), ("wide", 1)])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,ps", [(4, 2, 64, BF, 16), (4, 2, 128, BF, 48), (6, 2, 96, BF, 32), (8, 2, 256, BF, 16), (4, 2, 64, F32, 16), (4, 2, 64, BF, 7)])
def test_rows_alone(tree, q_len, Hq, Hkv, D, dtype, ps, poison):
    """Tables as wide as the longest node: CUDA cores, or tensor cores without tiles."""
    simt = dtype == F32 or ps % 16
    run(*TREES[tree], Hq, Hkv, D, dtype, ps, q_len, seed=1, poison=poison, kernels=("decode_simt",) if simt else ("decode_rows", "-decode_tile"))


@pytest.mark.parametrize("poison", [INF, -INF, 3e38])
@pytest.mark.parametrize("tree,q_len", [("crowd", 1), ("wide", 1), ("wide", 3), ("deep", 16)])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(4, 2, 64, 16), (4, 2, 128, 48), (6, 2, 96, 32), (8, 2, 128, 128)])
def test_with_tiles(tree, q_len, Hq, Hkv, D, ps, poison):
    """Tables so wide that nodes which many rows read go to the tile kernel,
    which clears the values behind the last token itself."""
    run(*TREES[tree], Hq, Hkv, D, BF, ps, q_len, seed=1, poison=poison, width=(1 << 18) // ps, kernels=("decode_tile",))
