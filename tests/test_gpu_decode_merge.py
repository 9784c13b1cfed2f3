"""The decoding attention's merge in each of its forms: few rows (four warps a
row), many (a warp a row), most (a warp for four heads), without and with tiles.
The row counts come from the thresholds in the source, so that a change of these
does not leave a form untested."""
import os
import re

import pytest
import torch

import prefix_tree_block_gb300 as pt
from decode_kept import run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SRC = open(os.path.join(os.path.dirname(pt.__file__), "csrc", "pt_decode.cu")).read()
MANY, MOST = (int(re.search(rf"\b{name} = (\d+)", SRC).group(1)) for name in ("kMergeManyRows", "kMergeMostRows"))


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


def _tree(samples):
    """A prompt, a second one for every other sample, and short continuations."""
    lens = [20, 17] + [1 + i % 13 for i in range(samples)]
    return lens, [[0, 1, 2 + i] if i % 2 else [0, 2 + i] for i in range(samples)]


@pytest.mark.parametrize("Hq,Hkv,D,dtype,ps", [
    (32, 8, 32, F32, 16), (32, 8, 33, F32, 16), (32, 8, 64, F32, 16), (32, 8, 65, F32, 16), (32, 8, 80, F32, 7), (32, 4, 128, F32, 16),
    (32, 8, 129, F32, 16), (32, 8, 256, F32, 16), (32, 8, 32, BF, 16), (32, 8, 64, BF, 16), (32, 4, 128, BF, 16), (32, 8, 136, BF, 16),
    (32, 8, 256, BF, 16), (32, 8, 64, BF, 7),
])
def test_four_heads_to_a_warp(Hq, Hkv, D, dtype, ps):
    samples = MOST // Hq
    assert samples * Hq >= MOST and Hq // Hkv % 4 == 0 and D <= 256
    run(*_tree(samples), Hq, Hkv, D, dtype, ps, seed=D, kernels=("-decode_tile",))
    run(*_tree(samples), Hq, Hkv, D, dtype, ps, q_count=[i % 3 > 0 for i in range(samples)], seed=D, kernels=("-decode_tile",))


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 32), (32, 8, 64), (32, 4, 96), (32, 8, 128)])
def test_four_heads_to_a_warp_with_tiles(Hq, Hkv, D):
    samples = MOST // Hq // 2
    run(*_tree(samples), Hq, Hkv, D, BF, 16, q_len=2, seed=D, width=4096, kernels=("decode_tile",))
    run(*_tree(samples), Hq, Hkv, D, BF, 16, q_len=2, q_count=[i % 3 for i in range(samples)], seed=D, width=4096, kernels=("decode_tile",))


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [
    (24, 8, 64, F32), (24, 8, 33, F32), (32, 8, 512, F32), (32, 8, 511, F32), (24, 8, 64, BF), (24, 8, 128, BF), (24, 8, 256, BF), (32, 8, 512, BF),
])
def test_most_rows_one_head_to_a_warp(Hq, Hkv, D, dtype):
    """Groups that four does not divide, and head dims over 256."""
    samples = -(-MOST // Hq)
    assert Hq // Hkv % 4 or D > 256
    run(*_tree(samples), Hq, Hkv, D, dtype, 16, seed=D, kernels=("-decode_tile",))


@pytest.mark.parametrize("D,dtype", [(64, F32), (77, F32), (64, BF), (320, BF)])
@pytest.mark.parametrize("less", [0, 1])
def test_at_the_threshold_of_many_rows(D, dtype, less):
    samples = MANY // 8 - less
    assert (samples * 8 >= MANY) == (less == 0)
    run(*_tree(samples), 8, 2, D, dtype, 16, seed=D, kernels=("-decode_tile",))
