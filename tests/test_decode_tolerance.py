"""The decoding tests' comparison finds wrong results whatever lies behind the
rows of the cache (CPU)."""
import numpy as np
import pytest
import torch

from decode_cases import cache_of, pages_of
from decode_kept import check_kept
from oracle import decode as OD

LENS, PATHS = [130, 31, 0, 64, 2, 3, 250, 1], [[0, 1, 4], [0, 1, 5], [0, 2, 6], [0, 3, 7], [0, 3], [0]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf"), 3e38, 0.0])
def test_wrong_results_are_found(dtype, poison):
    Hq, Hkv, D, ps = 4, 2, 64, 16
    tables, n_pages = pages_of(LENS, ps, np.random.default_rng(0))
    Kc, Vc = cache_of(LENS, tables, n_pages, Hkv, ps, D, dtype, 0, poison)
    Q = torch.randn(len(PATHS), Hq, D, generator=torch.Generator().manual_seed(1)).to(dtype)

    def right(lens):
        o, l = OD.attention(*(x.float().numpy() for x in (Q, Kc, Vc)), tables, lens, PATHS, 1)
        return torch.from_numpy(o).to(dtype), torch.from_numpy(l).float()

    def same(O, L):
        check_kept(O, L, Q, Kc, Vc, tables, LENS, PATHS, 1)

    O, L = right(LENS)
    same(O, L)
    wrong = [(torch.zeros_like(O), L), (O + 1e6, L), (O * 1.02, L), (O, L + 1e-3), (O, L + 1e6), (O, torch.full_like(L, -torch.inf))]
    wrong.append(right([n - 1 if n == 130 else n for n in LENS]))  # a mask that drops a token at the end of a node
    for o, l in wrong:
        with pytest.raises(AssertionError):
            same(o, l)
