"""Refusals of the calls on draft trees, rotary positions and token log
probabilities that return before any device work (no GPU needed), through the
C ABI and through the binding."""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from prefix_tree_block_gb300 import build as ptbuild

INV, UNS = pt.PT_ERR_INVALID_ARG, pt.PT_ERR_UNSUPPORTED
BUF = np.zeros(1 << 12, np.int64)
P = (BUF.ctypes.data + 15) // 16 * 16


@pytest.fixture(scope="module")
def lib():
    ptbuild.build()
    return pt.load_library()


def _rotary(lib, **kw):
    a = dict(X=P, xs=16, dt=pt.PT_BF16, T=3, H=2, D=8, pos=P, freq=P, rot=8, sections=None, axes=1, near=0, inv=0, Y=P + 4096, ys=16)
    a.update(kw)
    if isinstance(a["sections"], list):
        keep = np.array(a["sections"], np.int32)
        a["sections"] = keep.ctypes.data
    rc = lib.pt_rotary(*a.values(), None)
    assert rc == pt.PT_OK or b"pt_rotary" in lib.pt_last_error()
    return rc


@pytest.mark.parametrize("kw,want", [
    (dict(X=None), INV), (dict(Y=None), INV), (dict(pos=None), INV), (dict(freq=None), INV), (dict(dt=7), INV), (dict(T=-1), INV),
    (dict(H=-1), INV), (dict(D=0), INV), (dict(rot=7), INV), (dict(rot=0), INV), (dict(rot=10), INV), (dict(xs=15), INV), (dict(ys=15), INV),
    (dict(axes=0), INV), (dict(axes=5, sections=[1, 1, 1, 1, 0]), UNS), (dict(axes=2), INV), (dict(axes=2, sections=[2, 1]), INV),
    (dict(axes=2, sections=[-1, 5]), INV), (dict(axes=1, sections=[3]), INV), (dict(X=P + 1), INV), (dict(Y=P + 4097), INV),
    (dict(D=1026, H=1, xs=1026, ys=1026, rot=1026), UNS), (dict(H=1 << 20, D=1 << 10, xs=1 << 30, ys=1 << 30), INV),
    (dict(Y=P + 16), INV), (dict(Y=P, ys=24), INV), (dict(xs=24, ys=24, Y=P + 8), INV), (dict(xs=24, ys=24, Y=P + 2 * 24 + 8), INV),
    (dict(xs=24, ys=24, Y=P + 2 * 24 + 40), INV),
])
def test_rotary_refusals(lib, kw, want):
    assert _rotary(lib, **kw) == want


def test_rotary_of_nothing(lib):
    assert _rotary(lib, T=0, X=None, Y=None, pos=None) == pt.PT_OK
    assert _rotary(lib, H=0, X=None, Y=None, xs=0, ys=0) == pt.PT_OK


def _score(lib, **kw):
    a = dict(x=P, stride=100, dt=pt.PT_BF16, R=3, V=100, targets=P, row_ptr=None, index=None, N=3, scale=1.0, k=2, logp=P, lse=P, H=None, top=P, ids=P)
    a.update(kw)
    rc = lib.pt_token_logprobs(*a.values(), None)
    assert rc == pt.PT_OK or b"pt_token_logprobs" in lib.pt_last_error()
    return rc


BOTH = [(dict(x=None), INV), (dict(lse=None), INV), (dict(targets=None), INV), (dict(dt=7), INV), (dict(R=-1), INV),
        (dict(V=0), INV), (dict(N=-1), INV), (dict(N=2), INV), (dict(stride=99), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
        (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(scale=1e-31), INV), (dict(scale=1.1e30), INV),
        (dict(V=(1 << 30) + 1, stride=1 << 31), UNS), (dict(R=1 << 28, N=1 << 28), UNS), (dict(N=(1 << 30) + 1, row_ptr=P), UNS), (dict(x=P + 1), INV)]


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(logp=None), INV), (dict(top=None), INV), (dict(ids=None), INV), (dict(k=-1), INV), (dict(k=101), INV), (dict(k=65), UNS), (dict(R=0, row_ptr=P), INV),
])
def test_score_refusals(lib, kw, want):
    assert _score(lib, **kw) == want


def test_score_of_nothing(lib):
    assert _score(lib, R=0, N=0, x=None, lse=None) == pt.PT_OK


def _grad(lib, **kw):
    a = dict(g=P, dH=None, x=P, stride=100, dt=pt.PT_BF16, R=3, V=100, targets=P, row_ptr=None, index=None, N=3, scale=1.0, lse=P, H=None, d=P + 8192, ds=100)
    a.update(kw)
    rc = lib.pt_token_logprobs_bwd(*a.values(), None)
    assert rc == pt.PT_OK or b"pt_token_logprobs_bwd" in lib.pt_last_error()
    return rc


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(g=None), INV), (dict(d=None), INV), (dict(dH=P), INV), (dict(ds=99), INV), (dict(d=P + 8193), INV), (dict(d=P + 200), INV), (dict(d=P, ds=101), INV),
])
def test_grad_refusals(lib, kw, want):
    kw = dict(kw)
    if kw.get("stride", 0) > 1 << 30:
        kw["ds"] = kw["stride"]
    assert _grad(lib, **kw) == want


def test_grad_of_nothing(lib):
    assert _grad(lib, R=0, N=0, x=None, d=None) == pt.PT_OK


def test_null_plans(lib):
    assert lib.pt_draft_tree(P, P, None, None, None, P, P, None) == INV and b"plan is NULL" in lib.pt_last_error()
    assert lib.pt_cache_keep(P, None, P, P, 1, 0, 64, P, P, 1, 16, None, None) == INV and b"plan is NULL" in lib.pt_last_error()
    assert lib.pt_cache_keep(P, None, P, P, 1, 7, 64, P, P, 1, 16, None, None) == INV and b"dtype" in lib.pt_last_error()
    args = (P, 128, P, P, 0, 64, 1, 16, P, 1, P, None)
    assert lib.pt_attn_decode_drafts(*args, None, 0.0, None, P, P, P, 256, None) == INV and b"draft_mask is NULL" in lib.pt_last_error()
    assert lib.pt_attn_decode_drafts(*args, P, 0.0, None, P, P, P, 256, None) == INV and b"plan is NULL" in lib.pt_last_error()
    assert lib.pt_fold_successors(None, P, P, None) == INV


class _Plan:  # what the binding looks at before it calls the library
    n_samples, q_len, n_rows, n_nodes, Hq, Hkv, handle = 2, 3, 6, 4, 2, 2, None


def test_binding_refuses_host_tensors(lib):
    i = torch.zeros(6, dtype=torch.int32)
    with pytest.raises(TypeError):
        pt.draft_tree(i, i[:4], _Plan())
    with pytest.raises(TypeError):
        pt.cache_keep(i.view(2, 3), torch.zeros(1, 2, 16, 8), torch.zeros(1, 2, 16, 8), i.view(6, 1), i, _Plan())
    with pytest.raises(TypeError):
        pt.rotary(torch.zeros(2, 2, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(4))
    with pytest.raises(TypeError):
        pt.token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        pt.token_logprobs_bwd(torch.zeros(2), torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(2))


def test_binding_refuses_shapes_and_types(lib):
    with pytest.raises(ValueError):
        pt.rotary(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(4))
    with pytest.raises(ValueError):
        pt.token_logprobs(torch.zeros(8), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        pt.token_logprobs(torch.zeros(2, 8, dtype=torch.float16), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        pt.rotary(torch.zeros(2, 2, 8, dtype=torch.float16), torch.zeros(2, dtype=torch.int64), torch.zeros(4))
