"""Refusals of the cache and decoding calls that return before any device
work (no GPU needed), through the C ABI and through the binding."""
import ctypes

import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from prefix_tree_block_gb300 import build as ptbuild

INV, UNS = pt.PT_ERR_INVALID_ARG, pt.PT_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    ptbuild.build()
    return pt.load_library()


def _tables(lib, **kw):
    buf = np.zeros(1 << 12, np.int64)
    p = buf.ctypes.data
    a = dict(held=p, added=p + 512, start=None, n=4, ps=16, tables=p + 1024, mp=4, ring=p + 2048, cap=8, ctr=p + 2560, lens=p + 16384,
             row_ptr=p + 3584, slots=p + 4096, pos=p + 8192, new=32, out=p + 12288)
    a.update(kw)
    return lib.pt_cache_tables(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(held=None), INV), (dict(added=None), INV), (dict(tables=None), INV), (dict(ring=None), INV), (dict(ctr=None), INV),
    (dict(lens=None), INV), (dict(row_ptr=None), INV), (dict(slots=None), INV), (dict(out=None), INV),
    (dict(n=-1), INV), (dict(ps=0), INV), (dict(mp=-1), INV), (dict(cap=0), INV), (dict(new=-1), INV), (dict(new=(1 << 30) + 1), INV),
    (dict(n=1 << 18, mp=1 << 13), INV), (dict(mp=1 << 20, ps=1 << 11), INV), (dict(n=(1 << 18) + 1), UNS),
])
def test_tables_refusals(lib, kw, want):
    assert _tables(lib, **kw) == want
    assert b"pt_cache_tables" in lib.pt_last_error()


@pytest.mark.parametrize("a,b", [("held", "lens"), ("added", "lens"), ("ctr", "out"), ("held", "row_ptr"), ("added", "slots"), ("held", "tables"),
                                 ("held", "ring"), ("ctr", "pos")])
def test_tables_refuses_outputs_over_inputs(lib, a, b):
    buf = np.zeros(64, np.int64)
    assert _tables(lib, **{a: buf.ctypes.data, b: buf.ctypes.data}) == INV
    assert b"overlaps" in lib.pt_last_error()


def _write(lib, **kw):
    buf = np.zeros(64, np.int64)
    p = buf.ctypes.data
    a = dict(K=p, V=p, ks=16, vs=16, dt=pt.PT_BF16, T=1, Hkv=2, D=8, slots=p, Kc=p, Vc=p, pages=1, ps=1)
    a.update(kw)
    return lib.pt_cache_write(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(K=None), dict(V=None), dict(slots=None), dict(Kc=None), dict(Vc=None), dict(T=-1), dict(Hkv=0), dict(D=0),
                                dict(ps=0), dict(pages=-1), dict(dt=7), dict(ks=15), dict(vs=15), dict(Hkv=1 << 20, D=1 << 11, ks=1 << 31, vs=1 << 31)])
def test_write_refusals(lib, kw):
    assert _write(lib, **kw) == INV
    assert b"pt_cache_write" in lib.pt_last_error()


def test_write_of_nothing(lib):
    assert _write(lib, T=0, K=None, V=None, slots=None) == pt.PT_OK


@pytest.mark.parametrize("n,paths,kw,want", [
    (2, [[0, 2]], {}, INV), (2, [[0, -1]], {}, INV), (2, [[0], []], {}, INV), (2, [[0, 1, 0]], {}, INV),
    (2, [[0, 1]], dict(Hq=3, Hkv=2), INV), (2, [[0, 1]], dict(Hkv=0), INV), (2, [[0, 1]], dict(q_len=0), INV),
    (2, [[0, 1]], dict(Hq=1 << 15, Hkv=1, q_len=1 << 15), INV), ((1 << 16) + 1, [[0, 1]], {}, UNS), (-1, [], {}, INV),
])
def test_plan_refusals(lib, n, paths, kw, want):
    a = dict(Hq=4, Hkv=2, q_len=1)
    a.update(kw)
    ptr = np.cumsum([0] + [len(p) for p in paths])
    with pytest.raises(pt.PTError) as e:
        pt.decode_plan(n, ptr, [x for p in paths for x in p], stream=_S(), **a)
    assert e.value.status == want


class _S:
    cuda_stream = 0


def test_plan_binding_refuses_a_short_node_list(lib):
    with pytest.raises(ValueError):
        pt.decode_plan(4, [0, 3], [1, 2], 2, 2, stream=_S())


def test_null_plan(lib):
    assert lib.pt_attn_decode(None, 0, None, None, 0, 64, 1, 16, None, 1, None, None, 0.0, None, None, None, None, 0, None) == INV
    assert b"plan is NULL" in lib.pt_last_error()
    assert pt.PT_OK == 0 and lib.pt_decode_workspace_bytes(None, 64) == 256
    lib.pt_decodeplan_free(None)
    out = ctypes.c_void_p()
    assert lib.pt_decode_plan(0, None, None, 0, 1, 1, 1, None, ctypes.byref(out)) == INV


def test_binding_refuses_host_tensors(lib):
    i = torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(TypeError):
        pt.cache_tables(i, i, i.view(4, 1), i, c, 16, 4)
    k = torch.zeros(4, 2, 8)
    with pytest.raises(TypeError):
        pt.cache_write(k, k, torch.zeros(4, dtype=torch.int64), torch.zeros(1, 2, 16, 8), torch.zeros(1, 2, 16, 8))
