"""Rotary positions (pt_rotary) against the fp64 oracle.

Tolerance, from the arithmetic alone.  u = 2^-24.  The angle is exact to 2^-32 of
a turn (positions up to 2^31 times 2^-64, and the final 2^-64), its conversion to
fp32 half turns adds u of at most one, pi u of an angle; sincospif is good to 2
units in the last place, 2 * 2^-23 of a value up to 1: a sine or cosine is off by
c = (4 + 4) u at most.  a cos - b sin then takes three roundings: (c + 3 u)(|a| + |b|).
The output's rounding: u or 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt
from oracle import tokens as OT
from prefix_tree_block_gb300 import workloads as W

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U, UB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


def freqs(half, base=10000.0):
    return torch.tensor(base ** (-np.arange(half) / max(half, 1)), dtype=F32)


def positions_of(T, axes, seed, far=40000, low=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, far, (axes, T), generator=g)


def check(X, pos, f, sections=None, interleaved=False, inverse=False, **kw):
    x = X.double().cpu().numpy()
    before = X.clone()
    Y = pt.rotary(X, pos.cuda(), f.cuda(), sections=sections, interleaved=interleaved, inverse=inverse, **kw)
    torch.cuda.synchronize()
    half = f.numel()
    want = OT.rotary(x, pos.numpy(), f.numpy(), sections if sections is not None else [half], interleaved, inverse)
    size = np.abs(x)
    both = size.copy()
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
    both[:, :, a] = both[:, :, b] = size[:, :, a] + size[:, :, b]
    both[:, :, 2 * half:] = 0.0
    tol = 11 * U * both
    r = UB if X.dtype == BF else U
    tol = np.where(both > 0, tol * (1 + r) + r * np.abs(want), 0.0)
    bad = ~(np.abs(Y.double().cpu().numpy() - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}"
    if kw.get("out") is not X:
        assert torch.equal(X, before)
    return Y


def heads(T, H, D, dtype, seed):
    return torch.randn(T, H, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(2, 2), (4, 2), (6, 6), (7, 4), (8, 8), (10, 6), (32, 32), (64, 64), (64, 32), (64, 24), (80, 80), (96, 48), (128, 128), (256, 256), (512, 512), (1030, 1024)])
def test_head_dims(dtype, interleaved, D, rot):
    check(heads(5, 3, D, dtype, D), positions_of(5, 1, D)[0], freqs(rot // 2), interleaved=interleaved)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 64), (2, 7), (33, 1), (1000, 5), (4097, 2), (9, 200)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tokens_and_heads(T, H, dtype):
    check(heads(T, H, 64, dtype, T), positions_of(T, 1, T)[0], freqs(32), inverse=T % 2 == 0)


@pytest.mark.parametrize("sections", [[32], [16, 16], [16, 8, 8], [8, 8, 8, 8], [0, 32], [32, 0, 0], [1, 0, 30, 1]])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_axes(sections, interleaved, dtype):
    check(heads(21, 3, 64, dtype, 1), positions_of(21, len(sections), 2), freqs(32), sections=sections, interleaved=interleaved, inverse=True)
    check(heads(21, 3, 96, dtype, 1), positions_of(21, len(sections), 3), freqs(32), sections=sections, interleaved=interleaved)


@pytest.mark.parametrize("low,far", [(0, 4), (1 << 20, (1 << 20) + 1000), ((1 << 31) - 2000, (1 << 31) - 1), (-50000, 0), (-(1 << 31), -(1 << 30))])
def test_far_and_negative_positions(low, far):
    """Angles of positions up to 2^31 either way, with frequencies over 40 powers of two."""
    f = torch.tensor([1.0, 0.7, 1e-3, 1e-6, 3.14159274, 2.0 ** -40, 0.0, -0.25], dtype=F32)
    check(heads(300, 2, 16, F32, 3), positions_of(300, 1, 4, far, low)[0], f)


def test_large_frequencies():
    """Up to 2^20 a position: still exact to fp32."""
    f = torch.tensor([1048576.0, 1000.25, 65537.0, -12345.678], dtype=F32)
    check(heads(100, 1, 8, F32, 3), positions_of(100, 1, 4, 1 << 11)[0], f)


def test_frequencies_that_are_not_finite():
    f = torch.tensor([1.0, float("inf"), float("nan"), 0.5], dtype=F32)
    Y = pt.rotary(heads(4, 1, 8, F32, 3), positions_of(4, 1, 4).cuda()[0], f.cuda())
    assert torch.equal(Y[0, 0].isnan(), torch.tensor([False, True, True, False] * 2, device="cuda"))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_strides_and_places(dtype, interleaved, shift):
    """Slices of a fused projection, elements off the 16-byte boundaries, in
    place, into another slice; what lies beside them stays."""
    T, H, D = 19, 3, 64
    qkv = torch.full((T, (H + 4) * D + shift + 3), 5.0, dtype=dtype, device="cuda")
    X = qkv[:, shift:shift + H * D].view(T, H, D)
    X.copy_(heads(T, H, D, dtype, 5))
    pos, f = positions_of(T, 1, 6)[0], freqs(24)
    want = check(X, pos, f, interleaved=interleaved)
    out = torch.full((T, H + 1, D), 3.0, dtype=dtype, device="cuda")
    check(X, pos, f, interleaved=interleaved, out=out[:, 1:])
    assert torch.equal(out[:, 1:], want) and (out[:, 0] == 3.0).all()
    beside = qkv[:, shift + H * D:shift + 2 * H * D].view(T, H, D)
    pt.rotary(X, pos.cuda(), f.cuda(), interleaved=interleaved, out=beside)
    assert torch.equal(beside, want)
    beside.fill_(5.0)
    assert pt.rotary(X, pos.cuda(), f.cuda(), interleaved=interleaved, out=X) is X
    assert torch.equal(X, want)
    X.fill_(5.0)
    assert (qkv == 5.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_inverse_is_the_gradient(dtype):
    """<rotary(x), y> = <x, inverse(y)>, and the inverse undoes the rotation."""
    T, H, D = 50, 2, 64
    X, Y = heads(T, H, D, dtype, 7), heads(T, H, D, dtype, 8)
    pos, f = positions_of(T, 3, 9), freqs(32)
    kw = dict(sections=[10, 11, 11])
    a = check(X, pos, f, **kw)
    b = check(Y, pos, f, inverse=True, **kw)
    r = UB if dtype == BF else U
    # each side's outputs are off by (11 u + r) of at most |x| + |x'|, |y| + |y'|
    both = lambda t: (t.double().abs()[..., :32] + t.double().abs()[..., 32:]).repeat(1, 1, 2)  # noqa: E731
    tol = (12 * U + r * 1.01) * ((both(X) * Y.double().abs()).sum() + (both(Y) * X.double().abs()).sum())
    assert abs((a.double() * Y.double()).sum() - (X.double() * b.double()).sum()) <= tol
    back = pt.rotary(a, pos.cuda(), f.cuda(), inverse=True, **kw)
    assert ((back.double() - X.double()).abs() <= 3 * (12 * U + r * 1.01) * both(X)).all()


def test_folded_positions():
    """On a folded batch, with the position ids of the fold."""
    st = W.grpo_structure([(37, [5, 1, 12]), (9, [4, 9])])
    plan = pt.fold_plan(st.node_lengths, st.path_ptr, st.path_nodes, 60)
    check(heads(st.T, 4, 64, BF, 1), plan.positions().cpu(), freqs(32))


def test_far_tokens():
    """Tokens whose offsets pass 2^31 elements."""
    stride = (1 << 30) + 8
    X = torch.as_strided(torch.empty(2 * stride + 128, dtype=BF, device="cuda"), (3, 2, 64), (stride, 64, 1))
    X.copy_(heads(3, 2, 64, BF, 1))
    pos, f = positions_of(3, 1, 2)[0], freqs(32)
    want = check(X, pos, f)
    pt.rotary(X, pos.cuda(), f.cuda(), out=X)
    assert torch.equal(X, want)


def test_nothing():
    assert pt.rotary(heads(0, 2, 8, BF, 0), torch.zeros(0, dtype=torch.int64, device="cuda"), freqs(4).cuda()).shape == (0, 2, 8)
    assert pt.rotary(heads(3, 0, 8, BF, 0), torch.zeros(3, dtype=torch.int64, device="cuda"), freqs(4).cuda()).shape == (3, 0, 8)


def test_streams_and_graphs():
    X, pos, f = heads(77, 3, 64, BF, 1), positions_of(77, 1, 2)[0].cuda(), freqs(32).cuda()
    want = pt.rotary(X, pos, f)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [pt.rotary(X, pos, f, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(y, want) for y in got)
    x, p = X.clone(), pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pt.rotary(x, p, f)
    p.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pt.rotary(X, pos + 1, f))


def test_binding_refusals():
    X, pos, f = heads(6, 2, 8, BF, 0), torch.zeros(6, dtype=torch.int64, device="cuda"), freqs(4).cuda()
    for bad in (lambda: pt.rotary(X, pos[:5], f), lambda: pt.rotary(X, pos, f, sections=[2, 2]), lambda: pt.rotary(X, pos.view(2, 3), f),
                lambda: pt.rotary(X.transpose(0, 1), pos, f), lambda: pt.rotary(X, pos, f, out=X[:5])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: pt.rotary(X, pos.int(), f), lambda: pt.rotary(X, pos, f.double()), lambda: pt.rotary(X, pos, f, out=X.float()), lambda: pt.rotary(X, pos.cpu(), f)):
        with pytest.raises(TypeError):
            bad()
    two = pos.repeat(2, 1)
    for bad in (lambda: pt.rotary(X, two, f, sections=[2, 1]), lambda: pt.rotary(X, pos, torch.zeros(5, device="cuda")), lambda: pt.rotary(X, pos, torch.zeros(0, device="cuda")),
                lambda: pt.rotary(X[:5], pos[:5], f, out=X[1:])):
        with pytest.raises(pt.PTError) as e:
            bad()
        assert e.value.status == pt.PT_ERR_INVALID_ARG
