"""Pins of the oracle of draft trees, rotary positions and token log
probabilities: hand-worked cases, and its gradient against differences."""
import numpy as np
import pytest

from oracle import decode as OD
from oracle import tokens as OT


def test_draft_tree_by_hand():
    # 0 and 1 are roots, 2 below 0, 3 below 2, 4 below 1; the second sample has two drafts
    mask, pos = OT.draft_tree([[-1, -1, 0, 2, 1], [-1, 0, 9, 9, 9]], [5, 2], [100, 7])
    assert mask[:, 0].tolist() == [0b1, 0b10, 0b101, 0b1101, 0b10010, 0b1, 0b11, 0, 0, 0]
    assert pos.tolist() == [100, 100, 101, 102, 101, 7, 8, 0, 0, 0]


def test_draft_tree_words():
    mask, pos = OT.draft_tree([np.arange(70) - 1], [70], [0])
    assert mask.shape == (70, 3) and pos.tolist() == list(range(70))
    assert mask[69].view(np.uint32).tolist() == [0xffffffff, 0xffffffff, 0x3f] and mask[31].tolist() == [-1, 0, 0]


def test_attention_of_a_chain_is_the_causal_one():
    rng = np.random.default_rng(0)
    lens, paths, q = [5, 7, 3], [[0, 1], [0, 2]], 3
    tables = np.array([[0, 1], [2, 3], [4, 5]])
    Kc, Vc = rng.standard_normal((2, 6, 2, 4, 8))
    Q = rng.standard_normal((6, 4, 8))
    counts = [3, 2]
    want = OD.attention(Q, Kc, Vc, tables, lens, paths, q, counts)
    chain = [[list(range(j + 1)) for j in range(q)] for _ in paths]
    got = OT.attention(Q, Kc, Vc, tables, lens, paths, chain, q, counts)
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, rtol=1e-13, atol=1e-13)


def test_keep_by_hand():
    cache = np.arange(24.0).reshape(6, 1, 2, 2)  # pages of two tokens
    tables = np.array([[3, 0, 5]])
    out = OT.keep([[1, 3, -1, 0]], [4], [5], [0], tables, 2, cache)  # drafts are tokens 1 to 4
    want = cache.copy()
    want[3, :, 1] = cache[0, :, 0]  # draft 1 (token 2) to token 1
    want[0, :, 0] = cache[5, :, 0]  # draft 3 (token 4) to token 2
    np.testing.assert_array_equal(out, want)


def test_rotary_by_hand():
    x = np.array([[[1.0, 0.0, 2.0, 3.0, 9.0]]])
    q = np.pi / 2
    y = OT.rotary(x, [[1]], [q, 2 * q], [2], False, False)  # pairs (0, 2) and (1, 3)
    np.testing.assert_allclose(y[0, 0], [-2, 0, 1, -3, 9], atol=1e-12)
    y = OT.rotary(x, [[1], [2]], [q, q], [1, 1], True, False)  # pairs (0, 1) by axis 0, (2, 3) by axis 1
    np.testing.assert_allclose(y[0, 0], [0, 1, -2, -3, 9], atol=1e-12)
    np.testing.assert_allclose(OT.rotary(y, [[1], [2]], [q, q], [1, 1], True, True), x, atol=1e-12)


def test_successors_by_hand():
    # root 2, an empty node below it, two children of that, one of the root; a second tree of one token
    after, first = OT.successors([2, 0, 1, 2, 1, 1], [[0, 1, 2], [0, 1, 3], [0, 4], [5]])
    assert after == [[1], [2, 3, 5], [], [4], [], [], []] and first == [0, 6]


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_logprobs_against_plain_softmax(scale):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 9)) * 3
    x[1, 4] = -np.inf
    p = np.exp(scale * x) / np.exp(scale * x).sum(1, keepdims=True)
    logp, lse, H = OT.logprobs(x, [2, 8, -1, 0], [0, 1, 2, -1], scale)
    np.testing.assert_allclose(logp, [np.log(p[0, 2]), np.log(p[1, 8]), 0, 0], rtol=1e-12)
    np.testing.assert_allclose(lse, np.log(np.exp(scale * x).sum(1)), rtol=1e-12)
    np.testing.assert_allclose(H, -(p * np.log(np.where(p > 0, p, 1))).sum(1), rtol=1e-12)
    logp, lse, H = OT.logprobs(np.full((1, 4), -np.inf), [1], [0])
    assert logp[0] == -np.inf and lse[0] == -np.inf and H[0] == 0


def test_top_by_hand():
    assert OT.top([[1.0, 3.0, np.nan, 3.0, -np.inf]], 5).tolist() == [[1, 3, 0, 2, 4]]


@pytest.mark.parametrize("scale", [1.0, 1.3])
def test_gradient_against_differences(scale):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 6))
    targets, rows = [1, 1, 4, -1, 0], [0, 0, 0, 1, 2]
    g, dH = rng.standard_normal(5), rng.standard_normal(3)

    def f(y):
        logp, _, H = OT.logprobs(y, targets, rows, scale)
        return logp @ g + H @ dH

    d = OT.logprobs_grad(x, targets, rows, g, dH, scale)
    for i in np.ndindex(x.shape):
        h = np.zeros_like(x)
        h[i] = 1e-5
        # central differences: truncation below 1e-10 times a third derivative of order one, rounding about 1e-16 / 1e-5
        assert abs((f(x + h) - f(x - h)) / 2e-5 - d[i]) < 1e-8
