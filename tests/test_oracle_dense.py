"""Pins of the dense-attention oracle: closed forms, an independent mask-matrix form, invariants."""

import numpy as np

from oracle import dense_attention


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_first_token_and_equal_keys_have_closed_forms():
    g = _rng(0)
    q, k, v = g.standard_normal((5, 4, 8)), g.standard_normal((5, 2, 8)), g.standard_normal((5, 2, 8))
    out = dense_attention.prompt_attention(q, k, v, [0, 2, 5], 0.3)
    for first in (0, 2):  # the first token of a sequence sees itself alone
        np.testing.assert_allclose(out[first], v[first].repeat(2, 0), rtol=1e-14)
    flat = dense_attention.prompt_attention(q, np.ones_like(k), v, [0, 5], 0.3)
    np.testing.assert_allclose(flat[4, 3], v[:, 1].mean(0), rtol=1e-13)


def test_prompt_equals_a_masked_score_matrix():
    g = _rng(1)
    q, k, v = g.standard_normal((9, 3, 4)), g.standard_normal((9, 3, 4)), g.standard_normal((9, 3, 4))
    cu = [0, 4, 4, 8]
    out = dense_attention.prompt_attention(q, k, v, cu, -0.7)
    seq = np.array([0] * 4 + [1] * 4 + [2])
    mask = (seq[:, None] == seq[None]) & (np.arange(9)[None] <= np.arange(9)[:, None])
    s = np.where(mask, -0.7 * np.einsum("ihd,jhd->hij", q, k), -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    ref = np.einsum("hij,jhd->ihd", p / p.sum(-1, keepdims=True), v)
    np.testing.assert_allclose(out[:8], ref[:8], rtol=1e-12)
    assert np.isnan(out[8]).all()  # behind the last sequence


def test_tree_of_one_node_is_decoding_and_a_chain_is_a_prompt():
    g = _rng(2)
    q, kc, vc = g.standard_normal((1, 1, 4, 8)), g.standard_normal((1, 6, 2, 8)), g.standard_normal((1, 6, 2, 8))
    kd, vd = g.standard_normal((1, 1, 2, 8)), g.standard_normal((1, 1, 2, 8))
    out = dense_attention.tree_attention(q, kd, vd, [[-1]], kc, vc, [5], 0.5)
    K, V = np.concatenate([kc[0, :5], kd[0]]), np.concatenate([vc[0, :5], vd[0]])
    for h in range(4):
        s = 0.5 * K[:, h // 2] @ q[0, 0, h]
        w = np.exp(s) / np.exp(s).sum()
        np.testing.assert_allclose(out[0, 0, h], w @ V[:, h // 2], rtol=1e-12)
    n = 7
    q, k, v = g.standard_normal((n, 4, 8)), g.standard_normal((n, 2, 8)), g.standard_normal((n, 2, 8))
    chain = dense_attention.tree_attention(q[None], k[None], v[None], [list(range(-1, n - 1))],
                                           np.zeros((1, 0, 2, 8)), np.zeros((1, 0, 2, 8)), [0], 0.4)
    np.testing.assert_allclose(chain[0], dense_attention.prompt_attention(q, k, v, [0, n], 0.4),
                               rtol=1e-12)


def test_ancestors_by_hand():
    #        0       1
    #       / \      |
    #      2   3     4      5, 6 padding; 7 under padding; 8 points forward
    parents = [-1, -1, 0, 0, 1, -2, -7, 5, 8]
    want = [[0], [1], [0, 2], [0, 3], [1, 4], [], [], [], []]
    assert [dense_attention.ancestors(parents, i) for i in range(9)] == want
