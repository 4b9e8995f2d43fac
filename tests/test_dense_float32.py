"""Attention in float32 keeps the accuracy of float32: bounds that weights or operands rounded to
fewer bits anywhere on the way would break.

Bounds, fixed before the first run. u = 2^-24. Inputs are unit normals and scale is 1/sqrt(hd), so a
score's terms q_d k_d scale are about 1/sqrt(hd) each and its size about 1.

Root mean square, relative. Roundings are independent. A score is a chain of hd products: hd
roundings of partial sums of size up to 1, together at most u sqrt(hd). Its product with log2(e), up
to 8, rounds by 8 u at most, and the hardware exponential by 4 u. These act on the weights, one by
one, so on the output in the same proportion. The sums over n keys round n times, by u of partial
sums that are no larger than the output's own size but for common direction: u sqrt(n). Twice all
that:
    |got - ref| <= 2 u (sqrt(hd) + 12 + sqrt(n)) |ref|   (Frobenius).

Element by element: ``test_gpu_dense``'s bound with S = |scale| max_j sum_d |q_d k_jd| over the keys
that the row sees.
"""

import numpy as np
import pytest
import torch

U = 2.0 ** -24


def attend(q, k, v, see, scale, weights=lambda p: p):
    """(out, A, S) in float64: q (rows, n_q, hd), k / v (keys, n_kv, hd), see (rows, keys).
    ``weights`` may round the weights (relative to each row's largest)."""
    out, mag, smax = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    g = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        qq, kk, vv = q[:, h], k[:, h // g], v[:, h // g]
        s = np.where(see, scale * qq @ kk.T, -np.inf)
        p = weights(np.exp(s - s.max(1, keepdims=True)))
        p = p / p.sum(1, keepdims=True)
        out[:, h], mag[:, h] = p @ vv, p @ np.abs(vv)
        smax[:, h] = abs(scale) * np.where(see, np.abs(qq) @ np.abs(kk).T, 0).max(1)
    return out, mag, smax[..., None]


def within(got, ref, mag, smax, n, hd):
    """Whether both bounds hold."""
    e = 2 * (hd + 8) * U * smax
    tol = mag * (2 * e + 2.0 ** -20 + 2 * n * U + U) + U * np.abs(ref) + 2.0 ** -40
    rms = 2 * U * (np.sqrt(hd) + 12 + np.sqrt(n)) * np.linalg.norm(ref)
    return bool(np.all(np.abs(got - ref) <= tol)) and np.linalg.norm(got - ref) <= rms


def tree_sees(par, n):
    t = len(par)
    see = np.zeros((t, n + t), dtype=bool)
    see[:, :n] = True
    for i in range(t):
        cur = i
        while cur >= 0:
            see[i, n + cur] = True
            cur = par[cur]
    return see


def parents(seed, t):
    rng = np.random.default_rng(seed)
    return [int(rng.integers(-1, i)) if i else -1 for i in range(t)]


SHAPES = [(4, 1, 64), (4, 2, 128), (6, 3, 96), (2, 1, 256), (3, 1, 33)]
TREES = [([150], 7), ([0, 700], 40), ([1, 65, 1000], 5), ([3000], 100)]


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
def test_the_bounds_break_for_weights_of_fewer_bits(nq, nkv, hd):
    """The bounds hold for a float32 evaluation and break for weights of 14 bits and fewer."""
    g = np.random.default_rng(hd)
    n, t = 1000, 5
    q, k, v = (g.standard_normal((r, h, hd)).astype(np.float32).astype(np.float64)
               for r, h in ((t, nq), (n + t, nkv), (n + t, nkv)))
    see = tree_sees(parents(hd, t), n)
    ref, mag, smax = attend(q, k, v, see, hd ** -0.5)
    plain = attend(*(x.astype(np.float32) for x in (q, k, v)), see, np.float32(hd ** -0.5),
                   lambda p: p.astype(np.float32))[0]
    assert within(plain, ref, mag, smax, n + t, hd)
    for bits in (8, 11, 14):
        def cut(p, bits=bits):
            m, e = np.frexp(p)
            return np.ldexp(np.round(np.ldexp(m, bits)), e - bits)
        got = attend(q, k, v, see, hd ** -0.5, cut)[0]
        assert not within(got, ref, mag, smax, n + t, hd)


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("lens", [[300], [1, 64, 129, 700]])
def test_prompt(nq, nkv, hd, lens):
    from gpu_util import kv, np64
    from test_gpu_dense import gen, i32, randn
    K = kv()
    g, n = gen(sum(lens) + hd), sum(lens)
    q, k, v = (randn(g, n, h, hd, dtype=torch.float32) for h in (nq, nkv, nkv))
    cu = np.r_[0, np.cumsum(lens)]
    got = np64(K.prompt_attention(q, k, v, i32(cu.tolist())))
    q, k, v = map(np64, (q, k, v))
    for lo, hi in zip(cu[:-1], cu[1:]):
        see = np.tril(np.ones((hi - lo, hi - lo), dtype=bool))
        ref, mag, smax = attend(q[lo:hi], k[lo:hi], v[lo:hi], see, hd ** -0.5)
        assert within(got[lo:hi], ref, mag, smax, hi - lo, hd)


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("n_cached,t", TREES)
def test_tree(nq, nkv, hd, n_cached, t):
    from gpu_util import kv, np64
    from test_gpu_dense import i32, tree_inputs
    K = kv()
    b = len(n_cached)
    args = tree_inputs(hd + t, torch.float32, b, t, max(n_cached), nq, nkv, hd)
    par = [parents(t + i, t) for i in range(b)]
    got = np64(K.tree_attention(*args[:3], i32(par), *args[3:], i32(n_cached)))
    q, kd, vd, kc, vc = map(np64, args)
    for i, n in enumerate(n_cached):
        k, v = np.concatenate([kc[i, :n], kd[i]]), np.concatenate([vc[i, :n], vd[i]])
        ref, mag, smax = attend(q[i], k, v, tree_sees(par[i], n), hd ** -0.5)
        assert within(got[i], ref, mag, smax, n + t, hd)
