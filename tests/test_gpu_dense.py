"""Rotary embedding, prompt attention and tree attention against float64.

Tolerances, fixed before the first run. u = 2^-24; h = half a step of the element type (bf16 2^-8,
fp16 2^-11, float32 2^-24).

Attention, per element: scores of head_dim products summed in float32 are off by at most
e = 2 (hd + 8) u S, S = |scale| max_j sum_d |q_d k_jd| (the factor 2 allows a truncating
accumulator), so each weight by 2 e + 2^-20 (the hardware exponential and the joins) relatively, and
by h where two-byte probabilities enter the second product; n weights and products are summed with
2 n u. All of that acts on A = sum_j p_j |v_j|; the output rounds by h |out|:
    |error| <= A (2 e + 2^-20 + 2 n u + h) + h |out| + 2^-40.
(float32: the h of the probabilities is u.) Below fp16's smallest normal number, 2^-14, the steps
are 2^-24 apart whatever the value, so a result there rounds by up to 2^-25 and not by h |out|: that
much (``floor``: smallest normal x eps / 2, for bf16 and float32 below 2^-133) is added to both
bounds. In the mean the two-byte roundings are independent and
uniform: relative root mean square of at most h sqrt(2/3) for values without a common direction;
1.5 h is asked.

Rotation: hardware sine and cosine (two-byte) are off by 2^-21, sincospif by 2^-23, the angle by
2^-25; two products and a sum by 3 u, the result by h:
    |error| <= (|a| + |b|) (2^-20 or 2^-22) + h |out| + the float64 reference's own angle error,
    (|a| + |b|) |pos| 2^-52.
"""

import math

import numpy as np
import pytest
import torch

from gpu_util import bit, kv, np64
from oracle import dense_attention as od
from oracle import rope as orope

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float16, torch.float32]
SHAPE, NAN = 2, float("nan")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def floor(dtype):
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


def randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def check(got, ref, mag, smax, n, hd, dtype):
    """Error bound of the module's docstring; mag = A, smax = S (arrays that broadcast)."""
    u, h = 2.0 ** -24, half_step(dtype)
    e = 2 * (hd + 8) * u * smax
    tol = mag * (2 * e + 2.0 ** -20 + 2 * n * u + h) + h * np.abs(ref) + 2.0 ** -40 + floor(dtype)
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"worst error {np.max(err - tol)} above its bound"
    if h > u and n > 1:
        assert np.linalg.norm(got - ref) <= 1.5 * h * np.linalg.norm(ref)


def prompt_reference(q, k, v, cu, scale):
    """(out, A, S) in float64 by whole score matrices, per sequence."""
    out = np.zeros(q.shape)
    mag = np.zeros(q.shape)
    smax = np.zeros(q.shape[:2])
    g = q.shape[1] // k.shape[1]
    for lo, hi in zip(cu[:-1], cu[1:]):
        m = np.tril(np.ones((hi - lo, hi - lo), dtype=bool))
        for h in range(q.shape[1]):
            qq, kk, vv = q[lo:hi, h], k[lo:hi, h // g], v[lo:hi, h // g]
            if hi == lo:
                continue
            s = np.where(m, scale * qq @ kk.T, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[lo:hi, h], mag[lo:hi, h] = p @ vv, p @ np.abs(vv)
            smax[lo:hi, h] = abs(scale) * (np.abs(qq) @ np.abs(kk).T).max(1)
    return out, mag, smax[..., None]


def run_prompt(seed, dtype, lens, nq, nkv, hd, scale=None, gain=1.0):
    K = kv()
    g = gen(seed)
    n = sum(lens)
    q, k, v = (randn(g, n, nq, hd, dtype=dtype) * gain, randn(g, n, nkv, hd, dtype=dtype),
               randn(g, n, nkv, hd, dtype=dtype))
    cu = np.r_[0, np.cumsum(lens)].tolist()
    got = K.prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), scale)
    s = 1 / math.sqrt(hd) if scale is None else scale
    ref, mag, smax = prompt_reference(np64(q), np64(k), np64(v), cu, s)
    check(np64(got), ref, mag, smax, max(lens), hd, dtype)


def tree_reference(q, kd, vd, parents, kc, vc, nc, scale):
    ref = od.tree_attention(q, kd, vd, parents, kc, vc, nc, scale)
    mag = od.tree_attention(q, kd, np.abs(vd), parents, kc, np.abs(vc), nc, scale)
    top = max(np.abs(kd).max(), np.abs(kc).max() if kc.size else 0)
    smax = abs(scale) * np.abs(q).sum(-1, keepdims=True) * top
    return ref, mag, smax


def tree_parents(rng, t, live):
    return [(-1 if i == 0 else int(rng.integers(-1, i))) if i < live else -2 for i in range(t)]


def tree_inputs(seed, dtype, b, t, cap, nq, nkv, hd):
    g = gen(seed)
    return (randn(g, b, t, nq, hd, dtype=dtype), randn(g, b, t, nkv, hd, dtype=dtype),
            randn(g, b, t, nkv, hd, dtype=dtype), randn(g, b, cap, nkv, hd, dtype=dtype),
            randn(g, b, cap, nkv, hd, dtype=dtype))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_tree(seed, dtype, t, n_cached, nq, nkv, hd, live=None, cap=None, scale=None):
    K = kv()
    b = len(n_cached)
    cap = max(n_cached) + 3 if cap is None else cap
    q, kd, vd, kc, vc = tree_inputs(seed, dtype, b, t, cap, nq, nkv, hd)
    rng = np.random.default_rng(seed)
    par = [tree_parents(rng, t, t if live is None else live[i]) for i in range(b)]
    for i, n in enumerate(n_cached):  # rows that are not in use hold anything
        kc[i, n:] = NAN
        vc[i, n:] = NAN
    got = K.tree_attention(q, kd, vd, i32(par), kc, vc, i32(n_cached), scale)
    s = 1 / math.sqrt(hd) if scale is None else scale
    ref, mag, smax = tree_reference(np64(q), np64(kd), np64(vd), par, np.nan_to_num(np64(kc)),
                                    np.nan_to_num(np64(vc)), n_cached, s)
    check(np64(got), ref, mag, smax, max(n_cached) + t, hd, dtype)
    for i in range(b):
        for node in range(t):
            if not od.ancestors(par[i], node):
                assert not got[i, node].any()


# ------------------------------------------------------------------------------------------------
# Rotary embedding

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,heads,hd", [(1, 1, 2), (5, 3, 64), (33, 8, 128), (257, 5, 80), (7, 2, 6),
                                        (1000, 40, 128), (3, 1, 256), (129, 1, 96), (4, 1024, 8)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(dtype, n, heads, hd, inverse):
    K = kv()
    g = gen(n + hd)
    x = randn(g, n, heads, hd, dtype=dtype)
    p = np.random.default_rng(n).integers(-5, 1 << 17, n)
    p[0] = 0 if n == 1 else (1 << 31) - 1
    p[-1] = -(1 << 31) if n > 2 else p[-1]
    got = np64(K.apply_rope(x, i32(p), inverse=inverse))
    ref = orope.apply_rope(np64(x).reshape(n, -1), -p if inverse else p, heads, hd, 500000.0)
    ref = ref.reshape(n, heads, hd)
    a = np.abs(np64(x))
    size = np.tile(a[..., :hd // 2] + a[..., hd // 2:], 2)
    tol = (size * ((2.0 ** -22 if dtype == torch.float32 else 2.0 ** -20)
                   + np.abs(p)[:, None, None] * 2.0 ** -52) + half_step(dtype) * np.abs(ref)
           + floor(dtype))
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("dtype", DT)
def test_rope_on_views_in_place_and_back(dtype):
    """The query and key heads of one fused projection, rotated in place; odd strides; theta."""
    K = kv()
    buf = randn(gen(3), 50, 13, 64, dtype=dtype)
    keep = buf.clone()
    pos = torch.arange(100, 150, dtype=torch.int32, device="cuda")
    ref = K.apply_rope(buf[:, 1:9].contiguous(), pos, 10000.0)
    got = K.apply_rope(buf[:, 1:9], pos, 10000.0, out=buf[:, 1:9])
    assert got.data_ptr() == buf[:, 1:9].data_ptr() and torch.equal(got, ref)
    assert torch.equal(buf[:, 0], keep[:, 0]) and torch.equal(buf[:, 9:], keep[:, 9:])
    back = K.apply_rope(got, pos, 10000.0, inverse=True)
    h = half_step(dtype)
    a = keep[:, 1:9].double().abs()
    size = (a[..., :32] + a[..., 32:]).repeat(1, 1, 2)
    # two roundings by h of entries no larger than |a| + |b|, each turned once more by at most sqrt 2
    assert ((back.double() - keep[:, 1:9].double()).abs() <= 4 * size * (h + 2.0 ** -20)).all()
    odd = torch.empty(50 * 8 * 65 + 1, dtype=dtype, device="cuda")[1:].view(50, 8, 65)[..., :64]
    odd.copy_(keep[:, 1:9])  # rows that do not start on 16 bytes
    # the scalar and the vector form do the same arithmetic
    assert torch.equal(K.apply_rope(odd, pos, 10000.0), ref)


def test_rope_matches_the_reconstruction_and_prepares_the_selection():
    K = kv()
    n, heads, hd = 40, 2, 64
    rows = randn(gen(4), n, heads * hd, dtype=torch.float32)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    h = K.LowRankHistory(heads * hd, 16, 64, storage=torch.float32)
    dense = K.reconstruct(h, rows, pos, n, heads, hd, True, out_dtype=torch.float32)
    got = K.apply_rope(rows.view(n, heads, hd), pos)
    assert (got.view(n, -1) - dense).abs().max() <= 2.0 ** -20 * rows.abs().max()


# ------------------------------------------------------------------------------------------------
# Prompt attention

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("nq,nkv,hd", [(4, 1, 128), (2, 2, 64), (6, 2, 128), (5, 1, 64), (8, 1, 96),
                                       (3, 3, 80), (2, 1, 8), (2, 1, 256), (3, 1, 33), (64, 1, 64),
                                       (2, 1, 1)])
def test_prompt_head_layouts(dtype, nq, nkv, hd):
    run_prompt(nq * 1000 + hd, dtype, [37, 200], nq, nkv, hd)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [127, 128, 129], [0, 5, 0, 64, 0], [63, 65, 255, 257],
                                  [2] * 70, [600], [64], [128], [192]])
def test_prompt_lengths(dtype, lens):
    run_prompt(sum(lens), dtype, lens, 4, 2, 128)


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float16, 64)])
def test_prompt_long(dtype, hd):
    run_prompt(9, dtype, [2111, 700], 2, 1, hd)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("scale,gain", [(-0.1, 1.0), (0.0, 1.0), (0.09, 12.0), (2.0, 3.0)])
def test_prompt_scales(dtype, scale, gain):
    """Negative and zero scales, and scores whose running maximum moves far from tile to tile."""
    run_prompt(17, dtype, [300], 4, 1, 64, scale, gain)


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float16, 64),
                                      (torch.float32, 64), (torch.bfloat16, 33)])
def test_prompt_rising_scores(dtype, hd):
    """Keys whose scores grow along the prompt: every tile raises the maximum."""
    K = kv()
    n = 700
    q = torch.ones(n, 2, hd, device="cuda", dtype=dtype)
    k = (torch.arange(n, device="cuda")[:, None, None] / 16).expand(n, 1, hd).to(dtype).contiguous()
    v = randn(gen(1), n, 1, hd, dtype=dtype)
    got = K.prompt_attention(q, k, v, None, 4.0 / hd)
    ref, mag, smax = prompt_reference(np64(q), np64(k), np64(v), [0, n], 4.0 / hd)
    check(np64(got), ref, mag, smax, n, hd, dtype)


@pytest.mark.parametrize("dtype", DT)
def test_prompt_views_and_rows_outside(dtype):
    """Heads of one fused projection as strided views; an output view; rows between and behind the
    sequences keep what they hold, and what inputs hold there reaches nobody."""
    K = kv()
    rows, nq, nkv, hd = 300, 4, 2, 64
    buf = randn(gen(5), rows, nq + 2 * nkv, hd, dtype=dtype)
    cu = [3, 120, 290]
    buf[:3] = NAN
    buf[290:] = float("inf")
    q, k, v = buf[:, :nq], buf[:, nq:nq + nkv], buf[:, nq + nkv:]
    out = torch.full((rows, 2 * nq, hd), 7.0, dtype=dtype, device="cuda")
    K.prompt_attention(q, k, v, i32(cu), out=out[:, 1:1 + nq])
    ref, mag, smax = prompt_reference(np64(q), np64(k), np64(v), cu, 1 / math.sqrt(hd))
    sl = slice(3, 290)
    check(np64(out[sl, 1:1 + nq]), ref[sl], mag[sl], smax[sl], 170, hd, dtype)
    assert (out[:3] == 7).all() and (out[290:] == 7).all()
    assert (out[:, 0] == 7).all() and (out[:, 1 + nq:] == 7).all()


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float16, 64),
                                      (torch.float32, 64), (torch.float16, 20)])
@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("nq", [1, 4])
def test_prompt_values_that_are_not_finite_reach_only_their_readers(dtype, hd, bad, nq):
    K = kv()
    lens = [190, 260]
    g = gen(11)
    n = sum(lens)
    q, k, v = (randn(g, n, nq, hd, dtype=dtype), randn(g, n, 1, hd, dtype=dtype),
               randn(g, n, 1, hd, dtype=dtype))
    clean, where = np64(v), (190 + 100, 5)
    v[where[0], 0, where[1]] = bad
    got = np64(K.prompt_attention(q, k, v, i32([0, 190, n])))
    clean[where[0], 0, where[1]] = 0.0
    ref, mag, smax = prompt_reference(np64(q), np64(k), clean, [0, 190, n], 1 / math.sqrt(hd))
    hit = got[where[0]:, :, where[1]]
    assert np.isnan(hit).all() if bad != bad else (hit == bad).all()
    got[where[0]:, :, where[1]] = ref[where[0]:, :, where[1]]
    check(got, ref, mag, smax, 260, hd, dtype)
    # a key that is not finite: the rows from it on see it, the others do not
    v[where[0], 0, where[1]] = 0.0
    k[where[0], 0, 0] = NAN
    got = np64(K.prompt_attention(q, k, v, i32([0, 190, n])))
    assert np.isnan(got[where[0]:]).all()
    sl = slice(0, where[0])
    check(got[sl], ref[sl], mag[sl], smax[sl], 260, hd, dtype)


@pytest.mark.parametrize("dtype", DT)
def test_prompt_inconsistent_sequences_are_reported(dtype):
    K = kv()
    q = randn(gen(2), 64, 2, 64, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    out = torch.full_like(q, 7.0)
    # entries: [0, 10) fine, [10, 5) decreasing, [5, 5) empty, [5, 999) beyond the rows
    K.prompt_attention(q, q, q, i32([0, 10, 5, 5, 999]), out=out, status=status)
    assert status.item() == bit(SHAPE)
    fine = K.prompt_attention(q[:10], q[:10], q[:10])
    assert torch.equal(out[:10], fine) and (out[10:] == 7).all()
    status.zero_()
    K.prompt_attention(q, q, q, i32([-4, 3, 20]), out=out, status=status)
    assert status.item() == bit(SHAPE)


def test_prompt_many_sequences():
    """More sequences than a warp has lanes, among them the longest near the end."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 9, 300).tolist()
    lens[250] = 333
    run_prompt(21, torch.bfloat16, lens, 2, 1, 64)
    run_prompt(22, torch.float32, lens, 2, 1, 64)


# ------------------------------------------------------------------------------------------------
# Tree attention

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("nq,nkv,hd,t", [(4, 1, 128, 1), (8, 2, 64, 5), (2, 2, 128, 128), (6, 1, 80, 40),
                                         (32, 1, 64, 9), (5, 1, 256, 3), (3, 1, 21, 4), (12, 4, 96, 33),
                                         (4, 2, 128, 100), (64, 1, 64, 64)])
def test_tree_head_layouts(dtype, nq, nkv, hd, t):
    run_tree(hd + t, dtype, t, [150, 0, 77], nq, nkv, hd)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n_cached", [[0], [1], [127], [128], [129], [1000], [3, 500, 64, 0, 1]])
@pytest.mark.parametrize("t", [1, 13])
def test_tree_lengths(dtype, n_cached, t):
    run_tree(sum(n_cached) + t, dtype, t, n_cached, 4, 2, 128)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [2, 16])
def test_tree_padding(dtype, group):
    """Entries with fewer live nodes than the batch's trees, one with none and nothing cached."""
    run_tree(5, dtype, 20, [90, 0, 300], group, 1, 64, live=[20, 0, 7])


@pytest.mark.parametrize("dtype", DT)
def test_tree_last_row_block_is_short(dtype):
    """300 packed rows: row blocks of 256 and 44, the second without work for half of the kernel;
    more units than CTAs, so that a CTA meets both kinds in turn."""
    run_tree(12, dtype, 100, [5, 0, 260, 131, 40, 77, 10, 1] * 8, 3, 1, 64)
    run_tree(13, dtype, 100, [300, 1], 12, 4, 64)


@pytest.mark.parametrize("dtype", DT)
def test_tree_scales(dtype):
    run_tree(6, dtype, 6, [700], 4, 1, 64, scale=-0.2)
    run_tree(7, dtype, 6, [700], 4, 1, 64, scale=0.0)
    run_tree(8, dtype, 6, [700], 4, 1, 64, scale=3.0)


@pytest.mark.parametrize("dtype", DT)
def test_tree_units_cut_between_ctas(dtype):
    """Caches with room for more than seven tiles are cut into equal shares: units of one and of two
    row blocks, in two and in many parts, several whole ones per share, padding among the rows."""
    run_tree(40, dtype, 100, [1500, 3, 1100], 12, 4, 64)
    run_tree(41, dtype, 128, [2000], 2, 1, 128, live=[90])
    run_tree(42, dtype, 100, [5, 0, 260, 131, 40, 77, 10, 1] * 8, 3, 1, 64, cap=1000)
    run_tree(43, dtype, 20, [90, 0, 300, 999], 2, 1, 64, live=[20, 0, 7, 13], cap=1000)
    run_tree(44, dtype, 6, [1000] * 50, 6, 2, 80, cap=1001)
    run_tree(45, dtype, 1, [1200, 7], 64, 1, 33)


def test_tree_long_cache():
    run_tree(10, torch.bfloat16, 3, [20011], 2, 1, 128)
    run_tree(11, torch.float16, 2, [9000, 17], 2, 2, 64)


@pytest.mark.parametrize("dtype", DT)
def test_tree_bad_parents_and_lengths_are_reported(dtype):
    K = kv()
    q, kd, vd, kc, vc = tree_inputs(3, dtype, 2, 4, 70, 2, 1, 64)
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    par = [[-1, 0, 2, 2], [-1, -1, 1, 9]]  # node 2 its own parent (3 under it); node 3 of entry 1
    got = K.tree_attention(q, kd, vd, i32(par), kc, vc, i32([70, 30]), status=status)
    assert status.item() == bit(SHAPE)
    assert not got[0, 2:].any() and not got[1, 3].any()
    ref, mag, smax = tree_reference(*map(np64, (q, kd, vd)), par, np64(kc), np64(vc), [70, 30], 0.125)
    check(np64(got), ref, mag, smax, 74, 64, dtype)
    status.zero_()
    ok = i32([[-1, 0, 1, 2]] * 2)
    got = K.tree_attention(q, kd, vd, ok, kc, vc, i32([71, -5]), status=status)
    assert status.item() == bit(SHAPE)
    assert torch.equal(got, K.tree_attention(q, kd, vd, ok, kc, vc, i32([70, 0])))


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float16, 64),
                                      (torch.float32, 64), (torch.bfloat16, 12)])
@pytest.mark.parametrize("group", [2, 40])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
@pytest.mark.parametrize("cap", [200, 1000])
def test_tree_branch_that_is_not_finite_stays_in_its_branch(dtype, hd, group, bad, cap):
    K = kv()
    q, kd, vd, kc, vc = tree_inputs(4, dtype, 1, 6, cap, group, 1, hd)
    par = [[-1, 0, 0, 1, 2, -2]]  # branches 0-1-3 and 0-2-4, one padding node
    vd[0, 5], kd[0, 5], q[0, 5] = NAN, NAN, NAN
    clean = np64(vd)
    clean[0, 5], clean[0, 2, 0, 3] = 0.0, 0.0
    vd[0, 2, 0, 3] = bad
    got = np64(K.tree_attention(q, kd, vd, i32(par), kc, vc, i32([190])))
    q[0, 5] = 0
    ref, mag, smax = tree_reference(np64(q), np.nan_to_num(np64(kd)), clean, par, np64(kc),
                                    np64(vc), [190], hd ** -0.5)
    hit = got[0, [2, 4], :, 3]
    assert np.isnan(hit).all() if bad != bad else (hit == bad).all()
    got[0, [2, 4], :, 3] = ref[0, [2, 4], :, 3]
    assert np.isfinite(got).all()
    check(got, ref, mag, smax, 200, hd, dtype)


@pytest.mark.parametrize("dtype", DT)
def test_tree_views_broadcast_and_default_lengths(dtype):
    """One cache shared by every entry (stride 0), heads-first caches, one key head for all."""
    K = kv()
    q, kd, vd, kc, vc = tree_inputs(8, dtype, 3, 5, 130, 4, 2, 64)
    par = [[-1, 0, 1, 1, 0]] * 3
    shared_k, shared_v = kc[:1].expand(3, -1, -1, -1), vc[:1].expand(3, -1, -1, -1)
    got = K.tree_attention(q, kd, vd, i32(par), shared_k, shared_v)
    ref = K.tree_attention(q, kd, vd, i32(par), shared_k.contiguous(), shared_v.contiguous())
    assert torch.equal(got, ref)
    hk, hv = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kc, vc))
    out = torch.empty(3, 4, 5, 64, dtype=dtype, device="cuda").transpose(1, 2)
    K.tree_attention(q, kd, vd, i32(par), hk, hv, i32([130, 7, 64]), out=out)
    assert torch.equal(out, K.tree_attention(q, kd, vd, i32(par), kc, vc, i32([130, 7, 64])))
    one_k, one_v = kc[:, :, :1].expand(-1, -1, 2, -1), vc[:, :, :1].expand(-1, -1, 2, -1)
    got = K.tree_attention(q, kd, vd, i32(par), one_k, one_v)
    assert torch.equal(got, K.tree_attention(q, kd, vd, i32(par), one_k.contiguous(),
                                             one_v.contiguous()))


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_tree_without_a_cache(dtype, hd):
    K = kv()
    q, kd, vd, kc, vc = tree_inputs(9, dtype, 2, 5, 0, 4, 2, hd)
    par = [[-1, 0, 1, 1, 0]] * 2
    got = K.tree_attention(q, kd, vd, i32(par), kc, vc)
    ref, mag, smax = tree_reference(*map(np64, (q, kd, vd)), par, np64(kc), np64(vc), [0, 0],
                                    hd ** -0.5)
    check(np64(got), ref, mag, smax, 5, hd, dtype)


def test_offsets_beyond_32_bits():
    """Cache rows 2^20 elements apart: row 4,095 lies past 2^32 bytes and past 2^31 elements."""
    K = kv()
    n, step = 4096, 1 << 20
    flat = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
    kc = flat.view(1, n, step)[:, :, :128].view(1, n, 1, 128)
    vc = flat.view(1, n, step)[:, :, 256:384].view(1, n, 1, 128)
    q, kd, vd, k0, v0 = tree_inputs(12, torch.bfloat16, 1, 2, n, 4, 1, 128)
    kc.copy_(k0)
    vc.copy_(v0)
    par = i32([[-1, 0]])
    assert torch.equal(K.tree_attention(q, kd, vd, par, kc, vc),
                       K.tree_attention(q, kd, vd, par, k0, v0))
    kp, vp = kc[0], vc[0]
    qp = randn(gen(13), n, 4, 128, dtype=torch.bfloat16)
    cu = i32([0, n - 300, n])
    assert torch.equal(K.prompt_attention(qp, kp, vp, cu), K.prompt_attention(qp, k0[0], v0[0], cu))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    ref = K.apply_rope(k0[0], pos)
    assert torch.equal(K.apply_rope(kp, pos, out=kp), ref)


# ------------------------------------------------------------------------------------------------
# Streams, captured calls, repeated calls, the whole path

@pytest.mark.parametrize("dtype", DT)
def test_repeated_calls_are_bit_equal(dtype):
    K = kv()
    g = gen(14)
    q, k, v = (randn(g, 900, 4, 64, dtype=dtype), randn(g, 900, 2, 64, dtype=dtype),
               randn(g, 900, 2, 64, dtype=dtype))
    cu = i32([0, 500, 900])
    a = K.prompt_attention(q, k, v, cu)
    t = tree_inputs(15, dtype, 3, 9, 800, 4, 2, 64)
    par, nc = i32([[-1, 0, 1, 0, 3, 3, 2, 7, 7]] * 3), i32([800, 5, 400])
    b = K.tree_attention(*t[:3], par, *t[3:], nc)
    for _ in range(3):
        assert torch.equal(a, K.prompt_attention(q, k, v, cu))
        assert torch.equal(b, K.tree_attention(*t[:3], par, *t[3:], nc))


@pytest.mark.parametrize("dtype", DT)
def test_two_streams_at_once(dtype):
    """Calls that overlap on two streams, with no workspace given, do not disturb each other."""
    K = kv()
    ins = [tree_inputs(20 + i, dtype, 2, 9, 3001, 4, 2, 64) for i in range(2)]
    par, nc = i32([[-1, 0, 1, 0, 3, 3, 2, 7, 7]] * 2), i32([3001, 1234])
    want = [K.tree_attention(*t[:3], par, *t[3:], nc) for t in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(K.tree_attention(*ins[i][:3], par, *ins[i][3:], nc, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("dtype", DT)
def test_captured_calls_follow_their_inputs(dtype):
    """Two graphs of a step; replayed after the lengths, the tree and the data changed."""
    K = kv()
    t = tree_inputs(30, dtype, 2, 6, 500, 4, 2, 64)
    par, nc = i32([[-1, 0, 1, 0, 3, -2]] * 2), i32([100, 3])
    g = gen(31)
    q, k, v = (randn(g, 300, 4, 64, dtype=dtype), randn(g, 300, 2, 64, dtype=dtype),
               randn(g, 300, 2, 64, dtype=dtype))
    cu, pos = i32([0, 100, 300]), torch.arange(300, dtype=torch.int32, device="cuda")
    K.tree_attention(*t[:3], par, *t[3:], nc)  # loads the kernels
    K.prompt_attention(K.apply_rope(q, pos), k, v, cu)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        tree_out = K.tree_attention(*t[:3], par, *t[3:], nc)
    with torch.cuda.graph(gb):
        second = K.tree_attention(*t[:3], par, *t[3:], nc)
        prompt_out = K.prompt_attention(K.apply_rope(q, pos), k, v, cu)
    for lengths, cuts in (([500, 77], [0, 299, 300]), ([0, 1], [5, 6, 250])):
        nc.copy_(i32(lengths))
        cu.copy_(i32(cuts))
        par[0, 5] = 1 if lengths[0] else -2
        pos.add_(1000)
        prompt_out.zero_()
        q.mul_(-1.0)
        gb.replay()
        ga.replay()
        torch.cuda.synchronize()
        want = K.tree_attention(*t[:3], par, *t[3:], nc)
        assert torch.equal(tree_out, want) and torch.equal(second, want)
        full = torch.zeros_like(q)
        K.prompt_attention(K.apply_rope(q, pos), k, v, cu, out=full)
        assert torch.equal(prompt_out, full)


def test_default_stream_and_given_stream_agree():
    K = kv()
    x = randn(gen(40), 64, 2, 64, dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = K.prompt_attention(x, x, x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, K.prompt_attention(x, x, x))


def test_binding_refuses_on_the_device():
    K = kv()
    x = randn(gen(41), 8, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    for call in (lambda: K.apply_rope(x, pos.long()), lambda: K.apply_rope(x, pos[:4]),
                 lambda: K.apply_rope(x.transpose(1, 2), pos),
                 lambda: K.prompt_attention(x, x[:4], x),
                 lambda: K.prompt_attention(x, x, x, pos.cpu()),
                 lambda: K.prompt_attention(x, x, x, status=pos),
                 lambda: K.tree_attention(x[None], x[None], x[None], pos, x[None], x[None]),
                 lambda: K.tree_attention(x[None], x[None], x[None], pos[None], x[None], x[None],
                                          pos)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: K.prompt_attention(x, x.float(), x), lambda: K.apply_rope(x.double(), pos)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(K.IskvError):
        K.prompt_attention(x[:, :1].expand(8, 3, 64), x, x)  # 3 query heads over 2


def test_the_whole_path_of_a_layer():
    """Prompt: rotate, attend, select, partition, compress. Draft: reconstruct, attend over the tree;
    each step against float64 on the step's own inputs."""
    K = kv()
    L, nq, nkv, hd, T, W = 200, 4, 2, 64, 5, 8
    d, dt = nkv * hd, torch.float32
    g = gen(50)
    q, k, v = (randn(g, L, nq, hd, dtype=dt), randn(g, L, nkv, hd, dtype=dt),
               randn(g, L, nkv, hd, dtype=dt))
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    qr, kr = K.apply_rope(q, pos), K.apply_rope(k, pos)
    out = K.prompt_attention(qr, kr, v)
    ref, mag, smax = prompt_reference(np64(qr), np64(kr), np64(v), [0, L], hd ** -0.5)
    check(np64(out), ref, mag, smax, L, hd, dt)
    sel = K.select_prompt_blocks(kr, per_head=2, suffix_blocks=2, v_radius=8)
    n_pk, n_pv = (int(c) for c in sel["counts"][:2].tolist())
    sides = []
    for rows, P, win in ((k, sel["P_K"][:n_pk], 0), (v, sel["P_V"][:n_pv], W)):
        tab = K.ExactTable(d, 256, window=W, block=16, reorth_rows=0, dtype=dt)
        comp, cpos = K.cache_prefill(tab, rows.reshape(L, d).contiguous(), P, win)
        hist = K.LowRankHistory(d, d, 512, storage=dt)
        K.compress_prompt(hist, comp, cpos, block=16)
        sides.append((tab, hist))
    n = L
    cache = torch.zeros(2, 1, n, d, dtype=dt, device="cuda")
    exact = [t.exact() for t, _ in sides]
    K.reconstruct_batched([h for _, h in sides], [e[0] for e in exact], [e[1] for e in exact], n,
                          nkv, hd, [True, False], outs=[cache[0, 0], cache[1, 0]])
    # full rank: the cache is the prompt's own keys and values, to the fold's float32 accuracy
    assert (cache[0, 0].view(L, nkv, hd) - kr).norm() <= 1e-4 * kr.norm()
    par = [[-1, 0, 0, 1, 2]]
    depth = i32([0, 1, 1, 2, 2]) + n
    qd = K.apply_rope(randn(g, T, nq, hd, dtype=dt), depth)[None]
    kd = K.apply_rope(randn(g, T, nkv, hd, dtype=dt), depth)[None]
    vd = randn(g, 1, T, nkv, hd, dtype=dt)
    kc, vc = (c.view(1, n, nkv, hd) for c in cache)
    got = K.tree_attention(qd, kd, vd, i32(par), kc, vc)
    ref, mag, smax = tree_reference(*map(np64, (qd, kd, vd)), par, np64(kc), np64(vc), [n], hd ** -0.5)
    check(np64(got), ref, mag, smax, n + T, hd, dt)
    # one drafted token at position n: the same attention on the factors, plus the token itself
    one = K.tree_attention(qd[:, :1], kd[:, :1], vd[:, :1], i32([[-2]]), kc, vc)
    assert not one.any()
    flat = K.tree_attention(qd[:, :1], kc[:, -1:], vc[:, -1:], i32([[-1]]), kc, vc, i32([n - 1]))
    (kt, hk), (vt, hv) = sides
    comp = K.decode_attention(hk, hv, *kt.exact(), *vt.exact(), n, qd[0, 0].contiguous(), nkv, hd)
    assert (flat[0, 0] - comp).norm() <= 1e-4 * comp.norm()
