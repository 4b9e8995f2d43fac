"""Dense attention where calls meet: what follows a call on its stream, sequences whose bounds
contradict each other, extreme scales, errors without a status word, and the accuracy of float32.

References and element-wise bounds as in ``test_gpu_dense``.
"""

import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from gpu_util import bit, kv, np64
from test_gpu_dense import (SHAPE, check, gen, i32, prompt_reference, randn, tree_inputs,
                            tree_reference)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,b,t,cap,n_cached,nq,nkv", [
    (torch.bfloat16, 3, 5, 1000, 0, 4, 2),     # room for a long cache, nothing in it yet
    (torch.float32, 3, 5, 0, 0, 4, 2),         # no cache at all, CUDA cores
    (torch.float16, 2, 64, 1500, 0, 4, 1),     # two row blocks per head
    (torch.bfloat16, 37, 2, 1000, 1000, 8, 4),  # 148 equal units on 148 shares
    (torch.float32, 37, 2, 100, 100, 8, 8),    # 296 equal units on 296 shares
])
def test_work_behind_a_tree_call_without_cut_units(dtype, b, t, cap, n_cached, nq, nkv):
    """No unit is cut between CTAs, so the second kernel of the call has nothing to add up: a copy
    of the results that follows at once, called and captured, still finds them."""
    K = kv()
    q, kd, vd, kc, vc = tree_inputs(cap + b, dtype, b, t, cap, nq, nkv, 64)
    par, nc = i32([[i - 1 for i in range(t)]] * b), i32([n_cached] * b)
    out, snap = torch.empty_like(q), torch.empty_like(q)

    def call():
        out.fill_(float("nan"))
        K.tree_attention(q, kd, vd, par, kc, vc, nc, out=out)
        snap.copy_(out)

    call()
    torch.cuda.synchronize()
    want = out.clone()
    ref, mag, smax = tree_reference(*map(np64, (q, kd, vd)), par.tolist(), np64(kc), np64(vc),
                                    [n_cached] * b, 0.125)
    check(np64(want), ref, mag, smax, n_cached + t, 64, dtype)
    assert torch.equal(snap, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in (call, graph.replay):
        for _ in range(20):
            snap.zero_()
            step()
            assert torch.equal(snap, want)


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float16, 64),
                                      (torch.float32, 64)])
@pytest.mark.parametrize("cu,good", [
    ([0, 1000, 0, 1000], 1),             # the same rows twice
    ([0, 1000] * 8, 1),
    ([0, 10, 5, 15, 900], 1),            # overlapping by five rows
    ([40, 300, 1001, 700, 900], 1),      # beyond the rows, then inside again
    ([-1, 200, 400, 1000], 0),
    ([500, 400, 600, 1000], 0),
    ([300, -1], 0),
    (list(range(0, 80, 2)) + [0, 500, 1000], 39),  # past the first 32 sequences
])
def test_prompt_sequences_count_up_to_the_first_inconsistent_one(dtype, hd, cu, good):
    """Sequences ahead of the first broken pair are whole, all rows behind stay as they were."""
    K = kv()
    rows = 1000
    q, k, v = (randn(gen(70), rows, h, hd, dtype=dtype) for h in (4, 2, 2))
    out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int64, device="cuda")
    K.prompt_attention(q, k, v, i32(cu), out=out, status=status)
    assert status.item() == bit(SHAPE)
    want = torch.full_like(q, 7.0)
    if good:
        status.zero_()
        K.prompt_attention(q, k, v, i32(cu[:good + 1]), out=want, status=status)
        assert status.item() == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_errors_without_a_status_word_are_kept_by_the_device(dtype):
    K = kv()
    K.dense_status()
    q = randn(gen(71), 64, 2, 64, dtype=dtype)
    K.prompt_attention(q, q, q)
    K.tree_attention(q[None], q[None], q[None], i32([list(range(-1, 63))]), q[None], q[None])
    assert K.dense_status() == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    K.prompt_attention(q, q, q, i32([0, 10, 5]), stream=s)
    assert K.dense_status(reset=False) == K.dense_status("cuda:0") == bit(SHAPE)
    assert K.dense_status() == 0
    for parents, n in ([list(range(64)), 64], [list(range(-1, 63)), 65]):
        K.tree_attention(q[None], q[None], q[None], i32([parents]), q[None], q[None], i32([n]))
        assert K.dense_status() == bit(SHAPE)
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    K.prompt_attention(q, q, q, i32([0, 10, 5]), status=status)
    assert K.dense_status() == 0 and status.item() == bit(SHAPE)


def test_the_first_call_of_a_process_may_be_captured():
    """Kernels and the device's error word are found while a stream is captured."""
    kv()
    code = """
import torch, kv_cache_online_b200 as K
for dtype in (torch.bfloat16, torch.float32):
    q = torch.randn(64, 2, 64, device="cuda").to(dtype)
    cu = torch.tensor([0, 10, 5], dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = K.prompt_attention(q, q, q, cu)
    g.replay()
    assert K.dense_status() == 4, K.dense_status()
    assert torch.equal(out[:10], K.prompt_attention(q[:10], q[:10], q[:10]))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=os.environ, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_a_workspace_of_the_caller_s():
    K = kv()
    q, kd, vd, kc, vc = tree_inputs(72, torch.bfloat16, 2, 5, 1000, 4, 2, 64)
    par = i32([[-1, 0, 1, 1, 0]] * 2)
    n = K.tree_attention_workspace_size(5, 4, 2, 64)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(n, dtype=torch.uint8).pin_memory(),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)):
        with pytest.raises(ValueError):
            K.tree_attention(q, kd, vd, par, kc, vc, ws=ws)
    for ws in (torch.empty(0, dtype=torch.uint8, device="cuda"),
               torch.empty(n - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(n + 16, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(K.IskvError):
            K.tree_attention(q, kd, vd, par, kc, vc, ws=ws)
    # a tensor of any type and shape with enough bytes behind it
    ws = torch.empty(-(-n // 80), 10, dtype=torch.float64, device="cuda")
    want = K.tree_attention(q, kd, vd, par, kc, vc)
    assert torch.equal(K.tree_attention(q, kd, vd, par, kc, vc, ws=ws), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale,gain", [(1e-33, 1e33), (-2.0 ** -115, 2.0 ** 115), (0.0, 1e35),
                                        (1e-40, 1e35), (1e30, 1e-30), (2.0 ** 127, 2.0 ** -125)])
def test_scales_far_from_one(dtype, scale, gain):
    """Tiny scales of huge scores, the largest scale, and 0 whatever the scores: weights still
    follow the product of the two."""
    K = kv()
    nq, nkv, hd, lens = 4, 2, 64, [70, 300]
    g, n = gen(73), 370
    q, k, v = (randn(g, n, h, hd, dtype=dtype) for h in (nq, nkv, nkv))
    q *= gain
    got = K.prompt_attention(q, k, v, i32([0, 70, 370]), scale)
    ref, mag, smax = prompt_reference(np64(q), np64(k), np64(v), [0, 70, 370], scale)
    check(np64(got), ref, mag, smax, max(lens), hd, dtype)
    for t in (5, 100):  # both splits of a tree's rows
        par = [list(range(-1, t - 1))]
        args = [x[:t][None] for x in (q, k, v)]
        got = K.tree_attention(*args, i32(par), k[None], v[None], i32([300]), scale)
        ref, mag, smax = tree_reference(*map(np64, args), par, np64(k[None]), np64(v[None]), [300],
                                        scale)
        check(np64(got), ref, mag, smax, 300 + t, hd, dtype)


def test_heads_without_elements_are_refused_by_the_library():
    K = kv()
    x = torch.empty(4, 2, 0, device="cuda")
    for call in (lambda: K.prompt_attention(x, x, x),
                 lambda: K.tree_attention(x[None], x[None], x[None], i32([[-1, 0, 1, 2]]), x[None],
                                          x[None])):
        with pytest.raises(K.IskvError):
            call()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tensors_dropped_while_another_stream_still_reads_them(dtype):
    """Temporaries of the current stream in a call on another one that is busy: dropped right after
    the call, their memory asked for and overwritten at once."""
    K = kv()
    q, kd, vd, kc, vc = tree_inputs(74, dtype, 2, 9, 1500, 4, 2, 64)
    par, nc = i32([[-1, 0, 1, 0, 3, 3, 2, 7, 7]] * 2), i32([1500, 321])
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    calls = [
        (lambda a, s: K.tree_attention(*a, stream=s), (q, kd, vd, par, kc, vc, nc)),
        (lambda a, s: K.prompt_attention(*a, stream=s), (kc[0], kc[1], vc[0], i32([0, 700, 1500]))),
        (lambda a, s: K.apply_rope(*a, stream=s), (q[0], pos)),
    ]
    s = torch.cuda.Stream()
    for call, args in calls:
        want = call(args, None)
        temps = [x.clone() for x in args]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(50_000_000)
        got = call(temps, s)
        sizes = [x.numel() * x.element_size() for x in temps]
        del temps
        junk = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del junk
