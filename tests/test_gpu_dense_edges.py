"""Dense attention where calls meet: what follows a call on its stream, sequences whose bounds
contradict each other, extreme scales, errors without a status word, and the accuracy of float32.

References and element-wise bounds as in ``test_gpu_dense``.
"""

import pytest
import torch

from gpu_util import kv, np64
from test_gpu_dense import (check, i32, tree_inputs, tree_reference)

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
