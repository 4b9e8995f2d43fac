"""What the rotary embedding and the dense attention refuse, on the host before any CUDA call."""

import ctypes
import subprocess
import sys

import pytest
import torch

from conftest import ROOT


def _lib():
    from kv_cache_online_b200 import build
    build.build()
    from kv_cache_online_b200 import _lib as L
    return L, L.load()


ARG, SHAPE, WORKSPACE = 1, 2, 8
P = 0x10000  # never dereferenced


def _h(L, batch=4096, row=1024, head=128, data=P):
    return L.IskvHeads(data, batch, row, head)


def _rope(L, lib, x=None, pos=P, n=4, heads=8, hd=128, theta=1e4, dtype=1, out=None):
    return lib.iskv_rope(x or _h(L), pos, n, heads, hd, theta, 0, dtype, out or _h(L), None)


def _prompt(L, lib, q=None, k=None, v=None, cu=P, seqs=2, rows=16, nq=8, nkv=8, hd=128, scale=0.1,
            dtype=1, out=None, status=None):
    return lib.iskv_prompt_attention(q or _h(L), k or _h(L), v or _h(L), cu, seqs, rows, nq, nkv, hd,
                                     scale, dtype, out or _h(L), status, None)


def _tree(L, lib, q=None, kd=None, vd=None, parents=P, kc=None, vc=None, ncached=None, batch=2,
          nodes=4, cap=16, nq=8, nkv=8, hd=128, scale=0.1, dtype=1, out=None, status=None, ws=P,
          ws_bytes=1 << 30):
    return lib.iskv_tree_attention(q or _h(L), kd or _h(L), vd or _h(L), parents, kc or _h(L),
                                   vc or _h(L), ncached, batch, nodes, cap, nq, nkv, hd, scale, dtype,
                                   out or _h(L), status, ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (ARG, {"dtype": 7}), (SHAPE, {"hd": 127}), (SHAPE, {"hd": 0}), (SHAPE, {"hd": 258}),
    (SHAPE, {"heads": 0}), (SHAPE, {"heads": 1025}), (SHAPE, {"n": -1}), (SHAPE, {"n": 1 << 31}),
    (ARG, {"theta": 0.0}), (ARG, {"theta": float("nan")}), (ARG, {"theta": float("inf")}),
    (ARG, {"pos": None}), (ARG, {"pos": P + 2}), (ARG, {"x": (0, 1, 1, 0)}),
    (ARG, {"x": (0, 1024, 128, P + 1)}), (SHAPE, {"x": (0, -1, 128, P)}),
    (SHAPE, {"out": (0, 0, 128, 2 * P)}), (SHAPE, {"out": (0, 1024, 0, 2 * P)}),
    (ARG, {"out": (0, 2048, 128, P)}),  # in place with other strides
])
def test_rope_refuses(want, kw):
    L, lib = _lib()
    kw = {k: _h(L, *v) if isinstance(v, tuple) else v for k, v in kw.items()}
    assert _rope(L, lib, **kw) == want
    assert lib.iskv_last_error().startswith(b"iskv_rope")


@pytest.mark.parametrize("want,kw", [
    (ARG, {"dtype": -1}), (SHAPE, {"nq": 9}), (SHAPE, {"nq": 0}), (SHAPE, {"nkv": 0}),
    (SHAPE, {"nq": 65, "nkv": 1}), (SHAPE, {"nq": 1025, "nkv": 1025}), (SHAPE, {"hd": 0}),
    (SHAPE, {"hd": 257}), (ARG, {"scale": float("inf")}), (ARG, {"scale": float("nan")}),
    (SHAPE, {"rows": -1}), (SHAPE, {"rows": (1 << 24) + 1}), (SHAPE, {"seqs": -1}),
    (SHAPE, {"seqs": 4097}), (ARG, {"cu": None}), (ARG, {"cu": P + 1}), (ARG, {"status": P + 4}),
    (ARG, {"q": (0, 1, 1, 0)}), (ARG, {"k": (0, 1, 1, P + 1)}), (SHAPE, {"v": (0, 1, -1, P)}),
    (SHAPE, {"k": (0, 1 << 36, 1, P)}), (SHAPE, {"out": (0, 0, 128, P)}),
    (SHAPE, {"out": (0, 1024, 0, P)}), (SHAPE, {"rows": 1 << 24, "nq": 16384, "nkv": 256}),
])
def test_prompt_attention_refuses(want, kw):
    L, lib = _lib()
    kw = {k: _h(L, *v) if isinstance(v, tuple) else v for k, v in kw.items()}
    assert _prompt(L, lib, **kw) == want
    assert lib.iskv_last_error().startswith(b"iskv_prompt_attention")


@pytest.mark.parametrize("want,kw", [
    (ARG, {"dtype": 3}), (SHAPE, {"nq": 7}), (SHAPE, {"hd": 300}), (ARG, {"scale": float("-inf")}),
    (SHAPE, {"batch": -1}), (SHAPE, {"batch": 4097}), (SHAPE, {"nodes": -1}), (SHAPE, {"nodes": 129}),
    (SHAPE, {"cap": -1}), (SHAPE, {"cap": 1 << 31}), (ARG, {"parents": None}),
    (ARG, {"parents": P + 2}), (ARG, {"ncached": P + 2}), (ARG, {"status": P + 4}),
    (ARG, {"kc": (0, 1, 1, 0)}), (ARG, {"vd": (0, 1, 1, 0)}), (SHAPE, {"q": (-1, 1, 1, P)}),
    (SHAPE, {"out": (0, 1024, 128, P)}), (SHAPE, {"out": (4096, 0, 128, P)}),
    (SHAPE, {"out": (4096, 1024, 0, P)}),
    (SHAPE, {"batch": 4096, "nodes": 128, "nq": 512, "cap": 1 << 20}), (WORKSPACE, {"ws": None}), (WORKSPACE, {"ws": P + 16}),
    (WORKSPACE, {"ws_bytes": 4096}),
])
def test_tree_attention_refuses(want, kw):
    L, lib = _lib()
    kw = {k: _h(L, *v) if isinstance(v, tuple) else v for k, v in kw.items()}
    assert _tree(L, lib, **kw) == want
    assert lib.iskv_last_error().startswith(b"iskv_tree_attention")


def test_empty_calls_need_no_device():
    L, lib = _lib()
    nil = _h(L, data=0)
    assert _rope(L, lib, x=nil, pos=None, n=0, out=nil) == 0
    assert _prompt(L, lib, q=nil, k=nil, v=nil, cu=None, rows=0, out=nil) == 0
    assert _prompt(L, lib, seqs=0) == 0
    assert _tree(L, lib, batch=0, ws=None) == 0
    assert _tree(L, lib, nodes=0, ws=None) == 0


def test_workspace_query():
    _, lib = _lib()
    f = lib.iskv_tree_attention_workspace_size
    assert f(16, 32, 8, 128) > 0 and f(128, 64, 1, 256) > 0
    assert f(33, 4, 1, 128) > f(32, 4, 1, 128)  # 132 packed rows: larger units
    for bad in ((0, 8, 8, 128), (129, 8, 8, 128), (4, 9, 8, 128), (4, 8, 0, 128), (4, 8, 8, 0),
                (4, 8, 8, 257), (4, 65, 1, 64)):
        assert f(*bad) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    _lib()
    import kv_cache_online_b200 as kv
    x = torch.zeros(4, 2, 8)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kv.apply_rope(x, pos)
    with pytest.raises(ValueError):
        kv.apply_rope(x[0], pos)
    with pytest.raises(ValueError):
        kv.prompt_attention(x, x, x)
    with pytest.raises(ValueError):
        kv.tree_attention(x[None], x[None], x[None], pos[None], x[None], x[None])
    assert ctypes.sizeof(kv.IskvHeads) == 32


def test_the_device_s_error_word_needs_a_place():
    _, lib = _lib()
    assert lib.iskv_dense_status(None, 1) == ARG
    assert lib.iskv_last_error().startswith(b"iskv_dense_status")


def test_the_package_loads_without_cuda_in_torch():
    """The entry points of the host (workspace queries, plans) need no CUDA build of torch."""
    _lib()
    code = ("import torch\n"
            "for name in dir(torch._C):\n"
            "    if name.startswith('_cuda_getCurrent'): delattr(torch._C, name)\n"
            "import kv_cache_online_b200 as kv\n"
            "assert kv.tree_attention_workspace_size(16, 32, 8, 128) > 0\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_scales_beyond_2_to_127_are_refused():
    L, lib = _lib()
    for scale in (3e38, -3e38, 2.0 ** 127 * (1 + 2.0 ** -23)):
        assert _prompt(L, lib, scale=scale) == ARG and _tree(L, lib, scale=scale) == ARG
