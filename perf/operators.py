"""Cases and plain forms of the dense-attention operators that stand beside the compressed cache.

Three operators, as a program that serves a model through this package meets them:

- ``rope``: rotate-half rotary embedding of packed rows at given positions (queries and keys before
  a prompt's attention or a drafted tree's; ``inverse`` takes keys of a rotated cache back to the
  unrotated rows that the compression stores),
- ``prompt``: causal attention over whole prompts, packed one behind another, grouped heads,
- ``tree``: attention of a tree of drafted tokens over a dense (reconstructed) cache and over the
  drafted rows themselves; one drafted token is plain decoding.

``run`` with ``own`` false computes them with elementary torch operations in 32 bits (angles in 64),
rounded once at the end; with ``own`` true it makes the package's calls. ``exact`` computes them in
64 bits from the definition.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
THETA = 500000.0  # the package's default base

# The head layout of the benchmark's 32-layer model: 32 query heads over 8 key/value heads of 128
# (rows of d = 1024).
_MODEL = {"n_q": 32, "n_kv": 8, "hd": 128}


def _rope(name, dtype, tokens, heads, hd, start, seqs=1, inverse=False):
    return {"name": name, "op": "rope", "dtype": dtype, "tokens": tokens, "heads": heads, "hd": hd,
            "start": start, "seqs": seqs, "inverse": inverse}


def _prompt(name, dtype, lens, n_q, n_kv, hd):
    return {"name": name, "op": "prompt", "dtype": dtype, "lens": "+".join(map(str, lens)),
            "n_q": n_q, "n_kv": n_kv, "hd": hd}


def _tree(name, dtype, batch, nodes, ctx, n_q, n_kv, hd, ragged, absent):
    return {"name": name, "op": "tree", "dtype": dtype, "batch": batch, "nodes": nodes, "ctx": ctx,
            "n_q": n_q, "n_kv": n_kv, "hd": hd, "ragged": ragged, "absent": absent}


def listed():
    return [
        # 16 drafted tokens behind a cache of 19,584 rows: query and key heads of one fused
        # projection, rotated together. A launch's latency is all there is.
        _rope("rope_draft_bf16", "bf16", 16, 40, 128, 19584),
        # The query heads of a 32K-token prompt: pure bandwidth.
        _rope("rope_prompt_bf16", "bf16", 32768, 32, 128, 0),
        # Rotated float32 keys of three packed sequences, odd length and head size, taken back to
        # unrotated rows before they are compressed.
        _rope("rope_back_fp32", "fp32", 5001, 8, 96, 0, seqs=3, inverse=True),
        # One short chat turn: latency.
        _prompt("prompt_short_bf16", "bf16", [77], **_MODEL),
        # A serving batch of prompts of very different lengths, from one token to 5,000.
        _prompt("prompt_packed_bf16", "bf16", [1, 129, 4096, 517, 2048, 33, 5000, 777], **_MODEL),
        # fp16 with a key/value head per query head, small heads.
        _prompt("prompt_packed_fp16", "fp16", [2000, 2048, 1, 1500], 16, 16, 64),
        # A 32K-token prompt of the benchmark's model: one layer.
        _prompt("prompt_long_bf16", "bf16", [32768], **_MODEL),
        # float32 storage, the accuracy mode, a group of three query heads.
        _prompt("prompt_packed_fp32", "fp32", [700, 300, 65], 12, 4, 64),
        # Plain decoding of one token over a short cache: latency.
        _tree("tree_token_bf16", "bf16", 1, 1, 513, ragged=False, absent=False, **_MODEL),
        # 16 drafted tokens over one reconstructed cache of the benchmark's policy leg.
        _tree("tree_draft_bf16", "bf16", 1, 16, 19584, ragged=False, absent=False, **_MODEL),
        # A batch of eight sequences of different lengths, trees padded to 48 nodes.
        _tree("tree_batch_bf16", "bf16", 8, 48, 16384, ragged=True, absent=True, **_MODEL),
        # float32 storage, odd sizes, a group of five query heads.
        _tree("tree_batch_fp32", "fp32", 3, 7, 1501, 10, 2, 64, ragged=True, absent=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "tree"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    n_q, n_kv, hd = rng.choice([(32, 8, 128), (32, 8, 128), (32, 4, 128), (16, 16, 64), (28, 4, 128),
                                (8, 1, 64), (10, 2, 64), (6, 3, 96), (8, 2, 80), (12, 4, 64)])
    if op == "rope":
        tokens = _log(rng, 1, 32768)
        return _rope_case(rng, dtype, tokens, rng.choice([n_q, n_kv, n_q + n_kv]), hd)
    if op == "prompt":
        total = _log(rng, 1, 16384 if dtype != "fp32" else 2500)
        seqs = min(total, _log(rng, 1, 24))
        cuts = sorted(rng.sample(range(1, total), seqs - 1)) if seqs > 1 else []
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        case = _prompt("", dtype, lens, n_q, n_kv, hd)
    else:
        batch = _log(rng, 1, 16)
        ctx = _log(rng, 1, (131072 if dtype != "fp32" else 16384) // batch)
        nodes = _log(rng, 1, 64)
        case = _tree("", dtype, batch, nodes, ctx, n_q, n_kv, hd, rng.random() < 0.6,
                     rng.random() < 0.5)
    del case["name"]
    return case


def _rope_case(rng, dtype, tokens, heads, hd):
    case = _rope("", dtype, tokens, heads, hd, rng.choice([0, _log(rng, 1, 1 << 20)]),
                 seqs=min(tokens, rng.choice([1, 1, 3, 8])), inverse=rng.random() < 0.3)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------------
# Inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, gain=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(gain).to(dtype)


def _keys(g, lead, heads, hd, dtype):
    # Keys share a direction per head (the outlier channels of trained models' keys), so that
    # scores spread over several units and differ between keys.
    bias = torch.randn((heads, hd), generator=g, device="cuda")
    x = torch.randn((*lead, heads, hd), generator=g, device="cuda")
    return x.add_(bias, alpha=0.5).to(dtype)


def _cpu_rng(case, seed):
    import random
    return random.Random(repr((seed, sorted((k, v) for k, v in case.items() if k != "name"))))


def _parents(rng, nodes, absent):
    """A drafted tree in topological order: each node a child of one of the nodes just before it
    (or of the last cached token, -1); with ``absent`` the tail is padding (-2)."""
    live = nodes if not absent else rng.randint(max(1, nodes // 2), nodes)
    return [(-1 if i == 0 else max(-1, i - rng.randint(1, 4))) if i < live else -2
            for i in range(nodes)]


def prepare(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    if case["op"] == "rope":
        n, s = case["tokens"], case["seqs"]
        per = -(-n // s)
        pos = torch.arange(n, device="cuda") % per + case["start"]
        return {"case": case, "x": _keys(g, (n,), case["heads"], case["hd"], dt),
                "pos": pos.to(torch.int32)}
    n_q, n_kv, hd = case["n_q"], case["n_kv"], case["hd"]
    if case["op"] == "prompt":
        lens = [int(x) for x in case["lens"].split("+")]
        total = sum(lens)
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        return {"case": case, "lens": lens, "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
                "q": _randn(g, (total, n_q, hd), dt, 1.5), "k": _keys(g, (total,), n_kv, hd, dt),
                "v": _randn(g, (total, n_kv, hd), dt)}
    b, t, ctx = case["batch"], case["nodes"], case["ctx"]
    rng = _cpu_rng(case, seed)
    n_ctx = [rng.randint(max(1, ctx // 8), ctx) if case["ragged"] else ctx for _ in range(b)]
    parents = [_parents(rng, t, case["absent"]) for _ in range(b)]
    return {"case": case, "n_ctx": n_ctx,
            "n_cached": torch.tensor(n_ctx, dtype=torch.int32, device="cuda"),
            "parents": torch.tensor(parents, dtype=torch.int32, device="cuda"),
            "q": _randn(g, (b, t, n_q, hd), dt, 1.5), "k_draft": _keys(g, (b, t), n_kv, hd, dt),
            "v_draft": _randn(g, (b, t, n_kv, hd), dt),
            "k_cache": _keys(g, (b, ctx), n_kv, hd, dt),
            "v_cache": _randn(g, (b, ctx, n_kv, hd), dt)}


# ------------------------------------------------------------------------------------------------
# One pass

def run(state):
    op = state["case"]["op"]
    if own:
        import kv_cache_online_b200 as kv
        if op == "rope":
            return kv.apply_rope(state["x"], state["pos"], THETA, inverse=state["case"]["inverse"])
        if op == "prompt":
            return kv.prompt_attention(state["q"], state["k"], state["v"], state["cu"])
        return kv.tree_attention(state["q"], state["k_draft"], state["v_draft"], state["parents"],
                                 state["k_cache"], state["v_cache"], state["n_cached"])
    return {"rope": _plain_rope, "prompt": _plain_prompt, "tree": _plain_tree}[op](state)


def _plain_rope(state):
    x, pos = state["x"], state["pos"]
    hd = x.shape[-1]
    half = hd // 2
    freq = THETA ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / hd)
    ang = pos.double()[:, None] * freq
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if state["case"]["inverse"]:
        sin = -sin
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)


def _attend(q, k, v, visible, scale):
    """q (rows, n_q, hd), k and v (keys, n_kv, hd), visible (rows, keys) or None: softmax attention
    in 32 bits; rows that see nothing give zeros."""
    rows, n_q, hd = q.shape
    n_kv = k.shape[1]
    g = n_q // n_kv
    qh = q.float().view(rows, n_kv, g, hd).permute(1, 2, 0, 3).reshape(n_kv, g * rows, hd)
    s = torch.matmul(qh, k.float().permute(1, 2, 0)).mul_(scale).view(n_kv, g, rows, -1)
    if visible is not None:
        s.masked_fill_(~visible, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n_kv, g * rows, -1), v.float().permute(1, 0, 2)).view(n_kv, g, rows, hd)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(2, 0, 1, 3).reshape(rows, n_q, hd)


def _plain_prompt(state):
    q, k, v = state["q"], state["k"], state["v"]
    out = torch.empty_like(q)
    scale = 1.0 / math.sqrt(q.shape[-1])
    start = 0
    for n in state["lens"]:
        # Rows in chunks that keep the score matrix of all heads near 4 GB.
        step = max(1, min(n, (1 << 30) // (q.shape[1] * n)))
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            i = torch.arange(r0, r1, device=q.device)[:, None]
            j = torch.arange(r1, device=q.device)[None]
            out[start + r0:start + r1] = _attend(q[start + r0:start + r1], k[start:start + r1],
                                                 v[start:start + r1], j <= i, scale).to(q.dtype)
        start += n
    return out


def _closure(parents):
    """(batch, nodes, nodes) booleans: node i sees node j (itself or an ancestor of its own)."""
    b, t = parents.shape
    idx = torch.arange(t, device=parents.device)
    reach = ((parents[:, :, None] == idx) | (idx[:, None] == idx)).float()
    for _ in range(max(1, (t - 1).bit_length())):
        reach = (torch.matmul(reach, reach) > 0).float()
    return (reach > 0) & (parents > -2)[:, :, None]


def _plain_tree(state):
    q = state["q"]
    b, t, _, hd = q.shape
    sees = _closure(state["parents"])
    out = torch.empty_like(q)
    for i, n in enumerate(state["n_ctx"]):
        k = torch.cat([state["k_cache"][i, :n], state["k_draft"][i]])
        v = torch.cat([state["v_cache"][i, :n], state["v_draft"][i]])
        live = (state["parents"][i] > -2)[:, None].expand(t, n)
        vis = torch.cat([live, sees[i]], 1)
        out[i] = _attend(q[i], k, v, vis, 1.0 / math.sqrt(hd)).to(q.dtype)
    return out


# ------------------------------------------------------------------------------------------------
# Work and the exact values

def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "rope":
        elems = case["tokens"] * case["heads"] * case["hd"]
        return {"bytes": 2 * elems * e + 4 * case["tokens"], "flops": 3 * elems}
    n_q, n_kv, hd = case["n_q"], case["n_kv"], case["hd"]
    if case["op"] == "prompt":
        lens = [int(x) for x in case["lens"].split("+")]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": 2 * sum(lens) * (n_q + n_kv) * hd * e + 4 * (len(lens) + 1),
                "flops": 4 * hd * n_q * pairs}
    b, t = case["batch"], case["nodes"]
    # Ragged lengths are drawn evenly between an eighth of the longest and the longest.
    keys = b * case["ctx"] * (0.5625 if case["ragged"] else 1.0)
    live = 0.75 if case["absent"] else 1.0
    return {"bytes": int(2 * keys * n_kv * hd * e + 2 * b * t * (n_q + n_kv) * hd * e + 4 * b * (t + 1)),
            "flops": int(4 * hd * n_q * t * live * (keys + b * min(t, 8)))}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        x = st["x"].double()
        n, h, hd = x.shape
        half = hd // 2
        j = torch.arange(half, device="cuda", dtype=torch.float64)
        ang = torch.outer(st["pos"].double(), torch.exp(j * (-2.0 / hd * math.log(THETA))))
        z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
        turn = torch.polar(torch.ones_like(ang), -ang if case["inverse"] else ang)
        z = z * turn[:, None]
        return torch.cat([z.real, z.imag], -1)
    n_q, n_kv, hd = case["n_q"], case["n_kv"], case["hd"]
    group = n_q // n_kv
    scale = hd ** -0.5
    q = st["q"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")

    def one(qr, kk, vv, bias):
        # One head in 64 bits: rows x hd, keys x hd, additive 0 / -inf.
        s = qr.double() @ kk.double().T * scale + bias
        top = s.max(1, keepdim=True).values
        w = torch.exp(s - torch.clamp(top, min=-1e300))
        den = w.sum(1, keepdim=True)
        return torch.where(den > 0, (w @ vv.double()) / torch.clamp(den, min=1e-300), 0.0)

    if case["op"] == "prompt":
        base = 0
        for n in st["lens"]:
            for r0 in range(0, n, 4096):
                r1 = min(n, r0 + 4096)
                bias = torch.full((r1 - r0, r1), -math.inf, dtype=torch.float64, device="cuda")
                bias = torch.triu(bias, diagonal=r0 + 1)
                for h in range(n_q):
                    out[base + r0:base + r1, h] = one(
                        q[base + r0:base + r1, h], st["k"][base:base + r1, h // group],
                        st["v"][base:base + r1, h // group], bias)
            base += n
        return out
    for i, n in enumerate(st["n_ctx"]):
        par = st["parents"][i].tolist()
        t = len(par)
        bias = torch.full((t, n + t), -math.inf, dtype=torch.float64)
        for node, up in enumerate(par):
            if up < -1:
                continue
            bias[node, :n] = 0.0
            cur = node
            while cur >= 0:
                bias[node, n + cur] = 0.0
                cur = par[cur]
        bias = bias.cuda()
        for h in range(n_q):
            kk = torch.cat([st["k_cache"][i, :n, h // group], st["k_draft"][i, :, h // group]])
            vv = torch.cat([st["v_cache"][i, :n, h // group], st["v_draft"][i, :, h // group]])
            out[i, :, h] = one(q[i, :, h], kk, vv, bias)
    return out
