"""Dense attention around the compressed cache in float64 (Algorithm 1's exact prompt attention;
Algorithm 3 step 9 over a reconstructed cache, for a tree of drafted tokens)."""

import numpy as np


def _row(q, keys, values, scale):
    """One query row over the keys it sees; zeros when there are none."""
    if len(keys) == 0:
        return np.zeros(values.shape[1])
    s = scale * (keys @ q)
    p = np.exp(s - s.max())
    return (p @ values) / p.sum()


def prompt_attention(q, k, v, cu, scale):
    """q (rows, n_q, hd), k / v (rows, n_kv, hd); sequence s is rows cu[s]:cu[s + 1]. Rows outside
    every sequence stay NaN."""
    out = np.full(q.shape, np.nan)
    group = q.shape[1] // k.shape[1]
    for lo, hi in zip(cu[:-1], cu[1:]):
        for i in range(lo, hi):
            for h in range(q.shape[1]):
                out[i, h] = _row(q[i, h], k[lo:i + 1, h // group], v[lo:i + 1, h // group], scale)
    return out


def ancestors(parents, i):
    """Node i and its ancestors, or an empty list for padding (a chain that does not end in -1)."""
    seen, cur = [], i
    while cur >= 0:
        up = parents[cur]
        if up >= cur or up < -1:
            return []
        seen.append(cur)
        cur = up
    return sorted(seen)


def tree_attention(q, k_draft, v_draft, parents, k_cache, v_cache, n_cached, scale):
    """q (b, t, n_q, hd); drafts (b, t, n_kv, hd); parents (b, t); caches (b, n_cap, n_kv, hd)."""
    out = np.zeros(q.shape)
    group = q.shape[2] // k_draft.shape[2]
    for b in range(q.shape[0]):
        n = int(n_cached[b])
        for i in range(q.shape[1]):
            nodes = ancestors(list(parents[b]), i)
            if not nodes:
                continue
            for h in range(q.shape[2]):
                g = h // group
                keys = np.concatenate([k_cache[b, :n, g], k_draft[b, nodes, g]])
                values = np.concatenate([v_cache[b, :n, g], v_draft[b, nodes, g]])
                out[b, i, h] = _row(q[b, i, h], keys, values, scale)
    return out
