"""Float64 oracle of the calls on latent rows: attention on the rows of a paged
cache, products per head, attention of prompts with expanded keys and values.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A token's row is shared by all heads: keys and values are linear in its first
elements (what an absorbed query meets directly, what a prompt expands per
head), the rest is a part that carries positions and is a key's only.
"""

import numpy as np

from .tree import paths_to_root


def _attend(q, k, v, scale):
    """One row of queries [H, D] on keys [n, D] (or [n, H, D]) and values
    likewise: (out, spread, reach) as tree.tree_attention."""
    if k.ndim == 2:
        k, v = k[:, None].repeat(len(q), 1), v[:, None].repeat(len(q), 1)
    x = scale * np.einsum("nhd,hd->hn", k, q)
    with np.errstate(invalid="ignore"):
        w = np.exp(x - x.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
    reach = np.abs(scale) * np.einsum("nhd,hd->hn", np.abs(k), np.abs(q)).max(-1)
    return (np.einsum("hn,nhd->hd", w, v), np.einsum("hn,nhd->hd", w, np.abs(v)),
            np.stack((reach, np.full(len(q), float(k.shape[0]))), -1))


def cache_rows(cache, table, length):
    """The rows a sequence's table names; those on pages outside the pool are left out."""
    pages, ps, _ = cache.shape
    j = np.arange(int(np.clip(length, 0, len(table) * ps)))
    j = j[(table[j // ps] >= 0) & (table[j // ps] < pages)]
    return cache[table[j // ps], j % ps]


def attention(q, cache, table, lens, rows, parent=None, n_nodes=None, *, dim_v, scale):
    """(out [B, N, heads, dim_v], spread, reach [B, N, heads, 2]), float64."""
    B, N, H, _ = q.shape
    out, spread, reach = np.zeros((B, N, H, dim_v)), np.zeros((B, N, H, dim_v)), np.zeros((B, N, H, 2))
    chain = np.arange(N) - 1
    for b in range(B):
        n = N if n_nodes is None else int(np.clip(n_nodes[b], 0, N))
        ctx = cache_rows(cache, table[b], lens[b])
        for i, path in enumerate(paths_to_root(chain if parent is None else parent[b], n)):
            k = np.concatenate([ctx, rows[b, path]])
            out[b, i], spread[b, i], reach[b, i] = _attend(q[b, i], k, k[:, :dim_v], scale)
    return out, spread, reach


def head_product(x, w):
    """out[t, h] = w[h] x[t, h], and sum_k |x| |w| (what a rounding of the sum is worth)."""
    return np.einsum("thk,hmk->thm", x, w), np.einsum("thk,hmk->thm", np.abs(x), np.abs(w))


def prompt(q, cache, table, lens, q_start, w_k, w_v, scale=None):
    """(out [T, heads, dim_v], spread, reach, loose): as attention, with reach
    [T, heads, 3] = largest scale * sum |q k|, number of keys, and what float32
    sums over the latent dimensions and the smallest float16 are worth in a
    score; loose: the same for the values.  Rows of no sequence are NaN."""
    T, H, D = q.shape
    dv, R = w_v.shape[1:]
    scale = D ** -0.5 if scale is None else scale
    out, spread = np.full((T, H, dv), np.nan), np.zeros((T, H, dv))
    reach, loose = np.zeros((T, H, 3)), np.zeros((T, H, dv))
    for b in range(len(lens)):
        s, e = int(q_start[b]), int(q_start[b + 1])
        if not 0 <= s < e <= T:
            continue
        length = int(np.clip(lens[b], 0, table.shape[1] * cache.shape[1]))
        j = np.arange(length)
        pg = table[b, j // cache.shape[1]] if length else j
        j = j[(pg >= 0) & (pg < cache.shape[0])]
        c = cache_rows(cache, table[b], length)
        for h in range(H):
            k = np.concatenate([c[:, :R] @ w_k[h].T, c[:, R:]], 1)
            v = c[:, :R] @ w_v[h].T
            k_slack = np.concatenate([R * 2.0 ** -23 * (np.abs(c[:, :R]) @ np.abs(w_k[h]).T) + 2.0 ** -25,
                                      np.zeros((len(c), c.shape[1] - R))], 1)
            v_slack = R * 2.0 ** -23 * (np.abs(c[:, :R]) @ np.abs(w_v[h]).T) + 2.0 ** -25
            for t in range(s, e):
                n = int((j <= length - (e - t)).sum())
                if n == 0:
                    out[t, h] = 0.0
                    continue
                with np.errstate(invalid="ignore"):
                    x = scale * (k[:n] @ q[t, h])
                    w = np.exp(x - x.max())
                    w /= w.sum()
                out[t, h], spread[t, h], loose[t, h] = w @ v[:n], w @ np.abs(v[:n]), w @ v_slack[:n]
                a = abs(scale) * np.abs(q[t, h])
                reach[t, h] = (np.abs(k[:n]) @ a).max(), n, (k_slack[:n] @ a).max()
    return out, spread, reach, loose
