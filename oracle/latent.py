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
