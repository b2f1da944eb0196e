"""Float64 oracle of the tree round: attention of a drafted tree over a paged
cache, verification of the tree from given random numbers, commit and fork of
cache pages.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Sources: the page on LogitSpec (gist.science 2507.01449), section 2 (a draft
tree and its attention mask); the acceptance probability and the corrected
distribution of the page "Speculative Decoding للمحترف", section "التعريف
الرياضي من Leviathan et al."; the page "Faster LLM Inference via Sequential
Monte Carlo", section 2 (particles that share cache pages).

Readings taken where the pages are silent:
  * several drafted children of one node: each was drawn independently from
    the draft's row, and the rule is applied again after every refusal to the
    distribution that is left, renormalised (here literally, row by row);
    children that were chosen rather than drawn have a point mass as their
    draft distribution;
  * free pages are taken lowest number first, in the order of the sequences.
"""

from collections import Counter

import numpy as np


def paths_to_root(parent, n):
    """For each node the list [node, its parent, ...]; a parent outside
    [0, i) ends it."""
    out = []
    for i in range(n):
        path, at = [i], i
        while at > 0 and 0 <= parent[at] < at:
            at = int(parent[at])
            path.append(at)
        out.append(path)
    return out


def visible_rows(length, depth, window, sinks):
    """The cache rows a node at `depth` sees."""
    j = np.arange(length)
    if window <= 0:
        return j
    return j[(length + depth - j < window) | (j < sinks)]


def tree_attention(q, k_cache, v_cache, table, lens, k_tree, v_tree, parent, n_nodes=None, scale=None, window=0,
                   sinks=0):
    """Returns (out, spread, reach), float64: the outputs [B, N, heads, dim];
    sum_j w_j |v_j| / sum_j w_j, what a relative error of the weights is worth;
    and [B, N, heads] the largest scale * sum_d |q_d k_d| and the number of
    keys, what a rounding error of the scores is worth."""
    B, N, H, D = q.shape
    pages, ps, Hkv, _ = k_cache.shape
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros((B, N, H, D))
    spread = np.zeros((B, N, H, D))
    reach = np.zeros((B, N, H, 2))
    for b in range(B):
        n = N if n_nodes is None else int(np.clip(n_nodes[b], 0, N))
        length = int(np.clip(lens[b], 0, table.shape[1] * ps))
        for i, path in enumerate(paths_to_root(parent[b], n)):
            rows = visible_rows(length, len(path) - 1, window, sinks)
            rows = np.array([j for j in rows if 0 <= table[b, j // ps] < pages], dtype=np.int64)
            near = path if window <= 0 else path[:window]
            for h in range(H):
                e = h // (H // Hkv)
                k = np.concatenate([k_cache[table[b, rows // ps], rows % ps, e], k_tree[b, near, e]])
                v = np.concatenate([v_cache[table[b, rows // ps], rows % ps, e], v_tree[b, near, e]])
                x = scale * (k @ q[b, i, h])
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b, i, h] = w @ v
                spread[b, i, h] = w @ np.abs(v)
                reach[b, i, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, i, h])).max(), len(x)
    return out, spread, reach


def _prob_ok(x):
    return bool(np.all(np.isfinite(x)) and np.all(np.asarray(x) >= 0))


def verify_tree_row(p, q, tokens, parent, n, u_accept, u_final):
    """One sequence: (tokens, path, margins), or None if invalid.  p [N, V]
    and q [P, V] (or None) float64; margins: how near each decision was to
    going the other way (relative)."""
    N, V = p.shape
    if not 1 <= n <= N or not 0 <= u_final < 1:
        return None
    for i in range(1, n):
        ok = 0 <= parent[i] < i and 0 <= tokens[i] < V and 0 <= u_accept[i] < 1
        if q is not None:
            ok = ok and parent[i] < len(q)
        if not ok or not _prob_ok(p[parent[i], tokens[i]]):
            return None
        if q is not None and not _prob_ok(q[parent[i], tokens[i]]):
            return None
    here, path, said, margins = 0, [0], [], []
    while True:
        kids = [i for i in range(1, n) if parent[i] == here]
        # the distribution left after s refusals, kept as weights and their sum
        left, total = p[here].copy(), 1.0
        nxt = None
        for s, i in enumerate(kids):
            x = tokens[i]
            if q is None:
                r = left[x] / total if total > 0 else (np.inf if left[x] > 0 else 0.0)
                accept = u_accept[i] * total < left[x]
            else:
                want = u_accept[i] * q[here, x]
                r = left[x] / total / q[here, x] if q[here, x] > 0 and total > 0 else np.inf
                accept = want * total < left[x]
            if np.isfinite(r) and r > 0:  # 0 < 0 fails whatever the rounding
                margins.append(abs(u_accept[i] - r))
            if accept:
                nxt = i
                break
            if q is None:
                total -= left[x]
                left[x] = 0.0
            else:
                # p_{s+1} = max(0, p_s - q), renormalised before the next sibling
                if not (_prob_ok(p[here]) and _prob_ok(q[here])) and s + 1 < len(kids):
                    return None
                scaled = left / total if total > 0 else np.zeros(V)
                left = np.maximum(scaled - q[here], 0.0)
                total = left.sum()
        if nxt is None:
            break
        here = nxt
        path.append(here)
        said.append(int(tokens[here]))
    refused = any(parent[i] == here for i in range(1, n))
    if not _prob_ok(p[here]) or (q is not None and refused and not _prob_ok(q[here])):
        return None
    if not left.sum() > 0:
        left = p[here].copy()
    if not left.sum() > 0:
        return None
    cum = np.cumsum(left)
    at = int(np.searchsorted(cum, u_final * cum[-1], side="right"))
    if at >= V:
        at = int(np.nonzero(left > 0)[0][-1])
    # below the first id with weight there is no border: its running sum starts at 0 exactly
    before = cum[at - 1] if at else 0.0
    margins.append(abs(cum[at] / cum[-1] - u_final))
    if before > 0:
        margins.append(abs(u_final - before / cum[-1]))
    said.append(at)
    return said, path, margins


def verify_tree(p, q, tokens, parent, u_accept, u_final, n_nodes=None):
    """Returns (tokens [B, N], nodes [B, N], n_accepted [B], margin [B])."""
    B, N, _ = p.shape
    out_t, out_n = np.full((B, N), -1, np.int32), np.full((B, N), -1, np.int32)
    count, margin = np.full(B, -1, np.int32), np.ones(B)
    for b in range(B):
        r = verify_tree_row(p[b], None if q is None else q[b], tokens[b], parent[b], N if n_nodes is None else
                            int(n_nodes[b]), u_accept[b].astype(np.float64), float(u_final[b]))
        if r is None:
            continue
        said, path, m = r
        out_t[b, :len(said)], out_n[b, :len(path)] = said, path
        count[b], margin[b] = len(path) - 1, min(m)
    return out_t, out_n, count, margin


def _blocks(rows, ps):
    return -(-rows // ps)


def _lowest_free(rows, pages):
    used = {x for r in rows for x in r}
    return [x for x in range(pages) if x not in used]


def _as_table(rows, width):
    return np.array([list(r) + [-1] * (width - len(r)) for r in rows], dtype=np.int32)


def _unchanged(table, lens, ps, status):
    width = table.shape[1]
    live = [table[b, :_blocks(int(np.clip(n, 0, width * ps)), ps)] for b, n in enumerate(lens)]
    return _as_table(live, width), np.array(lens, dtype=np.int32), status


def cache_commit(k, v, table, lens, k_tree, v_tree, nodes, n_accepted):
    """In place on k and v [layers, pages, ps, heads, dim]; returns (table,
    lens, status)."""
    pages, ps, N = k.shape[1], k.shape[2], k_tree.shape[2]
    B, width = table.shape
    rows, move = [], []
    for b in range(B):
        take = max(0, int(n_accepted[b]) + 1)
        if not 0 <= lens[b] <= width * ps or take > N or lens[b] + take > width * ps:
            return _unchanged(table, lens, ps, -1)
        at = list(range(take)) if nodes is None else [int(x) for x in nodes[b, :take]]
        live = [int(x) for x in table[b, :_blocks(int(lens[b]), ps)]]
        if any(not 0 <= x < N for x in at) or any(not 0 <= x < pages for x in live):
            return _unchanged(table, lens, ps, -1)
        rows.append(live)
        move.append(at)
    # a page that is appended to belongs to one sequence only
    named = Counter(x for r in rows for x in r)
    if any(at and lens[b] % ps and named[rows[b][-1]] > 1 for b, at in enumerate(move)):
        return _unchanged(table, lens, ps, -1)
    free = _lowest_free(rows, pages)
    need = [_blocks(int(lens[b]) + len(move[b]), ps) - len(rows[b]) for b in range(B)]
    if sum(need) > len(free):
        return _unchanged(table, lens, ps, sum(need) - len(free))
    for b in range(B):
        rows[b], free = rows[b] + free[:need[b]], free[need[b]:]
        for j, node in enumerate(move[b]):
            at = int(lens[b]) + j
            k[:, rows[b][at // ps], at % ps] = k_tree[:, b, node]
            v[:, rows[b][at // ps], at % ps] = v_tree[:, b, node]
    return _as_table(rows, width), np.array([lens[b] + len(move[b]) for b in range(B)], dtype=np.int32), 0


def cache_fork(k, v, table, lens, ancestor):
    pages, ps = k.shape[1], k.shape[2]
    B, width = table.shape
    if any(not -1 <= a < B for a in ancestor) or any(not 0 <= n <= width * ps for n in lens):
        return _unchanged(table, lens, ps, -1)
    rows, copies, kept = [], [], set()
    for b, a in enumerate(ancestor):
        live = [] if a < 0 else [int(x) for x in table[a, :_blocks(int(lens[a]), ps)]]
        if any(not 0 <= x < pages for x in live):
            return _unchanged(table, lens, ps, -1)
        if a >= 0 and lens[a] % ps and a in kept:
            copies.append((b, live.pop(), int(lens[a]) % ps))
        kept.add(int(a))
        rows.append(live)
    free = _lowest_free(rows, pages)
    if len(copies) > len(free):
        return _unchanged(table, lens, ps, len(copies) - len(free))
    for (b, src, part), dst in zip(copies, free):
        rows[b].append(dst)
        k[:, dst, :part] = k[:, src, :part]
        v[:, dst, :part] = v[:, src, :part]
    return _as_table(rows, width), np.array([0 if a < 0 else lens[a] for a in ancestor], dtype=np.int32), 0
