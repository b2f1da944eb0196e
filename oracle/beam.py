"""Float64 oracle of a beam step and of the reservation of cache rows.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

from collections import Counter

import numpy as np

from .tree import _as_table, _blocks, _lowest_free, _unchanged


def log_softmax(x):
    d = x - x.max()
    return d - np.log(np.exp(d).sum())


def beam_select(logits, scores, finished=None, end=-1):
    """logits [B, W, V] float64, scores [B, W]; returns (tokens, ancestor,
    scores, finished, margin): margin [B] is the smallest distance between two
    different beams' candidates that decides something.  Equal scores come in the
    order of the beams, a beam's own ids in that of their logits (also where float64
    cannot tell their scores apart), then of their numbers."""
    B, W, V = logits.shape
    tokens, anc = np.full((B, W), -1, np.int32), np.full(B * W, -1, np.int32)
    out, fin, margin = np.full((B, W), -np.inf), np.zeros((B, W), np.int32), np.full(B, np.inf)
    for b in range(B):
        s, logit = np.full((W, V), -np.inf), np.zeros((W, V))
        for w in range(W):
            base = float(scores[b, w])
            if not np.isfinite(base):
                continue
            if finished is not None and finished[b, w]:
                s[w, end] = base
                continue
            x = logits[b, w]
            if np.isnan(x).any() or x.max() == np.inf or x.max() == -np.inf:
                continue
            with np.errstate(divide="ignore"):
                s[w] = (base + (x - x.max())) - np.log(np.exp(x - x.max()).sum())
            s[w][x == -np.inf] = -np.inf
            logit[w] = x
        flat = s.reshape(-1)
        at = np.arange(W * V)
        order = np.lexsort((at, -logit.reshape(-1), at // V, -flat))
        order = order[flat[order] > -np.inf]
        for k, c in enumerate(order[:W]):
            w, v = divmod(int(c), V)
            tokens[b, k], anc[b * W + k], out[b, k] = v, b * W + w, flat[c]
            fin[b, k] = v == end or (finished is not None and finished[b, w] != 0)
            for d in order[k + 1:k + 1 + 4 * W]:
                if d // V != w:
                    margin[b] = min(margin[b], flat[c] - flat[d])
    return tokens, anc, out, fin, margin


def cache_reserve(table, lens, n_new, pages, ps, rows):
    """(table, lens, start, slots, position, status)."""
    B, width = table.shape
    new = np.maximum(n_new, 0).astype(np.int64)
    nothing = (np.zeros(B + 1, np.int32), np.full(rows, -1, np.int32), np.full(rows, -1, np.int32))

    def refused(status):
        t, n, s = _unchanged(table, lens, ps, status)
        return (t, n) + nothing + (s,)

    if any(not 0 <= n <= width * ps for n in lens) or any(a + n > width * ps for a, n in zip(lens, new)) or \
            new.sum() > rows:
        return refused(-1)
    live = [[int(x) for x in table[b, :_blocks(int(lens[b]), ps)]] for b in range(B)]
    if any(not 0 <= x < pages for r in live for x in r):
        return refused(-1)
    named = Counter(x for r in live for x in r)
    if any(new[b] and lens[b] % ps and named[live[b][-1]] > 1 for b in range(B)):
        return refused(-1)
    free = _lowest_free(live, pages)
    need = [_blocks(int(lens[b] + new[b]), ps) - len(live[b]) for b in range(B)]
    if sum(need) > len(free):
        return refused(sum(need) - len(free))
    start, slots, position = [0], [], []
    for b in range(B):
        live[b], free = live[b] + free[:need[b]], free[need[b]:]
        for j in range(int(lens[b]), int(lens[b] + new[b])):
            slots.append(live[b][j // ps] * ps + j % ps)
            position.append(j)
        start.append(len(slots))
    pad = [-1] * (rows - len(slots))
    as32 = lambda x: np.array(x, dtype=np.int32)  # noqa: E731
    return (_as_table(live, width), as32([a + n for a, n in zip(lens, new)]), as32(start), as32(slots + pad),
            as32(position + pad), 0)
