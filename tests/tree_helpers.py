"""Inputs and tolerances shared by the tree round's tests."""

import numpy as np
import torch


def parents(kind, B, N, rng):
    """[B, N] int32: "chain", "star", a w-ary "levelW", or "random"."""
    out = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        if kind == "chain":
            out[:, i] = i - 1
        elif kind == "star":
            out[:, i] = 0
        elif kind.startswith("level"):
            out[:, i] = (i - 1) // int(kind[5:])
        else:
            out[:, i] = rng.integers(0, i, B)
    return out


def tables(lens, ps, rng, extra=0, spare=3):
    """(pages, table): every sequence's blocks at random pages, -1 behind."""
    blocks = [-(-int(n) // ps) for n in lens]
    pages = sum(blocks) + spare
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(blocks + [0]) + 1 + extra), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return pages, table


def attention_tolerance(spread, reach, out, dtype, D, vmax):
    """Largest |kernel - float64| the kernel's own arithmetic allows.

    With h half a step of the type (eps / 2): each weight is rounded once (h
    relative: at most h * spread in the quotient), the output once (h * |out|).
    Below that float32: a score's D-term dot product (2^-23 per term, the matrix
    unit's sums need not round to nearest) and its scaling, subtraction and
    exponential (4 more steps of 2^-23 relative to the score, and 2^-22 for the
    exponential's own error) change a weight by delta relative, and the sums
    over n keys by n 2^-23; numerator and denominator each once.  float16
    weights below 2^-14 are rounded absolutely, by 2^-25 against a largest weight
    of at least 1."""
    h = torch.finfo(dtype).eps / 2
    dots, n = reach[..., 0:1], reach[..., 1:2]
    delta = 2.0 ** -23 * ((D + 4) * dots + n + 4)
    tol = h * spread + 2 * delta * spread
    tol = tol + h * (np.abs(out) + tol)
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -25 * vmax + 2.0 ** -25
    return tol


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()
