"""spec_head_product and spec_latent_prompt on the GPU against the float64
oracle: sizes, widths, prefixes, ragged batches, strides, hidden rows that hold
NaN, rows that belong to no sequence."""

import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import latent as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import dev, f64, tables

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


# ---- products per head

def product_check(x, w, label, **kw):
    """Sums of K float32 terms (the matrix unit's need not round to nearest:
    2^-23 each), then one rounding."""
    out = binding.head_product(x, w, **kw)
    torch.cuda.synchronize()
    want, size = ref.head_product(f64(x), f64(w))
    h = torch.finfo(x.dtype).eps / 2
    tol = x.shape[2] * 2.0 ** -23 * size
    tol = tol + h * (np.abs(want) + tol) + (2.0 ** -25 if x.dtype == FP16 else 0.0)
    err = np.abs(f64(out) - want)
    say(f"[head product] {label}: worst error {float(np.max(err / np.maximum(tol, 1e-300), initial=0.0)):.3f} of its bound")
    assert (err <= tol).all(), label
    return out


def operands(T, H, K, M, dtype, seed=0):
    rng = np.random.default_rng(seed)
    return dev(rng.standard_normal((T, H, K)), dtype), dev(rng.standard_normal((H, M, K)), dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [1, 7, 31, 32, 33, 64, 127, 128, 129, 300])
@pytest.mark.parametrize("K,M", [(128, 512), (512, 128), (8, 8), (72, 136), (200, 64)])
def test_products(dtype, T, K, M):
    product_check(*operands(T, 3, K, M, dtype, T), f"T={T} K={K} M={M} {dtype}")


def test_product_of_no_tokens():
    x, w = operands(0, 3, 64, 32, BF16)
    assert binding.head_product(x, w).shape == (0, 3, 32)


@pytest.mark.parametrize("T", [5, 200])
def test_product_strides(T):
    """Slices of wider tensors, head-major tokens, a shared token row, and outputs laid out by the caller."""
    rng = np.random.default_rng(T)
    x = dev(rng.standard_normal((5, T, 96)), BF16).transpose(0, 1)[:, 1:4, 16:80]
    w = dev(rng.standard_normal((3, 48, 160)), BF16)[:, 8:, 64:128]
    full = torch.full((T, 5, 64), -7.0, dtype=BF16, device="cuda")
    out = full[:, 1:4, 8:48]
    assert product_check(x, w, "strides", out=out) is out
    keep = full.clone()
    keep[:, 1:4, 8:48] = -7.0
    assert (keep == -7.0).all()
    shared = dev(rng.standard_normal((T, 1, 64)), BF16).expand(T, 3, 64)
    product_check(shared, w, "a shared row")


def test_product_many_heads():
    product_check(*operands(40, 130, 64, 72, BF16), "130 heads")


# ---- prompts

def make(lens, new, H=3, dims=(128, 64, 128, 512), ps=16, dtype=BF16, seed=0, poison=True, gain=1.0, extra=0):
    """Inputs on the GPU; with `poison`, rows nothing may read hold NaN."""
    dn, dr, dv, R = dims
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
    pages, table = tables(lens, ps, rng, extra=extra)
    cache = rng.standard_normal((pages, ps, R + dr))
    if poison:
        used = np.zeros((pages, ps), bool)
        for b, n in enumerate(lens):
            j = np.arange(n)
            used[table[b, j // ps], j % ps] = True
        cache[~used] = np.nan
    T = int(new.sum())
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=dev(rng.standard_normal((T, H, dn + dr)) * gain, dtype), cache=dev(cache, dtype), table=dev(table),
                lens=dev(lens), start=dev(start), w_k=dev(rng.standard_normal((H, dn, R)) * R ** -0.5, dtype),
                w_v=dev(rng.standard_normal((H, dv, R)) * R ** -0.5, dtype), rows=int(lens.sum()))


def call(s, **kw):
    kw.setdefault("rows", s["rows"])
    return binding.latent_prompt(s["q"], s["cache"], s["table"], s["lens"], s["start"], s["w_k"], s["w_v"], **kw)


def check(s, label, scale=None, **kw):
    """The bound: keys, values and weights are rounded once to the type (h each),
    the output once; float32 sums over the latent dimensions (the oracle's
    slack), dot products, exponentials and sums over the keys as in
    tree_helpers.attention_tolerance.  A key's rounding moves a score by at most
    h * scale * sum |q k|."""
    out = call(s, scale=scale, **kw)
    torch.cuda.synchronize()
    host = lambda t: t.cpu().numpy()  # noqa: E731
    want, spread, reach, loose = ref.prompt(f64(s["q"]), f64(s["cache"]), host(s["table"]), host(s["lens"]),
                                            host(s["start"]), f64(s["w_k"]), f64(s["w_v"]), scale)
    got = f64(out)
    D, dt = s["q"].shape[2], s["q"].dtype
    h = torch.finfo(dt).eps / 2
    dots, n, slack = (reach[..., i:i + 1] for i in range(3))
    delta = h * dots + slack + 2.0 ** -23 * ((D + 4) * dots + n + 4)
    tol = 2 * h * (1 + h) * spread + loose + np.expm1(2 * delta) * spread * (1 + h)
    tol = tol + h * (np.abs(want) + tol)
    if dt == FP16:
        vmax = float(np.nanmax(spread, initial=0.0)) * 64
        tol = tol + n * 2.0 ** -25 * vmax + 2.0 ** -25
    mine = np.zeros(len(want), bool)
    start = host(s["start"])
    for b in range(len(start) - 1):
        if 0 <= start[b] < start[b + 1] <= len(want):
            mine[start[b]:start[b + 1]] = True
    seen = np.isfinite(want) & mine[:, None, None]
    assert (np.isfinite(got) == seen)[mine].all(), label
    err = np.abs(got - want)
    worst = float(np.max(err[seen] / np.maximum(tol[seen], 1e-300), initial=0.0))
    say(f"[latent prompt] {label}: worst error {worst:.3f} of its bound")
    assert (err[seen] <= tol[seen]).all(), (label, worst)
    return out


DIMS = [(128, 64, 128, 512), (64, 32, 64, 256), (80, 32, 72, 256), (96, 64, 96, 384), (8, 8, 8, 8), (64, 0, 128, 128),
        (96, 32, 128, 512), (128, 0, 8, 64)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dims", DIMS)
def test_dimensions(dtype, dims):
    check(make((150, 61), (150, 20), dims=dims, dtype=dtype), f"{dims} {dtype}")


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 100])
def test_lengths(n, prefix):
    check(make((n + prefix,), (n,), H=2, dims=(64, 32, 64, 128), ps=32, seed=n), f"{n} tokens behind {prefix}")


@pytest.mark.parametrize("ps", [1, 2, 8, 64, 1024])
def test_pages(ps):
    check(make((70, 3, 130), (70, 2, 1), H=2, dims=(64, 32, 64, 128), ps=ps), f"pages of {ps}")


def test_ragged_batch():
    """Empty sequences, sequences without queries, one long prefix."""
    check(make((0, 300, 5, 0, 64, 700), (0, 129, 5, 0, 0, 3), H=9), "ragged")


def test_many_sequences():
    rng = np.random.default_rng(3)
    new = rng.integers(0, 4, 1500)
    check(make(new + rng.integers(0, 5, 1500), new, H=1, dims=(8, 8, 8, 16), ps=4), "1500 sequences")


def test_scales():
    for scale in (0.0, -0.3, 0.7):
        check(make((90,), (90,), H=2, dims=(64, 32, 64, 128)), f"scale {scale}", scale=scale)
