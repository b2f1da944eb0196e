"""spec_latent_attention on the GPU against the float64 oracle: head counts,
row widths, tree shapes, lengths from none to many tiles, ragged batches,
strides, hidden rows that hold NaN, infinities among the values, HIP graphs,
other streams."""

import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import latent as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import attention_tolerance, dev, f64, parents, tables

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def make(B=2, N=5, H=4, C=576, dv=512, lens=(33, 7), ps=16, kind="random", dtype=BF16, n_nodes=None, seed=0,
         poison=True, extra=0, gain=2.0):
    """Inputs on the GPU; with `poison`, rows nothing may read hold NaN."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    pages, table = tables(lens, ps, rng, extra=extra)
    cache, rows = rng.standard_normal((pages, ps, C)), rng.standard_normal((B, N, C))
    q = rng.standard_normal((B, N, H, C)) * gain
    if poison:
        used = np.zeros((pages, ps), bool)
        for b in range(B):
            j = np.arange(lens[b])
            used[table[b, j // ps], j % ps] = True
        cache[~used] = np.nan
        if n_nodes is not None:
            for b in range(B):
                rows[b, max(0, n_nodes[b]):] = np.nan
                q[b, max(0, n_nodes[b]):] = np.nan
    return dict(q=dev(q, dtype), cache=dev(cache, dtype), rows=dev(rows, dtype), table=dev(table), lens=dev(lens),
                parent=None if kind is None else dev(parents(kind, B, N, rng)), dv=dv, scale=C ** -0.5,
                n_nodes=None if n_nodes is None else dev(np.asarray(n_nodes, np.int32)))


def call(s, **kw):
    return binding.latent_attention(s["q"], s["cache"], s["table"], s["lens"], s["rows"], s["parent"], s["n_nodes"],
                                    dim_v=s["dv"], scale=s["scale"], **kw)


def oracle_of(s):
    host = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    return ref.attention(f64(s["q"]), f64(s["cache"]), host(s["table"]), host(s["lens"]), f64(s["rows"]),
                         host(s["parent"]), host(s["n_nodes"]), dim_v=s["dv"], scale=s["scale"])


def check(s, label, out=None, **kw):
    out = call(s, **kw) if out is None else out
    torch.cuda.synchronize()
    want, spread, reach = oracle_of(s)
    got = f64(out)
    vmax = max(float(np.nanmax(np.abs(f64(s["cache"])), initial=0.0)), float(np.nanmax(np.abs(f64(s["rows"])))))
    tol = attention_tolerance(spread, reach, want, s["q"].dtype, s["q"].shape[-1], vmax)
    seen = np.isfinite(want)
    assert (np.isfinite(got) == seen).all(), label
    worst = float(np.max(np.abs(got - want)[seen] / np.maximum(tol[seen], 1e-300), initial=0.0))
    say(f"[latent attention] {label}: worst error {worst:.3f} of its bound")
    assert (np.abs(got - want)[seen] <= tol[seen]).all(), (label, worst)
    return out


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("C,dv", [(576, 512), (320, 256)])
@pytest.mark.parametrize("H,N", [(1, 1), (16, 1), (8, 5), (20, 3), (16, 8), (128, 1), (128, 3), (6, 64)])
def test_heads_and_nodes(dtype, C, dv, H, N):
    check(make(N=N, H=H, C=C, dv=dv, lens=(150, 61), dtype=dtype, seed=N), f"H={H} N={N} {C}/{dv} {dtype}")


@pytest.mark.parametrize("C,dv", [(8, 8), (72, 64), (288, 256), (320, 320), (328, 256), (448, 384), (512, 512),
                                  (576, 8), (568, 504)])
@pytest.mark.parametrize("H", [5, 40])
def test_row_widths(C, dv, H):
    check(make(N=2, H=H, C=C, dv=dv, lens=(140, 3)), f"rows of {C}, values {dv}")


@pytest.mark.parametrize("ps", [1, 4, 8, 16, 32, 64, 1024])
@pytest.mark.parametrize("length", [0, 1, 7, 8, 31, 32, 33, 64, 95, 96, 97, 300])
def test_lengths_and_pages(length, ps):
    check(make(B=1, N=4, lens=(length,), ps=ps, seed=length), f"len={length} page={ps}")


@pytest.mark.parametrize("H,N", [(3, 3), (12, 5), (16, 8), (64, 7)])
@pytest.mark.parametrize("C,dv", [(576, 512), (288, 256)])
def test_long_and_ragged(H, N, C, dv):
    """Lengths that differ by three orders of magnitude: parts cut across
    sequences, and single sequences over many parts."""
    check(make(B=6, N=N, H=H, C=C, dv=dv, lens=(2500, 0, 1, 700, 64, 1999), n_nodes=[N, 0, 1, N - 1, 2, N], seed=N),
          f"ragged H={H} N={N} {C}/{dv}")


@pytest.mark.parametrize("H", [1, 16, 48])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_one_long_sequence(H, dtype):
    check(make(B=1, N=1, H=H, lens=(9001,), dtype=dtype, kind=None), f"one sequence H={H}")


def test_more_sequences_than_a_workgroup_has_threads():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 600)
    lens[550] = 900
    check(make(B=600, N=1, H=2, C=64, dv=48, lens=lens), "B=600")


@pytest.mark.parametrize("kind", [None, "chain", "star", "level2", "random"])
@pytest.mark.parametrize("N", [2, 31, 33, 64])
def test_tree_shapes(kind, N):
    s = make(N=N, H=2, C=320, dv=256, kind=kind, lens=(20, 0))
    out = check(s, f"{kind} N={N}")
    if kind == "chain":
        s["parent"] = None
        assert torch.equal(call(s), out)
