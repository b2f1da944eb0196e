"""Pins of the oracle of latent rows, beams and reservations, and the host checks
of their entry points (no GPU): the absorbed form against the expanded one and
against a dense mask, beams against every path, pages by hand; every refused
argument."""

import ctypes
import itertools
import os

import numpy as np
import pytest
import torch

from oracle import beam as ref_beam
from oracle import latent as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import parents, tables

I32, I64, VP, F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from rejection_sampling_verifier_amd import build
        build.build(verbose=False)
    lib = binding.load()
    for name in ("spec_latent_attention_workspace", "spec_latent_prompt_workspace", "spec_beam_workspace",
                 "spec_cache_reserve_workspace"):
        getattr(lib, name).restype = I64
    return lib


# ---- the oracle itself

def test_attention_is_a_masked_softmax():
    """Against torch's softmax over all rows and a mask; 1e-12 is far above
    float64 rounding of a hundred terms."""
    rng = np.random.default_rng(1)
    B, N, H, C, dv, ps = 2, 6, 3, 24, 16, 4
    lens = np.array([13, 0], np.int32)
    pages, table = tables(lens, ps, rng)
    q, cache, rows = (rng.standard_normal(s) for s in ((B, N, H, C), (pages, ps, C), (B, N, C)))
    par = parents("random", B, N, rng)
    out, _, _ = ref.attention(q, cache, table, lens, rows, par, dim_v=dv, scale=0.3)
    for b in range(B):
        keys = np.concatenate([cache[table[b, np.arange(lens[b]) // ps], np.arange(lens[b]) % ps], rows[b]])
        sees = np.zeros((N, len(keys)), bool)
        sees[:, :lens[b]] = True
        for i in range(N):
            j = i
            while j >= 0:
                sees[i, lens[b] + j] = True
                j = par[b, j] if j > 0 else -1
        x = 0.3 * torch.from_numpy(np.einsum("nhd,kd->nhk", q[b], keys))
        w = torch.softmax(x.masked_fill(~torch.from_numpy(sees)[:, None], -torch.inf), -1).numpy()
        np.testing.assert_allclose(out[b], np.einsum("nhk,kd->nhd", w, keys[:, :dv]), atol=1e-12)


def test_absorbed_and_expanded_forms_agree():
    """Queries times the key weights on the rows themselves, and the result times
    the value weights, are the attention with expanded keys and values."""
    rng = np.random.default_rng(2)
    H, dn, dr, dv, R, ps, n = 3, 8, 4, 12, 20, 4, 11
    lens = np.array([n + 3], np.int32)
    pages, table = tables(lens, ps, rng)
    cache, q = rng.standard_normal((pages, ps, R + dr)), rng.standard_normal((n, H, dn + dr))
    w_k, w_v = rng.standard_normal((H, dn, R)), rng.standard_normal((H, dv, R))
    want = ref.prompt(q, cache, table, lens, np.array([0, n]), w_k, w_v, 0.2)[0]
    into = ref.head_product(q[..., :dn], w_k.transpose(0, 2, 1))[0]
    absorbed = np.concatenate([into, q[..., dn:]], -1)[None]
    rows = ref.cache_rows(cache, table[0], n + 3)[3:][None]
    mid = ref.attention(absorbed, cache, table, np.array([3], np.int32), rows, dim_v=R, scale=0.2)[0]
    np.testing.assert_allclose(ref.head_product(mid[0], w_v)[0], want, atol=1e-12)


def test_beams_of_full_width_find_the_best_paths():
    """With as many beams as prefixes nothing is lost: three steps give the best of
    all V^3 paths, in order."""
    rng = np.random.default_rng(3)
    V, W, steps = 3, 9, 3
    first, second = rng.standard_normal((V, V)), rng.standard_normal((V, V, V))
    start = rng.standard_normal(V)
    soft = lambda x: ref_beam.log_softmax(x)  # noqa: E731
    paths = sorted(((soft(start)[a] + soft(first[a])[b] + soft(second[a, b])[c], (a, b, c))
                    for a, b, c in itertools.product(range(V), repeat=3)), reverse=True)
    hist = np.zeros((W, 0), int)
    scores = np.full((1, W), -np.inf)
    scores[0, 0] = 0.0
    for s in range(steps):
        x = np.stack([start if s == 0 else first[h[0] % V] if s == 1 else second[h[0] % V, h[1] % V] for h in hist])
        tok, anc, scores, _, _ = ref_beam.beam_select(x[None], scores)
        hist = np.concatenate([hist[np.maximum(anc, 0)], tok[0][:, None]], 1)
    for k in range(W):
        np.testing.assert_allclose(scores[0, k], paths[k][0], atol=1e-12)
        assert tuple(hist[k]) == paths[k][1]


def test_reservation_by_hand():
    table = np.array([[4, 1, -1, -1], [-1, -1, -1, -1], [0, -1, -1, -1]], np.int32)
    got = ref_beam.cache_reserve(table, np.array([6, 0, 4], np.int32), np.array([3, 5, 0]), 7, 4, 10)
    assert got[0].tolist() == [[4, 1, 2, -1], [3, 5, -1, -1], [0, -1, -1, -1]]
    assert got[1].tolist() == [9, 5, 4] and got[2].tolist() == [0, 3, 8, 8] and got[5] == 0
    assert got[3].tolist() == [6, 7, 8, 12, 13, 14, 15, 20, -1, -1]
    assert got[4].tolist() == [6, 7, 8, 0, 1, 2, 3, 4, -1, -1]


# ---- argument blocks

def _struct(fields):
    return type("Block", (ctypes.Structure,), {"_fields_": fields})


ATTENTION = _struct([(n, I32) for n in ("dtype", "B", "N", "heads", "dim", "dim_v")] + [
    ("q", VP), ("q_stride", I64 * 3), ("rows", VP), ("rows_stride", I64 * 2), ("cache", VP), ("cache_stride", I64 * 2),
    ("pages", I32), ("page_size", I32), ("width", I32), ("table", VP), ("table_stride", I64), ("len", VP),
    ("parent", VP), ("n_nodes", VP), ("scale", F32), ("out", VP), ("out_stride", I64 * 3), ("workspace", VP),
    ("workspace_bytes", I64)])
PRODUCT = _struct([(n, I32) for n in ("dtype", "T", "heads", "K", "M")] + [
    ("x", VP), ("x_stride", I64 * 2), ("w", VP), ("w_stride", I64 * 2), ("out", VP), ("out_stride", I64 * 2)])
PROMPT = _struct([(n, I32) for n in ("dtype", "T", "B", "heads", "latent", "dim_k", "dim_p", "dim_v", "rows")] + [
    ("q", VP), ("q_stride", I64 * 2), ("cache", VP), ("cache_stride", I64 * 2), ("pages", I32), ("page_size", I32),
    ("width", I32), ("table", VP), ("table_stride", I64), ("len", VP), ("q_start", VP), ("w_k", VP),
    ("w_k_stride", I64 * 2), ("w_v", VP), ("w_v_stride", I64 * 2), ("scale", F32), ("out", VP),
    ("out_stride", I64 * 2), ("workspace", VP), ("workspace_bytes", I64)])
WRITE = _struct([("cache", VP), ("cache_stride", I64 * 2)] + [
    (n, I32) for n in ("dtype", "pages", "page_size", "T", "dim_a", "dim_b")] + [
    ("a", VP), ("a_stride", I64), ("b", VP), ("b_stride", I64), ("slots", VP)])


@pytest.mark.parametrize("pack,cls", [(binding._PACK_LATENT, ATTENTION), (binding._PACK_PRODUCT, PRODUCT),
                                      (binding._PACK_PROMPT, PROMPT), (binding._PACK_WRITE, WRITE)])
def test_packed_argument_blocks(pack, cls):
    """The binding packs what the C structures hold, field by field."""
    sizes = [t._length_ if hasattr(t, "_length_") else 1 for _, t in cls._fields_]
    values = list(range(1, sum(sizes) + 1))
    blob = pack(*values)
    assert len(blob) == ctypes.sizeof(cls)
    s, got = cls.from_buffer_copy(blob), []
    for name, _ in cls._fields_:
        x = getattr(s, name)
        got += list(x) if hasattr(x, "__len__") else [x]
    assert got == values


def _block(cls, base, kw):
    s = cls()
    for name, value in {**base, **kw}.items():
        t = dict(cls._fields_)[name]
        setattr(s, name, t(*value) if hasattr(t, "_length_") else value)
    return s


def attention(lib, **kw):
    base = dict(dtype=1, B=2, N=4, heads=8, dim=576, dim_v=512, q=0x10000, q_stride=(18432, 4608, 576), rows=0x20000,
                rows_stride=(2304, 576), cache=0x30000, cache_stride=(9216, 576), pages=10, page_size=16, width=40,
                table=0x40000, table_stride=40, len=0x50000, parent=0x60000, n_nodes=0x70000, scale=0.1, out=0x80000,
                out_stride=(16384, 4096, 512), workspace=0x90000, workspace_bytes=1 << 40)
    return lib.spec_latent_attention(ctypes.byref(_block(ATTENTION, base, kw)), None)


def attention_bytes(lib, **kw):
    base = dict(dtype=1, B=2, N=4, heads=8, dim=576, dim_v=512, pages=10, page_size=16, width=40)
    return lib.spec_latent_attention_workspace(ctypes.byref(_block(ATTENTION, base, kw)))


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), -3), (dict(dtype=3), -3), (dict(B=0), -2), (dict(B=65537), -2), (dict(N=0), -2), (dict(N=65), -2),
    (dict(heads=0), -2), (dict(heads=1025), -2), (dict(dim=0), -2), (dict(dim=12), -2), (dict(dim=584), -2),
    (dict(dim_v=0), -2), (dict(dim_v=4), -2), (dict(dim_v=520), -2), (dict(dim=256, dim_v=264), -2),
    (dict(pages=0), -2), (dict(page_size=0), -2), (dict(page_size=24), -2), (dict(page_size=2048), -2),
    (dict(width=-1), -2), (dict(width=1 << 25), -2), (dict(B=65536, N=64, heads=1024), -2),
    (dict(q=None), -1), (dict(rows=None), -1), (dict(cache=None), -1), (dict(table=None), -1), (dict(len=None), -1),
    (dict(out=None), -1), (dict(workspace=None), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(table_stride=-1), -1), (dict(q_stride=(-8, 4608, 576)), -1), (dict(rows_stride=(-8, 576)), -1),
    (dict(out_stride=(0, 4096, 512)), -1), (dict(out_stride=(16384, 0, 512)), -1),
    (dict(out_stride=(16384, 4096, 0)), -1), (dict(q_stride=(18432, 4608, 575)), -6),
    (dict(cache_stride=(9216, 572)), -6), (dict(rows_stride=(2304, 4)), -6), (dict(q=0x10008), -6),
    (dict(rows=0x20004), -6), (dict(cache=0x30002), -6), (dict(out=0x80008), -6), (dict(workspace=0x90008), -6),
    (dict(table=0x40002), -6), (dict(len=0x50001), -6), (dict(parent=0x60002), -6), (dict(n_nodes=0x70002), -6),
    (dict(workspace_bytes=64), -8), (dict(workspace_bytes=-1), -8), (dict(q_stride=(1 << 41, 4608, 576)), -2),
])
def test_attention_host_validation(lib, kw, code):
    assert attention(lib, **kw) == code


def test_attention_workspace(lib):
    assert lib.spec_latent_attention(None, None) == -1
    need = attention_bytes(lib)
    assert need > 0 and attention(lib, workspace_bytes=need - 1) == -8
    assert attention_bytes(lib, dim=12) == -2
    assert attention_bytes(lib, width=4) == 0  # a few tiles are not divided
    # the largest sizes do not overflow, and no GPU is needed to size them
    largest = dict(N=64, heads=1024, width=1 << 18, page_size=1024)
    assert 0 < attention_bytes(lib, B=8184, **largest) < 1 << 34
    assert attention_bytes(lib, B=8185, **largest) == -2  # eight more with the rounding: 2^23 tiles of rows


def product(lib, **kw):
    base = dict(dtype=1, T=5, heads=4, K=128, M=512, x=0x10000, x_stride=(512, 128), w=0x20000, w_stride=(65536, 128),
                out=0x30000, out_stride=(2048, 512))
    return lib.spec_head_product(ctypes.byref(_block(PRODUCT, base, kw)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), -3), (dict(dtype=9), -3), (dict(T=-1), -2), (dict(T=(1 << 24) + 1), -2), (dict(heads=0), -2),
    (dict(heads=1025), -2), (dict(K=0), -2), (dict(K=12), -2), (dict(K=65544), -2), (dict(M=0), -2), (dict(M=4), -2),
    (dict(M=65544), -2), (dict(T=1 << 24, heads=1024), -2), (dict(x=None), -1), (dict(w=None), -1), (dict(out=None), -1),
    (dict(x_stride=(-8, 128)), -1), (dict(out_stride=(0, 512)), -1), (dict(out_stride=(2048, 0)), -1),
    (dict(x=0x10008), -6), (dict(w=0x20004), -6), (dict(out=0x30008), -6), (dict(x_stride=(512, 124)), -6),
    (dict(w_stride=(65536, 129)), -6), (dict(out_stride=(2044, 512)), -6),
])
def test_product_host_validation(lib, kw, code):
    assert product(lib, **kw) == code


def test_product_of_no_tokens(lib):
    assert product(lib, T=0, x=None, w=None, out=None) == 0
    assert product(lib, T=0, K=12) == -2
    assert lib.spec_head_product(None, None) == -1


def prompt(lib, **kw):
    base = dict(dtype=1, T=50, B=2, heads=4, latent=512, dim_k=128, dim_p=64, dim_v=128, rows=100, q=0x10000,
                q_stride=(768, 192), cache=0x20000, cache_stride=(9216, 576), pages=10, page_size=16, width=5,
                table=0x30000, table_stride=5, len=0x40000, q_start=0x50000, w_k=0x60000, w_k_stride=(65536, 512),
                w_v=0x70000, w_v_stride=(65536, 512), scale=0.1, out=0x80000, out_stride=(512, 128),
                workspace=0x90000, workspace_bytes=1 << 40)
    return lib.spec_latent_prompt(ctypes.byref(_block(PROMPT, base, kw)), None)


def prompt_bytes(lib, **kw):
    base = dict(dtype=1, T=50, B=2, heads=4, latent=512, dim_k=128, dim_p=64, dim_v=128, rows=100, pages=10,
                page_size=16, width=5)
    return lib.spec_latent_prompt_workspace(ctypes.byref(_block(PROMPT, base, kw)))


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), -3), (dict(dtype=3), -3), (dict(T=-1), -2), (dict(T=(1 << 24) + 1), -2), (dict(B=0), -2),
    (dict(B=65537), -2), (dict(heads=0), -2), (dict(heads=1025), -2), (dict(dim_k=0), -2), (dict(dim_k=136), -2),
    (dict(dim_k=12), -2), (dict(dim_p=-8), -2), (dict(dim_p=72), -2), (dict(dim_p=4), -2), (dict(dim_v=0), -2),
    (dict(dim_v=136), -2), (dict(dim_v=20), -2), (dict(latent=0), -2), (dict(latent=520), -2), (dict(latent=500), -2),
    (dict(pages=0), -2), (dict(page_size=3), -2), (dict(page_size=2048), -2), (dict(width=-1), -2),
    (dict(width=1 << 25), -2), (dict(rows=-1), -2), (dict(rows=(1 << 26) + 1), -2), (dict(rows=1 << 26, heads=1024), -2),
    (dict(T=1 << 24, heads=1024, B=65536), -2),
    (dict(q=None), -1), (dict(cache=None), -1), (dict(table=None), -1), (dict(len=None), -1), (dict(q_start=None), -1),
    (dict(w_k=None), -1), (dict(w_v=None), -1), (dict(out=None), -1), (dict(workspace=None), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("-inf")), -1), (dict(table_stride=-1), -1),
    (dict(q_stride=(768, -8)), -1), (dict(w_k_stride=(-8, 512)), -1), (dict(out_stride=(0, 128)), -1),
    (dict(out_stride=(512, 0)), -1), (dict(q=0x10002), -6), (dict(cache=0x20008), -6), (dict(w_k=0x60004), -6),
    (dict(w_v=0x70008), -6), (dict(out=0x80004), -6), (dict(table=0x30002), -6), (dict(len=0x40002), -6),
    (dict(q_start=0x50001), -6), (dict(workspace=0x90004), -6), (dict(q_stride=(768, 188)), -6),
    (dict(w_v_stride=(65536, 516)), -6), (dict(cache_stride=(9216, 572)), -6), (dict(workspace_bytes=100), -8),
    (dict(workspace_bytes=-1), -8),
])
def test_prompt_host_validation(lib, kw, code):
    assert prompt(lib, **kw) == code


def test_prompt_workspace(lib):
    assert lib.spec_latent_prompt(None, None) == -1
    need = prompt_bytes(lib)
    assert need >= 4 * 100 * 256 * 2 and prompt(lib, workspace_bytes=need - 1) == -8
    assert prompt(lib, T=0, q=None, out=None) == 0
    assert prompt_bytes(lib, dim_k=12) == -2
    assert prompt_bytes(lib, rows=0) > 0
    assert 1 << 35 < prompt_bytes(lib, rows=1 << 20, heads=128) < 1 << 37


def write(lib, **kw):
    base = dict(cache=0x10000, cache_stride=(9216, 576), dtype=1, pages=10, page_size=16, T=5, dim_a=512, dim_b=64,
                a=0x20000, a_stride=512, b=0x30000, b_stride=64, slots=0x40000)
    return lib.spec_cache_write(ctypes.byref(_block(WRITE, base, kw)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -3), (dict(dtype=-1), -3), (dict(pages=0), -2), (dict(pages=(1 << 20) + 1), -2),
    (dict(page_size=0), -2), (dict(page_size=12), -2), (dict(T=-1), -2), (dict(T=(1 << 28) + 1), -2),
    (dict(dim_a=0), -2), (dict(dim_a=65537), -2), (dict(dim_b=-1), -2), (dict(dim_a=12), -6), (dict(dim_b=4), -6),
    (dict(cache=None), -1), (dict(a=None), -1), (dict(b=None), -1), (dict(slots=None), -1),
    (dict(cache_stride=(0, 576)), -1), (dict(cache_stride=(9216, 0)), -1), (dict(cache_stride=(-8, 576)), -1),
    (dict(a_stride=-8), -1), (dict(cache=0x10008), -6), (dict(a=0x20008), -6), (dict(b=0x30004), -6),
    (dict(slots=0x40002), -6), (dict(a_stride=508), -6), (dict(cache_stride=(9216, 580)), -6),
])
def test_write_host_validation(lib, kw, code):
    assert write(lib, **kw) == code


def test_write_of_no_rows(lib):
    assert write(lib, T=0, a=None, slots=None, cache=None) == 0
    assert lib.spec_cache_write(None, None) == -1


def select(lib, B=2, W=4, V=1000, dtype=0, data=0x10000, sb=None, sw=None, ptrs=None, end=-1, ws_bytes=1 << 40):
    l = binding.SvLogits(data, dtype, B, W, V, W * V if sb is None else sb, V if sw is None else sw)
    names = ("scores", "finished", "out_tokens", "out_ancestor", "out_scores", "out_finished", "ws")
    at = {n: 0x20000 + 0x1000 * i for i, n in enumerate(names)}
    at["finished"] = None
    at.update(ptrs or {})
    p = [VP(at[n]) for n in names]
    return lib.spec_beam_select(ctypes.byref(l), p[0], p[1], I32(end), *p[2:], I64(ws_bytes), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -2), (dict(W=0), -2), (dict(W=65), -2), (dict(B=1024, W=64), -2), (dict(V=0), -2),
    (dict(V=(1 << 24) + 1), -2), (dict(dtype=2), -3), (dict(data=0), -1), (dict(data=0x10002), -6),
    (dict(sb=-1), -1), (dict(ptrs=dict(scores=None)), -1), (dict(ptrs=dict(out_tokens=None)), -1),
    (dict(ptrs=dict(out_ancestor=None)), -1), (dict(ptrs=dict(out_scores=None)), -1),
    (dict(ptrs=dict(out_finished=None)), -1), (dict(ptrs=dict(ws=None)), -1), (dict(ptrs=dict(scores=0x20002)), -6),
    (dict(ptrs=dict(finished=0x21002), end=3), -6), (dict(ptrs=dict(out_ancestor=0x23001)), -6),
    (dict(ptrs=dict(ws=0x26004)), -6), (dict(end=-2), -1), (dict(end=1000), -1), (dict(ptrs=dict(finished=0x21000)), -1),
    (dict(ptrs=dict(out_scores=0x20000)), -1), (dict(ptrs=dict(finished=0x21000, out_finished=0x21000), end=3), -1),
    (dict(ws_bytes=16), -8), (dict(ws_bytes=-1), -8),
])
def test_beam_host_validation(lib, kw, code):
    assert select(lib, **kw) == code


def test_beam_workspace(lib):
    need = lib.spec_beam_workspace(2, 4, 1000)
    assert need > 0 and select(lib, ws_bytes=need - 1) == -8
    for bad in ((0, 4, 10), (1, 65, 10), (1, 4, 0), (1, 4, (1 << 24) + 1), (65535, 2, 10)):
        assert lib.spec_beam_workspace(*bad) == -2
    assert 0 < lib.spec_beam_workspace(1023, 64, 1 << 24) < 1 << 37


def reorder(lib, src=0x10000, src_stride=64, dst=0x20000, dst_stride=64, row=64, rows=4, anc=0x30000):
    return lib.spec_beam_reorder(VP(src), I64(src_stride), VP(dst), I64(dst_stride), I64(row), I32(rows), VP(anc), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), -2), (dict(rows=65536), -2), (dict(row=-1), -2), (dict(row=(1 << 40) + 1), -2),
    (dict(src_stride=-64), -1), (dict(dst_stride=-64), -1), (dict(dst_stride=63), -1), (dict(src=None), -1),
    (dict(dst=None), -1), (dict(dst=0x10000), -1), (dict(anc=None), -1), (dict(anc=0x30002), -6), (dict(row=0), 0),
])
def test_reorder_host_validation(lib, kw, code):
    assert reorder(lib, **kw) == code


RESERVE = ("table", "len", "n_new", "out_table", "out_len", "out_start", "out_slots", "out_position", "out_status", "ws")


def reserve(lib, B=3, width=4, pages=20, page_size=16, rows=50, ts=4, os=4, ws_bytes=1 << 30, **ptrs):
    at = {n: 0x10000 + 0x1000 * i for i, n in enumerate(RESERVE)}
    at.update(ptrs)
    p = {n: VP(at[n]) for n in RESERVE}
    return lib.spec_cache_reserve(p["table"], I64(ts), p["len"], p["n_new"], I32(B), I32(width), I32(pages),
                                  I32(page_size), I32(rows), p["out_table"], I64(os), p["out_len"], p["out_start"],
                                  p["out_slots"], p["out_position"], p["out_status"], p["ws"], I64(ws_bytes), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -2), (dict(B=65535), -2), (dict(width=0), -2), (dict(width=1 << 25), -2), (dict(pages=0), -2),
    (dict(pages=(1 << 20) + 1), -2), (dict(page_size=0), -2), (dict(page_size=24), -2), (dict(rows=-1), -2),
    (dict(rows=(1 << 30) + 1), -2), (dict(ts=-1), -1), (dict(os=3), -1), (dict(out_table=0x10000, ts=5, os=4), -1),
    (dict(ws_bytes=8), -8), (dict(ws_bytes=-1), -8)] +
    [({n: None}, -1) for n in RESERVE] + [({n: 0x90002}, -6) for n in RESERVE])
def test_reserve_host_validation(lib, kw, code):
    assert reserve(lib, **kw) == code


def test_reserve_workspace(lib):
    need = lib.spec_cache_reserve_workspace(3, 16, 50)
    assert need > 0 and need % 4 == 0 and reserve(lib, ws_bytes=need - 1) == -8
    for bad in ((0, 16, 5), (65535, 16, 5), (3, 0, 5), (3, 17, 5), (3, 16, -1), (3, 16, (1 << 30) + 1)):
        assert lib.spec_cache_reserve_workspace(*bad) == -2


def test_forced_launch_failure(lib, monkeypatch):
    monkeypatch.setenv("SPECVERIFY_FAIL_LAUNCH", "1")
    for call in (attention, product, prompt, write, select, reorder, reserve):
        assert call(lib) == -4, call.__name__
    assert attention(lib, dim=12) == -2


# ---- the binding

def test_binding_refuses_before_the_library():
    """Shapes and types the C interface cannot see."""
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731

    def refuses(f, ok, bad):
        for name, value in bad:
            with pytest.raises(ValueError):
                f(**{**ok, name: value})
        with pytest.raises(ValueError, match="GPU"):
            f(**ok)

    refuses(binding.latent_attention,
            dict(q=z(2, 4, 8, 96), cache=z(10, 16, 96), block_table=i(2, 5), seq_len=i(2), rows=z(2, 4, 96),
                 parent=i(2, 4), dim_v=64, scale=0.1),
            [("q", z(2, 4, 8, 96).float()), ("q", z(2, 4, 96)), ("q", z(2, 4, 8, 192)[..., ::2]),
             ("q", z(2, 4, 8, 96).requires_grad_()), ("cache", z(10, 16, 88)), ("cache", z(10, 16, 96).half()),
             ("block_table", i(3, 5)), ("block_table", i(2, 5).long()), ("seq_len", i(3)), ("rows", z(2, 3, 96)),
             ("parent", i(2, 3)), ("n_nodes", i(3)), ("out", z(2, 4, 8, 96))])
    refuses(binding.head_product, dict(x=z(5, 4, 16), w=z(4, 24, 16)),
            [("x", z(5, 4, 16).float()), ("x", z(4, 16)), ("w", z(3, 24, 16)), ("w", z(4, 24, 8)),
             ("w", z(4, 16, 24).transpose(1, 2)), ("out", z(5, 4, 16)), ("w", z(4, 24, 16).requires_grad_())])
    refuses(binding.latent_prompt,
            dict(q=z(9, 4, 24), cache=z(10, 16, 40), block_table=i(2, 5), seq_len=i(2), q_start=i(3), w_k=z(4, 16, 32),
                 w_v=z(4, 8, 32), rows=30),
            [("q", z(9, 4, 32)), ("q", z(9, 3, 24)), ("q", z(9, 4, 24).float()), ("cache", z(10, 16, 48)),
             ("w_k", z(4, 24, 32)), ("w_v", z(4, 8, 24)), ("w_v", z(5, 8, 32)), ("q_start", i(2)),
             ("q_start", i(3).long()), ("seq_len", i(2, 1)), ("out", z(9, 4, 16)), ("rows", 1 << 32)])
    refuses(binding.cache_write, dict(cache=z(10, 16, 40), slots=i(5), a=z(5, 32), b=z(5, 8)),
            [("a", z(5, 24)), ("a", z(4, 32)), ("a", z(5, 32).half()), ("b", z(5, 16)), ("b", None), ("slots", i(4)),
             ("slots", i(5).long()), ("cache", z(16, 40)), ("cache", z(10, 16, 40).long())])
    refuses(binding.cache_reserve,
            dict(block_table=i(2, 5), seq_len=i(2), n_new=i(2), pages=10, page_size=16, rows=30),
            [("block_table", i(3, 5)), ("seq_len", i(2).long()), ("n_new", i(3)), ("seq_len", i(2, 1)), ("rows", (1 << 32) + 30),
             ("pages", (1 << 32) + 10), ("page_size", (1 << 32) + 16)])
    refuses(binding.beam_select, dict(logits=torch.zeros(2, 4, 50), scores=torch.zeros(2, 4)),
            [("logits", torch.zeros(2, 4, 50).half()), ("logits", torch.zeros(4, 50)), ("scores", torch.zeros(2, 3)),
             ("scores", torch.zeros(2, 4).double()), ("finished", torch.zeros(2, 4)), ("scores", torch.zeros(2, 4, 1)), ("end", (1 << 32) + 3)])
    refuses(binding.beam_reorder, dict(state=i(8, 3), ancestor=i(8)),
            [("ancestor", i(7)), ("ancestor", i(8).long()), ("out", i(8, 4)), ("out", i(8, 3).long()),
             ("state", torch.zeros(8, 3, requires_grad=True)), ("state", i(3, 8, 4).transpose(0, 2))])
