"""Pins of the tree round's oracle and the host checks of its entry points
(no GPU): the law of the verified tokens, the closed form of repeated
refusals, attention against a dense mask, pages; every refused argument."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import tree as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import parents, tables


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from rejection_sampling_verifier_amd import build
        build.build(verbose=False)
    return binding.load()


def test_first_token_follows_the_target():
    """Whatever the draft: the first emitted token is the target's, with drawn
    children (three of them) and with chosen ones.  The law is summed exactly
    over the children and the acceptance path; 1e-12 is far above float64
    rounding of a few hundred terms."""
    rng = np.random.default_rng(0)
    V = 4
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))

    def law(left, draft, kids):
        """Probabilities of the emitted token when `kids` follow in order."""
        if not kids:
            return left / left.sum()
        x, dist = kids[0], left / left.sum()
        a = min(1.0, dist[x] / draft[x])
        out = np.zeros(V)
        out[x] = a
        if a < 1:
            out += (1 - a) * law(np.maximum(dist - draft, 0.0), draft, kids[1:])
        return out

    total = np.zeros(V)
    for x in np.ndindex(V, V, V):
        total += q[list(x)].prod() * law(p, q, list(x))
    np.testing.assert_allclose(total, p, atol=1e-12)
    # the oracle decides as that law says: each acceptance bound, from both sides
    for x in ((0, 1, 2), (3, 3, 1), (2, 0, 0)):
        left, u = p.copy(), np.zeros(4)
        for i, t in enumerate(x):
            a = min(1.0, left[t] / q[t])
            for side in (-1e-9, 1e-9):
                if not 0 < a + side < 1:
                    continue
                v = u.copy()
                v[i + 1] = a + side
                v[i + 2:] = 0.999999
                got = ref.verify_tree_row(np.stack([p] * 4), np.stack([q]), np.array([0, *x]),
                                          np.array([-1, 0, 0, 0]), i + 2, v, 0.5)
                assert (got[1] == [0, i + 1]) == (side < 0)
            if a >= 1:
                break
            u[i + 1] = (1 + a) / 2
            left = np.maximum(left - q, 0.0)
            left /= left.sum()


def test_refusals_in_closed_form():
    """After s refusals max(0, p - a_s q) with a_{s+1} = a_s + S_s is the
    repeatedly renormalised residual up to a factor."""
    rng = np.random.default_rng(1)
    p, q = rng.dirichlet(np.ones(30)), rng.dirichlet(np.ones(30) * 0.5)
    left, a, S = p.copy(), 0.0, 1.0
    for _ in range(4):
        left = np.maximum(left - q, 0.0)
        left /= left.sum()
        a += S
        w = np.maximum(p - a * q, 0.0)
        S = w.sum()
        np.testing.assert_allclose(w / S, left, rtol=1e-9, atol=1e-12)


def test_chosen_children_are_the_target_sampled():
    """With chosen children the accepted child x has probability p(x)."""
    p = np.array([0.4, 0.3, 0.2, 0.1])
    kids = [1, 0]
    first, n = np.zeros(4), 4000
    for i in range(n):
        u = np.array([0, (i + 0.5) / n, ((i * 1237) % n + 0.5) / n])
        got = ref.verify_tree_row(np.stack([p] * 3), None, np.array([0, *kids]), np.array([-1, 0, 0]), 3, u,
                                  ((i * 2741) % n + 0.5) / n)
        first[got[0][0]] += 1 / n
    # two-dimensional lattices of 4000 points: a box's share is off by about log(n)/n
    np.testing.assert_allclose(first, p, atol=0.01)


def test_attention_against_a_dense_mask():
    rng = np.random.default_rng(2)
    B, N, H, Hkv, D, ps = 2, 7, 4, 2, 8, 4
    lens = np.array([11, 0], np.int32)
    pages, table = tables(lens, ps, rng)
    k, v = rng.standard_normal((pages, ps, Hkv, D)), rng.standard_normal((pages, ps, Hkv, D))
    q, kt, vt = (rng.standard_normal((B, N, x, D)) for x in (H, Hkv, Hkv))
    par = parents("random", B, N, rng)
    for window, sinks in ((0, 0), (3, 2), (1, 0)):
        out, _, _ = ref.tree_attention(q, k, v, table, lens, kt, vt, par, None, window=window, sinks=sinks)
        for b in range(B):
            L = lens[b]
            depth = np.zeros(N, int)
            anc = np.eye(N, dtype=bool)
            for i in range(1, N):
                depth[i] = depth[par[b, i]] + 1
                anc[i] |= anc[par[b, i]]
            pos = np.concatenate([np.arange(L), L + depth])
            mask = np.concatenate([np.ones((N, L), bool), anc], 1)
            if window:
                far = (L + depth)[:, None] - pos[None] >= window
                far[:, :L] &= np.arange(L)[None] >= sinks
                mask &= ~far
            for h in range(H):
                e = h // (H // Hkv)
                kk = np.concatenate([k[table[b, np.arange(L) // ps], np.arange(L) % ps, e], kt[b, :, e]])
                vv = np.concatenate([v[table[b, np.arange(L) // ps], np.arange(L) % ps, e], vt[b, :, e]])
                x = np.where(mask, q[b, :, h] @ kk.T / np.sqrt(D), -np.inf)
                w = np.exp(x - x.max(-1, keepdims=True))
                np.testing.assert_allclose(out[b, :, h], w @ vv / w.sum(-1, keepdims=True), rtol=1e-12, atol=1e-13)


def test_pages_are_conserved():
    """Random commits and forks: no page lost or used twice, rows where the
    history says."""
    rng = np.random.default_rng(3)
    B, ps, pages, N = 4, 4, 60, 5
    k = np.zeros((1, pages, ps, 1, 1))
    v = np.zeros_like(k)
    table, lens = np.full((B, 30), -1, np.int32), np.zeros(B, np.int32)
    hist, stamp = [[] for _ in range(B)], 0
    for step in range(60):
        if step % 3 == 2:
            anc = rng.integers(-1, B, B)
            got = ref.cache_fork(k, v, table, lens, anc)
            if got[2] == 0:
                hist = [list(hist[a]) if a >= 0 else [] for a in anc]
        else:
            kt = stamp + 1 + np.arange(B * N, dtype=np.float64).reshape(1, B, N, 1, 1)
            stamp += B * N
            n = rng.integers(-1, 3, B)
            got = ref.cache_commit(k, v, table, lens, kt, -kt, None, n)
            if got[2] == 0:
                for b in range(B):
                    hist[b] += kt[0, b, :n[b] + 1, 0, 0].tolist()
        table, lens = got[0], got[1]
        for b in range(B):
            assert lens[b] == len(hist[b])
            at = np.arange(lens[b])
            assert k[0, table[b, at // ps], at % ps, 0, 0].tolist() == hist[b]
            assert (v[0, table[b, at // ps], at % ps, 0, 0] == -np.array(hist[b])).all()


# ------------------------------------------------------------ host checks

def _attn(**kw):
    a = binding.SvTreeAttention()
    d = dict(dtype=1, B=2, N=4, heads=8, kv_heads=2, dim=64, q=0x10000, k_tree=0x20000, v_tree=0x30000,
             k_cache=0x40000, v_cache=0x50000, pages=10, page_size=16, width=40, table=0x60000, table_stride=40,
             len=0x70000, parent=0x80000, n_nodes=None, scale=0.125, window=0, sinks=0, out=0x90000,
             workspace=0xA0000, workspace_bytes=1 << 40)
    d.update(kw)
    for f in ("q", "k_tree", "v_tree", "k_cache", "v_cache", "out"):
        s = d.pop(f + "_stride", (4096, 512, 64))
        setattr(a, f + "_stride", (ctypes.c_int64 * 3)(*s))
    for f, x in d.items():
        setattr(a, f, x)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), -3), (dict(dtype=3), -3),
    (dict(q_stride=(1 << 41, 512, 64)), -2), (dict(heads=1026), -2),
    (dict(B=0), -2), (dict(B=65537), -2), (dict(N=0), -2), (dict(N=65), -2), (dict(heads=0), -2),
    (dict(kv_heads=0), -2), (dict(heads=7), -2), (dict(dim=0), -2), (dict(dim=12), -2), (dict(dim=136), -2),
    (dict(pages=0), -2), (dict(page_size=0), -2), (dict(page_size=24), -2), (dict(page_size=2048), -2),
    (dict(width=-1), -2), (dict(width=1 << 25), -2),
    (dict(q=None), -1), (dict(k_tree=None), -1), (dict(v_tree=None), -1), (dict(k_cache=None), -1),
    (dict(v_cache=None), -1), (dict(table=None), -1), (dict(len=None), -1), (dict(parent=None), -1),
    (dict(out=None), -1), (dict(workspace=None), -1), (dict(window=-1), -1), (dict(sinks=-1), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(table_stride=-1), -1),
    (dict(q_stride=(-8, 512, 64)), -1), (dict(q_stride=(4096, 512, 63)), -6), (dict(out_stride=(4096, 516, 64)), -6),
    (dict(k_cache_stride=(4, 512, 64)), -6), (dict(q=0x10008), -6), (dict(v_cache=0x50002), -6),
    (dict(out=0x90004), -6), (dict(workspace=0xA0008), -6), (dict(len=0x70002), -6), (dict(parent=0x80001), -6),
    (dict(n_nodes=0x80002), -6), (dict(table=0x60002), -6), (dict(workspace_bytes=100), -8),
    (dict(workspace_bytes=-1), -8),
])
def test_attention_host_validation(lib, kw, code):
    assert lib.spec_tree_attention(_attn(**kw), None) == code


@pytest.mark.parametrize("stride", [(0, 512, 64), (4096, 0, 64), (4096, 512, 0)])
def test_expanded_output_is_refused(lib, stride):
    """Rows written on top of each other; inputs may be expanded."""
    assert lib.spec_tree_attention(_attn(out_stride=stride), None) == -1
    size = dict(zip((0, 1, 2), ("B", "N", "heads")))[stride.index(0)]
    one = {"B": dict(B=1), "N": dict(N=1), "heads": dict(heads=1, kv_heads=1)}[size]
    assert lib.spec_tree_attention(_attn(out_stride=stride, workspace_bytes=-1, **one), None) == -8
    assert lib.spec_tree_attention(_attn(q_stride=stride, workspace_bytes=-1), None) == -8


def test_launches_stay_below_the_largest_grid(lib):
    big = dict(B=65536, N=1, width=4, kv_heads=256, dim=8)
    assert lib.spec_tree_attention_workspace(_attn(heads=256, **big)) == -2
    assert lib.spec_tree_attention_workspace(_attn(heads=255, **{**big, "kv_heads": 255})) == 0
    assert lib.spec_tree_attention_workspace(_attn(**{**big, "N": 64, "heads": 512, "kv_heads": 128})) == -2
    assert _verify(lib, B=1 << 22) == -2
    assert lib.spec_verify_tree_workspace(1 << 22, 4, 100, 0, 1) == -2
    assert lib.spec_verify_tree_workspace((1 << 22) - 1, 4, 100, 0, 1) == 0


@pytest.mark.parametrize("out", ["out_tokens", "out_nodes", "out_n"])
def test_verify_outputs_on_inputs_are_refused(lib, out):
    """Another workgroup of a team may still read them."""
    for at in (0x3000, 0x4000, 0x5000):
        assert _verify(lib, ptrs={out: at}) == -1
    assert _verify(lib, ptrs=dict(out_tokens=0x9000, out_nodes=0x9000)) == -1


def test_attention_workspace(lib):
    assert lib.spec_tree_attention_workspace(_attn()) > 0
    assert lib.spec_tree_attention_workspace(_attn(dim=12)) == -2
    # contexts of a few tiles are not divided
    assert lib.spec_tree_attention_workspace(_attn(width=4)) == 0
    # no GPU is needed to size it, and the largest sizes do not overflow
    assert 0 < lib.spec_tree_attention_workspace(_attn(B=65536, N=64, heads=128, kv_heads=8, dim=128, width=1 << 18,
                                                       page_size=1024)) < 1 << 34


def _verify(lib, B=2, N=4, P=3, V=100, dtype=0, ddtype=0, tdata=0x1000, ddata=0x2000, draft=True, ptrs=None, dV=None,
            ws_bytes=1 << 30):
    t = binding.SvLogits(tdata, dtype, B, N, V, N * V, V)
    d = binding.SvLogits(ddata, ddtype, B, P, V if dV is None else dV, P * V, V)
    names = ("tokens", "parent", "n_nodes", "u_accept", "u_final", "out_tokens", "out_nodes", "out_n", "ws")
    at = {n: 0x3000 + 0x1000 * i for i, n in enumerate(names)}
    at.update(ptrs or {})
    return lib.spec_verify_tree(t, d if draft else None, *[at[n] for n in names], ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -2), (dict(N=0, P=1), -2), (dict(N=65), -2), (dict(V=0), -2), (dict(V=(1 << 21) + 1), -2), (dict(P=0), -2),
    (dict(P=5), -2), (dict(dV=99), -2), (dict(dtype=2), -3), (dict(ddtype=1), -3), (dict(tdata=0), -1),
    (dict(ddata=0), -1), (dict(tdata=0x1002), -6), (dict(ptrs=dict(tokens=None)), -1),
    (dict(ptrs=dict(parent=None)), -1), (dict(ptrs=dict(u_accept=None)), -1), (dict(ptrs=dict(u_final=None)), -1),
    (dict(ptrs=dict(out_tokens=None)), -1), (dict(ptrs=dict(out_nodes=None)), -1), (dict(ptrs=dict(out_n=None)), -1),
    (dict(V=50000, ptrs=dict(ws=None)), -1), (dict(V=50000, ptrs=dict(ws=0xB004)), -6), (dict(V=50000, ws_bytes=64), -8),
    (dict(ptrs=dict(tokens=0x3002)), -6), (dict(ptrs=dict(n_nodes=0x5001)), -6), (dict(ptrs=dict(out_n=0xA002)), -6),
])
def test_verify_host_validation(lib, kw, code):
    assert _verify(lib, **kw) == code


def test_verify_workspace(lib):
    assert lib.spec_verify_tree_workspace(1, 8, 128256, 0, 1) > 0
    for none in ((300, 8, 128256, 0, 1), (1, 8, 100, 0, 1), (1, 8, 128256, 0, 0)):
        assert lib.spec_verify_tree_workspace(*none) == 0
    for bad, code in (((0, 8, 100, 0), -2), ((1, 65, 100, 0), -2), ((1, 8, 0, 0), -2), ((1, 8, 100, 2), -3)):
        assert lib.spec_verify_tree_workspace(*bad, 1) == code


def _cache_call(lib, fork=False, N=4, kts=(4096, 2048, 512, 64), ws_bytes=1 << 20, out_stride=9, **kw):
    c = binding.SvCache()
    d = dict(k=0x10000, v=0x20000, dtype=1, layers=2, pages=50, page_size=16, heads=2, dim=64, table=0x30000,
             table_stride=9, len=0x40000, B=3, width=9)
    ptr = dict(kt=0x50000, vt=0x60000, nodes=0x70000, n=0x80000, out_table=0x90000, out_len=0xA0000, status=0xB0000,
               ws=0xC0000, ancestor=0xD0000)
    c.k_stride = (ctypes.c_int64 * 4)(*kw.pop("k_stride", (65536, 2048, 128, 64)))
    c.v_stride = (ctypes.c_int64 * 4)(65536, 2048, 128, 64)
    for f, x in kw.items():
        (ptr if f in ptr else d)[f] = x
    for f, x in d.items():
        setattr(c, f, x)
    if fork:
        return lib.spec_cache_fork(c, ptr["ancestor"], ptr["out_table"], out_stride, ptr["out_len"], ptr["status"],
                                   ptr["ws"], ws_bytes, None)
    st = (ctypes.c_int64 * 4)(*kts)
    return lib.spec_cache_commit(c, ptr["kt"], ptr["vt"], st, st, N, ptr["nodes"], ptr["n"], ptr["out_table"],
                                 out_stride, ptr["out_len"], ptr["status"], ptr["ws"], ws_bytes, None)


BOTH = [
    (dict(dtype=5), -3), (dict(B=0), -2), (dict(B=65535), -2), (dict(layers=0), -2), (dict(layers=65535), -2),
    (dict(heads=0), -2), (dict(dim=0), -2), (dict(pages=0), -2), (dict(pages=(1 << 20) + 1), -2),
    (dict(page_size=12), -2), (dict(width=0), -2), (dict(width=1 << 28), -2),
    (dict(table=None), -1), (dict(len=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out_table=None), -1),
    (dict(out_len=None), -1), (dict(status=None), -1), (dict(ws=None), -1), (dict(out_stride=8), -1),
    (dict(dim=4), -6), (dict(dim=60), -6), (dict(k=0x10008), -6), (dict(k_stride=(65536, 2048, 124, 64)), -6),
    (dict(k_stride=(65536, -2048, 128, 64)), -1), (dict(ws=0xC0002), -6), (dict(status=0xB0001), -6),
    (dict(ws_bytes=20), -8),
]


@pytest.mark.parametrize("fork", [False, True])
@pytest.mark.parametrize("kw,code", BOTH)
def test_cache_host_validation(lib, fork, kw, code):
    assert _cache_call(lib, fork=fork, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), -2), (dict(N=65), -2), (dict(kt=None), -1), (dict(vt=None), -1), (dict(n=None), -1),
    (dict(kts=(4096, 2048, 512, 60)), -6), (dict(kts=(4096, 2048, -512, 64)), -1), (dict(nodes=0x70002), -6),
    (dict(out_table=0x30000, out_stride=10), -1),
])
def test_commit_host_validation(lib, kw, code):
    assert _cache_call(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ancestor=None), -1), (dict(ancestor=0xD0002), -6), (dict(out_table=0x30000), -1), (dict(out_len=0x40000), -1),
])
def test_fork_host_validation(lib, kw, code):
    assert _cache_call(lib, fork=True, **kw) == code


@pytest.mark.parametrize("fork", [False, True])
def test_cache_rows_written_twice_or_uncountable_are_refused(lib, fork):
    """An expanded cache; more 16-byte vectors per sequence than 32 bits count."""
    for stride in ((0, 2048, 128, 64), (65536, 0, 128, 64), (65536, 2048, 0, 64), (65536, 2048, 128, 0)):
        assert _cache_call(lib, fork=fork, k_stride=stride) == -1
    assert _cache_call(lib, fork=fork, heads=4096, dim=65536, page_size=1024, N=64, ws_bytes=20) == -2
    assert _cache_call(lib, fork=fork, heads=4096, dim=65536, page_size=32, N=32, ws_bytes=20) == -8


def test_cache_workspace(lib):
    assert lib.spec_cache_workspace(3, 4, 16) > 0
    for bad in ((0, 4, 16), (3, -1, 16), (3, 4, 0), (3, 4, 3)):
        assert lib.spec_cache_workspace(*bad) == -2


def test_forced_launch_failure(lib, monkeypatch):
    monkeypatch.setenv("SPECVERIFY_FAIL_LAUNCH", "1")
    assert lib.spec_tree_attention(_attn(), None) == -4
    assert _verify(lib) == -4 and _verify(lib, draft=False) == -4
    assert _cache_call(lib) == -4 and _cache_call(lib, fork=True) == -4
    assert lib.spec_tree_attention(_attn(dim=12), None) == -2


def test_packed_argument_blocks():
    """The binding packs what the C structures hold, field by field."""
    def flat(s):
        out = []
        for name, _ in s._fields_:
            x = getattr(s, name)
            out += list(x) if hasattr(x, "__len__") else [x or 0]
        return out

    for pack, cls, n in ((binding._PACK_LOGITS, binding.SvLogits, 7), (binding._PACK_CACHE, binding.SvCache, 21),
                         (binding._PACK_ATTENTION, binding.SvTreeAttention, 43)):
        values = list(range(1, n + 1))
        blob = pack(*values)
        assert len(blob) == ctypes.sizeof(cls)
        assert flat(cls.from_buffer_copy(blob)) == values


def test_binding_refuses_before_the_library():
    """Shapes and types the C interface cannot see."""
    q = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16)
    kt = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16)
    kc = torch.zeros((10, 16, 2, 64), dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(q=q, k_cache=kc, v_cache=kc, block_table=i(2, 5), seq_len=i(2), k_tree=kt, v_tree=kt, parent=i(2, 4))
    for name, bad in (("q", q.float()), ("q", q[0]), ("k_tree", kt[:, :3]), ("v_tree", kt.half()),
                      ("k_cache", kc[0]), ("v_cache", kc[:, :8]), ("block_table", i(3, 5)),
                      ("block_table", i(2, 5).long()), ("block_table", i(5, 2).t()), ("seq_len", i(3)),
                      ("parent", i(2, 3)), ("parent", i(2, 8)[:, ::2]),
                      ("k_tree", torch.zeros((2, 4, 2, 128), dtype=torch.bfloat16)[..., ::2]),
                      ("q", q.clone().requires_grad_())):
        with pytest.raises(ValueError):
            binding.tree_attention(**{**ok, name: bad})
    with pytest.raises(ValueError, match="GPU"):
        binding.tree_attention(**ok)
    p = torch.zeros((2, 4, 50))
    ok = dict(target_probs=p, draft_probs=p[:, :3], tokens=i(2, 4), parent=i(2, 4), u_accept=torch.zeros(2, 4),
              u_final=torch.zeros(2))
    for name, bad in (("target_probs", p.half()), ("target_probs", p[0]), ("tokens", i(2, 3)), ("parent", i(2, 4).long()),
                      ("u_accept", torch.zeros(2, 4, dtype=torch.float64)), ("u_final", torch.zeros(2, 1))):
        with pytest.raises(ValueError):
            binding.verify_tree(**{**ok, name: bad})
    with pytest.raises(ValueError, match="GPU"):
        binding.verify_tree(**ok)
    c = torch.zeros((2, 10, 16, 2, 64), dtype=torch.bfloat16)
    t = torch.zeros((2, 2, 4, 2, 64), dtype=torch.bfloat16)
    ok = dict(k_cache=c, v_cache=c, block_table=i(2, 5), seq_len=i(2), k_tree=t, v_tree=t, nodes=i(2, 4),
              n_accepted=i(2))
    for name, bad in (("k_cache", c[0]), ("v_cache", c.float()), ("k_tree", t[:1]), ("v_tree", t[..., :32]),
                      ("nodes", i(2, 3)), ("n_accepted", i(1)), ("block_table", i(2, 5).float())):
        with pytest.raises(ValueError):
            binding.cache_commit(**{**ok, name: bad})
    with pytest.raises(ValueError):
        binding.cache_fork(c, c, i(2, 5), i(2), i(3))
    with pytest.raises(ValueError, match="GPU"):
        binding.cache_fork(c, c, i(2, 5), i(2), i(2))


def test_a_line_of_tiles_stays_below_32_bits(lib):
    """1024 key heads of 2^28 cache rows and the tree's tile are 2^32 + 1024
    tiles of 64 keys: refused, where the kernel's count would wrap to head 0."""
    big = dict(B=1, heads=1024, kv_heads=1024, dim=64, page_size=1024, table_stride=1 << 18)
    assert lib.spec_tree_attention_workspace(_attn(N=33, width=1 << 18, **big)) == -2
    assert lib.spec_tree_attention(_attn(N=33, width=1 << 18, **big), None) == -2
    assert lib.spec_tree_attention_workspace(_attn(N=33, width=(1 << 18) - 1, **big)) > 0
    assert lib.spec_tree_attention_workspace(_attn(N=32, width=1 << 18, **big)) > 0  # tiles of 128 keys
    fewer = dict(big, heads=1023, kv_heads=1023)
    assert lib.spec_tree_attention_workspace(_attn(N=33, width=1 << 18, **fewer)) > 0


def test_rounded_launches_stay_below_the_largest_grid(lib):
    """Several row tiles are launched in groups of eight parts: 5592405 parts of
    three tiles are fewer than 2^24 workgroups, rounded up they are not."""
    big = dict(width=4, dim=8, N=48, table_stride=4)  # 384 rows per key head
    assert lib.spec_tree_attention_workspace(_attn(B=46995, heads=952, kv_heads=119, **big)) == -2
    assert lib.spec_tree_attention(_attn(B=46995, heads=952, kv_heads=119, **big), None) == -2
    assert lib.spec_tree_attention_workspace(_attn(B=46994, heads=952, kv_heads=119, **big)) == 0


def test_commit_into_a_shared_page_is_refused():
    """A partly filled page that two live entries name is not appended to;
    shared full pages, and a shared page nobody appends to, are fine."""
    k = np.zeros((1, 12, 4, 1, 1))
    kt = np.arange(1.0, 7).reshape(1, 3, 2, 1, 1)
    lens = np.array([6, 6, 4], np.int32)
    apart = np.array([[3, 5, -1], [3, 6, -1], [3, -1, -1]], np.int32)
    for table, n, want in ((apart, [0, 1, 0], 0),
                           ([[3, 5, -1], [3, 5, -1], [3, -1, -1]], [0, 1, 0], -1),   # both append
                           ([[3, 5, -1], [3, 5, -1], [3, -1, -1]], [0, -1, 0], -1),  # one does
                           ([[3, 5, -1], [3, 5, -1], [3, -1, -1]], [-1, -1, 0], 0),  # neither
                           ([[3, 5, -1], [3, 6, -1], [5, -1, -1]], [0, 0, -1], -1),  # another's full page
                           ([[5, 5, -1], [3, 6, -1], [3, -1, -1]], [0, -1, -1], -1),  # its own
                           ([[3, 5, 5], [3, 6, 6], [3, 6, 5]], [0, 0, 0], 0)):  # entries behind the live ones
        kk, vv = k.copy(), k.copy()
        t, m, status = ref.cache_commit(kk, vv, np.array(table, np.int32), lens, kt, -kt, None, np.array(n, np.int32))
        assert status == want, (table, n)
        if want:
            assert not kk.any() and (m == lens).all() and (t[:, :2] == np.array(table)[:, :2])[:2].all()
        else:
            assert (m == lens + np.array(n) + 1).all()


def test_kept_workspace_sizes_are_bounded(monkeypatch):
    """A decoder whose tables grow with its batch asks for ever new sizes."""
    monkeypatch.setattr(binding, "_workspaces", {})
    asked = []
    for i in range(5000):
        for _ in range(2):
            assert binding._workspace_bytes(None, ("sizes", i), lambda: asked.append(i) or i) == i
    assert asked == list(range(5000))
    assert len(binding._workspaces) <= 1024
    a = dict(index=0, B=1, N=2, heads=4, kv_heads=2, dim=64, page_size=16, width=5)
    assert binding._workspace_bytes(None, tuple(a.values()), lambda: 7) == 7


def test_refused_sizes_are_not_kept(lib, monkeypatch):
    monkeypatch.setattr(binding, "_workspaces", {})
    for _ in range(2):
        with pytest.raises(binding.SpecVerifyError):
            binding._workspace_bytes(lib, ("bad",), lambda: -2)
    assert not binding._workspaces
