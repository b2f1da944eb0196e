"""spec_cache_commit and spec_cache_fork on the GPU against the oracle: tables,
lengths, status and every byte of the cache; refusals leave all as it was."""

import numpy as np
import pytest
import torch

from oracle import tree as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import dev, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def make(lens, N=5, layers=2, ps=8, Hkv=2, D=64, dtype=torch.bfloat16, spare=40, seed=0, head_major=False, extra=4):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    B = len(lens)
    pages, table = tables(lens, ps, rng, extra=extra, spare=spare)
    g = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype).cuda()  # noqa: E731
    pool = (lambda: g(layers, pages, Hkv, ps, D).transpose(2, 3)) if head_major else (lambda: g(layers, pages, ps, Hkv, D))
    n = rng.integers(-1, N, B).astype(np.int32)
    nodes = np.full((B, N), -1, np.int32)
    for b in range(B):
        if n[b] >= 0:
            nodes[b, :n[b] + 1] = [0] + sorted(rng.choice(np.arange(1, N), n[b], replace=False).tolist())
    return dict(k=pool(), v=pool(), table=dev(table), lens=dev(lens), kt=g(layers, B, N, Hkv, D),
                vt=g(layers, B, N, Hkv, D), nodes=dev(nodes), n=dev(n))


def bits(t):
    t = t.contiguous()
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32).cpu().numpy()


def commit(s, **kw):
    return binding.cache_commit(s["k"], s["v"], s["table"], s["lens"], s["kt"], s["vt"], s["nodes"], s["n"], **kw)


def fork(s, anc, **kw):
    return binding.cache_fork(s["k"], s["v"], s["table"], s["lens"], anc, **kw)


def same(s, run, oracle):
    """run(s) and oracle(arrays) leave the same tables, lengths, status, caches."""
    k, v = bits(s["k"]).copy(), bits(s["v"]).copy()
    want = oracle(k, v)
    got = run()
    torch.cuda.synchronize()
    assert int(got[2]) == want[2]
    np.testing.assert_array_equal(got[0].cpu().numpy(), want[0])
    np.testing.assert_array_equal(got[1].cpu().numpy(), want[1])
    np.testing.assert_array_equal(bits(s["k"]), k)
    np.testing.assert_array_equal(bits(s["v"]), v)
    return got


def check_commit(s, **kw):
    h = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    tab, lens = h(s["table"]).copy(), h(s["lens"]).copy()
    return same(s, lambda: commit(s, **kw), lambda k, v: ref.cache_commit(
        k, v, tab, lens, bits(s["kt"]), bits(s["vt"]), h(s["nodes"]), h(s["n"])))


def check_fork(s, anc):
    a = dev(np.asarray(anc, np.int32))
    return same(s, lambda: fork(s, a), lambda k, v: ref.cache_fork(k, v, s["table"].cpu().numpy(),
                                                                   s["lens"].cpu().numpy(), anc))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ps", [1, 2, 8, 64, 1024])
@pytest.mark.parametrize("head_major", [False, True])
def test_commit(dtype, ps, head_major):
    check_commit(make([0, 1, 7, 8, 9, 30, 63, 64], ps=ps, dtype=dtype, head_major=head_major, seed=ps))


@pytest.mark.parametrize("D,Hkv,layers,N", [(8, 1, 1, 1), (80, 3, 5, 64), (128, 8, 3, 17)])
def test_commit_shapes(D, Hkv, layers, N):
    check_commit(make([5, 100, 0, 31], D=D, Hkv=Hkv, layers=layers, N=N, extra=12, spare=60))


def test_commit_chain_and_in_place():
    s = make([5, 100, 0, 31])
    s["nodes"] = None
    check_commit(s)
    s = make([5, 100, 0, 31], seed=3)
    got = check_commit(s, out_table=s["table"], out_len=s["lens"])
    assert got[0] is s["table"] and got[1] is s["lens"]


def test_commit_many_sequences():
    rng = np.random.default_rng(1)
    check_commit(make(rng.integers(0, 40, 2100), layers=1, Hkv=1, D=8, spare=4000))


def test_commit_refusals_change_nothing():
    s = make([8, 16, 24], ps=8, spare=2)
    s["n"].fill_(2)
    s["nodes"][:, :3] = torch.arange(3, dtype=torch.int32)
    assert int(check_commit(s)[2]) == 1  # three pages wanted, two free
    for change in ("node", "count", "length", "page", "width"):
        s = make([8, 16, 24], ps=8)
        s["n"].fill_(2)
        s["nodes"][:, :3] = torch.arange(3, dtype=torch.int32)
        if change == "node":
            s["nodes"][1, 1] = 5
        elif change == "count":
            s["n"][1] = 5
        elif change == "length":
            s["lens"][2] = 10 ** 6
        elif change == "page":
            s["table"][0, 0] = -2
        else:
            s["lens"][2] = s["table"].shape[1] * 8
            s["table"].clamp_(min=0)
        assert int(check_commit(s)[2]) == -1, change


@pytest.mark.parametrize("ps", [1, 4, 16, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_fork(ps, dtype):
    for seed in range(3):
        rng = np.random.default_rng(seed)
        lens = rng.integers(0, 70, 9)
        check_fork(make(lens, ps=ps, dtype=dtype, seed=seed, head_major=seed == 1),
                   np.sort(rng.integers(-1, 9, 9)) if seed else rng.integers(-1, 9, 9))


def test_fork_identity_all_from_one_and_free():
    s = make([5, 16, 30], ps=8)
    got = check_fork(s, [0, 1, 2])
    assert torch.equal(got[0], s["table"]) and torch.equal(got[1], s["lens"])
    check_fork(s, [2, 2, 2])
    got = check_fork(s, [-1, -1, -1])
    assert (got[0] == -1).all() and (got[1] == 0).all()


def test_fork_reuses_the_pages_of_dropped_slots():
    # no spare page: the copies go to the pages the dropped slot leaves
    s = make([13, 21], ps=8, spare=0)
    got = check_fork(s, [0, 0])
    assert int(got[2]) == 0


def test_fork_refusals_change_nothing():
    s = make([13, 13, 13], ps=8, spare=0)
    s["lens"][1] = 0  # its two pages are free now, four copies are wanted by none: two of [0, 0, 0]
    check_fork(s, [0, 0, 0])
    s = make([13, 3], ps=8, spare=0)
    assert int(check_fork(s, [1, 0])[2]) == 0
    s = make([13] * 6, ps=8, spare=0)
    for b in range(1, 6):
        s["table"][b] = s["table"][0]  # one sequence's pages only
    s["table"][5, 0] = s["table"][0, 0]
    for bad in ([0, 1, 6, 3, 4, 5], [0, 1, -2, 3, 4, 5]):
        assert int(check_fork(s, bad)[2]) == -1
    s["table"][2, 0] = 10 ** 5
    assert int(check_fork(s, [0, 1, 2, 3, 4, 5])[2]) == -1
    s = make([13] * 4, ps=8, spare=0)
    s["k"], s["v"] = s["k"][:, :8].contiguous(), s["v"][:, :8].contiguous()
    used = s["table"][:, :2].flatten().tolist()
    assert sorted(used) == list(range(8))
    big = make([13, 12, 11], ps=8, spare=0)  # 6 pages: sequence 0 thrice wants 2 + 2, has 6: fits
    assert int(check_fork(big, [0, 0, 0])[2]) == 0
    tight = make([9, 9, 9], ps=8, spare=0)
    tight["table"][1], tight["table"][2] = tight["table"][0], tight["table"][0]
    tight["k"], tight["v"] = tight["k"][:, :6].contiguous(), tight["v"][:, :6].contiguous()
    assert int(check_fork(tight, [0, 0, 0])[2]) == 0


def test_fork_lacking_pages():
    s = make([9], ps=8, spare=0)  # two pages in all
    two = dict(s, table=s["table"].repeat(4, 1).contiguous(), lens=s["lens"].repeat(4).contiguous())
    assert int(check_fork(two, [0, 0, 0, 0])[2]) == 3


def test_large_page_numbers():
    """The largest pool: page numbers up to 2^20 - 1."""
    pages = 1 << 20
    k = torch.zeros((1, pages, 1, 1, 8), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    lens = np.array([3, 2], np.int32)
    table = np.full((2, 8), -1, np.int32)
    table[0, :3], table[1, :2] = [pages - 1, 0, 1], [2, 1 << 19]
    s = dict(k=k, v=v, table=dev(table), lens=dev(lens), kt=torch.randn((1, 2, 2, 1, 8), device="cuda").bfloat16(),
             vt=torch.randn((1, 2, 2, 1, 8), device="cuda").bfloat16(), nodes=None, n=dev(np.array([1, 0], np.int32)))
    t, n, st = commit(s)
    assert int(st) == 0 and t[0, :5].tolist() == [pages - 1, 0, 1, 3, 4] and t[1, :3].tolist() == [2, 1 << 19, 5]
    assert torch.equal(k[0, 3:6, 0], torch.stack([s["kt"][0, 0, 0], s["kt"][0, 0, 1], s["kt"][0, 1, 0]]))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes per layer: the last page's rows."""
    pages, ps, H, D = 70000, 16, 16, 128  # 2 bytes each: 4.6 GB
    k = torch.zeros((1, pages, ps, H, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = np.full((2, 4), -1, np.int32)
    table[0, 0], table[1, 0] = pages - 1, pages - 2
    kt, vt = torch.randn((1, 2, 3, H, D), device="cuda").bfloat16(), torch.randn((1, 2, 3, H, D), device="cuda").bfloat16()
    s = dict(k=k, v=v, table=dev(table), lens=dev(np.array([4, 1], np.int32)), kt=kt, vt=vt, nodes=None,
             n=dev(np.array([2, 2], np.int32)))
    t, n, st = commit(s)
    assert int(st) == 0 and n.tolist() == [7, 4]
    assert torch.equal(k[0, pages - 1, 4:7], kt[0, 0]) and torch.equal(v[0, pages - 2, 1:4], vt[0, 1])
    q = torch.randn((2, 1, H, D), device="cuda").bfloat16()
    out = binding.tree_attention(q, k[0], v[0], t, n, kt[0, :, :1], vt[0, :, :1],
                                 torch.full((2, 1), -1, dtype=torch.int32, device="cuda"))
    for b, (pg, m) in enumerate(((pages - 1, 7), (pages - 2, 4))):
        kk = torch.cat((k[0, pg, :m], kt[0, b, :1])).double()
        vv = torch.cat((v[0, pg, :m], vt[0, b, :1])).double()
        w = torch.softmax((kk * q[b].double()).sum(-1) * D ** -0.5, 0)
        want = (w.unsqueeze(-1) * vv).sum(0)
        assert (out[b, 0].double() - want).abs().max() <= 2 * 2.0 ** -8 * vv.abs().max()


def test_graph_replays():
    s = make([5, 100, 0, 31], seed=6)
    anc = dev(np.array([1, 1, 0, 3], np.int32))
    k0, v0 = s["k"].clone(), s["v"].clone()
    fork(s, anc)
    commit(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t1, n1, st1 = fork(s, anc)
        t2, n2, st2 = binding.cache_commit(s["k"], s["v"], t1, n1, s["kt"], s["vt"], s["nodes"], s["n"])
    for rep in range(4):
        s["k"].copy_(k0)
        s["v"].copy_(v0)
        anc.copy_(dev(np.array([[1, 1, 0, 3], [3, 3, 3, 3], [-1, 1, 1, 0], [0, 1, 2, 3]][rep], np.int32)))
        e = fork(s, anc)
        e2 = binding.cache_commit(s["k"], s["v"], e[0], e[1], s["kt"], s["vt"], s["nodes"], s["n"])
        want = (s["k"].clone(), s["v"].clone())
        s["k"].copy_(k0)
        s["v"].copy_(v0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((t1, n1, st1, t2, n2, st2, s["k"], s["v"]), (*e, *e2, *want)):
            assert torch.equal(a, b), rep


@pytest.mark.parametrize("B", [3, 1500])  # one thread per sequence, and more sequences than threads
@pytest.mark.parametrize("how", ["both", "one", "neither", "full", "itself", "behind"])
def test_commit_into_a_shared_page_is_refused(how, B):
    """Two live entries name a partly filled page that is appended to: nothing
    is.  Its neighbours in the batch lie anywhere in it."""
    s = make([14] * B, ps=8, N=3, Hkv=1, layers=1, spare=2 * B + 4, seed=5)
    s["nodes"] = None
    s["n"].fill_(1)
    a, b = B // 3, B - 1
    s["table"][b, 0] = s["table"][a, 0]  # a shared full page
    if how in ("both", "one", "neither"):
        s["table"][b, 1] = s["table"][a, 1]
        s["n"][a] = 1 if how == "both" else -1
        s["n"][b] = -1 if how == "neither" else 1
    elif how == "full":
        s["lens"][b], s["n"][b] = 16, -1
        s["table"][b, 1] = s["table"][a, 1]
    elif how == "itself":
        s["table"][a, 0] = s["table"][a, 1]
    else:
        s["table"][b, 2:] = s["table"][a, 1]  # not live
    got = check_commit(s)
    assert int(got[2]) == (0 if how in ("neither", "behind") else -1)


def test_commit_after_a_fork_owns_its_pages():
    """spec_cache_fork leaves every partly filled page to one slot."""
    s = make([13, 16, 21, 3], ps=8, spare=20, N=4)
    got = check_fork(s, [2, 2, 0, 2])
    s["table"], s["lens"] = got[0], got[1]
    s["nodes"] = None
    s["n"].fill_(2)
    assert int(check_commit(s)[2]) == 0


def test_most_sequences_and_most_layers():
    """The limits the header states: 65534 sequences, 65534 layers."""
    rng = np.random.default_rng(2)
    B = 65534
    s = make(rng.integers(0, 8, B), N=2, ps=2, layers=1, Hkv=1, D=8, spare=2 * B, extra=2)
    assert int(check_commit(s)[2]) == 0
    s["n"].fill_(-1)
    anc = rng.integers(-1, B, B)
    assert int(check_fork(s, anc)[2]) == 0
    s = make([3, 0, 2], N=3, ps=2, layers=65534, Hkv=1, D=8, spare=8)
    assert int(check_commit(s)[2]) == 0
    assert int(check_fork(s, [0, 0, 2])[2]) == 0


def test_expanded_tree_rows():
    """The same tree rows for every sequence and head."""
    s = make([5, 100, 0, 31], Hkv=4)
    s["kt"], s["vt"] = s["kt"][:, :1, :, :1].expand(-1, 4, -1, 4, -1), s["vt"][:, :, :, 1:2].expand(-1, -1, -1, 4, -1)
    assert int(check_commit(s)[2]) == 0
