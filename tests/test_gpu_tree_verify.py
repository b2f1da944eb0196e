"""spec_verify_tree on the GPU against the float64 oracle: equal outputs at
every decision further than float64 rounding from its border, invalid
sequences, odd vocabularies and strides, and HIP graphs."""

import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import tree as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import dev, f64, parents

pytestmark = pytest.mark.gpu

# Decisions are float64 comparisons of sums of at most V + V terms: the sums'
# relative rounding is below 2 V 2^-53, 5e-10 at the largest V, and a walk
# repeats it at most 63 times.
BAND = 3e-8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def make(B, N, V, kind="level2", draft=True, dtype=torch.float32, seed=0, n_nodes=None, noise=0.7):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((B, N, V)) * 2
    par = parents(kind, B, N, rng)
    soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
    p = torch.from_numpy(soft(logits)).to(dtype)
    P = max(1, int(par.max()) + 1)
    q = torch.from_numpy(soft(logits[:, :P] + noise * rng.standard_normal((B, P, V)))).to(dtype) if draft else None
    tok = np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(1, N):
            if draft:
                row = q[b, par[b, i]].double().numpy()
                tok[b, i] = rng.choice(V, p=row / row.sum())
            else:
                order = np.argsort(-p[b, par[b, i]].double().numpy(), kind="stable")
                tok[b, i] = order[min(V - 1, int((par[b, :i] == par[b, i]).sum()))]
    return dict(p=p.cuda(), q=None if q is None else q.cuda(), tok=dev(tok), par=dev(par),
                ua=dev(rng.random((B, N), np.float32)), uf=dev(rng.random(B, np.float32)),
                n=None if n_nodes is None else dev(np.asarray(n_nodes, np.int32)))


def call(s, **kw):
    return binding.verify_tree(s["p"], s["q"], s["tok"], s["par"], s["ua"], s["uf"], s["n"], **kw)


def check(s, label):
    got = [t.cpu().numpy() for t in call(s)]
    h = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    t, nd, n, margin = ref.verify_tree(f64(s["p"]), None if s["q"] is None else f64(s["q"]), h(s["tok"]), h(s["par"]),
                                       h(s["ua"]), h(s["uf"]), h(s["n"]))
    clear = margin > BAND
    assert clear.mean() > 0.9
    say(f"[tree verify] {label}: accepted {n.tolist()[:8]}, {int((~clear).sum())} of {len(n)} within the band")
    np.testing.assert_array_equal(got[2][clear], n[clear])
    np.testing.assert_array_equal(got[1][clear], nd[clear])
    np.testing.assert_array_equal(got[0][clear], t[clear])
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 255, 256, 257, 1000, 4099, 20001])
def test_vocabularies(V, draft, dtype):
    check(make(6, 7, V, draft=draft, dtype=dtype, seed=V), f"V={V} draft={draft} {dtype}")


@pytest.mark.parametrize("kind", ["chain", "star", "level2", "level4", "random"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("N", [1, 2, 16, 64])
def test_tree_shapes(kind, draft, N):
    check(make(12, N, 300, kind=kind, draft=draft, seed=N), f"{kind} N={N} draft={draft}")


def test_ragged_and_empty_trees():
    s = make(6, 9, 500, n_nodes=[9, 1, 0, 5, 10, -1])
    got = check(s, "ragged")
    assert (got[2][[2, 4, 5]] == -1).all() and got[2][1] == 0


@pytest.mark.parametrize("draft", [True, False])
def test_many_refusals(draft):
    """Far-off drafts: every sibling costs a sum."""
    s = make(16, 12, 700, kind="star", draft=draft, noise=6.0, seed=3)
    s["ua"].clamp_(min=0.6)
    got = check(s, f"refusals draft={draft}")
    assert (got[2] == 0).any()


def test_repeated_children():
    """The same id twice among siblings: refused once, refused again."""
    for draft in (True, False):
        s = make(8, 6, 50, kind="star", draft=draft, noise=3.0, seed=4)
        s["tok"][:, 2:] = s["tok"][:, 1:2]
        check(s, f"repeated draft={draft}")


def test_equal_distributions_accept_everything():
    s = make(5, 8, 999, kind="chain")
    s["q"] = s["p"][:, :7].contiguous()
    got = check(s, "p = q")
    assert (got[2] == 7).all()


def test_nothing_left_falls_back_to_the_target():
    # q >= p everywhere and refused: the residual is zero
    p = torch.zeros((1, 2, 4))
    p[0, :, 1], p[0, :, 2] = 0.25, 0.25
    q = torch.full((1, 1, 4), 0.5)
    one = dict(p=p.cuda(), q=q.cuda(), tok=dev(np.array([[0, 1]], np.int32)), par=dev(np.array([[-1, 0]], np.int32)),
               ua=dev(np.array([[0, 0.9]], np.float32)), uf=dev(np.array([0.75], np.float32)), n=None)
    t, nd, n = check(one, "zero residual")
    assert n[0] == 0 and t[0, 0] == 2
    one["q"] = None
    p[0, 0, 2], p[0, 0, 1] = 0.0, 0.5
    one["p"] = p.cuda()
    t, nd, n = [x.cpu().numpy() for x in call(one)]
    assert n[0] == 0 and t[0, 0] == 1
    p.zero_()
    one["p"] = p.cuda()
    assert [x.cpu().numpy().tolist() for x in call(one)] == [[[-1, -1]], [[-1, -1]], [-1]]


def test_random_numbers_at_the_ends():
    s = make(4, 5, 400, kind="chain")
    s["ua"].zero_()
    s["uf"].zero_()
    check(s, "zeros")
    s["ua"].fill_(1 - 2.0 ** -24)
    s["uf"].fill_(1 - 2.0 ** -24)
    check(s, "next to one")


def test_invalid_sequences():
    base = lambda: make(10, 6, 300, kind="level2", seed=8)  # noqa: E731
    s = base()
    s["tok"][0, 3], s["tok"][1, 5] = -1, 300
    s["par"][2, 4], s["par"][3, 2], s["par"][4, 1] = 4, -1, 1
    s["ua"][5, 1], s["ua"][6, 2], s["uf"][7], s["uf"][8] = 1.0, float("nan"), -0.25, float("nan")
    s["par"][9, 0], s["tok"][9, 0], s["ua"][9, 0] = 77, -5, 9.0  # the root's are not read
    got = check(s, "invalid indices")
    assert (got[2][:9] == -1).all() and got[2][9] >= 0
    for bad in (float("nan"), float("inf"), -1e-3):
        s = base()
        s["p"][:, :, 17] = bad
        got = [t.cpu().numpy() for t in call(s)]
        assert (got[2] == -1).all() and (got[0] == -1).all() and (got[1] == -1).all()
    s = base()
    s["q"] = s["q"][:, :1].contiguous()  # children of nodes without a draft row
    assert (call(s)[2] == -1).all()


def test_strides_and_alignment():
    for dtype in (torch.float32, torch.bfloat16):
        s = make(4, 6, 1003, dtype=dtype, seed=2)
        want = call(s)
        wide = torch.full((4, 7, 1010), float("nan"), dtype=dtype, device="cuda")
        wide[:, :6, 3:1006] = s["p"]
        s["p"] = wide[:, :6, 3:1006]
        for a, b in zip(call(s), want):
            assert torch.equal(a, b)


def test_largest_vocabulary():
    V = 1 << 21
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.softmax(torch.randn((1, 2, V), device="cuda", generator=g), -1)
    q = torch.softmax(torch.randn((1, 1, V), device="cuda", generator=g), -1)
    for uf in (0.0, 0.3, 0.999999):
        s = dict(p=p, q=q, tok=dev(np.array([[0, 5]], np.int32)), par=dev(np.array([[-1, 0]], np.int32)),
                 ua=dev(np.array([[0, 1 - 2.0 ** -24]], np.float32)), uf=dev(np.array([uf], np.float32)), n=None)
        check(s, f"V=2^21 u={uf}") if uf else call(s)


@pytest.mark.parametrize("looks", ["0", "1", "64"])
def test_teams_do_not_depend_on_each_other(monkeypatch, looks):
    """However often a workgroup looks for the others' sums (0: it computes
    every one itself), the result is the same."""
    for B, V, dtype in ((1, 70001, torch.float32), (9, 50000, torch.bfloat16), (40, 30000, torch.float32)):
        s = make(B, 10, V, kind="level3", noise=3.0, dtype=dtype, seed=B)
        assert binding.load().spec_verify_tree_workspace(B, 10, V, 1 if dtype == torch.bfloat16 else 0, 1) > 0
        want = check(s, f"team B={B} V={V}")
        monkeypatch.setenv("SPECVERIFY_VERIFY_LOOKS", looks)
        got = [t.cpu().numpy() for t in call(s)]
        monkeypatch.delenv("SPECVERIFY_VERIFY_LOOKS")
        for a, b in zip(got, want):
            np.testing.assert_array_equal(a, b)


def test_two_teams_at_once():
    a, b = make(1, 8, 60000, seed=1), make(3, 8, 60000, kind="star", noise=4.0, seed=2)
    want_a, want_b = [[t.clone() for t in call(x)] for x in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        oa, ob = call(a, stream=s1), call(b, stream=s2)
        s1.synchronize()
        s2.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(oa, want_a))
        assert all(torch.equal(x, y) for x, y in zip(ob, want_b))


def test_graph_replays_and_streams():
    s = make(8, 7, 20000, seed=1)
    call(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(s)
    stream = torch.cuda.Stream()
    for rep in range(4):
        n = make(8, 7, 20000, seed=20 + rep)
        for k in ("p", "q", "tok", "ua", "uf"):
            s[k].copy_(n[k])
        want = call(s)
        graph.replay()
        torch.cuda.synchronize()
        other = call(s, stream=stream)
        stream.synchronize()
        for a, b, c in zip(outs, want, other):
            assert torch.equal(a, b) and torch.equal(c, b), rep


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V,first", [(1, 1 << 21, 1234567), (3, 128256, 100000), (300, 20001, 19999), (2, 700, 0)])
def test_draw_at_zero_is_the_first_id_with_weight(B, V, first, dtype):
    """u_final = 0 draws the first id of which something is left, whatever the
    order of the sums: exact, there is no border below it."""
    g = torch.Generator(device="cuda").manual_seed(V)
    p = torch.softmax(torch.randn((B, 2, V), device="cuda", generator=g), -1).to(dtype)
    q = p[:, :1].clone()
    q[:, :, first:] = torch.softmax(torch.randn((B, 1, V), device="cuda", generator=g), -1).to(dtype)[:, :, first:]
    q[:, 0, -1] = p[:, 0, -1] * 4  # the child: refused at u next to 1
    q[:, 0, first] = p[:, 0, first] / 2
    s = dict(p=p, q=q, tok=dev(np.tile(np.array([[0, V - 1]], np.int32), (B, 1))),
             par=dev(np.tile(np.array([[-1, 0]], np.int32), (B, 1))),
             ua=dev(np.tile(np.array([[0, 1 - 2.0 ** -24]], np.float32), (B, 1))), uf=dev(np.zeros(B, np.float32)), n=None)
    want = (f64(p[:, 0]) - f64(q[:, 0]) > 0).argmax(-1)
    assert (want == first).all()
    t, nd, n = [x.cpu().numpy() for x in call(s)]
    assert (n == 0).all() and (nd == np.array([0, -1])).all()
    np.testing.assert_array_equal(t[:, 0], want)
    # chosen children: the first id but the refused one
    p[:, 0, :first] = 0.0
    s.update(q=None, tok=dev(np.tile(np.array([[0, first]], np.int32), (B, 1))))
    t, nd, n = [x.cpu().numpy() for x in call(s)]
    assert (n == 0).all()
    np.testing.assert_array_equal(t[:, 0], np.full(B, first + 1))


def test_largest_batch():
    """2^22 - 1 sequences of one node: the token is the inverse CDF's."""
    B, V = (1 << 22) - 1, 3
    g = torch.Generator(device="cuda").manual_seed(0)
    p = torch.rand((B, 1, V), device="cuda", generator=g)
    uf = torch.rand((B,), device="cuda", generator=g)
    z = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    t, nd, n = binding.verify_tree(p, None, z, z, torch.zeros((B, 1), device="cuda"), uf)
    cum = p[:, 0].double().cumsum(-1)
    at = uf.double() * cum[:, -1]
    clear = ((cum[:, :2] - at.view(B, 1)).abs() > 1e-12).all(-1)
    assert clear.float().mean() > 0.999
    want = (cum[:, :2] <= at.view(B, 1)).sum(-1).int()
    assert torch.equal(t[clear, 0], want[clear])
    assert not nd.any() and not n.any()


@pytest.mark.parametrize("draft", [True, False])
def test_expanded_inputs(draft):
    """One set of rows for all sequences; one row for all nodes."""
    s = make(5, 9, 2003, draft=draft, seed=6)
    e = dict(s, p=s["p"][:1].expand(5, -1, -1), q=s["q"][:1, :1].expand(5, 8, -1) if draft else None)
    check(e, "expanded over the batch")
    e = dict(s, p=s["p"][:, :1].expand(-1, 9, -1))
    check(e, "expanded over the nodes")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [300, 70001])
def test_smallest_and_largest_probabilities(V, draft, dtype):
    """Rows of denormal numbers, and rows (not distributions) near the largest."""
    for factor in (2.0 ** -130, 2.0 ** 125):
        s = make(3, 6, V, draft=draft, dtype=dtype, seed=V)
        s["p"] = (s["p"].double() / s["p"].double().amax() * factor).to(dtype)
        if draft:
            s["q"] = (s["q"].double() / s["q"].double().amax() * factor).to(dtype)
        check(s, f"times {factor:.0e}")
